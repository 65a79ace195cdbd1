"""GPU parity of appending by position and reading back.  The append must leave the same bytes as the pack
by slots (itself checked against the oracle) and as the oracle, at every combination of norm and rotation,
ragged counts around the kernel's switch to several tokens per warp, empty sequences and windows; the
read-back is exact.  Metadata out of range is reported and touches nothing else."""
import numpy as np
import pytest
import torch

import oracle
from fp4_compressed_sparse_kv_b200 import csa, synth
from runs_helpers import Run, random_layer, values64

pytestmark = pytest.mark.gpu

CACHES = ("codes", "scales", "keys", "swa", "swa_scale")


def header_ws():
    ws = torch.empty(csa.HEADER_BYTES, dtype=torch.uint8, device="cuda")
    csa.workspace_init(ws)
    return ws


def inputs(rows, positions, seed):
    rng = np.random.default_rng(seed)
    lat = synth.bf16_bits((rng.standard_normal((rows, 512)) * np.exp(rng.uniform(-5, 5, (rows, 1)))).astype(np.float32))
    lat[::53] = 0
    key = synth.index_keys(rng, rows)
    w = rng.uniform(-1.5, 1.5, 512).astype(np.float32)
    ang = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(32) / 32.0)
    table = np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)
    return lat, key, w, table


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a)).view(torch.bfloat16).cuda()


SHAPES = [([1], [1]), ([1, 1, 1], [70, 1, 129]), ([0, 5, 0, 200, 1], [9, 5, 1, 300, 64]), ([130, 127, 128], [130, 500, 129]),
          ([1] * 40, list(range(1, 41))), ([0] * 30 + [3] + [0] * 1000 + [2], [1] * 30 + [66] + [1] * 1000 + [2]),
          ([2500, 1603], [2500, 3001]), ([4099], [4100])]


@pytest.mark.parametrize("norm,rope", [(True, True), (False, False), (True, False), (False, True)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_append_equals_pack_by_slots(shape, norm, rope):
    n, lens = SHAPES[shape]
    r = Run(n, lens, 10 + shape)
    lat, key, w, table = inputs(r.rows, max(lens), 20 + shape)
    seq, pos = r.positions()
    a, b = csa.KVLayer(r.num_pages, r.B), csa.KVLayer(r.num_pages, r.B)
    for layer in (a, b):        # stale bytes stay where no row goes
        for name in CACHES:
            getattr(layer, name).fill_(7)
    ws = header_ws()
    dw, dt = torch.from_numpy(w).cuda(), torch.from_numpy(table).cuda()
    csa.kv_append_fp4(a, r.batch, r.cu_rows, bf16(lat), bf16(key), ws, norm_weight=dw if norm else None,
                      rope_table=dt if rope else None)
    assert csa.check_device_error(ws)[0] == 0
    slot = torch.from_numpy(np.array([r.slots(s, p) for s, p in zip(seq, pos)], np.int64)).cuda()
    ring = np.where(pos >= np.array(lens)[seq] - 128, seq * 128 + pos % 128, -1).astype(np.int32)
    if norm or rope:            # a missing step is the identity: unit weight has no norm, so only compare what exists
        cs = table[pos] if rope else np.broadcast_to(np.array([1.0, 0.0], np.float32), (r.rows, 32, 2))
        if norm:
            csa.kv_norm_rope_pack_fp4(b, bf16(lat), dw, torch.from_numpy(np.ascontiguousarray(cs)).cuda(), bf16(key), slot,
                                      torch.from_numpy(ring).cuda(), ws)
        else:                   # the rotation alone, in the order the append fixes, on the CPU in binary32
            x = synth.bf16_to_f32(lat).copy()
            u, v = x[:, 448::2].copy(), x[:, 449::2].copy()
            x[:, 448::2] = u * cs[..., 0] - v * cs[..., 1]
            x[:, 449::2] = u * cs[..., 1] + v * cs[..., 0]
            csa.kv_pack_fp4(b, bf16(synth.bf16_bits(x)), bf16(key), slot, torch.from_numpy(ring).cuda(), ws)
    else:
        csa.kv_pack_fp4(b, bf16(lat), bf16(key), slot, torch.from_numpy(ring).cuda(), ws)
    for name in CACHES:
        assert torch.equal(getattr(a, name), getattr(b, name)), name


def test_append_equals_oracle():
    n, lens = [5, 0, 333], [90, 3, 400]
    r = Run(n, lens, 1)
    lat, key, w, table = inputs(r.rows, 400, 2)
    seq, pos = r.positions()
    layer, ws = csa.KVLayer(r.num_pages, r.B), header_ws()
    csa.kv_append_fp4(layer, r.batch, r.cu_rows, bf16(lat), bf16(key), ws, norm_weight=torch.from_numpy(w).cuda(),
                      rope_table=torch.from_numpy(table).cuda())
    ref = oracle.pack_tokens(oracle.norm_rope(lat, w, np.ascontiguousarray(table[pos])), key)
    slot = np.array([r.slots(s, p) for s, p in zip(seq, pos)])
    assert np.array_equal(layer.codes.view(-1, 256).cpu().numpy()[slot], ref["codes"])
    assert np.array_equal(layer.scales.view(-1, 32).cpu().numpy()[slot], ref["scales"])
    assert np.array_equal(layer.keys.view(-1, 128).cpu().numpy()[slot], ref["key8"])
    keep = pos >= np.array(lens)[seq] - 128
    ring = (seq * 128 + pos % 128)[keep]
    assert np.array_equal(layer.swa.view(-1, 512).cpu().numpy()[ring], ref["swa"][keep])
    assert np.array_equal(layer.swa_scale.view(-1).cpu().numpy()[ring], ref["swa_scale"][keep])


@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_unpack_is_exact_and_leaves_other_rows(shape):
    n, lens = SHAPES[shape]
    r = Run(n, lens, 30 + shape, pad_rows=5)
    layer, ws = random_layer(r.num_pages, 31 + shape), header_ws()
    out = torch.full((r.rows, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    csa.kv_unpack_fp4(layer, r.batch, r.cu_rows, out, ws)
    assert csa.check_device_error(ws)[0] == 0
    seq, pos = r.positions()
    slot = np.array([r.slots(s, p) for s, p in zip(seq, pos)])
    assert torch.equal(out[:-5].double(), values64(layer, slot))
    assert (out[-5:] == 3.0).all()


def test_every_code_and_scale_reads_back():
    layer, ws = csa.KVLayer(4, 1), header_ws()
    e = torch.arange(256, device="cuda", dtype=torch.uint8)
    layer.codes.view(256, 256).copy_(e[None, :].expand(256, 256))
    layer.scales.view(256, 32).copy_(e[:, None].expand(256, 32))
    r = Run([256], [256], 3, spare=0)
    out = torch.empty((256, 512), dtype=torch.bfloat16, device="cuda")
    csa.kv_unpack_fp4(layer, r.batch, r.cu_rows, out, ws)
    ref = values64(layer, r.slots(0, np.arange(256)))
    assert torch.equal(torch.nan_to_num(out.double(), nan=1e30), torch.nan_to_num(ref, nan=1e30))


def test_bad_metadata_is_reported_and_skipped():
    n, lens = [4, 4, 4], [100, 100, 100]
    lat, key, w, table = inputs(12, 100, 5)
    for what in ("page", "long", "rows", "short table", "swa row"):
        r = Run(n, lens, 6)
        layer, ws = csa.KVLayer(r.num_pages, 3), header_ws()
        dt = torch.from_numpy(table).cuda()
        skipped = [1]
        if what == "page":
            r.batch.block_table[1, 1] = r.num_pages
        elif what == "long":
            r.batch.seq_len[1] = 3                      # four new rows of a sequence of three
        elif what == "rows":
            r.cu_rows[2], r.cu_rows[3] = 8, 13          # past the arrays: the last sequence is left out
            skipped = [2]
        elif what == "short table":
            dt = dt[:96].contiguous()
            skipped = [0, 1, 2]
        else:
            r.batch.swa_row[1] = 3
            skipped = []
        csa.kv_append_fp4(layer, r.batch, r.cu_rows, bf16(lat), bf16(key), ws,
                          norm_weight=torch.from_numpy(w).cuda(), rope_table=dt)
        assert csa.check_device_error(ws)[0] == 5, what
        for b in range(3):
            touched = bool(layer.scales.view(-1, 32)[torch.from_numpy(r.slots(b, np.arange(96, 100))).cuda()].any())
            assert touched == (b not in skipped), (what, b)
        assert not layer.swa[1].any() if what == "swa row" else True
        if what in ("page", "long", "rows"):
            out = torch.full((12, 512), 3.0, dtype=torch.bfloat16, device="cuda")
            csa.kv_unpack_fp4(layer, r.batch, r.cu_rows, out, ws)
            assert csa.check_device_error(ws)[0] == 5, what
            assert (out[4 * skipped[0]:4 * skipped[0] + 4] == 3.0).all()


def test_no_window_and_long_pools():
    """swa_row -1 writes no window; pages whose byte offsets pass 32 bits."""
    pool = 300_000                                       # 4.9 GB of codes
    r = Run([70, 3], [200, 77], 7, pool=pool)
    r.batch.swa_row[1] = -1
    lat, key, w, table = inputs(73, 200, 8)
    layer, ws = csa.KVLayer(pool, 2), header_ws()
    csa.kv_append_fp4(layer, r.batch, r.cu_rows, bf16(lat), bf16(key), ws)
    out = torch.empty((73, 512), dtype=torch.bfloat16, device="cuda")
    csa.kv_unpack_fp4(layer, r.batch, r.cu_rows, out, ws)
    assert csa.check_device_error(ws)[0] == 0
    assert int(r.bt[r.bt >= 0].min()) * 64 * 256 > 2 ** 32
    seq, pos = r.positions()
    ref = oracle.pack_tokens(lat, key)
    want = torch.from_numpy(oracle.dequant_main(ref["codes"], ref["scales"])).double().cuda()
    assert torch.equal(out.double(), want)
    assert layer.swa[0].any() and not layer.swa[1].any()


def test_captured_and_replayed_on_another_stream():
    r = Run([3, 1], [130, 64], 9)
    lat, key, w, table = inputs(4, 130, 10)
    layer, ws = csa.KVLayer(r.num_pages, 2), header_ws()
    dl, dk = bf16(lat), bf16(key)
    out = torch.zeros((4, 512), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        csa.kv_append_fp4(layer, r.batch, r.cu_rows, dl, dk, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            csa.kv_append_fp4(layer, r.batch, r.cu_rows, dl, dk, ws)
            csa.kv_unpack_fp4(layer, r.batch, r.cu_rows, out, ws)
        dl.neg_()
        g.replay()
    torch.cuda.synchronize()
    ref = oracle.pack_tokens(lat ^ np.uint16(0x8000), key)
    assert torch.equal(out.double(), torch.from_numpy(oracle.dequant_main(ref["codes"], ref["scales"])).double().cuda())


def test_binding_refuses_and_takes_streams_and_threads():
    """Non-contiguous and host tensors are refused with nothing written; a side stream and two host threads at once give
    the same entries."""
    import threading
    r = Run([5, 70], [9, 100], 81)
    g = torch.Generator(device="cuda").manual_seed(82)
    latent = torch.randn((75, 512), generator=g, device="cuda").bfloat16()
    key = torch.randn((75, 128), generator=g, device="cuda").bfloat16()
    new_ws = lambda: torch.zeros(csa.HEADER_BYTES, dtype=torch.uint8, device="cuda")
    want, ws = csa.KVLayer(r.num_pages, 2), new_ws()
    csa.workspace_init(ws)
    wide = torch.zeros((75, 1024), dtype=torch.bfloat16, device="cuda")[:, ::2]
    for bad in (dict(latent=wide), dict(idx_key=key.cpu()), dict(cu_rows=r.cu_rows.cpu()), dict(norm_weight=torch.ones(512))):
        with pytest.raises(ValueError):
            csa.kv_append_fp4(**{**dict(layer=want, batch=r.batch, cu_rows=r.cu_rows, latent=latent, idx_key=key, ws=ws), **bad})
    with pytest.raises(ValueError):
        csa.kv_unpack_fp4(want, r.batch, r.cu_rows, wide, ws)
    assert not want.codes.any() and not wide.any()
    csa.kv_append_fp4(want, r.batch, r.cu_rows, latent, key, ws)
    assert csa.check_device_error(ws)[0] == 0
    torch.cuda.synchronize()
    layers = [csa.KVLayer(r.num_pages, 2) for _ in range(4)]
    outs = [torch.zeros_like(latent) for _ in range(4)]
    spaces = [new_ws() for _ in range(4)]
    for w in spaces:
        csa.workspace_init(w)
    torch.cuda.synchronize()

    def work(i):
        side = torch.cuda.Stream()
        for _ in range(50):
            csa.kv_append_fp4(layers[i], r.batch, r.cu_rows, latent, key, spaces[i], stream=side)
            csa.kv_unpack_fp4(layers[i], r.batch, r.cu_rows, outs[i], spaces[i], stream=side)
        side.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    back = torch.zeros_like(latent)
    csa.kv_unpack_fp4(want, r.batch, r.cu_rows, back, ws)
    for l, o, w in zip(layers, outs, spaces):
        assert csa.check_device_error(w)[0] == 0
        for name in ("codes", "scales", "keys", "swa", "swa_scale"):
            assert torch.equal(getattr(l, name), getattr(want, name)), name
        assert torch.equal(o, back)
