"""GPU parity of the attention over the whole FP4 cache against its formula in 64 bits.

Tolerance of a row, from the roundings of the call.  With W = sum p|v| / sum p and A = max_j sm_scale *
sum |q||v_j| of the row and N the positions:
  - a score is a binary32 sum of 512 exact products in some order: |dz| <= 2^-15 A (512 * 2^-24); scaling,
    cap and bias round it a few more times: 2^-21 (max |z| + cap).  A change dz of every score moves out by
    at most 2 |dz| W;
  - P is rounded to fp16, 2^-11 of itself, below fp16's normal range by at most 2^-25 against a largest
    P of at least 2^7: N 2^-32 max |v| in all;
  - sums of N terms in binary32: N 2^-24 W each for numerator and denominator; exp2 and 1/x: 2^-20 W;
  - out is rounded to bf16: 2^-8 |out|.
"""
import math

import numpy as np
import pytest
import torch

from fp4_compressed_sparse_kv_b200 import csa
from runs_helpers import Run, random_layer, values64

pytestmark = pytest.mark.gpu

TAU = 1.0 / math.sqrt(512)


def reference(layer, r, q, spans, cap, slopes, tau=TAU):
    """(out, lse, tolerance of out, tolerance of lse) of every row that belongs to a sequence, in float64."""
    H = q.shape[1]
    outs, lses, tols, ltols = [], [], [], []
    at = 0
    for b, (n, L) in enumerate(zip(r.n, r.lens)):
        if n == 0:
            continue
        v = values64(layer, r.slots(b, np.arange(L)))
        qq = q[at:at + n].double().reshape(n * H, 512)
        p = torch.arange(L - n, L, device="cuda")
        j = torch.arange(L, device="cuda")
        lo, hi = (torch.zeros_like(p), p + 1) if spans is None else spans[at:at + n].long().unbind(1)
        seen = ((j >= lo[:, None]) & (j < hi[:, None])).repeat_interleave(H, 0)
        z = tau * (qq @ v.T)
        a = tau * (qq.abs() @ v.abs().T)
        if cap:
            z = cap * torch.tanh(z / cap)
        if slopes is not None:
            z = z - (slopes.double()[None, :, None] * (p[:, None] - j).abs()[:, None, :]).reshape(n * H, L)
        z = torch.where(seen, z, -math.inf)
        lse = torch.logsumexp(z, 1)
        w = torch.where(seen, torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[:, None]), 0.0)
        out = w @ v
        W = w @ v.abs()
        zmax = torch.where(seen, z.abs(), 0.0).amax(1)
        dz = 2.0 ** -15 * torch.where(seen, a, 0.0).amax(1) + 2.0 ** -21 * (zmax + cap)
        rel = 2 * dz + 2.0 ** -11 + 2 * L * 2.0 ** -24 + 2.0 ** -20
        outs.append(out)
        lses.append(lse)
        tols.append(2.0 ** -8 * out.abs() + rel[:, None] * W * (1 + 2.0 ** -8) + L * 2.0 ** -32 * v.abs().max())
        ltols.append(dz + L * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -21 * torch.where(lse == -math.inf, 0.0, lse).abs())
        at += n
    shape = lambda x: torch.cat(x).reshape(at, H, -1)
    return shape(outs), shape(lses)[..., 0], shape(tols), shape(ltols)[..., 0]


def queries(rows, H, seed, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn((rows, H, 512), generator=g, device="cuda")).bfloat16()


def make_spans(r, kind, seed):
    if kind == "causal":
        return None
    rng = np.random.default_rng(seed)
    seq, pos = r.positions()
    L = np.array(r.lens)[seq]
    if kind == "window":
        s = np.stack([pos - 99, pos + 1], 1)             # negative lo counts as 0
    elif kind == "all":
        s = np.stack([0 * pos, L + 1000], 1)             # hi past the end counts as the end
    else:                                                # documents, prefixes, rows that see nothing
        lo = pos // 150 * 150
        s = np.stack([lo, np.maximum(pos + 1, np.minimum(lo + 40, L))], 1)
        s[rng.random(pos.size) < 0.1] = [5, 5]
        s[::17] = [2 ** 31 - 1, -(2 ** 31)]
        s[5:9] = [0, 1]
    return torch.from_numpy(s.astype(np.int32)).cuda()


def attend(layer, r, q, spans=None, cap=0.0, slopes=None, ws=None, fill=7.0, **kw):
    out = torch.full(q.shape, fill, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], fill, device="cuda")
    ws = csa.dense_attn_workspace() if ws is None else ws
    csa.dense_attn(layer, r.batch, r.cu_rows, q, out, lse, ws, softcap=cap, slopes=slopes, spans=spans, **kw)
    return out, lse, ws


def assert_close(got, ref, what=""):
    out, lse, tol, ltol = ref
    n = out.shape[0]
    err = (got[0][:n].double() - out).abs() - tol
    assert not torch.isnan(err).any(), what
    assert float(err.max()) <= 0, "%s: out off by %.3g more than its tolerance" % (what, float(err.max()))
    empty = lse == -math.inf
    assert torch.equal(got[1][:n] == -math.inf, empty), what
    lerr = torch.where(empty, 0.0, (got[1][:n].double() - torch.where(empty, 0.0, lse)).abs() - ltol)
    assert float(lerr.max()) <= 0, "%s: lse off by %.3g more than its tolerance" % (what, float(lerr.max()))
    assert not got[0][:n][empty].any(), what


CASES = [  # heads, new rows, lengths, mask, cap, slopes
    (1, [1], [1], "causal", 0.0, False),
    (64, [1], [64], "causal", 0.0, False),
    (16, [1], [4096], "causal", 0.0, False),
    (64, [1, 1, 1], [65, 1, 640], "causal", 0.0, False),
    (128, [3, 0, 5], [3, 10, 200], "causal", 0.0, False),
    (24, [7, 1], [130, 3001], "causal", 30.0, True),
    (1, [200], [333], "causal", 0.0, True),
    (33, [63, 2, 0], [63, 129, 7], "all", 0.0, False),
    (96, [70], [1000], "window", 0.0, False),
    (40, [100, 0, 300], [100, 1, 301], "documents", 50.0, False),
    (64, [129], [400], "documents", 0.0, True),
    (127, [2], [63], "documents", 0.0, False),
    (32, [4, 4, 4, 4], [2000, 1999, 64, 4], "causal", 20.0, False),
    (64, [1] * 300, [64 + (i * 37) % 200 for i in range(300)], "causal", 0.0, False),
    (8, [0] * 50 + [9] + [0] * 50, [1] * 50 + [900] + [1] * 50, "causal", 0.0, False),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_formula(case):
    H, n, lens, mask, cap, biased = CASES[case]
    r = Run(n, lens, 100 + case, pad_rows=3)
    layer = random_layer(r.num_pages, 200 + case)
    q = queries(r.rows, H, 300 + case)
    spans = make_spans(r, mask, 400 + case)
    if spans is not None:
        spans = torch.cat([spans, spans.new_zeros((3, 2))])
    slopes = 2.0 ** (-8.0 * (torch.arange(H, device="cuda") + 1) / H) if biased else None
    got = attend(layer, r, q, spans, cap, slopes)
    assert csa.check_device_error(got[2])[0] == 0
    assert_close(got, reference(layer, r, q, spans, cap, slopes))
    assert (got[0][-3:] == 7.0).all() and (got[1][-3:] == 7.0).all()   # rows behind the last sequence
    again = attend(layer, r, q, spans, cap, slopes, ws=got[2])
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


def test_long_sequence_splits_over_the_gpu():
    """One row tile over every CTA, and a page count that divides unevenly."""
    r = Run([1, 2], [60001, 12345], 11)
    layer = random_layer(r.num_pages, 12)
    q = queries(3, 64, 13)
    assert_close(attend(layer, r, q), reference(layer, r, q, None, 0.0, None))


def test_maximum_jumps_in_late_tiles():
    """Each row's largest score comes last and outweighs all before it by far (O rescaled between tiles)."""
    r = Run([1], [1000], 14)
    layer = random_layer(r.num_pages, 15)
    q = queries(1, 64, 16)
    v = values64(layer, r.slots(0, np.arange(1000)))
    for h in range(64):
        q[0, h] += ((3 + h % 4) * v[999 - 13 * h]).bfloat16()
    assert_close(attend(layer, r, q), reference(layer, r, q, None, 0.0, None))


@pytest.mark.parametrize("biased", [False, True])
def test_maximum_grows_page_by_page(biased):
    """Every page outweighs those before it, whichever end the pages are taken from (a bias reverses their order): O is
    rescaled at each page."""
    r = Run([1, 3], [1500, 700], 43)
    layer = random_layer(r.num_pages, 44)
    q = queries(4, 64, 45)
    slopes = torch.full((64,), 1e-3, device="cuda") if biased else None
    at = 0
    for b, n in enumerate(r.n):
        v = values64(layer, r.slots(b, np.arange(r.lens[b])))
        top = v[3 if biased else -5]
        # entries grow along the way the pages are taken: scales double every other page, codes stay
        pages = (r.lens[b] + 63) // 64
        for k in range(pages):
            step = k if not biased else pages - 1 - k
            page = int(r.bt[b, k])
            layer.scales[page] = 0x08 + 8 * min(8, step // 2) + (step % 2) * 4
        v = values64(layer, r.slots(b, np.arange(r.lens[b])))
        q[at:at + n] = (4 * torch.sign(top)[None, None] * torch.rand((n, 64, 1), device="cuda")).bfloat16()
        at += n
    got = attend(layer, r, q, slopes=slopes)
    assert csa.check_device_error(got[2])[0] == 0
    assert_close(got, reference(layer, r, q, None, 0.0, slopes))


def test_scales_of_queries_in_one_tile():
    """Rows 80 binades apart share a row tile; zero rows give the plain average."""
    r = Run([4], [300], 17)
    layer = random_layer(r.num_pages, 18)
    q = queries(4, 16, 19)
    q[0] *= 2.0 ** -60
    q[1] *= 2.0 ** 4
    q[2] = 0
    assert_close(attend(layer, r, q), reference(layer, r, q, None, 0.0, None))


def test_garbage_in_hidden_places_stays_there():
    """NaN scales behind a sequence's end, in unmapped pages and in entries that a row does not see; rows
    of infinite or NaN q: only rows that see such an entry, or are such a row, are NaN."""
    r = Run([6], [200], 20)
    layer = random_layer(r.num_pages, 21)
    q = queries(6, 16, 22)
    spans = torch.tensor([[0, 150], [0, 101], [101, 200], [100, 200], [0, 100], [7, 7]], dtype=torch.int32, device="cuda")
    clean = reference(layer, r, q, spans, 0.0, None)
    used = set(r.slots(0, np.arange(200)).tolist())
    flat = layer.scales.view(-1, 32)
    for s in range(flat.shape[0]):
        if s not in used:
            flat[s] = 0x7F
    for bad in (0x7F, 0xFF):
        flat[int(r.slots(0, [100])[0]), 17] = bad
        got = attend(layer, r, q, spans)
        assert csa.check_device_error(got[2])[0] == 0
        sees = torch.tensor([True, True, False, True, False, False], device="cuda")
        assert torch.isnan(got[0][sees].float()).all() and torch.isnan(got[1][sees]).all()
        keep = (~sees).nonzero()[:, 0]
        assert_close([x[keep] for x in got[:2]], [x[keep] for x in clean])
    flat[int(r.slots(0, [100])[0]), 17] = 0x38
    clean = reference(layer, r, q, spans, 0.0, None)
    q[2, 3, 5], q[4, 15] = math.inf, math.nan
    got = attend(layer, r, q, spans)
    sick = torch.zeros((6, 16), dtype=torch.bool, device="cuda")
    sick[2, 3] = sick[4, 15] = True
    assert torch.isnan(got[0][sick].float()).all()
    keep = ~sick
    assert_close([x[keep][None] for x in got[:2]], [x[keep][None] for x in clean])


def test_bad_metadata_is_reported_and_skipped():
    for what in ("page", "long", "order", "too many"):
        r = Run([2, 2, 2], [200, 200, 200], 23)
        layer = random_layer(r.num_pages, 24)
        q = queries(6, 16, 25)
        ref = reference(layer, r, q, None, 0.0, None)
        skipped = [1]
        if what == "page":
            r.batch.block_table[1, 2] = -5             # its positions are left out; the rows are still written
        elif what == "long":
            r.batch.seq_len[1] = 201                   # past max_seq_len
        elif what == "order":
            r.cu_rows[1] = 5
            skipped = [0, 1, 2]
        else:
            r.cu_rows[3] = 7
            skipped = [0, 1, 2]
        got = attend(layer, r, q)
        assert csa.check_device_error(got[2])[0] == 5, what
        for b in range(3):
            rows = slice(2 * b, 2 * b + 2)
            if b not in skipped:
                assert_close([x[rows] for x in got[:2]], [x[rows] for x in ref], what)
            elif what != "page":
                assert (got[0][rows] == 7.0).all() and (got[1][rows] == 7.0).all(), what
        if what == "page":
            spans = torch.tensor([[0, 128], [0, 128]], dtype=torch.int32, device="cuda")
            short = Run([2], [200], 0)
            short.bt = r.bt[1:2]
            left = values64(layer, r.slots(1, np.r_[0:128, 192:200]))
            z = TAU * (q[2:4].double().reshape(32, 512) @ left.T)
            z[:16, 135] = -math.inf                    # the first row ends one position earlier
            assert (got[1][2:4].double().flatten() - torch.logsumexp(z, 1)).abs().max() < 1e-3
            assert spans is not None


def test_pools_past_32_bit_offsets():
    pool = 300_000
    r = Run([2], [300], 26, pool=pool)
    layer = random_layer(pool, 27)
    q = queries(2, 64, 28)
    assert int(r.bt[r.bt >= 0].min()) * 64 * 256 > 2 ** 32
    assert_close(attend(layer, r, q), reference(layer, r, q, None, 0.0, None))


def test_agrees_with_sparse_attention_over_every_block():
    """Every block selected and no window: the sparse decode attention computes the same thing."""
    L, H = 1000, 64
    r = Run([1, 1], [L, 777], 29)
    layer = random_layer(r.num_pages, 30)
    q = queries(2, H, 31)
    r.batch.swa_row.fill_(-1)
    nb = (L + 7) // 8
    blocks = torch.arange(nb, dtype=torch.int32, device="cuda").repeat(2, 1).contiguous()
    count = torch.tensor([nb, (777 + 7) // 8], dtype=torch.int32, device="cuda")
    out = torch.empty((2, H, 512), device="cuda")
    lse = torch.empty((2, H), device="cuda")
    ws = csa.workspace(2, H, L, nb)
    csa.sparse_decode_attn(layer, r.batch, q, TAU, blocks, count, out, lse, ws)
    got = attend(layer, r, q)
    assert (got[0].float() - out).abs().max() <= (2.0 ** -8 + 2e-3) * out.abs().max()
    assert (got[1] - lse).abs().max() <= 1e-3


def test_streams_graphs_and_two_calls_at_once():
    """Captured and replayed on new inputs; two calls overlap on two streams, each with its workspace."""
    runs = [Run([1, 1], [5000, 300], 32), Run([40], [900], 33)]
    layers = [random_layer(r.num_pages, 34 + i) for i, r in enumerate(runs)]
    qs = [queries(r.rows, 64, 36 + i) for i, r in enumerate(runs)]
    want = [attend(l, r, q)[:2] for l, r, q in zip(layers, runs, qs)]
    new = [queries(r.rows, 64, 38 + i) for i, r in enumerate(runs)]
    want_new = [attend(l, r, q)[:2] for l, r, q in zip(layers, runs, new)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    graphs, outs = [], []
    for i, r in enumerate(runs):
        ws = csa.dense_attn_workspace()
        out, lse = torch.zeros_like(want[i][0]), torch.zeros_like(want[i][1])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            csa.dense_attn(layers[i], r.batch, r.cu_rows, qs[i], out, lse, ws)
        graphs.append(g)
        outs.append((out, lse, ws))
    for k, w in enumerate((want, want_new)):
        for i in range(2):
            if k:
                qs[i].copy_(new[i])
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                for _ in range(5):
                    graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i][0], w[i][0]) and torch.equal(outs[i][1], w[i][1])
            assert csa.check_device_error(outs[i][2])[0] == 0


def test_append_attend_unpack_together():
    """A prompt written and attended in chunks, then a decoded token, equals one call over everything."""
    import oracle
    from fp4_compressed_sparse_kv_b200 import synth
    L, H = 333, 32
    rng = np.random.default_rng(40)
    lat = synth.bf16_bits(rng.standard_normal((L, 512)).astype(np.float32))
    key = synth.index_keys(rng, L)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).view(torch.bfloat16).cuda()
    whole = Run([L], [L], 41)
    layer, ws = csa.KVLayer(whole.num_pages, 1), csa.dense_attn_workspace()
    q = queries(L, H, 42)
    outs, at = [], 0
    for n in (200, 1, 131, 1):
        at += n
        seq_len = torch.tensor([at], dtype=torch.int32, device="cuda")
        batch = csa.Batch(seq_len, whole.batch.block_table, whole.batch.swa_row, L)
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        rows = slice(at - n, at)
        csa.kv_append_fp4(layer, batch, cu, dev(lat[rows]), dev(key[rows]), ws)
        out, lse = torch.empty((n, H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((n, H), device="cuda")
        csa.dense_attn(layer, batch, cu, q[rows].contiguous(), out, lse, ws)
        outs.append((out, lse))
    back = torch.empty((L, 512), dtype=torch.bfloat16, device="cuda")
    csa.kv_unpack_fp4(layer, whole.batch, whole.cu_rows, back, ws)
    assert csa.check_device_error(ws)[0] == 0
    ref = oracle.pack_tokens(lat, key)
    assert torch.equal(back.double(), torch.from_numpy(oracle.dequant_main(ref["codes"], ref["scales"])).double().cuda())
    got = [torch.cat([o[i] for o in outs]) for i in range(2)]
    assert_close(got, reference(layer, whole, q, None, 0.0, None))


def test_as_many_sequences_as_a_batch_holds():
    """16,384 sequences, most without a row: the division's tables fill the shared memory they are given."""
    B = 16384
    rng = np.random.default_rng(50)
    n = np.where(rng.random(B) < 0.05, 1, 0)
    n[[0, 7000, B - 1]] = [2, 40, 3]
    lens = np.where(n > 0, rng.integers(1, 100, B), 1) + n
    r = Run(n.tolist(), lens.tolist(), 51)
    layer = random_layer(r.num_pages, 52)
    q = queries(r.rows, 8, 53)
    got = attend(layer, r, q)
    assert csa.check_device_error(got[2])[0] == 0
    assert_close(got, reference(layer, r, q, None, 0.0, None))


@pytest.mark.parametrize("H,n,L", [(1, 700, 1000), (3, 500, 700), (128, 9, 9)])
def test_spans_of_many_tokens_in_one_row_tile(H, n, L):
    """Up to 128 tokens share a row tile; each has its own span, some see nothing, whole tiles among them."""
    r = Run([n], [L], 54 + H)
    layer = random_layer(r.num_pages, 55 + H)
    q = queries(n, H, 56 + H)
    rng = np.random.default_rng(57 + H)
    lo = rng.integers(-5, L, n)
    s = np.stack([lo, np.minimum(lo + rng.integers(0, 200, n), L + 3)], 1)
    s[n // 3:n // 3 + 260] = 11                              # two row tiles in a row that see nothing (one head)
    spans = torch.from_numpy(s.astype(np.int32)).cuda()
    got = attend(layer, r, q, spans, cap=5.0)
    assert csa.check_device_error(got[2])[0] == 0
    assert_close(got, reference(layer, r, q, spans, 5.0, None))


def test_non_finite_queries_under_a_cap():
    """The cap maps infinite scores to finite ones; a row of infinite q is NaN all the same, and only that row."""
    r = Run([4], [150], 58)
    layer = random_layer(r.num_pages, 59)
    layer.codes |= 0x11                                      # no zero among the entries' values
    q = queries(4, 16, 60)
    clean = reference(layer, r, q, None, 3.0, None)
    q[1, 5] = math.inf
    q[2, 0, 300] = -math.inf
    got = attend(layer, r, q, cap=3.0)
    sick = torch.zeros((4, 16), dtype=torch.bool, device="cuda")
    sick[1, 5] = sick[2, 0] = True
    assert torch.isnan(got[0][sick].float()).all() and torch.isnan(got[1][sick]).all()
    assert_close([x[~sick][None] for x in got[:2]], [x[~sick][None] for x in clean])


def test_other_streams_workspaces_and_orders():
    """The caller's stream argument; one workspace for calls of different sizes in turn, many times over."""
    runs = [Run([1], [3000], 61), Run([33, 0, 90], [400, 5, 90], 62), Run([1] * 20, [700] * 20, 63)]
    layers = [random_layer(r.num_pages, 64 + i) for i, r in enumerate(runs)]
    qs = [queries(r.rows, 40, 66 + i) for i, r in enumerate(runs)]
    want = [attend(l, r, q)[:2] for l, r, q in zip(layers, runs, qs)]
    torch.cuda.synchronize()
    side, ws = torch.cuda.Stream(), csa.dense_attn_workspace()
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for l, r, q in zip(layers, runs, qs):
            out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
            side.wait_stream(torch.cuda.current_stream())
            csa.dense_attn(l, r.batch, r.cu_rows, q, out, lse, ws, stream=side)
            outs.append((out, lse))
    side.synchronize()
    for i, (out, lse) in enumerate(outs):
        assert torch.equal(out, want[i % 3][0]) and torch.equal(lse, want[i % 3][1])
    assert csa.check_device_error(ws)[0] == 0


@pytest.mark.parametrize("width", [1, 2, 2500])
def test_scores_of_large_magnitude(width):
    """Slopes, or a scale, that put every visible score below -2^100: the largest score takes all of the weight, so out
    is that entry (its product with a power of two and the division by it are exact) and lse that score."""
    n, L, H = 5, 2600, 6
    r = Run([n], [L], 70)
    layer = random_layer(r.num_pages, 71)
    v = values64(layer, r.slots(0, np.arange(L)))
    pos = np.arange(L - n, L)
    hi = pos - np.array([0, 1, 5, 63, 64])                   # the row's own position is not among those it sees
    s = np.stack([hi - width, hi], 1)
    spans = torch.from_numpy(s.astype(np.int32)).cuda()
    slopes = 2.0 ** (101 + torch.arange(H, device="cuda").float())
    got = attend(layer, r, queries(n, H, 72), spans, slopes=slopes)
    nearest = torch.from_numpy(hi - 1).cuda()
    want = v[nearest][:, None].expand(n, H, 512)
    lse = -slopes.double()[None] * torch.from_numpy(pos - hi + 1).cuda()[:, None]
    assert torch.equal(got[0].double(), want)
    assert float(((got[1].double() - lse) / lse).abs().max()) <= 2.0 ** -20     # the scores vanish beside the bias
    # the same by the scale: q opposite to the entry, which is at least 2^100 of the score away from zero
    q = -(v[nearest][:, None] * 2.0 ** torch.arange(H, device="cuda")[:, None]).bfloat16()
    one = torch.stack([nearest, nearest + 1], 1).int()
    got = attend(layer, r, q, one, sm_scale=1e30)
    assert torch.equal(got[0].double(), want)
    lse = 1e30 * (q.double() * v[nearest][:, None]).sum(-1)
    assert float(lse.max()) < -1e32
    assert float(((got[1].double() - lse) / lse).abs().max()) <= 2.0 ** -15     # terms of one sign: 512 roundings
    assert csa.check_device_error(got[2])[0] == 0
