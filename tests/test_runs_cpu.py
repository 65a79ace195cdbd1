"""Host checks of the ragged-run entry points, without a GPU: they return before any launch."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from fp4_compressed_sparse_kv_b200 import build, csa
    build.build()
    return csa.lib()


def handles():
    from fp4_compressed_sparse_kv_b200 import csa
    lay = csa.KVLayerC(0x1000, 0x1000, 0x1000, 0x1000, 0x1000, 64, 1)
    bat = csa.BatchC(2, 0x1000, 0x1000, 64, 0x1000, 4096)
    return ctypes.byref(lay), ctypes.byref(bat), lay, bat


OK, ODD, BIG = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008), 1 << 40


def test_no_rows_is_a_no_op_and_bad_arguments_are_refused(lib):
    l, b, lay, bat = handles()
    calls = {
        "append": lambda l=l, b=b, cu=OK, rows=4, x=OK, key=OK, w=None, rope=None, npos=0, ws=OK, wsb=256:
            lib.csa_kv_append_fp4(l, b, cu, rows, x, key, w, rope, npos, ws, wsb, None),
        "unpack": lambda l=l, b=b, cu=OK, rows=4, x=OK, ws=OK, wsb=256: lib.csa_kv_unpack_fp4(l, b, cu, rows, x, ws, wsb, None),
        "attend": lambda l=l, b=b, cu=OK, rows=4, x=OK, H=64, tau=0.1, cap=0.0, slopes=None, spans=None, out=OK, lse=OK, ws=OK,
        wsb=BIG: lib.csa_dense_attn(l, b, cu, rows, x, H, tau, cap, slopes, spans, out, lse, ws, wsb, None),
    }
    for name, f in calls.items():
        assert f(l=None, b=None, cu=None, rows=0, x=None, ws=None) == 0, name
        for bad in (dict(rows=-1), dict(rows=(1 << 24) + 1), dict(l=None), dict(b=None), dict(cu=None), dict(cu=ODD),
                    dict(x=None), dict(x=ODD), dict(ws=None), dict(ws=ODD)):
            assert f(**bad) == 1, (name, bad)
        assert f(wsb=255) == 3, name
    f = calls["append"]
    for bad in (dict(key=None), dict(key=ODD), dict(w=ODD), dict(rope=ODD, npos=9), dict(rope=OK, npos=0)):
        assert f(**bad) == 1, bad
    f = calls["attend"]
    for bad in (dict(out=None), dict(lse=ODD), dict(slopes=ODD), dict(spans=ODD), dict(tau=0.0), dict(tau=-1.0),
                dict(tau=float("nan")), dict(tau=float("inf")), dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf"))):
        assert f(**bad) == 1, bad
    for H in (0, 129, -3):
        assert f(H=H) == 2, H
    assert f(wsb=lib.csa_dense_attn_workspace_bytes() - 1) == 3
    bat.max_pages = 63                                       # fewer than max_seq_len needs
    for name, f in calls.items():
        assert f() == 1, name


def test_binding_checks_shapes_and_types():
    from fp4_compressed_sparse_kv_b200 import csa
    layer = csa.KVLayer(2, 1, device="cpu")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    batch = csa.Batch(i32(3), i32(0).view(1, 1), i32(0), 64)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8)
    cu = i32(0, 3)
    for a in (dict(cu_rows=i32(0, 1, 3)), dict(cu_rows=cu.long()), dict(latent=bf(3, 511)), dict(latent=bf(3, 512).float()),
              dict(idx_key=bf(2, 128)), dict(norm_weight=torch.zeros(511)), dict(norm_weight=bf(512)),
              dict(rope_table=torch.zeros(9, 64)), dict(rope_table=torch.zeros(9, 32, 2, dtype=torch.float64))):
        with pytest.raises(ValueError):
            csa.kv_append_fp4(**{**dict(layer=layer, batch=batch, cu_rows=cu, latent=bf(3, 512), idx_key=bf(3, 128), ws=ws), **a})
    with pytest.raises(ValueError):
        csa.kv_unpack_fp4(layer, batch, cu, bf(3, 512).float(), ws)
    with pytest.raises(ValueError):                          # right shapes, but not on a GPU
        csa.kv_unpack_fp4(layer, batch, cu, bf(3, 512), ws)
    good = dict(layer=layer, batch=batch, cu_rows=cu, q=bf(3, 8, 512), out=bf(3, 8, 512), lse=torch.zeros(3, 8), ws=ws)
    for a in (dict(q=bf(3, 8, 512).half()), dict(out=bf(3, 9, 512)), dict(out=torch.zeros(3, 8, 512)), dict(lse=bf(3, 8)),
              dict(lse=torch.zeros(3, 9)), dict(slopes=torch.zeros(7)), dict(spans=torch.zeros(3, 2)),
              dict(spans=torch.zeros(2, 2, dtype=torch.int32)), dict()):
        with pytest.raises(ValueError):
            csa.dense_attn(**{**good, **a})
