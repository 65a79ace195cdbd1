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


def test_pack_quotients_round_as_the_divisions_do():
    """The pack's quotients (a product with the rounded reciprocal, then 11 significant bits, half up) land on the same
    side of every border of E2M1 and E4M3 as the binary32 divisions x / s and amax / 6: every bf16 value, every scale."""
    import numpy as np
    x = (np.arange(0x7F82, dtype=np.uint32) << 16).view(np.float32)          # 0 .. infinity, one NaN

    def near(a, inv):
        with np.errstate(over="ignore", invalid="ignore"):
            q = (a * inv).astype(np.float32)
        return ((q.view(np.uint32) + np.uint32(0x1000)) & np.uint32(0xFFFFE000)).view(np.float32)

    def nearest(y, grid):                                                    # index of the nearest, even index on a tie
        mid = ((grid[1:].astype(np.float64) + grid[:-1]) / 2).astype(np.float32)
        lo, hi = np.searchsorted(mid, y, side="left"), np.searchsorted(mid, y, side="right")
        return np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))

    e4m3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    e2m1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float32)
    six = np.float32(6)
    with np.errstate(over="ignore"):
        assert np.array_equal(nearest(near(x[:-1], np.float32(1) / six), e4m3), nearest(x[:-1] / six, e4m3))
        for s in e4m3[1:]:
            inv = np.float32(1) / s
            y, z = near(x, inv), x / s
            assert np.array_equal(nearest(y[:-1], e2m1), nearest(z[:-1], e2m1)), s
            assert np.isnan(y[-1]) and np.isnan(z[-1])


def test_softcap_has_a_range(lib):
    l, b, lay, bat = handles()
    f = lambda cap, rows: lib.csa_dense_attn(l, b, OK, rows, OK, 64, 0.1, cap, None, None, OK, OK, OK, BIG, None)
    for cap in (1e-21, -1e-21, 1e31):
        assert f(cap, 4) == 1, cap
        assert f(cap, 0) == 0, cap                           # no rows: nothing is looked at


def test_arrays_of_a_run_are_on_the_current_device(monkeypatch):
    """Tensors of another device than the current one are refused before anything is launched (devices faked)."""
    from fp4_compressed_sparse_kv_b200 import csa

    class On:
        def __init__(self, device):
            self.device_index = device

        def get_device(self):
            return self.device_index

    monkeypatch.setattr(csa.torch, "Tensor", On)
    monkeypatch.setattr(csa.torch.cuda, "current_device", lambda: 0)
    assert csa._run_device(On(0), "ws") == 0
    with pytest.raises(ValueError, match="not the current one"):
        csa._run_device(On(1), "ws")
    monkeypatch.setattr(csa, "_ptr", lambda t, name: 1)
    with pytest.raises(ValueError, match="not on the current device"):
        csa._run_ptr(On(1), "latent", 0)
    assert csa._run_ptr(None, "slopes", 0) == 0


def test_binding_of_append_and_unpack_refuses_before_the_library_is_called():
    """The extension's own checks: what is no tensor, a workspace on the CPU, lengths that do not fit, missing attributes,
    a wrong number of arguments."""
    from fp4_compressed_sparse_kv_b200 import csa
    mod = csa._runs()
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    layer = csa.KVLayer(2, 1, device="cpu")
    batch = csa.Batch(torch.zeros(1, dtype=torch.int32), torch.zeros((1, 2), dtype=torch.int32),
                      torch.zeros(1, dtype=torch.int32), 128)
    cu, ws = torch.zeros(2, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    good = dict(layer=layer, batch=batch, cu_rows=cu, latent=bf(3, 512), idx_key=bf(3, 128), ws=ws)
    for a in (dict(latent=[1.0]), dict(idx_key=None), dict(cu_rows=(0, 3)), dict(ws=b"ws"), dict(norm_weight=1.0)):
        with pytest.raises(TypeError, match="torch tensor"):
            csa.kv_append_fp4(**{**good, **a})
    with pytest.raises(ValueError, match="ws must be a CUDA tensor"):
        csa.kv_append_fp4(**good)
    with pytest.raises(ValueError, match=r"idx_key must be torch.bfloat16 of shape \[3, 128\]"):
        csa.kv_append_fp4(**{**good, "idx_key": bf(128, 3)})
    with pytest.raises(ValueError):
        csa.kv_unpack_fp4(layer, batch, cu, torch.tensor(0.0).bfloat16(), ws)
    batch.B = 2 ** 40
    with pytest.raises(OverflowError):
        csa.kv_append_fp4(**good)
    del batch.B
    with pytest.raises(AttributeError):
        csa.kv_append_fp4(**good)
    for f, n in ((mod.kv_append_fp4, 8), (mod.kv_unpack_fp4, 7), (mod.bind, 1)):
        with pytest.raises(TypeError):
            f(*[None] * n)
    with pytest.raises(ValueError):
        mod.bind(0, 0)
