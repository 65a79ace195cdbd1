"""Dense attention where the block table has bad pages (every position of one is left out, in out and in lse), and runs
whose rows do not begin at the first row of the arrays."""
import math

import numpy as np
import pytest
import torch

from fp4_compressed_sparse_kv_b200 import csa
from runs_helpers import Run, random_layer, values64
from test_gpu_dense_attn import TAU, assert_close, attend, queries, reference

pytestmark = pytest.mark.gpu


def reference_of(v, q, pos, seen, slopes):
    """(out, lse, tolerances) of queries q [n, H, 512] at positions pos over entries v where seen [n, L], in float64; the
    tolerance is test_gpu_dense_attn's, with the entries that are seen."""
    n, H, _ = q.shape
    L = v.shape[0]
    qq = q.double().reshape(n * H, 512)
    s = seen.repeat_interleave(H, 0)
    z, a = TAU * (qq @ v.T), TAU * (qq.abs() @ v.abs().T)
    if slopes is not None:
        far = (pos[:, None] - torch.arange(L, device="cuda")).abs()
        z = z - (slopes.double()[None, :, None] * far[:, None, :]).reshape(n * H, L)
    zmax = torch.where(s, z.abs(), 0.0).amax(1)
    dz = 2.0 ** -15 * torch.where(s, a, 0.0).amax(1) + 2.0 ** -21 * zmax
    z = torch.where(s, z, -math.inf)
    lse = torch.logsumexp(z, 1)
    w = torch.where(s, torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[:, None]), 0.0)
    out, W = w @ v, w @ v.abs()
    rel = 2 * dz + 2.0 ** -11 + 2 * L * 2.0 ** -24 + 2.0 ** -20
    tol = 2.0 ** -8 * out.abs() + rel[:, None] * W * (1 + 2.0 ** -8) + L * 2.0 ** -32 * v.abs().max()
    ltol = dz + L * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -21 * torch.where(lse == -math.inf, 0.0, lse).abs()
    shape = lambda x: x.reshape(n, H, -1)
    return shape(out), shape(lse)[..., 0], shape(tol), shape(ltol)[..., 0]


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("bad", [[0], [2], [10], [0, 1, 2], [9, 10], [1, 3, 5, 7, 9], list(range(11))])
@pytest.mark.parametrize("H", [16, 128])
def test_positions_of_bad_pages_are_left_out(H, bad, biased):
    n, L = 3, 700
    r = Run([2, n], [90, L], 140)
    layer = random_layer(r.num_pages, 141)
    v = values64(layer, r.slots(1, np.arange(L)))
    q = queries(r.rows, H, 142)
    slopes = 2.0 ** (-8.0 * (torch.arange(H, device="cuda") + 1) / H) if biased else None
    first = [x[:2] for x in reference(layer, r, q, None, 0.0, slopes)]
    for i, k in enumerate(bad):
        r.batch.block_table[1, k] = (-5, r.num_pages, 2 ** 31 - 1)[i % 3]
    pos, j = torch.arange(L - n, L, device="cuda"), torch.arange(L, device="cuda")
    left = torch.tensor([k not in bad for k in range((L + 63) // 64)], device="cuda")[j // 64]
    ref = reference_of(v, q[2:], pos, (j <= pos[:, None]) & left, slopes)
    got = attend(layer, r, q, slopes=slopes)
    assert csa.check_device_error(got[2])[0] == 5
    assert_close([x[2:] for x in got[:2]], ref)
    assert_close([x[:2] for x in got[:2]], first)


@pytest.mark.parametrize("before", [1, 37, 500])
def test_rows_before_the_first_sequence(before):
    """cu_rows[0] > 0: append, read-back and attention leave the rows before it alone, as those behind the last."""
    n, lens, H, behind = [40, 0, 3], [70, 9, 300], 24, 5
    r = Run(n, lens, 143)
    layer, ws = random_layer(r.num_pages, 144, num_rows=3), csa.dense_attn_workspace()
    rows = before + sum(n) + behind
    cu = torch.from_numpy(r.cu + np.int32(before)).cuda()
    inner = slice(before, before + sum(n))
    g = torch.Generator(device="cuda").manual_seed(145)
    lat = torch.randn((rows, 512), generator=g, device="cuda").bfloat16()
    key = torch.randn((rows, 128), generator=g, device="cuda").bfloat16()
    twin = csa.KVLayer(r.num_pages, 3)
    for name in ("codes", "scales", "keys", "swa", "swa_scale"):
        getattr(twin, name).copy_(getattr(layer, name))
    csa.kv_append_fp4(layer, r.batch, cu, lat, key, ws)
    csa.kv_append_fp4(twin, r.batch, r.cu_rows, lat[inner].contiguous(), key[inner].contiguous(), ws)
    for name in ("codes", "scales", "keys", "swa", "swa_scale"):
        assert torch.equal(getattr(layer, name), getattr(twin, name)), name
    back = torch.full((rows, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    csa.kv_unpack_fp4(layer, r.batch, cu, back, ws)
    seq, pos = r.positions()
    slot = np.array([r.slots(s, p) for s, p in zip(seq, pos)])
    assert torch.equal(back[inner].double(), values64(layer, slot))
    q = queries(rows, H, 146)
    out = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 3.0, device="cuda")
    csa.dense_attn(layer, r.batch, cu, q, out, lse, ws)
    assert csa.check_device_error(ws)[0] == 0
    assert_close((out[inner], lse[inner]), reference(layer, r, q[inner], None, 0.0, None))
    for x in (back, out, lse):
        assert (x[:before] == 3.0).all() and (x[-behind:] == 3.0).all()
