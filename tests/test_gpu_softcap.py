"""Capped scores over the whole range of caps against the formula in 64 bits.

The tolerance of a score holds no term of the cap.  With x = s / cap:
  - |x| < 0.25: s (1 + x^2 P(x^2)), the series of tanh to x^7: the next term is 62/2835 x^8 <= 2^-21.5; x^2 P is at
    most 0.021, so its own roundings are below 2^-26, and the last operation's is 2^-24;
  - otherwise 1 - 2 / (1 + e^2x): e^2x to 2^-22 and the rounding of its argument, the reciprocal and 1 + e^2x to 2^-23
    and 2^-24, at most 1.55 * 2^-22 of 1 in all where |tanh x| >= 0.244;
so a capped score z is within 2^-19 |z|, two more roundings of s / cap and the cap included.  The score before the cap
is within 2^-15 A (512 roundings of binary32, A = sm_scale sum |q||v|), which the cap does not enlarge.  The rest
(P in fp16, sums, exp2, bf16) is as for uncapped scores."""
import math

import numpy as np
import pytest
import torch

from fp4_compressed_sparse_kv_b200 import csa
from runs_helpers import Run, random_layer, values64
from test_gpu_dense_attn import assert_close, attend, queries

pytestmark = pytest.mark.gpu


def capped_reference(layer, r, q, cap, slopes, tau):
    """(out, lse, tolerance of out, tolerance of lse) of the rows of a single sequence, causal, in float64."""
    (n,), (L,), H = r.n, r.lens, q.shape[1]
    v = values64(layer, r.slots(0, np.arange(L)))
    qq = q.double().reshape(n * H, 512)
    p, j = torch.arange(L - n, L, device="cuda"), torch.arange(L, device="cuda")
    seen = (j <= p[:, None]).repeat_interleave(H, 0)
    s = tau * (qq @ v.T)
    z = cap * torch.tanh(s / cap)
    a = torch.where(seen, tau * (qq.abs() @ v.abs().T), 0.0).amax(1)
    dz = 2.0 ** -15 * a + 2.0 ** -19 * torch.where(seen, z.abs(), 0.0).amax(1)
    if slopes is not None:
        z = z - (slopes.double()[None, :, None] * (p[:, None] - j).abs()[:, None, :]).reshape(n * H, L)
    dz = dz + 2.0 ** -21 * torch.where(seen, z.abs(), 0.0).amax(1)
    z = torch.where(seen, z, -math.inf)
    lse = torch.logsumexp(z, 1)
    w = torch.exp(z - lse[:, None])
    out, W = w @ v, w @ v.abs()
    rel = 2 * dz + 2.0 ** -11 + 2 * L * 2.0 ** -24 + 2.0 ** -20
    tol = 2.0 ** -8 * out.abs() + rel[:, None] * W * (1 + 2.0 ** -8) + L * 2.0 ** -32 * v.abs().max()
    ltol = dz + L * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -21 * lse.abs()
    shape = lambda x: x.reshape(n, H, -1)
    return shape(out), shape(lse)[..., 0], shape(tol), shape(ltol)[..., 0]


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("cap", [1e-20, 1e-3, 0.3, 1.0, 4.0, 50.0, 1e3, 1e4, 1e6, 1e8, 1e20, 1e30])
def test_cap_of_any_size(cap, biased):
    n, L, H = 5, 333, 24
    r = Run([n], [L], 110)
    layer = random_layer(r.num_pages, 111)
    q = queries(n, H, 112)
    q[1] *= 2.0 ** -6                                     # scores far below the cap
    slopes = 2.0 ** (-8.0 * (torch.arange(H, device="cuda") + 1) / H) if biased else None
    got = attend(layer, r, q, cap=cap, slopes=slopes)
    assert csa.check_device_error(got[2])[0] == 0
    assert_close(got, capped_reference(layer, r, q, cap, slopes, 1.0 / math.sqrt(512)))


def test_scores_on_both_sides_of_the_forms():
    """One entry per row (lse is its score): scores of 2^-20 to 2^6 caps, the crossing between the two forms among them."""
    H, n = 128, 4
    r = Run([n], [n], 113)
    layer = csa.KVLayer(r.num_pages, 1)
    layer.codes.fill_(0x22)                               # every value 1
    layer.scales.fill_(0x38)
    spans = torch.stack([torch.arange(n), torch.arange(n) + 1], 1).int().cuda()
    x = 2.0 ** torch.linspace(-20, 6, H * n // 2, dtype=torch.float64)
    x[: H // 2] = torch.linspace(0.2, 0.3, H // 2, dtype=torch.float64)
    x = torch.cat([x, -x]).reshape(n, H).cuda()
    q = torch.zeros((n, H, 512), dtype=torch.bfloat16, device="cuda")
    for cap in (1e-3, 1.0, 30.0, 1e7):
        q[:, :, 5] = (x * cap).bfloat16()
        want = cap * torch.tanh(q[:, :, 5].double() / cap)
        got = attend(layer, r, q, spans, cap=cap, sm_scale=1.0)
        assert csa.check_device_error(got[2])[0] == 0
        # the product is exact; to base 2 and back: 5 roundings of |z|; lse = (m - 7) ln 2 + log(2^7): a half unit of
        # 4.85 for the product, one for the logarithm, 2^-22 for exp2: below 2^-19
        err = (got[1].double() - want).abs() - (2.0 ** -19 + 2.0 ** -21) * want.abs() - 2.0 ** -19
        assert float(err.max()) <= 0, cap
