"""q of the sparse attention written by a kernel that releases its dependents early (a long read-back, whose last rows
are q), with one short kernel of the library between the two: the attention may begin early, but not before q is there."""
import math

import numpy as np
import pytest
import torch

from fp4_compressed_sparse_kv_b200 import csa
from runs_helpers import Run, random_layer

pytestmark = pytest.mark.gpu

B, H, LONG = 4, 64, 60000


@pytest.mark.parametrize("between", ["append", "unpack", "reuse", "topk", "dense"])
def test_q_from_an_early_releasing_kernel_two_launches_before(between):
    lens = [700, 64, 513, 129]
    r, long = Run([1] * B, lens, 120), Run([LONG], [LONG], 121)
    layer, values = random_layer(r.num_pages, 122, num_rows=B), random_layer(long.num_pages, 123)
    values.scales.clamp_(max=0x30)
    nb = max((L + 7) // 8 for L in lens)
    g = torch.Generator(device="cuda").manual_seed(124)
    cap = nb
    blocks = torch.arange(nb, dtype=torch.int32, device="cuda").repeat(B, 1).contiguous()
    count = torch.tensor([(L + 7) // 8 for L in lens], dtype=torch.int32, device="cuda")
    scores = torch.randn((B, nb), generator=g, device="cuda")
    r.batch.swa_row.fill_(-1)
    ws, hws = csa.workspace(B, H, max(lens), cap), csa.dense_attn_workspace()
    lat = torch.randn((B, 512), generator=g, device="cuda").bfloat16()
    key = torch.randn((B, 128), generator=g, device="cuda").bfloat16()
    small = torch.empty((B, 512), dtype=torch.bfloat16, device="cuda")
    got_blocks, got_count = torch.zeros_like(blocks), torch.zeros_like(count)
    dq = torch.randn((B, 16, 512), generator=g, device="cuda").bfloat16()
    dout, dlse = torch.empty_like(dq), torch.empty((B, 16), device="cuda")
    table = torch.empty((LONG, 512), dtype=torch.bfloat16, device="cuda")
    q = table[LONG - B * H:].view(B, H, 512)

    def middle():
        if between == "append":
            csa.kv_append_fp4(layer, r.batch, r.cu_rows, lat, key, hws)
        elif between == "unpack":
            csa.kv_unpack_fp4(layer, r.batch, r.cu_rows, small, hws)
        elif between == "reuse":
            csa.index_reuse(blocks, count, got_blocks, got_count, hws)
        elif between == "topk":
            csa.topk_blocks(r.batch, scores, cap, got_blocks, got_count, hws)
        else:
            csa.dense_attn(layer, r.batch, r.cu_rows, dq, dout, dlse, hws)

    def attend():
        out, lse = torch.empty((B, H, 512), device="cuda"), torch.empty((B, H), device="cuda")
        csa.sparse_decode_attn(layer, r.batch, q, 1.0 / math.sqrt(512), blocks, count, out, lse, ws)
        return out, lse

    csa.kv_unpack_fp4(values, long.batch, long.cu_rows, table, hws)
    torch.cuda.synchronize()
    middle()
    torch.cuda.synchronize()
    want = attend()
    torch.cuda.synchronize()
    assert np.isfinite(want[1].cpu().numpy()).all()
    for _ in range(10):
        table.fill_(1.0)
        torch.cuda.synchronize()
        csa.kv_unpack_fp4(values, long.batch, long.cu_rows, table, hws)
        middle()
        got = attend()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert csa.check_device_error(ws)[0] == 0 and csa.check_device_error(hws)[0] == 0
