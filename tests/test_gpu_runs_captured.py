"""The run operators captured where what precedes them is no kernel of theirs: copies and fills, and a join of two
streams that append to two layers."""
import numpy as np
import pytest
import torch

from fp4_compressed_sparse_kv_b200 import csa
from runs_helpers import Run
from test_gpu_dense_attn import assert_close, queries, reference

pytestmark = pytest.mark.gpu


def test_captured_behind_copies_and_a_join():
    n, lens, H = [40, 1], [64, 200], 32
    r = Run(n, lens, 150)
    rows = r.rows
    layers = [csa.KVLayer(r.num_pages, 2) for _ in range(2)]
    ws = [csa.dense_attn_workspace() for _ in range(2)]
    host = torch.empty((rows, 512), dtype=torch.bfloat16).pin_memory()
    lat = torch.zeros((rows, 512), dtype=torch.bfloat16, device="cuda")
    key = torch.zeros((rows, 128), dtype=torch.bfloat16, device="cuda")
    q = queries(rows, H, 151)
    outs = [(torch.zeros_like(q), torch.zeros((rows, H), device="cuda")) for _ in range(2)]
    backs = [torch.zeros_like(lat) for _ in range(2)]
    side, main = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        lat.copy_(host, non_blocking=True)                     # a copy, then the append
        side.wait_stream(main)
        csa.kv_append_fp4(layers[0], r.batch, r.cu_rows, lat, key, ws[0])
        with torch.cuda.stream(side):
            csa.kv_append_fp4(layers[1], r.batch, r.cu_rows, lat, key, ws[1])
        main.wait_stream(side)                                 # the join, then an attention over the other stream's layer
        csa.dense_attn(layers[1], r.batch, r.cu_rows, q, *outs[1], ws[1])
        backs[0].zero_()                                       # a fill, then the read-back
        csa.kv_unpack_fp4(layers[0], r.batch, r.cu_rows, backs[0], ws[0])
        csa.kv_unpack_fp4(layers[1], r.batch, r.cu_rows, backs[1], ws[1])
        csa.dense_attn(layers[0], r.batch, r.cu_rows, q, *outs[0], ws[0])
    rng = np.random.default_rng(152)
    for _ in range(3):
        host.copy_(torch.from_numpy(rng.standard_normal((rows, 512)).astype(np.float32)))
        with torch.cuda.stream(main):
            g.replay()
        torch.cuda.synchronize()
        twin = csa.KVLayer(r.num_pages, 2)
        csa.kv_append_fp4(twin, r.batch, r.cu_rows, host.cuda(), key, ws[0])
        want = torch.zeros_like(lat)
        csa.kv_unpack_fp4(twin, r.batch, r.cu_rows, want, ws[0])
        ref = reference(twin, r, q, None, 0.0, None)
        for i in range(2):
            assert torch.equal(backs[i], want) and torch.equal(layers[i].codes, twin.codes)
            assert_close(outs[i], ref)
            assert csa.check_device_error(ws[i])[0] == 0
