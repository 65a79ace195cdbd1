"""Row tiles one after the other in one cluster's share of the dense attention: a full row tile, many sequences without
a row, then a row tile of few rows and pages, so that one CTA of a cluster can be at the end of the second while the
other still stores the first."""
import pytest
import torch

from fp4_compressed_sparse_kv_b200 import csa
from runs_helpers import Run, random_layer
from test_gpu_dense_attn import assert_close, attend, queries, reference

pytestmark = pytest.mark.gpu

CLUSTERS = 74


@pytest.mark.parametrize("tokens,length", [(1, 60), (2, 64), (4, 100), (6, 128)])
def test_few_rows_behind_a_full_row_tile(tokens, length):
    """Each cluster's share is 8 tokens of 16 heads (one whole row tile), 200 sequences without a row, and `tokens` more
    tokens on one or two pages: quarters of the second row tile have no rows, and must not touch what the first needs."""
    H, empty = 16, 200
    r = Run(([8] + [0] * empty + [tokens]) * CLUSTERS, ([60] + [1] * empty + [length]) * CLUSTERS, 90)
    layer = random_layer(r.num_pages, 91)
    q = queries(r.rows, H, 92)
    ref = reference(layer, r, q, None, 0.0, None)
    ws = csa.dense_attn_workspace()
    first = None
    for _ in range(20):
        got = attend(layer, r, q, ws=ws)
        if first is None:
            assert_close(got, ref)
            first = got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    assert csa.check_device_error(ws)[0] == 0
