"""A NaN or an infinity among the channels of a group: the NaN's code is what the conversion gives for a NaN (the largest
magnitude, 6), infinities saturate, and the group's other channels are packed as without it.  The same by slots and by
position."""
import numpy as np
import pytest
import torch

from fp4_compressed_sparse_kv_b200 import csa, synth
from runs_helpers import Run

pytestmark = pytest.mark.gpu

CODE_OF_MAX = 7


def codes_of(layer, slot):
    c = layer.codes.view(-1, 256)[torch.from_numpy(slot).cuda()].cpu().numpy()
    return np.stack([c & 15, c >> 4], -1).reshape(c.shape[0], 512)


@pytest.mark.parametrize("by_position", [False, True])
@pytest.mark.parametrize("rows", [5, 5000])
def test_non_finite_channels(rows, by_position):
    rng = np.random.default_rng(130)
    r = Run([rows], [rows], 131)
    lat = synth.bf16_bits(rng.standard_normal((rows, 512)).astype(np.float32))
    lat[:, ::16] = 0x3F80                                    # no group of zeros alone
    key = synth.index_keys(rng, rows)
    where = rng.integers(0, 512, rows)
    at = (np.arange(rows), where)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).view(torch.bfloat16).cuda()
    slot = r.slots(0, np.arange(rows))
    ws = torch.empty(csa.HEADER_BYTES, dtype=torch.uint8, device="cuda")
    csa.workspace_init(ws)
    none = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    r.batch.swa_row.fill_(-1)

    def pack(x):
        layer = csa.KVLayer(r.num_pages, 1)
        if by_position:
            csa.kv_append_fp4(layer, r.batch, r.cu_rows, dev(x), dev(key), ws)
        else:
            csa.kv_pack_fp4(layer, dev(x), dev(key), torch.from_numpy(slot).cuda(), none, ws)
        assert csa.check_device_error(ws)[0] == 0
        return codes_of(layer, slot), layer.scales.view(-1, 32)[torch.from_numpy(slot).cuda()].cpu().numpy()

    lat[at] = 0                                              # a group's maximum passes over its NaN
    clean, clean_scales = pack(lat)
    for bits in (0x7FC0, 0xFFC0, 0x7F81):
        x = lat.copy()
        x[at] = bits
        codes, scales = pack(x)
        assert np.array_equal(scales, clean_scales), hex(bits)
        assert (codes[at] == CODE_OF_MAX).all(), hex(bits)
        codes[at] = clean[at]
        assert np.array_equal(codes, clean), hex(bits)
    for bits, want in ((0x7F80, CODE_OF_MAX), (0xFF80, 8 + CODE_OF_MAX)):
        x = lat.copy()
        x[at] = bits
        codes, scales = pack(x)
        assert (codes[at] == want).all() and (scales[np.arange(rows), where // 16] == 0x7E).all(), hex(bits)
