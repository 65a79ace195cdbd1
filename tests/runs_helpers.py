"""Ragged runs for the tests: cu_rows, lengths, scattered pages, and random FP4 entries with their values in
64 bits."""
import numpy as np
import torch

from fp4_compressed_sparse_kv_b200 import csa

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


class Run:
    """Lengths of a run on the device: n[b] new rows of seq_len[b] positions, pages scattered over a pool
    that has `spare` more pages (the last ones when top is set)."""

    def __init__(self, n, lens, seed, spare=3, pad_rows=0, pool=None):
        rng = np.random.default_rng(seed)
        self.n, self.lens, self.B = list(n), list(lens), len(n)
        self.rows = sum(n) + pad_rows
        self.cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        need = [(x + 63) // 64 for x in lens]
        total = sum(need) + spare
        ids = rng.permutation(total) if pool is None else pool - 1 - rng.permutation(total)
        self.num_pages = total if pool is None else pool
        self.max_pages = max(need)
        self.bt = np.full((self.B, self.max_pages), -1, np.int32)
        at = 0
        for b, k in enumerate(need):
            self.bt[b, :k] = ids[at:at + k]
            at += k
        self.cu_rows = torch.from_numpy(self.cu).cuda()
        self.batch = csa.Batch(torch.tensor(self.lens, dtype=torch.int32).cuda(), torch.from_numpy(self.bt).cuda(),
                               torch.arange(self.B, dtype=torch.int32).cuda(), max(lens))

    def positions(self):
        """(sequence, position) of every row that belongs to a sequence."""
        seq = np.repeat(np.arange(self.B), self.n)
        pos = np.concatenate([np.arange(L - k, L) for k, L in zip(self.n, self.lens)] or [[]]).astype(np.int64)
        return seq, pos

    def slots(self, b, pos):
        return self.bt[b, np.asarray(pos) // 64].astype(np.int64) * 64 + np.asarray(pos) % 64


def random_layer(num_pages, seed, num_rows=1):
    """A layer of random codes and scales between 1/16 and 2 (some zero, some subnormal)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    layer = csa.KVLayer(num_pages, num_rows)
    layer.codes.random_(0, 256, generator=g)
    layer.scales.random_(0x18, 0x41, generator=g)
    odd = torch.rand(layer.scales.shape, generator=g, device="cuda") < 0.02
    layer.scales[odd] = torch.randint(0, 8, (int(odd.sum()),), generator=g, device="cuda", dtype=torch.uint8)
    return layer


def values64(layer, slots):
    """float64 values [len(slots), 512] of cache entries."""
    s = torch.as_tensor(slots, device=layer.codes.device)
    c = layer.codes.view(-1, 256)[s].int()
    lut = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64, device=c.device)
    v = torch.stack([lut[c % 16], lut[c // 16]], -1).flatten(1)
    return v * layer.scales.view(-1, 32)[s].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
