"""Shared by the key/value cache tests: batches of sequences with their pages, a
numpy mirror of the cache, and bfloat16 inputs as keys and values come."""
import numpy as np
import torch

from oracle import kv, nf4


class Case:
    """Sequences with n new rows each at the end of kv_len cached tokens; pages in
    random order; `pad` rows behind the last sequence."""

    def __init__(self, n, kv_len, page_size=16, pad=0, spare=2, seed=0, max_pages=None):
        rng = np.random.default_rng(seed)
        self.n, self.kv_len, self.page_size, self.pad = list(n), list(kv_len), page_size, pad
        per = [-(-k // page_size) for k in kv_len]
        self.num_pages = sum(per) + spare
        order = rng.permutation(self.num_pages)
        width = max_pages or max(1, max(per))
        self.table = np.full((len(kv_len), width), -7, np.int32)
        at = 0
        for b, p in enumerate(per):
            self.table[b, :p] = order[at:at + p]
            at += p
        self.start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.tokens = int(self.start[-1]) + pad

    def batch(self, api):
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()
        return api.KVBatch(dev(self.start), dev(self.kv_len), dev(self.table))

    def slots(self):
        """(row, sequence, position, page, slot) of every owned row whose position is not negative."""
        for b, n in enumerate(self.n):
            for i in range(n):
                p = self.kv_len[b] - n + i
                if p >= 0:
                    yield self.start[b] + i, b, p, self.table[b, p // self.page_size], p % self.page_size


def bf16(x) -> torch.Tensor:
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def bits(t: torch.Tensor) -> np.ndarray:
    return t.detach().contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def f64(t: torch.Tensor) -> np.ndarray:
    return nf4.bf16_to_f64(bits(t))


def inputs(rng, tokens, heads, dim):
    """Gaussian with a few strong channels per head."""
    x = rng.standard_normal((tokens, heads, dim)) * (1 + 4 * (rng.random((heads, dim)) < 0.03))
    return bf16(x)


def filled_cache(api, case, heads, dim, codebook, rng, garbage=True):
    """A cache whose sequences hold random tokens, written by the oracle, and its mirror
    {(b): (k, v)} in float64 [len, heads, dim].  Slots of no sequence hold NaN constants."""
    c = api.alloc_kv_cache(case.num_pages, heads, dim, case.page_size, codebook)
    shape = (case.num_pages, heads, case.page_size)
    host = {}
    for side in "kv":
        host[side] = (rng.integers(0, 256, shape + (dim // 2,)).astype(np.uint8),
                      np.full(shape + (dim // 64,), 0x7FC0 if garbage else 0, np.uint16))
    mirror = {}
    for b, length in enumerate(case.kv_len):
        both = []
        for side in "kv":
            codes, absmax = kv.encode(bits(inputs(rng, length, heads, dim)), codebook)
            p = np.arange(length)
            page, slot = case.table[b, p // case.page_size], p % case.page_size
            host[side][0][page, :, slot] = codes
            host[side][1][page, :, slot] = absmax
            both.append(kv.decode(codes, absmax, codebook))
        mirror[b] = tuple(both)
    for side in "kv":
        getattr(c, side + "_codes").copy_(torch.from_numpy(host[side][0]))
        getattr(c, side + "_absmax").copy_(torch.from_numpy(host[side][1].view(np.int16)).view(torch.bfloat16))
    return c, mirror
