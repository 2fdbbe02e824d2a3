"""Oracle for the 4-bit key/value cache and the attention over it, in float64.
TEST INFRASTRUCTURE ONLY (see the package docstring).

The cache stores every 64-channel block of a key or value as the weight
quantiser stores a block ("QLoRA: Efficient Finetuning of Quantized LLMs",
intuitivepapers.ai, §Quantize in blocks, §NormalFloat): the block's absmax and
the nearest level of float32(x / absmax), ties to the lower index.  The absmax
is kept in bfloat16, where it is exact for bfloat16 inputs.

Attention uses level * absmax unrounded.  ``attention`` also returns a bound on
what the kernel's roundings can add, element by element (see there).
"""
from __future__ import annotations

import numpy as np

from . import formats, nf4

BLOCK = 64


def encode(x_bits: np.ndarray, codebook: str):
    """bfloat16 bits [..., D] (finite) -> (packed codes uint8 [..., D/2], absmax
    bfloat16 bits [..., D/64])."""
    shape = x_bits.shape
    codes, c = formats.quantize_codes(x_bits.reshape(-1), formats.codebook(codebook), BLOCK)
    codes = codes.reshape(*shape[:-1], shape[-1] // 2, 2).astype(np.uint8)
    absmax = (c.view(np.uint32) >> 16).astype(np.uint16)
    assert np.array_equal(absmax.astype(np.uint32) << 16, c.view(np.uint32))  # exact
    return (codes[..., 0] << 4) | codes[..., 1], absmax.reshape(*shape[:-1], shape[-1] // BLOCK)


def decode(codes: np.ndarray, absmax: np.ndarray, codebook: str) -> np.ndarray:
    """Stored form -> float64 values level * absmax [..., D]."""
    idx = np.stack([codes >> 4, codes & 15], axis=-1).reshape(*codes.shape[:-1], codes.shape[-1] * 2)
    lv = formats.codebook(codebook).astype(np.float64)
    return lv[idx] * np.repeat(nf4.bf16_to_f64(absmax), BLOCK, axis=-1)


def read(codes: np.ndarray, absmax: np.ndarray, codebook: str) -> np.ndarray:
    """bf16_rn(float32(level * absmax)) as bits."""
    import torch
    x = decode(codes, absmax, codebook).astype(np.float32)  # float32 product: exact in float64, rounded once
    return torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, causal: bool, window: int, nf4_levels: bool):
    """One sequence.  q [n, Hq, D], k and v [len, H, D], all float64; the rows are
    the last n positions.  Returns (out [n, Hq, D], bound [n, Hq, D]).

    The bound: a score is off by at most ds = S * (2^-10 + 2^-14) with S = scale *
    sum |q_d k_d|: for NF4 alone the levels are rounded to fp16 (half a step, 2^-11)
    and, where many rows share the decoded keys, level * constant once more (2^-11;
    the other code books' levels are multiples of at most 3 bits, exact in both);
    float32 sums of D products, exponents and logarithms: 2^-14.  So a softmax weight
    is off by a factor within exp(+-2 ds).  Weights are rounded to fp16 (2^-11), and
    for NF4 alone the values' levels (2^-11) and, where many rows share them, level *
    constant (2^-11); a token's weight that is 2^-31 of the largest vanishes, and its
    value may be 2^8 times the largest one's (2^-23 for each token); float32 sums and
    the joins of parts add 2^-14; the output is rounded to bfloat16 (2^-8, and half
    the smallest subnormal).
    """
    n, hq, d = q.shape
    length, h, _ = k.shape
    g = hq // h
    out = np.zeros((n, hq, d))
    bound = np.zeros((n, hq, d))
    pos = np.arange(length - n, length)
    j = np.arange(length)
    see = np.ones((n, length), bool)
    if causal:
        see &= j[None, :] <= pos[:, None]
    if window:
        see &= j[None, :] > pos[:, None] - window
    if length == 0:
        return out, bound
    for x in range(hq):
        kk, vv = k[:, x // g], v[:, x // g]
        s = scale * (q[:, x] @ kk.T)
        mag = scale * (np.abs(q[:, x]) @ np.abs(kk).T)
        s = np.where(see, s, -np.inf)
        any_ = see.any(1)
        top = np.where(any_, s.max(1, initial=-np.inf), 0.0)
        p = np.exp(s - top[:, None])
        total = p.sum(1)
        p = p / np.where(total > 0, total, 1.0)[:, None]
        out[:, x] = p @ vv
        ds = np.where(see, mag, 0.0).max(1) * ((2.0 ** -10 if nf4_levels else 0.0) + 2.0 ** -14)
        with np.errstate(over="ignore"):
            rel = np.expm1(2 * ds) + 2.0 ** -11 * (3 if nf4_levels else 1) + 2.0 ** -14
        spread = p @ np.abs(vv)
        # contributions to a block of 64 channels: weight times the block's largest magnitude
        big = np.abs(vv).reshape(length, -1, BLOCK).max(2)
        most = (p[:, :, None] * big[None]).max(1)
        lost = np.repeat(most, BLOCK, axis=1) * length * 2.0 ** -23
        # two averages of the visible values are never further apart than twice the largest
        span = 2 * np.where(see[:, :, None], np.abs(vv)[None], 0.0).max(1)
        with np.errstate(over="ignore", invalid="ignore"):
            moved = rel[:, None] * spread
        bound[:, x] = np.minimum(np.where(np.isnan(moved), np.inf, moved), span) + lost
        bound[:, x] += 2.0 ** -8 * (np.abs(out[:, x]) + bound[:, x]) + 2.0 ** -133
    return out, bound
