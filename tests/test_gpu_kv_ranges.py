"""GPU parity of qlora_kv_attention where the values' constants and the scores lie far
apart: zero blocks of values under high scores, steps of very different sizes, blocks of
one head of very different sizes, peaked softmax.

The inputs are exact in every format on the way (Int4 codes +-7, constants that are
bfloat16 numbers, queries of ones), so the oracle's bound is a few parts in a thousand of
what the visible values weigh, and tells a right output from a wrong one."""
import numpy as np
import pytest
import torch

from oracle import kv
from tests.gpu_util import api, check_dev_err
from tests.kv_util import Case, bf16, f64

pytestmark = pytest.mark.gpu

DIMS = [64, 128, 256]


def _step(dim):
    """Cached tokens that the many-row kernel weighs together."""
    return 64 if dim == 256 else 128


def _fill(a, t, size, heads, dim, signs, case):
    """A cache with one sequence: the keys of token j give every row the score t[j] (in powers of two),
    its values are size[j, block] with a sign per channel; every head the same."""
    length = len(t)
    c = a.alloc_kv_cache(case.num_pages, heads, dim, case.page_size, "int4")
    whole = Case([length], [length], page_size=case.page_size)
    whole.table = case.table[:1]
    K = np.repeat(np.asarray(t, np.float64)[:, None, None], dim, axis=2)
    V = (np.repeat(np.asarray(size, np.float64), 64, axis=1) * signs)[:, None]
    for x in (K, V):
        assert np.array_equal(f64(bf16(x)), x)
    a.qlora_kv_append(c, whole.batch(a), *(bf16(x).cuda().expand(-1, heads, -1) for x in (K, V)))
    return c, K, V


def _scale(dim):
    return float(np.float32(np.log(2.0) / dim))


def _off(out, K, V, dim, extra=0.0):
    """How far past its bound the furthest output is; every row and head sees the same."""
    want, bound = kv.attention(np.ones((1, 1, dim)), K, V, _scale(dim), False, 0, False)
    got = f64(out)
    assert np.all(np.isfinite(got)), "non-finite output"
    return (np.abs(got - want) - bound - extra).max(), want, bound


def _run(t, size, n, heads, group, dim, extra=0.0):
    a = api()
    signs = np.where(np.random.default_rng(len(t)).random(dim) < 0.5, -1.0, 1.0)
    case = Case([n], [len(t)], page_size=16, seed=30)
    c, K, V = _fill(a, t, size, heads, dim, signs, case)
    Q = torch.ones(n, heads * group, dim, dtype=torch.bfloat16, device="cuda")
    err = a.new_error_word()
    out = a.qlora_kv_attention(c, case.batch(a), Q, scale=_scale(dim), causal=False, dev_err=err)
    check_dev_err(err)
    off, want, bound = _off(out, K, V, dim, extra)
    assert off <= 0, off
    return want, bound


def _near(rng, length, spread=2.0):
    """Scores that differ by a few binades (sixteenths: exact in bfloat16)."""
    return np.round(rng.uniform(-spread, spread, length) * 16) / 16


@pytest.mark.parametrize("n", [1, 2, 60])
@pytest.mark.parametrize("dim", DIMS)
def test_zero_values_under_the_highest_score(dim, n):
    """The token with the highest score has an all-zero block of values; the others' weights lie 130
    binades below and vanish in float32 (a weight below 2^-126 of the largest: `extra`)."""
    for size in (2.0, 4.0, 2.0 ** 20, 2.0 ** 100):
        t, values = np.full(90, -130.0), np.full((90, dim // 64), size)
        t[7], values[7] = 0.0, 1.0
        values[7, 0] = 0.0
        _run(t, values, n, 2, 4, dim, extra=90 * 2.0 ** -126 * size)


@pytest.mark.parametrize("n", [1, 2, 60])
@pytest.mark.parametrize("dim", DIMS)
def test_huge_value_far_below_the_highest_score(dim, n):
    """A value of 2^123 whose weight, 2^-150, vanishes in float32 beside ordinary tokens."""
    t, values = _near(np.random.default_rng(31), 90), np.ones((90, dim // 64))
    t[40], values[40] = -150.0, 2.0 ** 123
    _run(t, values, n, 2, 4, dim, extra=2.0 ** (123 - 148))


# ---------------------------------------------------------------- prompt chunks: several steps of one item
# With 160 heads a worker does whole items; with one head every step has a worker of its own and the
# parts are joined.
@pytest.mark.parametrize("heads", [160, 1])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("first,second", [(40, -100), (100, -50), (8, -126), (3, -120), (60, -80), (-100, 40), (-80, 60)])
def test_steps_of_very_different_sizes(dim, first, second, heads):
    """What tokens weigh in the softmax does not depend on the size of their values."""
    rng, step = np.random.default_rng(32), _step(dim)
    length = 2 * step + 37
    size = np.full((length, dim // 64), 2.0 ** second)
    size[:step] = 2.0 ** first
    _run(_near(rng, length), size, 60, heads, 4, dim)


@pytest.mark.parametrize("heads", [160, 1])
@pytest.mark.parametrize("exponent", [-17, -30, -100])
@pytest.mark.parametrize("at", [0, 1, 2])
@pytest.mark.parametrize("dim", DIMS)
def test_step_of_zero_values(dim, at, exponent, heads):
    """A whole step of tokens without values, with the highest scores, before, between and after small values."""
    rng, step = np.random.default_rng(33), _step(dim)
    length = 3 * step + 20
    t, size = _near(rng, length), np.full((length, dim // 64), 1.3125 * 2.0 ** exponent)
    t[at * step:(at + 1) * step] += 8
    size[at * step:(at + 1) * step] = 0.0
    want, bound = _run(t, size, 60, heads, 4, dim)
    assert (bound <= 0.02 * np.abs(want)).all()


def test_values_of_nothing_but_zeros():
    for n in (1, 60):
        want, _ = _run(_near(np.random.default_rng(34), 300), np.zeros((300, 2)), n, 2, 4, 128)
        assert not want.any()


@pytest.mark.parametrize("far", [0, 1])
@pytest.mark.parametrize("dim", DIMS)
def test_highest_score_of_small_values_before_larger_contributions(dim, far):
    """The first step has the highest scores and the smallest values, the second contributes 2^8 times as
    much; with `far` one key of the second is 2^-14 of the others (its constants are apart)."""
    rng, step = np.random.default_rng(35), _step(dim)
    length = 2 * step
    size = np.full((length, dim // 64), 1.3125 * 2.0 ** 20)
    t = np.round(rng.uniform(-1.5, 1.5, length) * 2) / 2  # (eight bits of significand, with what is added)
    t[step:] += 30
    if far:
        t[step + 3] = 2.0 ** -10
    t[:step] += 100
    size[:step] = 2.0 ** -60
    want, bound = _run(t, size, 60, 160, 4, dim)
    assert (bound <= 0.02 * np.abs(want)).all()


@pytest.mark.parametrize("heads", [160, 1])
@pytest.mark.parametrize("above", [12, 30, 60, 110, 120, 250])
@pytest.mark.parametrize("dim", DIMS)
def test_token_without_values_above_all_others(dim, above, heads):
    """One token of a step has zero values and takes nearly all the weight: what the others contribute keeps
    its precision."""
    rng, step = np.random.default_rng(36), _step(dim)
    length = 2 * step + 11
    t, size = _near(rng, length), np.full((length, dim // 64), 1.3125)
    t[step + 5], size[step + 5] = above, 0.0
    want, bound = _run(t, size, 60, heads, 4, dim)
    assert above == 250 or (bound <= 0.05 * np.abs(want)).all()


@pytest.mark.parametrize("heads", [160, 1])
@pytest.mark.parametrize("at", [0, 1, 2])
@pytest.mark.parametrize("larger", [10, 20, 31, 70])
@pytest.mark.parametrize("dim", [128, 256])
def test_blocks_of_very_different_sizes(dim, larger, at, heads):
    """In one step the first 64 channels' values are 2^larger times the others'; each block keeps its precision."""
    rng, step = np.random.default_rng(37), _step(dim)
    length = 3 * step
    t, size = _near(rng, length), np.full((length, dim // 64), 1.3125)
    size[at * step:(at + 1) * step, 0] *= 2.0 ** larger
    want, bound = _run(t, size, 60, heads, 4, dim)
    assert (bound <= 0.02 * np.abs(want)).all()


@pytest.mark.parametrize("dim", [128, 256])
def test_blocks_that_every_step_has_far_apart(dim):
    """A block 2^40 smaller throughout, and one of zeros."""
    rng = np.random.default_rng(38)
    for small in (2.0 ** -40, 0.0):
        length = 2 * _step(dim) + 50
        size = np.full((length, dim // 64), 1.3125)
        size[:, -1] = 1.3125 * small
        _run(_near(rng, length), size, 60, 160, 4, dim)


def _weird_and_ordinary(a, dim=128, heads=2, n=60):
    """Two sequences of three steps, the first with blocks far apart, and a single token over the second; the
    caches' values and the expected outputs' ingredients."""
    rng, step = np.random.default_rng(39), _step(dim)
    length = 3 * step
    signs = np.where(rng.random(dim) < 0.5, -1.0, 1.0)
    case = Case([n, n, 1], [length, length, length], page_size=16, seed=31)
    case.table[2] = case.table[1]
    both = []
    c = None
    for b in range(2):
        t, size = _near(rng, length), np.full((length, dim // 64), 1.3125)
        if b == 0:
            size[:step, 0] *= 2.0 ** 31
        one = Case([length], [length], page_size=16)
        one.num_pages, one.table = case.num_pages, case.table[b:b + 1]
        filled, K, V = _fill(a, t, size, heads, dim, signs, one)
        if c is None:
            c = filled
        else:
            pages = torch.from_numpy(one.table[0].astype(np.int64)).cuda()
            for name in ("k_codes", "k_absmax", "v_codes", "v_absmax"):
                getattr(c, name)[pages] = getattr(filled, name)[pages]
        both.append((K, V))
    return case, c, both, signs


def test_other_sequences_of_the_call_keep_their_bits():
    """A sequence whose blocks lie far apart beside an ordinary one, which comes out as it does alone; and
    in a graph, whose replays follow what the cache holds."""
    a = api()
    dim, heads, group, n = 128, 2, 4, 60
    case, c, both, _ = _weird_and_ordinary(a)
    batch = case.batch(a)
    Q = torch.ones(case.tokens, heads * group, dim, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(Q, 7.0)
    err = a.new_error_word()
    ws = torch.empty(a.qlora_kv_attention_workspace_size(c, 3, case.tokens, heads * group), dtype=torch.uint8, device="cuda")
    attend = lambda: a.qlora_kv_attention(c, batch, Q, scale=_scale(dim), causal=False, out=out, ws=ws, dev_err=err)

    def check(first):
        torch.cuda.synchronize()
        check_dev_err(err)
        for rows, which in ((slice(0, n), first), (slice(n, 2 * n + 1), 1)):
            off, _, _ = _off(out[rows], *both[which], dim)
            assert off <= 0, off

    attend()
    check(0)
    direct = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attend()
    ws.fill_(0xFF)
    out.fill_(7.0)
    graph.replay()
    check(0)
    assert torch.equal(out.view(torch.int16), direct.view(torch.int16))
    batch.page_table[0] = batch.page_table[1]  # the first sequence becomes an ordinary one
    graph.replay()
    check(1)
    assert torch.equal(out[n:].view(torch.int16), direct[n:].view(torch.int16))
    assert torch.equal(out[:n].view(torch.int16), direct[n:2 * n].view(torch.int16))
    batch.page_table.copy_(torch.from_numpy(case.table))
    graph.replay()
    check(0)
    assert torch.equal(out.view(torch.int16), direct.view(torch.int16))


@pytest.mark.parametrize("n", [1, 2, 60])
@pytest.mark.parametrize("dim", DIMS)
def test_peaked_softmax(dim, n):
    """Scores of 0 to 250 binades in no order, so that references move again and again, by little and
    by much; the outputs are told from those of any other order of weights."""
    rng = np.random.default_rng(40)
    for top in (20, 60, 250):
        length = 3 * _step(dim) + 7
        t = np.round(rng.uniform(0, top, length))
        size = rng.choice([0.5, 1.0, 1.3125, 3.0], (length, dim // 64))
        want, bound = _run(t, size, n, 3, 4, dim)
        assert (bound <= 0.1 * np.abs(want)).all()


@pytest.mark.parametrize("n", [1, 2, 60])
@pytest.mark.parametrize("larger", [10, 20, 36, 40, 100])
@pytest.mark.parametrize("dim", [128, 256])
def test_key_blocks_of_very_different_sizes(dim, larger, n):
    """The first 64 channels of some keys are 2^larger times the others, and the queries zero there: the scores
    come from the small blocks alone."""
    a = api()
    rng, step, heads, group = np.random.default_rng(41), _step(dim), 3, 4
    length = 2 * step + 9
    t, signs = _near(rng, length, 5.0), np.where(rng.random(dim) < 0.5, -1.0, 1.0)
    case = Case([n], [length], page_size=16, seed=32)
    c, K, V = _fill(a, t, np.full((length, dim // 64), 1.3125), heads, dim, signs, case)
    V = V * rng.choice([0.5, 1.0, 3.0], (length, 1, 1))  # (values that differ, so that the weights show)
    K[::3, :, :64] = 2.0 ** larger
    whole = Case([length], [length], page_size=16)
    whole.table = case.table
    a.qlora_kv_append(c, whole.batch(a), *(bf16(x).cuda().expand(-1, heads, -1) for x in (K, V)))
    q = np.ones((1, 1, dim))
    q[..., :64] = 0.0
    out = a.qlora_kv_attention(c, case.batch(a), bf16(q).cuda().expand(n, heads * group, -1), scale=_scale(dim), causal=False)
    want, bound = kv.attention(q, K, V, _scale(dim), False, 0, False)
    assert (bound <= 0.02 * np.abs(want)).all()
    off = (np.abs(f64(out) - want) - bound).max()
    assert off <= 0, off


def test_random_ranges_and_masks():
    """Sizes, scores, zeros, masks and lengths drawn at random; every row against the oracle.  A weight
    below 2^-126 of its row's largest is 0 in float32: what such tokens would add is allowed for."""
    a = api()
    for seed in range(200):
        rng = np.random.default_rng(9000 + seed)
        dim = int(rng.choice(DIMS))
        step, blocks = _step(dim), dim // 64
        group, heads = int(rng.choice([1, 4, 7])), int(rng.choice([1, 3, 160]))
        length = int(rng.choice([1, 17, 90, step, 2 * step + 5, 3 * step + 70]))
        n = int(min(rng.choice([1, 2, 5, 20, 60, 130]), length + 3))
        causal, window = bool(rng.random() < 0.6), int(rng.choice([0, 0, 1, 40, 200]))
        t = np.round(rng.uniform(-0.5, 0.5, length) * rng.choice([4, 20, 100, 250]))
        span = int(rng.choice([0, 3, 8, 12, 30, 60, 100]))
        shape = [(length, blocks), (length, 1), (1, blocks)][rng.integers(3)]
        size = rng.choice([1.0, 1.25, 1.75], (length, blocks)) * 2.0 ** rng.integers(-span, span + 1, shape)
        size[rng.random((length, blocks)) < rng.choice([0, 0.02, 0.3])] = 0.0
        if rng.random() < 0.3:
            size[:step] = 0.0
        case = Case([n], [length], page_size=16, seed=seed)
        signs = np.where(rng.random(dim) < 0.5, -1.0, 1.0)
        c, K, V = _fill(a, t, size, heads, dim, signs, case)
        Q = torch.ones(n, heads * group, dim, dtype=torch.bfloat16, device="cuda")
        out = a.qlora_kv_attention(c, case.batch(a), Q, scale=_scale(dim), causal=causal, window=window)
        want, bound = kv.attention(np.ones((n, 1, dim)), K, V, _scale(dim), causal, window, False)
        pos, j = np.arange(length - n, length)[:, None], np.arange(length)
        see = (j <= pos if causal else np.ones((n, length), bool)) & ((j > pos - window) if window else True)
        below = np.where(see, t, -np.inf)
        below = below - np.maximum(below.max(1, keepdims=True), -1e9)  # (-inf throughout where nothing is seen)
        gone = np.where(see & (below < -124), 2.0 ** np.maximum(below, -1000.0), 0.0) @ np.abs(V[:, 0])
        off = np.abs(f64(out) - want) - bound - 1.01 * gone[:, None]
        assert np.all(off <= 0), (seed, off.max())
