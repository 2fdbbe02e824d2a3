"""GPU parity of qlora_kv_attention against the float64 oracle, element by element
within the bound that oracle/kv.py derives from the kernel's roundings."""
import numpy as np
import pytest
import torch

from oracle import formats, kv, linear, nf4
from tests.gpu_util import api, check_dev_err
from tests.kv_util import Case, bf16, bits, f64, filled_cache, inputs

pytestmark = pytest.mark.gpu


def _verify(case, mirror, Q, out, scale, causal, window, codebook, only=None):
    q, got = f64(Q), f64(out)
    for b, n in enumerate(case.n):
        if only is not None and b not in only:
            continue
        rows = slice(int(case.start[b]), int(case.start[b]) + n)
        want, bound = kv.attention(q[rows], *mirror[b], scale, causal, window, codebook == "nf4")
        assert np.all(np.isfinite(got[rows])), f"sequence {b}: non-finite output"
        far = np.abs(got[rows] - want) - bound
        assert n == 0 or far.max() <= 0, f"sequence {b}: {far.max():.3e} past the bound at {np.unravel_index(far.argmax(), far.shape)}"


def _run(case, heads, group, dim, codebook="nf4", causal=True, window=0, scale=None, seed=0, q_scale=1.0):
    a = api()
    rng = np.random.default_rng(seed + 1000)
    c, mirror = filled_cache(a, case, heads, dim, codebook, rng)
    Q = bf16(rng.standard_normal((case.tokens, heads * group, dim)) * q_scale).cuda()
    err = a.new_error_word()
    out = torch.full((case.tokens, heads * group, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    a.qlora_kv_attention(c, case.batch(a), Q, scale=scale, causal=causal, window=window, out=out, dev_err=err)
    check_dev_err(err)
    _verify(case, mirror, Q, out, dim ** -0.5 if scale is None else scale, causal, window, codebook)
    assert torch.all(out[case.tokens - case.pad:] == 7.0), "rows behind the last sequence were written"
    return c, mirror, Q, out


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,group,page", [(1, 1, 16), (2, 7, 64), (8, 8, 32), (3, 16, 128), (32, 1, 256), (1, 40, 16)])
def test_single_tokens(dim, heads, group, page):
    """Decode: lengths around every boundary of the kernel (16-token tiles, 32 per warp, 128 per step)."""
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 300, 1000]
    _run(Case([1] * len(lens), lens, page_size=page, pad=2, seed=page), heads, group, dim)


@pytest.mark.parametrize("codebook", formats.CODEBOOKS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_code_books(codebook, dim):
    _run(Case([1, 3, 1], [77, 200, 513], page_size=64, seed=1), 4, 4, dim, codebook)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 33), (True, 100), (False, 0), (False, 50)])
@pytest.mark.parametrize("heads,group", [(2, 5), (4, 1)])
def test_several_tokens_and_masks(dim, causal, window, heads, group):
    """Rows of one sequence with different limits; more rows than cached tokens (rows that see
    nothing); sequences without rows, without tokens; a prompt from position 0."""
    case = Case([4, 0, 7, 3, 30, 1, 5], [200, 50, 5, 0, 30, 1, 129], page_size=16, pad=1, seed=2)
    _run(case, heads, group, dim, causal=causal, window=window)


@pytest.mark.parametrize("dim,heads,group", [(128, 2, 4), (64, 4, 1), (256, 1, 8), (128, 1, 7)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 200)])
def test_prompt_chunks(dim, heads, group, causal, window):
    """Hundreds of rows per sequence, beside single tokens in the same call; more rows than cached
    tokens, and none cached."""
    case = Case([257, 1, 130, 64, 1, 100, 90], [600, 333, 130, 1000, 2, 40, 0], page_size=64, pad=3, seed=3)
    _run(case, heads, group, dim, causal=causal, window=window)


def test_one_long_sequence():
    """Every group of warps of the GPU shares each item; the parts are joined."""
    _run(Case([1], [20_011], page_size=128, seed=4), 2, 8, 128)


def test_rounding_of_levels_cancels_over_a_long_cache():
    """100000 tokens with nearly equal weights: the outputs are averages of values of random signs,
    360 times smaller than they, and any common bias of the decoded values would show.  The error's
    2-norm over the outputs': bfloat16 rounding at most 2^-8 / sqrt(3) in the mean square (half a step
    is 2^-8, uniform); levels and weights 2^-11 / sqrt(3) each, independent from token to token; the
    levels' mean error, 2.3e-6 of the values' root mean square, grows by sqrt(100000) against it: 7.3e-4
    (the keys' move the weights together and cancel in the softmax)."""
    a = api()
    length, heads, group, dim = 100_000, 4, 4, 128
    case = Case([1], [length], page_size=256, seed=20)
    c, mirror = filled_cache(a, case, heads, dim, "nf4", np.random.default_rng(96))
    Q = bf16(np.random.default_rng(97).standard_normal((1, heads * group, dim)) * 0.1).cuda()
    out = a.qlora_kv_attention(c, case.batch(a), Q)
    want, _ = kv.attention(f64(Q), *mirror[0], dim ** -0.5, True, 0, True)
    off = np.linalg.norm(f64(out) - want) / np.linalg.norm(want)
    assert off <= np.sqrt(2.0 ** -16 / 3 + 3 * 2.0 ** -22 / 3 + 7.3e-4 ** 2), off


def test_long_prompt():
    _run(Case([1500], [2100], page_size=64, seed=5), 1, 4, 128)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_items_of_many_parts(dim):
    """A long cache under a single token and under a chunk of two row tiles, in one call: each item is
    shared by more workers than a warp has lanes."""
    _run(Case([1, 100, 1], [20_011, 20_500, 3], page_size=128, pad=1, seed=21), 1, 4, dim)


@pytest.mark.parametrize("others", [0, 5])
@pytest.mark.parametrize("n", [2, 16, 17, 32, 33, 129, 130])
def test_rows_around_the_limits_between_kernels(n, others):
    """64 rows and 512 of four query heads each are where the choice of kernel changes; alone, and beside single
    tokens and empty sequences."""
    _run(Case([n] + [1, 0, 1, 1, 0][:others], [n + 100] + [70, 9, 300, 1, 0][:others], page_size=32, seed=22), 2, 4, 128)


def test_many_sequences():
    n = [b % 3 % 2 for b in range(4096)]
    case = Case(n, [(5 * b) % 23 + x for b, x in enumerate(n)], page_size=16, pad=2, seed=6)
    _run(case, 1, 2, 64)


@pytest.mark.parametrize("scale,q_scale", [(1.0, 1.0), (0.5, 1e-30), (3e-4, 300.0), (0.088, 1e4), (2.0 ** -100, 2.0 ** 100)])
def test_scales(scale, q_scale):
    """Flat and peaked softmax, tiny and huge queries (scores of several hundred)."""
    _run(Case([1, 2], [100, 400], page_size=32, seed=7), 2, 4, 128, scale=scale, q_scale=q_scale)


def _constants_of_any_size(dim, n, side, exps):
    """The constants of token j's keys or values times 2^exps[j]."""
    a = api()
    rng = np.random.default_rng(50)
    case = Case([n], [90], page_size=16, seed=8)
    c, mirror = filled_cache(a, case, 1, dim, "nf4", rng)
    p = np.arange(90)
    page, slot = case.table[0, p // 16], p % 16
    absmax = getattr(c, side + "_absmax")
    full = bits(absmax).copy()
    full[page, :, slot] = bits(bf16(nf4.bf16_to_f64(full[page, :, slot]) * 2.0 ** exps[:, None, None]))
    absmax.copy_(torch.from_numpy(full.view(np.int16)).view(torch.bfloat16))
    k, v = mirror[0]
    if side == "k":
        k = k * 2.0 ** exps[:, None, None]
    else:
        v = v * 2.0 ** exps[:, None, None]
    Q = bf16(rng.standard_normal((n, 4, dim))).cuda()
    out = a.qlora_kv_attention(c, case.batch(a), Q)
    _verify(case, {0: (k, v)}, Q, out, dim ** -0.5, True, 0, "nf4")


@pytest.mark.parametrize("n", [2, 60])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_values_of_any_size(dim, n):
    """Constants of the values far apart: from 2^-100 to 1, and a token of 2^100 that all rows but the
    last may not see; all of them huge, tiny, zero; a few binades apart."""
    rng = np.random.default_rng(51)
    exps = rng.integers(-100, 0, 90)
    exps[[3, 88]] = -100
    _constants_of_any_size(dim, n, "v", exps)
    exps[89] = 100
    _constants_of_any_size(dim, n, "v", exps)
    for e in (-125, -100, 100, 118, -400):
        _constants_of_any_size(dim, n, "v", np.full(90, e))
    _constants_of_any_size(dim, n, "v", rng.integers(-9, 1, 90))


@pytest.mark.parametrize("n", [2, 40])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_maximum_that_jumps_within_a_step(dim, n):
    """The scores of one step rise by 7 binades after a quarter of it and by 18 more after three quarters:
    what was weighed before has weights of 2^-18 then, but there are many and their values 2^7 times the
    last ones' (1/32 of the output; with 256 channels and steps half as long, 1/64)."""
    a = api()
    quarter = 16 if dim == 256 else 32
    case = Case([n], [4 * quarter], page_size=16, seed=24)
    c, _ = filled_cache(a, case, 1, dim, "int4", np.random.default_rng(1))
    kc, vc = np.full(4 * quarter, 1.0), np.full(4 * quarter, 1.0)
    kc[quarter:3 * quarter], vc[quarter:3 * quarter] = 1.21875, 128.0  # 7 / 32 more
    kc[3 * quarter + 5] = 1.78125                                     # 25 / 32 more
    K, V = (np.repeat(x[:, None, None], dim, axis=2) for x in (kc, vc))
    whole = Case([4 * quarter], [4 * quarter], page_size=16, seed=24)
    whole.table = case.table
    a.qlora_kv_append(c, whole.batch(a), bf16(K).cuda(), bf16(V).cuda())
    Q = torch.ones(n, 2, dim, dtype=torch.bfloat16, device="cuda")
    scale = float(np.float32(32 * np.log(2) / dim))
    out = a.qlora_kv_attention(c, case.batch(a), Q, scale=scale, causal=False)
    want, bound = kv.attention(f64(Q), K, V, scale, False, 0, False)
    assert bound.max() < np.abs(want - 1).min()  # tells them from nothing
    off = (np.abs(f64(out) - want) - bound).max()
    assert off <= 0, off


@pytest.mark.parametrize("n", [2, 60])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_keys_of_any_size(dim, n):
    """Constants of the keys far apart (a huge key hidden from all rows but the last), zero, tiny."""
    rng = np.random.default_rng(52)
    _constants_of_any_size(dim, n, "k", rng.integers(-60, 1, 90))
    exps = rng.integers(-3, 1, 90)
    exps[89] = 60
    _constants_of_any_size(dim, n, "k", exps)
    for e in (-125, -400):
        _constants_of_any_size(dim, n, "k", np.full(90, e))
    _constants_of_any_size(dim, n, "k", rng.integers(-13, 1, 90))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n,group", [(2, 4), (40, 8)])
def test_nan_stays_where_it_is_seen(n, group, dim):
    """A NaN key makes exactly the rows that see it NaN, a NaN value constant its 64 channels of those
    rows; NaN in a query its own row.  Everything else stays within its bound."""
    a = api()
    rng = np.random.default_rng(60)
    case = Case([n, 1], [150, 100], page_size=16, seed=9)
    heads, scale = 2, dim ** -0.5
    c, mirror = filled_cache(a, case, heads, dim, "nf4", rng)
    Q = bf16(rng.standard_normal((case.tokens, heads * group, dim)))

    def check(got, nan):
        assert torch.equal(torch.isnan(got.float()), nan)
        for b in range(2):
            rows = slice(int(case.start[b]), int(case.start[b + 1]))
            want, bound = kv.attention(f64(Q[rows]), *mirror[b], scale, True, 0, True)
            far = np.abs(f64(got[rows]) - want) - bound
            assert far[~nan[rows].numpy()].max() <= 0

    last = case.table[0, 149 // 16], 149 % 16  # the last position: row n - 1 alone sees it
    for side, block in (("k", 0), ("v", dim // 64 - 1)):
        absmax = getattr(c, side + "_absmax")
        keep = absmax.clone()
        absmax[last[0], 1, last[1], block] = float("nan")
        got = a.qlora_kv_attention(c, case.batch(a), Q.cuda()).cpu()
        nan = torch.zeros(got.shape, dtype=torch.bool)
        nan[n - 1, group:, (64 * block if side == "v" else 0):] = True
        check(got, nan)
        absmax.copy_(keep)
    for poison in (float("nan"), float("inf")):
        Q2 = Q.clone()
        Q2[0, 1, 17] = poison
        got = a.qlora_kv_attention(c, case.batch(a), Q2.cuda()).cpu()
        nan = torch.zeros(got.shape, dtype=torch.bool)
        nan[0, 1] = True
        check(got, nan)


def test_strided_queries_and_error_free_padding():
    """Q as the first slice of a fused projection; rows behind the last sequence hold NaN."""
    a = api()
    rng = np.random.default_rng(70)
    case = Case([1, 2], [40, 70], pad=2, seed=10)
    c, mirror = filled_cache(a, case, 2, 128, "nf4", rng)
    fused = bf16(rng.standard_normal((case.tokens, 12, 128))).cuda()
    fused[3:] = float("nan")
    Q = fused[:, :8]
    out = torch.full((case.tokens, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    a.qlora_kv_attention(c, case.batch(a), Q, out=out)
    _verify(case, mirror, Q, out, 128 ** -0.5, True, 0, "nf4")
    assert torch.all(out[3:] == 7.0)
    Qt = Q.transpose(0, 1).contiguous().transpose(0, 1)  # head-major in memory
    out2 = torch.full_like(out, 7.0)
    a.qlora_kv_attention(c, case.batch(a), Qt, out=out2)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16))


def test_entries_out_of_range():
    """Reported; the sequences with sound entries are right all the same."""
    a = api()
    rng = np.random.default_rng(80)
    for n in (1, 60):
        case = Case([n, n, n], [60, 90, 200], seed=11)
        c, mirror = filled_cache(a, case, 2, 64, "nf4", rng)
        Q = bf16(rng.standard_normal((case.tokens, 4, 64))).cuda()
        for change in ("page_high", "page_negative", "kv_len_high", "kv_len_negative", "start"):
            batch = case.batch(a)
            if change == "page_high":
                batch.page_table[1, 2] = case.num_pages
            elif change == "page_negative":
                batch.page_table[1, 0] = -3
            elif change == "kv_len_high":
                batch.kv_len[1] = 1 << 30
            elif change == "kv_len_negative":
                batch.kv_len[1] = -1
            else:
                batch.token_start[3] = case.tokens + 5
            err = a.new_error_word()
            out = a.qlora_kv_attention(c, batch, Q, dev_err=err)
            torch.cuda.synchronize()
            assert int(err[0]) == a.QLORA_DEVERR_KV_INDEX, change
            _verify(case, mirror, Q, out, 64 ** -0.5, True, 0, "nf4", only=[0] if change == "start" else [0, 2])


def test_identical_bits_and_a_dirty_workspace():
    """Whatever the workspace held, and however often: the same bits."""
    a = api()
    rng = np.random.default_rng(90)
    case = Case([1, 5, 1, 200], [3000, 700, 1, 900], page_size=64, seed=12)
    c, _ = filled_cache(a, case, 2, 128, "nf4", rng)
    Q = bf16(rng.standard_normal((case.tokens, 16, 128))).cuda()
    batch = case.batch(a)
    need = a.qlora_kv_attention_workspace_size(c, 4, case.tokens, 16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    first = None
    for fill in (0, 0xFF, 0x7F, 1, 1, 1):
        ws.fill_(fill)
        out = a.qlora_kv_attention(c, batch, Q, ws=ws)
        first = out if first is None else first
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))


def test_two_streams_with_a_workspace_each():
    a = api()
    rng = np.random.default_rng(91)
    case = Case([1, 1], [5000, 3000], page_size=64, seed=13)
    c, mirror = filled_cache(a, case, 4, 128, "nf4", rng)
    Qs = [bf16(rng.standard_normal((2, 16, 128))).cuda() for _ in range(2)]
    batch = case.batch(a)
    need = a.qlora_kv_attention_workspace_size(c, 2, 2, 16)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [[], []]
    wss = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(a.qlora_kv_attention(c, batch, Qs[i], ws=wss[i]))
    torch.cuda.synchronize()
    for i in range(2):
        _verify(case, mirror, Qs[i], outs[i][0], 128 ** -0.5, True, 0, "nf4")
        assert all(torch.equal(o, outs[i][0]) for o in outs[i])


def test_decode_loop_in_a_graph():
    """Append and attend captured once; each replay reads the new token and length written in place."""
    a = api()
    rng = np.random.default_rng(92)
    heads, group, dim = 2, 4, 128
    case = Case([1, 1], [32, 70], page_size=16, seed=14, spare=6)
    c, mirror = filled_cache(a, case, heads, dim, "nf4", rng)
    table = np.full((2, 8), -7, np.int32)
    table[:, : case.table.shape[1]] = case.table
    free = [p for p in range(case.num_pages) if p not in case.table]
    table[0, 2:4] = free[:2]
    table[1, 5] = free[2]
    case.table = table
    batch = case.batch(a)
    K, V = (torch.zeros(2, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    Q = torch.zeros(2, heads * group, dim, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(a.qlora_kv_attention_workspace_size(c, 2, 2, heads * group), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(Q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    keep = [t.clone() for t in (c.k_codes, c.k_absmax, c.v_codes, c.v_absmax)]
    with torch.cuda.stream(side):
        a.qlora_kv_append(c, batch, K, V)
        a.qlora_kv_attention(c, batch, Q, out=out, ws=ws)
    side.synchronize()
    for t, k in zip((c.k_codes, c.k_absmax, c.v_codes, c.v_absmax), keep):
        t.copy_(k)
    with torch.cuda.graph(graph):
        a.qlora_kv_append(c, batch, K, V)
        a.qlora_kv_attention(c, batch, Q, out=out, ws=ws)
    state = {b: [x for x in mirror[b]] for b in mirror}
    for step in range(4):
        kx, vx = inputs(rng, 2, heads, dim), inputs(rng, 2, heads, dim)
        K.copy_(kx), V.copy_(vx), Q.copy_(bf16(rng.standard_normal(tuple(Q.shape))))
        lens = [33 + step, 71 + step]
        batch.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for b in range(2):
            for s, x in enumerate((kx, vx)):
                codes, absmax = kv.encode(bits(x[b]), "nf4")
                state[b][s] = np.concatenate([state[b][s], kv.decode(codes, absmax, "nf4")[None]])
        now = Case([1, 1], lens, page_size=16)
        _verify(now, {b: tuple(state[b]) for b in state}, Q, out, dim ** -0.5, True, 0, "nf4")


def test_prompt_chunks_in_a_graph():
    """A captured call (on the capture's own stream) gives the bits of a direct one, and follows the batch
    arrays when they are rewritten."""
    a = api()
    case = Case([200, 1, 90], [700, 300, 400], page_size=64, pad=2, seed=23)
    c, mirror = filled_cache(a, case, 2, 128, "nf4", np.random.default_rng(98))
    Q = bf16(np.random.default_rng(99).standard_normal((case.tokens, 8, 128))).cuda()
    batch = case.batch(a)
    out = torch.zeros(case.tokens, 8, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(a.qlora_kv_attention_workspace_size(c, 3, case.tokens, 8), dtype=torch.uint8, device="cuda")
    err = a.new_error_word()
    a.qlora_kv_attention(c, batch, Q, out=out, ws=ws, dev_err=err)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.qlora_kv_attention(c, batch, Q, out=out, ws=ws, dev_err=err)
    for shorter in (0, 130):
        batch.kv_len.sub_(shorter)
        graph.replay()
        graph.replay()
        got = out.clone()
        direct = a.qlora_kv_attention(c, batch, Q)
        assert np.array_equal(bits(got)[: case.tokens - case.pad], bits(direct)[: case.tokens - case.pad])
    check_dev_err(err)


def test_pool_larger_than_4_gib():
    a = api()
    rng = np.random.default_rng(93)
    heads, dim, page = 8, 128, 64
    pages = 140_000
    case = Case([1, 60], [100, 130], page_size=page, seed=15)
    small, mirror = filled_cache(a, case, heads, dim, "nf4", rng)
    c = a.alloc_kv_cache(pages, heads, dim, page, "nf4")
    assert c.k_codes.numel() > 1 << 32
    moved = case.batch(a)
    for name in ("k_codes", "k_absmax", "v_codes", "v_absmax"):
        getattr(c, name)[pages - case.num_pages:] = getattr(small, name)
    moved.page_table.add_(pages - case.num_pages)
    Q = bf16(rng.standard_normal((case.tokens, 32, dim))).cuda()
    err = a.new_error_word()
    out = a.qlora_kv_attention(c, moved, Q, dev_err=err)
    check_dev_err(err)
    _verify(case, mirror, Q, out, dim ** -0.5, True, 0, "nf4")
    assert torch.equal(out, a.qlora_kv_attention(small, case.batch(a), Q))


def test_a_layer_of_a_quantised_model():
    """The operators as they are used together: the frozen NF4 projection with its adapter gives q, k
    and v; k and v are appended; attention reads them; the output projection follows.  Every stage is
    checked against the oracle on the stage's own inputs: a prompt first, then two decode steps."""
    a = api()
    rng = np.random.default_rng(94)
    heads, group, dim, r = 2, 2, 64, 8
    hidden, hq = 256, heads * group
    n_qkv = (hq + 2 * heads) * dim
    weights = {}
    for name, rows, cols in (("qkv", n_qkv, hidden), ("o", hidden, hq * dim)):
        w = a.qlora_quantize(bf16(rng.standard_normal((rows, cols)) * 0.06).cuda())
        A = bf16(rng.standard_normal((cols, r)) * 0.05).cuda()
        B = bf16(rng.standard_normal((r, rows)) * 0.05).cuda()
        weights[name] = (w, A, B, bits(a.qlora_dequantize(w)))

    def project(name, x):
        w, A, B, hat = weights[name]
        y, _ = a.qlora_linear_forward(w, x, A, B, 0.5)
        ref = linear.forward(bits(x), hat, bits(A), bits(B), 0.5)["Y"]
        assert np.linalg.norm(f64(y) - ref) <= 1e-2 * np.linalg.norm(ref)
        return y

    c = a.alloc_kv_cache(12, heads, dim, 16, "nf4")
    lens, mirror = [0, 0], {0: None, 1: None}
    table = np.arange(12, dtype=np.int32).reshape(2, 6)[:, ::-1].copy()
    for n in ([33, 20], [1, 1], [1, 1]):
        lens = [x + y for x, y in zip(lens, n)]
        case = Case(n, lens, page_size=16)
        case.table = table
        batch = case.batch(a)
        qkv = project("qkv", bf16(rng.standard_normal((case.tokens, hidden))).cuda()).view(case.tokens, -1, dim)
        Q, K, V = qkv[:, :hq], qkv[:, hq:hq + heads], qkv[:, hq + heads:]
        err = a.new_error_word()
        a.qlora_kv_append(c, batch, K, V, dev_err=err)
        out = a.qlora_kv_attention(c, batch, Q, dev_err=err)
        check_dev_err(err)
        for b in range(2):
            rows = slice(int(case.start[b]), int(case.start[b + 1]))
            new = [kv.decode(*kv.encode(bits(x[rows]), "nf4"), "nf4") for x in (K, V)]
            mirror[b] = tuple(new) if mirror[b] is None else tuple(np.concatenate(x) for x in zip(mirror[b], new))
        _verify(case, mirror, Q, out, dim ** -0.5, True, 0, "nf4")
        project("o", out.reshape(case.tokens, -1))
