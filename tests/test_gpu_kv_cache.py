"""GPU parity of qlora_kv_append and qlora_kv_read against the oracle: codes,
constants and read-back values bit for bit, and nothing else touched."""
import numpy as np
import pytest
import torch

from oracle import formats, kv
from tests.gpu_util import api, check_dev_err
from tests.kv_util import Case, bf16, bits, inputs

pytestmark = pytest.mark.gpu


def _blank(a, case, heads, dim, codebook):
    """A cache full of a recognisable pattern."""
    c = a.alloc_kv_cache(case.num_pages, heads, dim, case.page_size, codebook)
    for t in (c.k_codes, c.v_codes):
        t.fill_(0xA5)
    for t in (c.k_absmax, c.v_absmax):
        t.view(torch.int16).fill_(0x1234)
    return c


def _expected(case, heads, dim, codebook, x, page_codes, page_absmax):
    codes, absmax = kv.encode(bits(x), codebook)
    for row, _, _, page, slot in case.slots():
        page_codes[page, :, slot] = codes[row]
        page_absmax[page, :, slot] = absmax[row]


def _check(a, case, heads, dim, codebook, K, V, expect_err=0):
    """Append strided slices of one buffer, compare the whole pool, read back, compare."""
    c = _blank(a, case, heads, dim, codebook)
    batch = case.batch(a)
    err = a.new_error_word()
    a.qlora_kv_append(c, batch, K, V, dev_err=err)
    torch.cuda.synchronize()
    assert int(err[0]) == expect_err
    want = {}
    for side, x in (("k", K), ("v", V)):
        codes = np.full(tuple(c.k_codes.shape), 0xA5, np.uint8)
        absmax = np.full(tuple(c.k_absmax.shape), 0x1234, np.uint16)
        _expected(case, heads, dim, codebook, x, codes, absmax)
        assert np.array_equal(getattr(c, side + "_codes").cpu().numpy(), codes), f"{side} codes"
        assert np.array_equal(bits(getattr(c, side + "_absmax")), absmax), f"{side} constants"
        want[side] = kv.read(codes, absmax, codebook)
    err.zero_()
    outs = [torch.full((case.tokens, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    a.qlora_kv_read(c, batch, case.tokens, *outs, dev_err=err)
    torch.cuda.synchronize()
    assert int(err[0]) == expect_err
    sevens = bits(bf16([7.0]))[0]
    for side, out in zip("kv", outs):
        ref = np.full((case.tokens, heads, dim), sevens, np.uint16)
        for row, _, _, page, slot in case.slots():
            ref[row] = want[side][page, :, slot]
        assert np.array_equal(bits(out), ref), f"{side} read back"
    # one side alone gives the same
    only = torch.full_like(outs[1], 7.0)
    assert a.qlora_kv_read(c, batch, case.tokens, V_out=only)[0] is None
    assert torch.equal(only.view(torch.int16), outs[1].view(torch.int16))
    only.fill_(7.0)
    a.qlora_kv_read(c, batch, case.tokens, K_out=only)
    assert torch.equal(only.view(torch.int16), outs[0].view(torch.int16))


def _fused(rng, case, heads, dim, extra=0):
    """K and V as slices of one projection's output (rows strided)."""
    both = inputs(rng, case.tokens, 2 * heads + extra, dim).cuda()
    return both[:, extra:extra + heads], both[:, extra + heads:]


@pytest.mark.parametrize("codebook", formats.CODEBOOKS)
def test_every_ratio_of_bfloat16_values(codebook):
    """Every quotient of two bfloat16 significands, at every exponent distance that matters
    (down to 2^-9) and both signs, gets the definition's code: 128 absmax significands, each in enough
    blocks to hold all numerators."""
    a = api()
    nums = np.concatenate([np.arange(128, 256) * 2.0 ** -k for k in range(0, 10)])
    nums = np.concatenate([nums, -nums, [0.0, -0.0]])
    rows = []
    for b in range(128, 256):
        ok = nums[np.abs(nums) <= b]
        ok = np.concatenate([ok, np.zeros(-len(ok) % 63)]).reshape(-1, 63)
        rows.append(np.concatenate([np.full((len(ok), 1), float(b)), ok], 1))
    x = np.concatenate(rows)
    x = np.concatenate([x, np.zeros((-len(x) % 4, 64))]).reshape(-1, 4, 64)
    case = Case([len(x)], [len(x)], page_size=256)
    _check(a, case, 4, 64, codebook, bf16(x).cuda(), bf16(-x * 2.0 ** -20).cuda())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page,heads,codebook", [(16, 1, "nf4"), (64, 3, "fp4_e2m1"), (256, 8, "nf4"), (32, 5, "int4"),
                                                 (128, 32, "fp4_e3m0")])
def test_append_and_read_ragged(dim, page, heads, codebook):
    rng = np.random.default_rng(dim + page)
    # single tokens, nothing, a page's end inside the rows, rows behind the last sequence
    case = Case([1, 0, 17, 1, 70, 0, 5], [1, 40, 33, 128, 70, 0, 300], page_size=page, pad=3, seed=page)
    _check(api(), case, heads, dim, codebook, *_fused(rng, case, heads, dim, extra=2))


@pytest.mark.parametrize("heads,dim", [(32, 128), (40, 256), (7, 64), (512, 64)])
def test_single_tokens(heads, dim):
    """One new token per sequence; with 40 heads of 256 channels a row is split over CTAs."""
    rng = np.random.default_rng(heads)
    lens = [1, 15, 16, 17, 64, 65, 200]
    case = Case([1] * len(lens), lens, page_size=16, seed=1)
    _check(api(), case, heads, dim, "nf4", *_fused(rng, case, heads, dim))


def test_prompt_of_several_thousand_tokens():
    rng = np.random.default_rng(5)
    case = Case([2500, 1, 1777], [2500, 900, 1800], page_size=64, seed=2)
    _check(api(), case, 2, 128, "nf4", *_fused(rng, case, 2, 128))


def test_many_sequences():
    """The largest batch: 4096 sequences, every third without rows."""
    n = [0 if b % 3 == 2 else 1 + b % 2 for b in range(4096)]
    case = Case(n, [1 + (7 * b) % 20 + x for b, x in enumerate(n)], page_size=16, pad=1, seed=3)
    rng = np.random.default_rng(6)
    _check(api(), case, 1, 64, "nf4", *_fused(rng, case, 1, 64))


def test_strides_of_head_major_and_expanded_inputs():
    rng = np.random.default_rng(7)
    case = Case([9, 4], [20, 4], seed=4)
    K = inputs(rng, 3, case.tokens, 128).cuda().transpose(0, 1)          # [heads][tokens][channels] in memory
    V = inputs(rng, case.tokens, 1, 128).cuda().expand(-1, 3, -1)        # one value head broadcast: head stride 0
    _check(api(), case, 3, 128, "nf4", K, V)


@pytest.mark.parametrize("exp", [-133, -120, -97, -96, -95, -60, 60, 95, 96, 97, 126])
def test_extreme_magnitudes(exp):
    """Blocks from the smallest subnormals to the largest finite values."""
    rng = np.random.default_rng(200 + exp)
    x = rng.standard_normal((6, 2, 128))
    x /= np.abs(x).reshape(6, 2, 2, 64).max(-1).repeat(64, -1).reshape(6, 2, 128)
    K = torch.from_numpy(np.ldexp(x, exp + 1)).to(torch.float32).to(torch.bfloat16)
    K = torch.where(torch.isfinite(K), K, torch.full_like(K, 3.3895e38) * K.sign()).cuda()
    case = Case([6], [6], seed=5)
    _check(api(), case, 2, 128, "nf4", K, (-K).contiguous())


def test_zero_blocks_and_negative_zero():
    K = torch.zeros(4, 1, 128, dtype=torch.bfloat16)
    K[1] = -0.0
    K[2, 0, 70] = -3.0
    K[3, 0, 0] = 1.0
    case = Case([4], [4], seed=6)
    for codebook in formats.CODEBOOKS:
        _check(api(), case, 1, 128, codebook, K.cuda(), (-K).cuda())


def test_non_finite_blocks_read_back_as_nan_alone():
    a = api()
    rng = np.random.default_rng(8)
    case = Case([3], [3], seed=7)
    K, V = inputs(rng, 3, 2, 128), inputs(rng, 3, 2, 128)
    clean = [t.clone() for t in (K, V)]
    K[0, 1, 5] = float("inf")
    K[1, 0, 127] = float("nan")
    V[2, 1, 64] = float("-inf")
    c = _blank(a, case, 2, 128, "nf4")
    err = a.new_error_word()
    batch = case.batch(a)
    a.qlora_kv_append(c, batch, K.cuda(), V.cuda(), dev_err=err)
    k, v = a.qlora_kv_read(c, batch, 3)
    assert int(err[0]) == a.QLORA_DEVERR_NONFINITE
    a.qlora_kv_append(c, batch, clean[0].cuda(), clean[1].cuda())
    k0, v0 = a.qlora_kv_read(c, batch, 3)
    for got, ref, x in ((k, k0, K), (v, v0, V)):
        hurt = ~torch.isfinite(x.float().reshape(3, 2, 2, 64)).all(-1)
        assert torch.equal(torch.isnan(got.cpu().float().reshape(3, 2, 2, 64)).all(-1), hurt)
        assert torch.equal(torch.isnan(got.cpu().float().reshape(3, 2, 2, 64)).any(-1), hurt)
        keep = ~hurt.repeat_interleave(64, -1).reshape(3, 2, 128)
        assert torch.equal(got.cpu()[keep], ref.cpu()[keep])


def test_entries_out_of_range_are_skipped():
    """Pages, lengths and row offsets that only the device sees: reported, the rest done."""
    a = api()
    rng = np.random.default_rng(9)
    heads, dim = 2, 64
    case = Case([3, 2, 4], [20, 18, 4], seed=8)
    bad = a.QLORA_DEVERR_KV_INDEX
    K, V = _fused(rng, case, heads, dim)
    for change in ("page_high", "page_negative", "kv_len_short"):
        broken = Case([3, 2, 4], [20, 18, 4], seed=8)
        if change == "page_high":
            broken.table[1, 1] = case.num_pages
        elif change == "page_negative":
            broken.table[1, 1] = -1
        else:
            broken.kv_len[1] = 1  # two rows, one cached token: row 0 has position -1
        c = _blank(a, case, heads, dim, "nf4")
        err = a.new_error_word()
        a.qlora_kv_append(c, broken.batch(a), K, V, dev_err=err)
        torch.cuda.synchronize()
        assert int(err[0]) == bad, change
        codes, absmax = kv.encode(bits(K), "nf4")
        want = np.full(tuple(c.k_codes.shape), 0xA5, np.uint8)
        for row, b, p, page, slot in broken.slots():
            if 0 <= page < case.num_pages:
                want[page, :, slot] = codes[row]
        assert np.array_equal(c.k_codes.cpu().numpy(), want), change
        err.zero_()
        out = torch.full((case.tokens, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
        a.qlora_kv_read(c, broken.batch(a), case.tokens, K_out=out, dev_err=err)
        torch.cuda.synchronize()
        assert int(err[0]) == bad, change
    for start, kv_len in (([0, 3, 2, 9], [20, 18, 4]), ([0, 3, 5, 40], [20, 18, 4]), ([-1, 3, 5, 9], [20, 18, 4]),
                          ([0, 3, 5, 9], [20, 10 ** 6, 4]), ([0, 3, 5, 9], [20, -5, 4])):
        broken = Case([3, 2, 4], [20, 18, 4], seed=8)
        broken.start, broken.kv_len = np.array(start, np.int32), kv_len
        c = _blank(a, case, heads, dim, "nf4")
        err = a.new_error_word()
        a.qlora_kv_append(c, broken.batch(a), K, V, dev_err=err)
        a.qlora_kv_read(c, broken.batch(a), case.tokens, dev_err=err)
        torch.cuda.synchronize()
        assert int(err[0]) & bad, (start, kv_len)


def test_pool_larger_than_4_gib():
    """Byte offsets past 32 bits: the sequence's pages lie at the end of a 4.6 GB pool of codes."""
    a = api()
    rng = np.random.default_rng(10)
    heads, dim, page = 8, 128, 64
    pages = 140_000                                  # 32 KiB of codes each
    case = Case([70], [70], page_size=page, seed=9)
    case.table[0, :2] = [pages - 1, pages - 2]
    c = a.alloc_kv_cache(pages, heads, dim, page, "nf4")
    assert c.k_codes.numel() > 1 << 32
    K, V = _fused(rng, case, heads, dim)
    batch = case.batch(a)
    a.qlora_kv_append(c, batch, K, V)
    k, v = a.qlora_kv_read(c, batch, 70)
    for got, x in ((k, K), (v, V)):
        codes, absmax = kv.encode(bits(x), "nf4")
        assert np.array_equal(bits(got), kv.read(codes, absmax, "nf4"))
    codes, _ = kv.encode(bits(K), "nf4")
    assert np.array_equal(c.k_codes[pages - 1].cpu().numpy(), codes[:64].transpose(1, 0, 2))


def test_on_a_side_stream_and_in_a_graph():
    """Captured once, replayed with other inputs and lengths rewritten in place."""
    a = api()
    rng = np.random.default_rng(11)
    heads, dim = 4, 128
    first, second = Case([1, 1, 1], [5, 16, 40], seed=10), Case([1, 1, 1], [6, 17, 41], seed=10)
    second.table = first.table  # room for one more token in the same pages
    c = _blank(a, first, heads, dim, "nf4")
    K, V = (inputs(rng, 3, heads, dim).cuda() for _ in range(2))
    batch = first.batch(a)
    out = [torch.empty(3, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.qlora_kv_append(c, batch, K, V)
        a.qlora_kv_read(c, batch, 3, *out)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.qlora_kv_append(c, batch, K, V)
        a.qlora_kv_read(c, batch, 3, *out)
    for step in range(2):
        K.copy_(inputs(rng, 3, heads, dim))
        V.copy_(inputs(rng, 3, heads, dim))
        batch.kv_len.copy_(torch.tensor([5 + step, 15 + step, 40 + step], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for got, x in zip(out, (K, V)):
            codes, absmax = kv.encode(bits(x), "nf4")
            assert np.array_equal(bits(got), kv.read(codes, absmax, "nf4"))
