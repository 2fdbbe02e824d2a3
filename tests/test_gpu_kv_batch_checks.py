"""Batch entries that only the device sees are reported by all three operators of the
key/value cache, also those that no token row of the call leads to."""
import numpy as np
import pytest
import torch

from tests.gpu_util import api
from tests.kv_util import Case, bf16

pytestmark = pytest.mark.gpu

SOUND = ([0, 3, 3, 9], [20, 7, 20])


@pytest.mark.parametrize("start,kv_len", [
    ([0, 5, 3, 9], [20, 18, 20]),       # descends between two sequences that share out all rows
    ([0, 3, 3, 9], [20, 10 ** 6, 20]),  # a length past the table, of a sequence without rows
    ([0, 3, 3, 9], [20, -5, 20]),
    ([0, 9, 9, 12], [20, 7, 20]),       # rows behind the call's
    ([-4, -4, 0, 9], [20, 7, 20])])
def test_every_entry_is_checked(start, kv_len):
    a = api()
    heads, dim = 2, 64
    x = bf16(np.random.default_rng(1).standard_normal((9, heads, dim))).cuda()
    case = Case([3, 0, 6], [20, 7, 20], seed=12)
    cache = a.alloc_kv_cache(case.num_pages, heads, dim, 16, "nf4")
    for sound in (True, False):
        case.start, case.kv_len = (np.array(v) for v in (SOUND if sound else (start, kv_len)))
        batch = case.batch(a)
        for call in (lambda err: a.qlora_kv_append(cache, batch, x, x, dev_err=err),
                     lambda err: a.qlora_kv_read(cache, batch, 9, dev_err=err),
                     lambda err: a.qlora_kv_read(cache, batch, 9, K_out=torch.empty_like(x), dev_err=err),
                     lambda err: a.qlora_kv_attention(cache, batch, x, dev_err=err)):
            err = a.new_error_word()
            call(err)
            torch.cuda.synchronize()
            assert int(err[0]) == (0 if sound else a.QLORA_DEVERR_KV_INDEX)


@pytest.mark.parametrize("wrong", [0, 1, 2500, 4095])
def test_one_wrong_length_of_4096(wrong):
    """More sequences than a CTA has threads; the wrong one has no rows."""
    a = api()
    n = [1] * 4096
    n[wrong] = 0
    case = Case(n, [1] * 4096, page_size=16, seed=13)
    x = bf16(np.zeros((4095, 1, 64))).cuda()
    cache = a.alloc_kv_cache(case.num_pages, 1, 64, 16, "nf4")
    for bad in (False, True):
        case.kv_len[wrong] = -1 if bad else 1
        batch = case.batch(a)
        for call in (lambda err: a.qlora_kv_append(cache, batch, x, x, dev_err=err),
                     lambda err: a.qlora_kv_read(cache, batch, 4095, dev_err=err)):
            err = a.new_error_word()
            call(err)
            torch.cuda.synchronize()
            assert int(err[0]) == (a.QLORA_DEVERR_KV_INDEX if bad else 0)
