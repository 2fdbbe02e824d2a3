"""Host-side refusals of the key/value cache entry points (no GPU needed): every
call here is turned away before the device is touched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def api():
    from bit_nf4_quantised_codebook_b200 import build
    build.build()
    from bit_nf4_quantised_codebook_b200 import api as a
    return a


INVALID, SHAPE, MISALIGNED, WORKSPACE = 1, 2, 3, 5


def _cache(api, pages=4, page=16, heads=2, dim=64, codebook=0, k=4096, ka=8192, v=12288, va=16384):
    return api._KVCache(pages, page, heads, dim, codebook, k, ka, v, va)


def _batch(api, batch=1, max_pages=2, tokens=1, start=32, length=64, table=128):
    return api._KVBatch(batch, max_pages, tokens, start, length, table)


def _append(api, c, b, K=1 << 20, kt=128, kh=64, V=1 << 21, vt=128, vh=64):
    return api.lib().qlora_kv_append(c, b, K, kt, kh, V, vt, vh, None, None)


def _attend(api, c, b, Q=1 << 20, hq=4, qt=256, qh=64, scale=1.0, window=0, out=1 << 22, ws=1 << 23, ws_bytes=1 << 30):
    return api.lib().qlora_kv_attention(c, b, Q, hq, qt, qh, ctypes.c_float(scale), 1, window, out, ws, ws_bytes, None,
                                        None)


@pytest.mark.parametrize("change,status", [
    (dict(pages=0), INVALID), (dict(heads=0), INVALID), (dict(dim=0), INVALID), (dict(page=0), INVALID),
    (dict(codebook=4), INVALID), (dict(codebook=-1), INVALID), (dict(k=0), INVALID), (dict(va=0), INVALID),
    (dict(page=24), SHAPE), (dict(page=8), SHAPE), (dict(page=512), SHAPE), (dict(dim=96), SHAPE),
    (dict(dim=512), SHAPE), (dict(heads=513), SHAPE), (dict(pages=(1 << 30) + 1), SHAPE),
    (dict(k=4100), MISALIGNED), (dict(ka=8194), MISALIGNED)])
def test_cache_refusals(api, change, status):
    c, b = _cache(api, **change), _batch(api)
    assert _append(api, c, b) == status
    assert api.lib().qlora_kv_read(c, b, 1 << 20, 1 << 21, None, None) == status
    assert _attend(api, c, b) == status


@pytest.mark.parametrize("change,status", [
    (dict(batch=0), INVALID), (dict(max_pages=0), INVALID), (dict(tokens=-1), INVALID), (dict(start=0), INVALID),
    (dict(length=0), INVALID), (dict(table=0), INVALID), (dict(batch=4097), SHAPE), (dict(tokens=(1 << 30) + 1), SHAPE),
    (dict(start=34), MISALIGNED), (dict(table=129), MISALIGNED)])
def test_batch_refusals(api, change, status):
    c, b = _cache(api), _batch(api, **change)
    assert _append(api, c, b) == status
    assert api.lib().qlora_kv_read(c, b, 1 << 20, 1 << 21, None, None) == status
    assert _attend(api, c, b) == status


def test_argument_refusals(api):
    c, b = _cache(api), _batch(api)
    assert _append(api, c, b, K=None) == INVALID
    assert _append(api, c, b, V=None) == INVALID
    assert _append(api, c, b, kt=-128) == INVALID
    assert _append(api, c, b, K=(1 << 20) + 8) == MISALIGNED
    assert _append(api, c, b, kt=132) == MISALIGNED
    assert _append(api, c, b, vh=60) == MISALIGNED
    L = api.lib()
    assert L.qlora_kv_read(c, b, None, None, None, None) == INVALID
    assert L.qlora_kv_read(c, b, 8, None, None, None) == MISALIGNED
    assert _attend(api, c, b, Q=None) == INVALID
    assert _attend(api, c, b, out=None) == INVALID
    assert _attend(api, c, b, hq=0) == INVALID
    assert _attend(api, c, b, hq=3) == SHAPE
    assert _attend(api, c, b, hq=258) == SHAPE
    assert _attend(api, c, b, window=-1) == INVALID
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _attend(api, c, b, scale=scale) == INVALID
    assert _attend(api, c, b, out=(1 << 22) + 2) == MISALIGNED
    assert _attend(api, c, b, qt=250) == MISALIGNED
    assert _attend(api, c, b, out=1 << 20) == INVALID               # out over Q
    assert _attend(api, c, b, out=(1 << 20) + 256) == INVALID
    many = _batch(api, tokens=1 << 29)
    assert _attend(api, c, many, hq=8) == SHAPE                     # tokens * q_heads / heads


def test_sizes(api):
    L = api.lib()
    x, y = ctypes.c_size_t(), ctypes.c_size_t()
    assert L.qlora_kv_cache_sizes(10, 64, 8, 128, ctypes.byref(x), ctypes.byref(y)) == 0
    assert (x.value, y.value) == (10 * 64 * 8 * 64, 10 * 64 * 8 * 2 * 2)
    assert L.qlora_kv_cache_sizes(10, 64, 8, 100, None, None) == SHAPE
    n = ctypes.c_size_t()
    c = _cache(api)
    assert L.qlora_kv_attention_workspace_size(c, 1, 1, 4, ctypes.byref(n)) == 0 and n.value > 0
    assert L.qlora_kv_attention_workspace_size(c, 1, 1, 4, None) == INVALID
    assert L.qlora_kv_attention_workspace_size(c, 0, 1, 4, ctypes.byref(n)) == INVALID
    assert L.qlora_kv_attention_workspace_size(c, 4097, 1, 4, ctypes.byref(n)) == SHAPE


def test_python_refusals(api):
    import torch
    with pytest.raises(api.QloraError, match="unsupported shape"):
        api.alloc_kv_cache(4, 2, 96, device="cpu")
    with pytest.raises(api.QloraError, match="k_codes"):                      # not on a GPU
        api.alloc_kv_cache(4, 2, 64, 16, device="cpu")
    with pytest.raises(api.QloraError, match="codebook"):
        api.alloc_kv_cache(4, 2, 64, 16, codebook="nf5", device="cpu")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(api.QloraError, match="page_table"):
        api.KVBatch(i32(3), i32(2), i32(4))
    with pytest.raises(api.QloraError, match="token_start"):
        api.KVBatch(i32(2), i32(2), i32(2, 2))
    with pytest.raises(api.QloraError, match="contiguous channels"):
        api._kv_rows(torch.zeros(4, 2, 128, dtype=torch.bfloat16)[:, :, ::2], 2, 64, "K")
    with pytest.raises(api.QloraError, match="bfloat16"):
        api._kv_rows(torch.zeros(4, 2, 64), 2, 64, "K")
