"""What the Python entry points of the key/value cache hand to the C ABI, and what they
turn away (no GPU needed: the library is replaced by one that records its calls)."""
from types import SimpleNamespace

import pytest
import torch


class _Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def kv(monkeypatch):
    """The module with a recording library, and a cache and a batch on the CPU (device -1)."""
    from bit_nf4_quantised_codebook_b200 import api
    library = _Library()
    monkeypatch.setattr(api, "lib", lambda: library)
    monkeypatch.setattr(api, "_kv_stream", lambda device: 0)
    cache = SimpleNamespace(_c="cache", _device=-1, heads=2, head_dim=64)
    batch = SimpleNamespace(batch=1, _device=-1, c_struct=lambda tokens: ("batch", tokens))
    return SimpleNamespace(api=api, library=library, cache=cache, batch=batch,
                           Q=torch.zeros(3, 4, 64, dtype=torch.bfloat16), out=torch.zeros(3, 4, 64, dtype=torch.bfloat16),
                           ws=torch.zeros(4096, dtype=torch.uint8))


def _attention_args(kv, monkeypatch, **change):
    monkeypatch.setattr(kv.api, "_need", lambda *a: None)  # (refuses what is not on a GPU)
    kv.api.qlora_kv_attention(kv.cache, kv.batch, kv.Q, out=kv.out, ws=kv.ws, **change)
    (name, args), = kv.library.calls
    assert name == "qlora_kv_attention"
    names = ["cache", "batch", "Q", "q_heads", "token_stride", "head_stride", "scale", "causal", "window", "out", "ws",
             "ws_bytes", "dev_err", "stream"]
    return dict(zip(names, args))


@pytest.mark.parametrize("window,passed", [(0, 0), (5, 5), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                                           (2 ** 32 + 5, 2 ** 31 - 1), (2 ** 63, 2 ** 31 - 1), (-1, -1), (-2 ** 32 + 3, -1)])
def test_window_reaches_the_library_as_an_int(kv, monkeypatch, window, passed):
    """Longer than an int holds is longer than any cache; negative stays negative (and is refused there)."""
    assert _attention_args(kv, monkeypatch, window=window)["window"] == passed


@pytest.mark.parametrize("causal,passed", [(True, True), (False, False), (2 ** 32, True)])
def test_causal_is_a_truth_value(kv, monkeypatch, causal, passed):
    assert _attention_args(kv, monkeypatch, causal=causal)["causal"] is passed


def test_workspace_of_sizes_past_an_int_is_refused():
    from bit_nf4_quantised_codebook_b200 import api, build
    build.build()
    cache = SimpleNamespace(_c=api._KVCache(4, 16, 2, 64, 0, 4096, 8192, 12288, 16384))
    assert api.qlora_kv_attention_workspace_size(cache, 1, 1, 4) > 0
    for batch, q_heads in ((2 ** 32 + 1, 4), (1, 2 ** 32 + 4), (1 - 2 ** 32, 4)):
        with pytest.raises(api.QloraError):
            api.qlora_kv_attention_workspace_size(cache, batch, 1, q_heads)


def _error_words():
    whole = torch.zeros(8, dtype=torch.uint8)
    return [torch.zeros(4, dtype=torch.int64), whole[1:5], torch.zeros(0, dtype=torch.int32),
            torch.zeros(4, dtype=torch.float32)]


@pytest.mark.parametrize("which", range(4))
def test_error_word_of_another_type_is_refused(kv, monkeypatch, which):
    """Kernels add bits to one int32: anything else would be written beside, or at no multiple of four bytes."""
    monkeypatch.setattr(kv.api, "_need", lambda *a: None)
    wrong, api = _error_words()[which], kv.api
    K = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: api.qlora_kv_append(kv.cache, kv.batch, K, K, dev_err=wrong),
                 lambda: api.qlora_kv_read(kv.cache, kv.batch, 3, K_out=K, dev_err=wrong),
                 lambda: api.qlora_kv_attention(kv.cache, kv.batch, kv.Q, out=kv.out, ws=kv.ws, dev_err=wrong)):
        with pytest.raises(api.QloraError, match="dev_err"):
            call()
    assert kv.library.calls == []


def test_workspace_without_memory_of_its_own_is_refused(kv, monkeypatch):
    """An expanded or strided tensor counts bytes that it does not have side by side."""
    monkeypatch.setattr(kv.api, "_need", lambda *a: None)
    for wrong in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), kv.ws[::2]):
        with pytest.raises(kv.api.QloraError, match="ws"):
            kv.api.qlora_kv_attention(kv.cache, kv.batch, kv.Q, out=kv.out, ws=wrong)
    assert kv.library.calls == []


def test_sound_scratch_passes(kv, monkeypatch):
    word = torch.zeros(4, dtype=torch.int32)
    args = _attention_args(kv, monkeypatch, dev_err=word)
    assert (args["dev_err"], args["ws"], args["ws_bytes"]) == (word.data_ptr(), kv.ws.data_ptr(), 4096)


@pytest.mark.parametrize("apart,fits", [(0, False), (16, False), (3 * 2 * 64 * 2 - 16, False), (3 * 2 * 64 * 2, True)])
def test_read_outputs_that_overlap_are_refused(apart, fits):
    """Keys and values written to the same memory would be a mixture of both (the call is turned away, or
    goes on to the check of the device)."""
    from bit_nf4_quantised_codebook_b200 import api, build
    build.build()
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: for machines without a GPU")
    c = api._KVCache(4, 16, 2, 64, 0, 4096, 8192, 12288, 16384)
    b = api._KVBatch(1, 2, 3, 32, 64, 128)
    for k, v in ((1 << 20, (1 << 20) + apart), ((1 << 20) + apart, 1 << 20)):
        status = api.lib().qlora_kv_read(c, b, k, v, None, None)
        assert (status != 1) is fits
    assert api.lib().qlora_kv_read(c, b, 1 << 20, None, None, None) != 1
