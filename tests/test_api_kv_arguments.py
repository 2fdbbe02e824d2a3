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
