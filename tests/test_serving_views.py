"""Views that the operators around the KV cache accept and refuse, on the CPU: a
refused call enqueues nothing, so it needs no GPU."""
import ctypes

import pytest
import torch

from lossless_bf16_kv_gb300 import _build, serving
from lossless_bf16_kv_gb300 import splitzip as sz

FAKE = 1 << 20   # aligned, never dereferenced: every call below is refused


@pytest.fixture(scope="module")
def lib():
    _build.build_library()
    return serving.library()


def test_cache_rows_between_sequences():
    kv = torch.empty((3, 2, 40, 2, 64), dtype=torch.bfloat16)
    assert serving._cache_rows(kv[:, 0], "k") == (200, 128, 64, 80)          # the values lie between
    assert serving._cache_rows(kv[:1, 0], "k") == (40, 128, 64, 0)           # one sequence
    assert serving._cache_rows(kv[0], "k") == (80, 128, 64, 0)               # sequences without gaps
    assert serving._cache_rows(kv[0, 0], "k") == (40, 128, 64, 0)
    heads_first = torch.empty((3, 2, 40, 64), dtype=torch.bfloat16).transpose(1, 2)
    assert serving._cache_rows(heads_first, "k") == (200, 64, 2560, 80)


@pytest.mark.parametrize("kw", [dict(cache_step=40, cache_tokens=41), dict(cache_step=40, cache_tokens=40, cache_rows=(1 << 32) + 1)])
def test_norm_rope_refuses_sequences_that_do_not_fit(lib, kw):
    view = (FAKE, 0, 1024, 128)
    a = serving.NormRopeArgs(view, view, view, None, None, FAKE, FAKE, FAKE, view, view, view, 10, 10, 5, 8, 2, 128, 128,
                             0, 0, 1e-6)
    for k, v in kw.items():
        setattr(a, k, v)
    assert lib.splitzip_qk_norm_rope(ctypes.byref(a), None) == sz.ERR_INVALID_ARG


def test_norm_rope_refuses_caches_that_a_slot_addresses_differently(monkeypatch):
    """The binding's own check, in front of the library (which is never reached: the
    tensors are on the CPU and only said to be elsewhere)."""
    bf = lambda *shape: torch.empty(shape, dtype=torch.bfloat16)  # noqa: E731
    whole = bf(2, 40, 2, 64)
    pairs = [(whole, bf(2, 48, 2, 64)[:, :40]), (bf(2, 48, 2, 64)[:, :40], whole),      # 40 and 48 tokens apart
             (whole, bf(4, 20, 2, 64)), (bf(2, 2, 40, 2, 64)[:, 0], bf(2, 2, 40, 2, 64)[:, 0, :39]),
             (bf(2, 48, 2, 64)[:, :40], bf(88, 2, 64)), (bf(88, 2, 64), bf(2, 48, 2, 64)[:, :40])]
    fine = [(whole, bf(2, 40, 2, 64)), (whole, bf(80, 2, 64)), (bf(2, 2, 40, 2, 64)[:, 0], bf(2, 2, 40, 2, 64)[:, 1]),
            (bf(2, 2, 40, 64).transpose(1, 2), bf(2, 80, 2, 64)[:, :40]), (bf(1, 40, 2, 64), bf(50, 2, 64))]
    reached = []
    monkeypatch.setattr(serving, "_fn_norm_rope", lambda a, s: reached.append(a) or 0)
    monkeypatch.setattr(serving, "_stream_of", lambda s: 0)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    x, y, slots = bf(3, 4, 64), bf(3, 2, 64), torch.arange(3)
    for i, (k, v) in enumerate(pairs):
        with pytest.raises(sz.SplitZipError) as err:
            serving.splitzip_qk_norm_rope(x, y, y, None, None, None, None, slots, x, k, v)
        assert err.value.status == sz.ERR_INVALID_ARG and not reached, i
    for k, v in fine:
        serving.splitzip_qk_norm_rope(x, y, y, None, None, None, None, slots, x, k, v)
    assert len(reached) == len(fine)


def test_outputs_are_not_shared_by_a_batch(lib):
    """A batch stride of 0 is one sequence for the whole batch: an input's only."""
    view, shared = (FAKE, 1 << 16, 1 << 10, 128), (FAKE, 0, 1 << 10, 128)
    a = serving.AttentionArgs(view, view, view, shared, None, None, 2, 3, 64, 8, 2, 128, 0, 0, 0, 1.0)
    need = lib.splitzip_attention_workspace_bytes(ctypes.byref(a))
    assert need and lib.splitzip_attention(ctypes.byref(a), FAKE, need, None) == sz.ERR_INVALID_ARG
    for kw in (dict(k_out=shared), dict(v_out=shared)):
        a = serving.EvictArgs(view, view, view, view, FAKE, None, FAKE, None, None, 2, 64, 2, 128, 8, 2, 2, 0)
        for k, v in kw.items():
            setattr(a, k, v)
        assert lib.splitzip_evict(ctypes.byref(a), None) == sz.ERR_INVALID_ARG


def test_attention_refuses_tokens_whose_tiles_pass_32_bits(lib):
    """From 2^31 - 255 slots on the end of the last tile of slots is no signed 32-bit
    number: the few-row kernel took such a tile for one inside the cache, and read
    past it."""
    view, inv = (FAKE, 0, 128, 1 << 20), sz.ERR_INVALID_ARG
    for kw in (dict(kv_tokens=(1 << 31) - 1), dict(kv_tokens=(1 << 31) - 255), dict(q_tokens=(1 << 31) - 255),
               dict(q_tokens=(1 << 30) - 127, q_heads=2)):
        a = serving.AttentionArgs(view, view, view, view, FAKE, None, 1, 1, 64, 1, 1, 64, 0, 0, 1, 1.0)
        for k, v in kw.items():
            setattr(a, k, v)
        assert lib.splitzip_attention_workspace_bytes(ctypes.byref(a)) == 0
        assert lib.splitzip_attention(ctypes.byref(a), FAKE, 1 << 40, None) == inv
        assert lib.splitzip_attention_weights(ctypes.byref(a), None, FAKE, None) == inv
        a.kv_tokens, a.q_tokens = min(a.kv_tokens, (1 << 31) - 256), min(a.q_tokens, ((1 << 31) - 256) // a.q_heads)
        assert lib.splitzip_attention_workspace_bytes(ctypes.byref(a)) > 0


def test_status_refuses_what_is_no_workspace(lib, monkeypatch):
    """The status is a word of the workspace's header: a shorter tensor has none, and
    the word behind it is someone else's."""
    q = torch.empty((1, 1, 1, 64), dtype=torch.bfloat16)
    least = serving.splitzip_attention_workspace_bytes(q, q)
    assert least == serving._HEADER
    reached = []
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    monkeypatch.setattr(serving, "_stream_of", lambda s: 0)
    monkeypatch.setattr(lib, "splitzip_attention_status", lambda w, s: reached.append(w) or 0)
    for n in (0, 16, least - 1):
        with pytest.raises(sz.SplitZipError) as err:
            serving.splitzip_attention_status(torch.zeros(n, dtype=torch.uint8))
        assert err.value.status == sz.ERR_INVALID_ARG and not reached
    assert serving.splitzip_attention_status(torch.zeros(least, dtype=torch.uint8)) == 0 and len(reached) == 1
