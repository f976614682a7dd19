"""Integers that the C interface's 32 bits cannot hold, or that are negative, are refused by the binding: passed on, the
lowest 32 bits of -(2**32) + 5 would be read as 5."""
import pytest
import torch

from speculative_sampling_verification_spec_gb300 import SPEC_BF16, SpecError, kv_cache, kv_pages

WRAPS = (-(1 << 32) + 5, -(1 << 31) - 1, -(1 << 31), -1, 1 << 31, (1 << 32) + 4, -(1 << 63), 1 << 64)


class Calls:
    """Stands in for the library: no call may reach it."""

    def __getattr__(self, name):
        raise AssertionError("%s was called" % name)


@pytest.mark.parametrize("name", ["T", "window", "sinks"])
@pytest.mark.parametrize("value", WRAPS)
def test_hold(name, value, monkeypatch):
    monkeypatch.setattr(kv_pages, "_on_device", lambda refs, stream: True)
    monkeypatch.setattr(kv_pages, "_stream_of", lambda stream, device: 0)
    monkeypatch.setattr(kv_pages, "_lib", Calls)
    refs, table, seq = torch.zeros(4, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(SpecError):
        kv_pages.spec_kv_hold(refs, table, seq, page_size=16, **{name: value})


class Cache:
    _index, device, head_dim, kv_heads, _packed = -1, torch.device("cpu"), 64, 1, b""


@pytest.mark.parametrize("name", ["window", "sinks"])
@pytest.mark.parametrize("value", WRAPS)
def test_attention(name, value, monkeypatch):
    monkeypatch.setattr(kv_cache, "_current_device", lambda: -1)
    monkeypatch.setattr(kv_cache, "_first_check", lambda name, t, heads: SPEC_BF16)
    monkeypatch.setattr(kv_cache, "_stream_of", lambda stream, device: 0)
    monkeypatch.setattr(kv_cache, "_lib", Calls)
    q, table, seq = torch.zeros(2, 1, 1, 64), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(SpecError):
        kv_cache.spec_kv_attention(q, Cache, table, seq, **{name: value})


@pytest.mark.gpu
def test_on_the_device():
    """The same through the calls as they are."""
    import speculative_sampling_verification_spec_gb300 as sv
    cache = sv.PagedKVCache.empty(4, 16, 1, 64)
    q = torch.zeros(2, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    refs, table, seq = (torch.zeros(*n, dtype=torch.int32, device="cuda") for n in ((4,), (2, 3), (2,)))
    for value in WRAPS:
        for name in ("T", "window", "sinks"):
            with pytest.raises(sv.SpecError):
                sv.spec_kv_hold(refs, table, seq, page_size=16, **{name: value})
        for name in ("window", "sinks"):
            with pytest.raises(sv.SpecError):
                sv.spec_kv_attention(q, cache, table, seq, **{name: value})
    assert not refs.any() and not table.any()
