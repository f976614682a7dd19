"""The paged cache at the edges of what it is given: evicted pages, scales and scores of extreme size, devices, streams
and workspaces."""
import math

import numpy as np
import pytest
import torch

from test_kv_cache import DT, Setup, assert_attention

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("T,Hq,Hkv,D,S,seq,window", [(5, 8, 2, 128, 16, 700, 100), (1, 4, 4, 64, 16, 333, 33),
                                                     (4, 4, 2, 64, 32, 1203, 300), (150, 4, 2, 128, 16, 411, 70)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_before_the_window_may_be_gone(T, Hq, Hkv, D, S, seq, window, dtype):
    """Pages that no query sees need no place in the table: -1 there is no error.  The first page that one sees does."""
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(300, 2, T, Hq, Hkv, D, S, [seq, seq // 2], [T, T], dtype)
    cache = s.cache()
    s.append(cache)
    s.ref_append()
    want = s.ref_attention(window=window)
    q = s.dev(s.q)
    table, lens, new = s.idx()
    first = [max(0, int(n) + 1 - window) // S for n in s.seq]
    assert min(first) > 0
    for b in range(2):
        table[b, :first[b]] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = sv.spec_kv_attention(q, cache, table, lens, new, window=window, return_lse=True, status=status)
    assert_attention(out, lse, want)
    assert status.item() == 0
    table[0, first[0]] = -1
    out, lse = sv.spec_kv_attention(q, cache, table, lens, new, window=window, return_lse=True, status=status)
    assert status.item() == 8
    assert torch.isnan(out[0, 0]).all() and torch.isnan(lse[0, 0]).all() and torch.isfinite(out[1]).all()
