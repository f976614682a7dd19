"""Pages that no query sees, but whose numbers are still in the table, have no influence through their scales either."""
import numpy as np
import pytest
import torch

from test_kv_cache import Setup, assert_attention
from test_kv_sinks import run, sink_attention


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 96), ("f32", 64)])
@pytest.mark.parametrize("sinks", [0, 5])
@pytest.mark.parametrize("T,seq,window", [(1, 700, 33), (3, 1003, 200), (40, 500, 17), (2, 20015, 9100)])
@pytest.mark.parametrize("scale", [2.0 ** 100, 2.0 ** -100, np.nan, np.inf])
def test_scales_before_the_window(dtype, D, sinks, T, seq, window, scale):
    """Every page before the first query's window (behind the sinks) gets this scale, those of its first tile too."""
    S = 16
    s = Setup(1500, 1, T, 4, 2, D, S, [seq], [T], dtype)
    s.append(s.cache())
    s.ref_append()
    want = sink_attention(s, window, sinks)
    first = (seq + 1 - window) // S
    assert first * S % 128                # the window begins inside a tile of 128 tokens
    gone = s.table[0, -(-sinks // S):first]
    s.ks[gone] = s.vs[gone] = scale
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert_attention(*run(s, window, sinks, status=status), want)
    assert status.item() == 0
