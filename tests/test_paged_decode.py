"""The example's decode loop over the paged cache: drafting, scoring in one pass, verification, dropped tokens."""
import os
import sys

import numpy as np
import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_greedy_rounds_emit_the_tokens_of_single_steps(dtype):
    """Greedy speculative decoding emits what the target alone would, one token at a time.  The scales that rejected
    tokens leave behind and the order of sums differ between the two, so a sequence is compared up to its first
    position whose two best logits are closer than the two runs' logits can be apart (0.1; logits are of order 1)."""
    import paged_decode as ex
    B, K, rounds = 5, 3, 12
    a = ex.Target(vocab=97, batch=B, max_tokens=96, dtype=dtype, seed=3)
    first = torch.arange(B, device="cuda", dtype=torch.int32)
    emitted, accepted = ex.decode(a, first, K, rounds, greedy=True)
    b = ex.Target(vocab=97, batch=B, max_tokens=96, dtype=dtype, seed=3)
    last, compared = first, 0
    alive = np.ones(B, bool)
    want = emitted.cpu().numpy()
    for t in range(rounds):
        logits = b(last[:, None], torch.full((B,), t, dtype=torch.int32, device="cuda"))[:, 0]
        top = logits.topk(2, dim=-1).values
        alive &= ((top[:, 0] - top[:, 1]) > 0.1).cpu().numpy()
        last = logits.argmax(-1).to(torch.int32)
        got = last.cpu().numpy()
        assert np.array_equal(got[alive], want[alive, t]), t
        compared += int(alive.sum())
    assert compared >= 2 * B
    assert (accepted >= 0).all() and accepted.float().mean() > 0


def test_sampled_rounds_and_rollback():
    """Sampling: every round emits between 1 and K + 1 tokens, all of the vocabulary, and the same seed the same ones."""
    import paged_decode as ex
    runs = []
    for _ in range(2):
        t = ex.Target(vocab=64, batch=4, max_tokens=80, seed=1)
        runs.append(ex.decode(t, torch.arange(4, device="cuda", dtype=torch.int32), 4, 10, seed=5))
    (tok, acc), (tok2, acc2) = runs
    assert torch.equal(tok, tok2) and torch.equal(acc, acc2)
    assert ((acc >= 0) & (acc <= 4)).all()
    for b in range(4):
        n = int((acc[:, b] + 1).sum())
        row = tok[b].cpu().numpy()
        assert np.all((row[:n] >= 0) & (row[:n] < 64)) and np.all(row[n:] == -1)


def test_the_example_runs():
    import paged_decode as ex
    argv, sys.argv = sys.argv, ["paged_decode.py", "--batch", "3", "--rounds", "4"]
    try:
        ex.main()
    finally:
        sys.argv = argv
