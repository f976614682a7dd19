"""The operators of long streams as they are used together: pages held, norms and append, attention with a window and sinks,
forks, round after round with the lengths on the device."""
import os
import sys
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import kv_ref
from conftest import ROOT
from test_kv_cache import DT, assert_attention
from test_kv_norm import EPS, normalise, weights
from test_kv_pages import dev, ref_fork, ref_hold, same
from test_kv_sinks import sink_attention

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.parametrize("dtype,D,S", [("bf16", 64, 16), ("bf16", 128, 32), ("f32", 64, 16)])
def test_rounds(dtype, D, S):
    """Every round on the device: hold, append with norms, attention, what verification leaves, and now and then forks;
    against the same steps in numpy: tables, counts, codes and scales equal, attention within its bounds.  The pool has no
    page more than it needs and is never cleared, so what was released is used again with what it held."""
    import speculative_sampling_verification_spec_gb300 as sv
    g = np.random.default_rng(800 + D + S)
    B, T, Hq, Hkv, P, window, sinks, rounds = 4, 5, 4, 2, 160 // S, 40, 5, 60
    each = -(-sinks // S) + (window + T - 2) // S + 2
    N = B * each
    f = np.float32
    refs, table, seq = np.zeros(N, np.int32), np.full((B, P), -1, np.int32), np.zeros(B, np.int32)
    kc, vc = (np.full((N, Hkv, S, D), 0x7F, np.uint8) for _ in range(2))
    ks, vs = (np.full((N, Hkv), np.nan, f) for _ in range(2))
    ang = np.arange(P * S)[:, None] * 10000.0 ** (-np.arange(D // 2) / (D // 2))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(f)
    qw, kw = weights(g, D), weights(g, D)
    cache = sv.PagedKVCache(dev(kc), dev(vc), dev(ks), dev(vs))
    d = dict(refs=dev(refs), table=dev(table), seq=dev(seq), cs=dev(cs), qw=dev(qw), kw=dev(kw))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def values(*shape):
        x = g.standard_normal(shape).astype(f) * f(2)
        return kv_ref.bf16_round(x) if dtype == "bf16" else x

    for step in range(rounds):
        new = g.integers(0, T + 1, B).astype(np.int32)
        new = np.minimum(new, P * S - seq).astype(np.int32)
        q, k, v = values(B, T, Hq, D), values(B, T, Hkv, D), values(B, T, Hkv, D)
        kept = np.array([g.integers(0, n + 1) for n in new], np.int32)
        parents = np.full(B, -1, np.int32)
        if step % 4 == 3:
            parents[g.integers(1, B)] = 0

        # the device's round
        t = [dev(x).to(DT[dtype]) for x in (q, k, v)]
        n = dev(new)
        sv.spec_kv_hold(d["refs"], d["table"], d["seq"], n, page_size=S, window=window, sinks=sinks, status=status)
        qr = sv.spec_kv_append(*t, cache, d["table"], d["seq"], n, cos_sin=d["cs"], q_norm=d["qw"], k_norm=d["kw"],
                               norm_eps=EPS, status=status)
        out, lse = sv.spec_kv_attention(qr, cache, d["table"], d["seq"], n, window=window, sinks=sinks, return_lse=True,
                                        status=status)
        d["seq"] += dev(kept)
        sv.spec_kv_hold(d["refs"], d["table"], d["seq"], page_size=S, window=window, sinks=sinks, status=status)
        sv.spec_kv_fork(cache, d["refs"], d["table"], d["seq"], dev(parents), status=status)

        # the same in numpy
        assert ref_hold(refs, table, seq, new, S, window, sinks)[1] == 0
        with np.errstate(invalid="ignore"):
            qn = kv_ref.append(normalise(q, qw, EPS), normalise(k, kw, EPS), v, kc, vc, ks, vs, table, seq, new, cs, D, False,
                               dtype, S)
        assert np.array_equal(qr.float().cpu().numpy(), qn), step
        want = sink_attention(SimpleNamespace(q=qn, kc=kc, vc=vc, ks=ks, vs=vs, table=table, seq=seq, new=new, S=S,
                                              dtype=dtype), window, sinks)
        assert_attention(out, lse, want, step)
        seq = seq + kept
        assert ref_hold(refs, table, seq, np.zeros(B), S, window, sinks)[1] == 0
        assert ref_fork(refs, table, seq, parents, S, [kc, ks, vc, vs])[1] == 0
        same(d["table"], table)
        same(d["refs"], refs)
        same(d["seq"], seq)
        for got, ref in ((cache.k_codes, kc), (cache.v_codes, vc)):
            a, b = got.cpu().numpy() & 0x7F, ref & 0x7F
            assert np.array_equal(a, b) and np.array_equal((got.cpu().numpy() ^ ref)[a != 0x7F] & 0x80, 0 * a[a != 0x7F]), step
        assert np.array_equal(cache.k_scale.cpu().numpy(), ks, equal_nan=True)
        assert np.array_equal(cache.v_scale.cpu().numpy(), vs, equal_nan=True)
    assert status.item() == 0 and seq.max() > window + sinks


def test_the_round_replays_from_a_graph():
    """A round captured once and replayed while the lengths grow gives what the calls give outright."""
    import speculative_sampling_verification_spec_gb300 as sv
    B, T, D, S, P, N, window, sinks = 3, 4, 64, 16, 12, 20, 48, 4
    g = torch.Generator(device="cuda").manual_seed(9)
    x = [torch.randn(B, T, h, D, generator=g, device="cuda").to(torch.bfloat16) for h in (4, 2, 2)]
    w = torch.ones(D, device="cuda")
    runs = []
    for graphed in (False, True):
        cache = sv.PagedKVCache.empty(N, S, 2, D)
        refs, table = torch.zeros(N, dtype=torch.int32, device="cuda"), torch.full((B, P), -1, dtype=torch.int32, device="cuda")
        seq, out = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, T, 4, D, dtype=torch.bfloat16, device="cuda")

        def once():
            sv.spec_kv_hold(refs, table, seq, T=T, page_size=S, window=window, sinks=sinks)
            q = sv.spec_kv_append(*x, cache, table, seq, q_norm=w, k_norm=w)
            sv.spec_kv_attention(q, cache, table, seq, window=window, sinks=sinks, out=out)
            seq.add_(3)
        if graphed:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                once()
        got = []
        for _ in range(40):
            graph.replay() if graphed else once()
            got.append(out.clone())
        runs.append((torch.stack(got), table.clone(), refs.clone(), cache.k_codes.view(torch.uint8).clone()))
    assert torch.isfinite(runs[0][0]).all()
    for a, b in zip(*runs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_example_with_a_window(dtype):
    """Greedy rounds with a window over a small pool emit the tokens of single steps (compared up to a sequence's first
    position whose two best logits are closer than the two runs' logits can be apart; see test_paged_decode)."""
    import paged_decode as ex
    B, K, rounds = 4, 3, 30
    args = dict(vocab=97, batch=B, max_tokens=160, dtype=dtype, seed=3, window=24, sinks=3)
    a = ex.Target(new_tokens=K + 1, **args)
    assert a.refs.numel() < B * 160 // 16
    first = torch.arange(B, device="cuda", dtype=torch.int32)
    emitted, accepted = ex.decode(a, first, K, rounds, greedy=True)
    b = ex.Target(new_tokens=1, **args)
    last, compared = first, 0
    alive = np.ones(B, bool)
    want = emitted.cpu().numpy()
    for t in range(rounds):
        logits = b(last[:, None], torch.full((B,), t, dtype=torch.int32, device="cuda"))[:, 0]
        top = logits.topk(2, dim=-1).values
        alive &= ((top[:, 0] - top[:, 1]) > 0.1).cpu().numpy()
        last = logits.argmax(-1).to(torch.int32)
        assert np.array_equal(last.cpu().numpy()[alive], want[alive, t]), t
        compared += int(alive.sum())
    assert compared >= 2 * B
    argv, sys.argv = sys.argv, ["paged_decode.py", "--batch", "3", "--rounds", "8", "--window", "16", "--sinks", "2"]
    try:
        ex.main()
    finally:
        sys.argv = argv
