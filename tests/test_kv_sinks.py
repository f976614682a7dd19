"""Attention over the paged cache with a window and first tokens that stay visible (sinks), against float64 within a bound
that follows from the roundings."""
import math

import numpy as np
import pytest
import torch

import kv_ref
from test_kv_cache import DT, L, Setup, _pack, assert_attention  # noqa: F401

gpu = pytest.mark.gpu


def sink_attention(s, window, sinks, scale=None):
    """out, lse and their tolerances as kv_ref.attention gives them: a row's sum over its own tokens, max of the scores
    taken off.  The bounds are kv_ref.attention's, with the tokens that the row sees in place of all before it."""
    B, T, Hq, D = s.q.shape
    Hkv, S, U = s.kc.shape[1], s.S, kv_ref.U
    G, scale = Hq // Hkv, 1 / math.sqrt(D) if scale is None else scale
    out, lse = np.zeros((B, T, Hq, D)), np.full((B, T, Hq), -np.inf)
    tol, tol_lse = np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq))
    for b in range(B):
        n, L0 = int(s.new[b]), int(s.seq[b])
        for t in range(n):
            p = L0 + t
            j = np.arange(p + 1)
            j = j[(j > p - window) | (j < sinks)] if window else j
            pages = s.table[b, j // S].astype(np.int64)
            for h in range(Hkv):
                k = kv_ref.CODE_VALUES[s.kc[pages, h, j % S]] * s.ks[pages, h].astype(np.float64)[:, None]
                v = kv_ref.CODE_VALUES[s.vc[pages, h, j % S]] * s.vs[pages, h].astype(np.float64)[:, None]
                x = s.q[b, t, h * G:(h + 1) * G].astype(np.float64)
                a = scale * (x @ k.T)
                m = a.max(axis=1, keepdims=True)
                w = np.exp(a - m)
                l = w.sum(axis=1, keepdims=True)
                at = (b, t, slice(h * G, (h + 1) * G))
                out[at], lse[at] = (w @ v) / l, (m + np.log(l))[:, 0]
                A = abs(scale) * (np.abs(x) @ np.abs(k).T).max(axis=1, keepdims=True)
                e = 2 * ((D + 4) * U * A + 2.0 ** -21) + len(j) * U
                mass = (w @ np.abs(v)) / l
                tol[at] = 2 * e * mass
                if s.dtype == "bf16":
                    e = e + 2 * 2.0 ** -17 * abs(scale) * np.abs(x).max(axis=1, keepdims=True) * np.abs(k).sum(axis=1).max()
                    tol[at] = (2 * e + 2.0 ** -8) * mass + 2.0 ** -17 * np.abs(v).sum(axis=0) / l + 2.0 ** -8 * np.abs(out[at])
                tol_lse[at] = e[:, 0] + 4 * U * np.abs(lse[at])
    return out, lse, tol, tol_lse


def evict(s, window, sinks, hole=-1):
    """Takes the pages that no query sees out of the table and fills them with NaN codes."""
    for b in range(s.B):
        first = max(0, int(s.seq[b]) + 1 - window) // s.S
        for i in range(-(-sinks // s.S), first):
            s.kc[s.table[b, i]], s.vc[s.table[b, i]] = 0x7F, 0x7F
            s.ks[s.table[b, i]], s.vs[s.table[b, i]] = np.nan, np.nan
            s.table[b, i] = hole


def run(s, window, sinks, cache=None, **kw):
    import speculative_sampling_verification_spec_gb300 as sv
    return sv.spec_kv_attention(s.dev(s.q), s.cache() if cache is None else cache, *s.idx(), window=window, sinks=sinks,
                                return_lse=True, **kw)


# --------------------------------------------------------------------------
# refusals (CPU)

def test_refuses(L):  # noqa: F811
    for over, sinks, code in ((dict(window=4), -1, 1), ({}, -1, 1), (dict(window=-1), 4, 1), (dict(T=0), 4, 1),
                              (dict(workspace=0), 4, 1), (dict(q2=-1, window=5), 4, 1), (dict(B=0, window=4), 4, 0),
                              (dict(B=0, window=4), (1 << 31) - 1, 0), (dict(max_pages=1 << 28), 4, 6)):
        c, p = _pack(over)
        assert L.spec_kv_attention_sinks(0x8000, c, p, sinks, 0x9000, None) == code, over
    c, p = _pack(dict(window=4))
    assert L.spec_kv_attention_sinks(None, c, p, 4, 0x9000, None) == 1
    assert L.spec_kv_attention_sinks(0x8000, c, p, 4, None, None) == 1
    assert L.spec_kv_attention_sinks(0x8000, None, p, 4, 0x9000, None) == 1


# --------------------------------------------------------------------------
# values

CASES = [
    # B, T, Hq, Hkv, S, seq, new, window, sinks
    (1, 1, 8, 2, 16, [1000], [1], 100, 4),                        # sinks end inside a page, one tile of them
    (1, 1, 8, 2, 16, [1000], [1], 1, 1),                          # a query that sees itself and the first token
    (3, 5, 8, 2, 16, [0, 3, 700], [5, 2, 5], 64, 4),              # sequences shorter than sinks and window
    (3, 5, 8, 2, 16, [126, 127, 128], [5, 5, 5], 3, 127),         # the window just behind, inside and across the sinks
    (4, 9, 8, 2, 32, [900, 400, 300, 260], [9, 0, 4, 9], 130, 129),   # sinks of more than a tile
    (2, 4, 4, 4, 64, [1500, 800], [4, 4], 256, 300),
    (2, 4, 4, 4, 128, [1500, 800], [4, 4], 37, 128),              # sinks that end with a tile and a page
    (2, 4, 4, 4, 16, [300, 250], [4, 4], 16, 5000),               # sinks beyond every length
    (2, 150, 4, 2, 32, [500, 77], [150, 150], 40, 10),            # row tiles whose windows begin at different tiles
    (1, 300, 6, 1, 16, [0], [300], 16, 2),                        # a prompt from its beginning
    (2, 3, 12, 1, 64, [2000, 1023], [3, 3], 513, 64),
]


@gpu
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 96), ("f32", 64), ("f32", 256)])
@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("hole", [-1, 1 << 30])
def test_against_64_bits(i, dtype, D, hole):
    B, T, Hq, Hkv, S, seq, new, window, sinks = CASES[i]
    s = Setup(500 + i, B, T, Hq, Hkv, D, S, seq, new, dtype)
    s.append(cache := s.cache())
    s.ref_append()
    want = sink_attention(s, window, sinks)
    evict(s, window, sinks, hole)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = run(s, window, sinks, status=status)
    assert_attention(out, lse, want, (i, dtype, D))
    assert status.item() == 0
    # the cache as append left it, with the pages still there: the same bits
    t = Setup(500 + i, B, T, Hq, Hkv, D, S, seq, new, dtype)
    out2, lse2 = run(t, window, sinks, cache=cache)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,seq,window,sinks", [(5, 60000, 20000, 3000), (1, 30000, 64, 20000), (40, 20011, 9000, 700)])
def test_shared_by_many_ranges(dtype, T, seq, window, sinks):
    """One sequence cut into many ranges, some of which hold first tokens only, some both."""
    s = Setup(520, 1, T, 4, 1, 64, 64, [seq], [T], dtype)
    s.append(s.cache())
    s.ref_append()
    want = sink_attention(s, window, sinks)
    evict(s, window, sinks)
    assert_attention(*run(s, window, sinks), want)


@gpu
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_limits_are_the_calls_that_were_there(dtype, D):
    """No sinks, sinks without a window and sinks that fill the gap to the window: the bits of calls without them."""
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(530, 2, 5, 8, 2, D, 16, [900, 90], [5, 5], dtype)
    cache = s.cache()
    s.append(cache)
    q, idx = s.dev(s.q), s.idx()
    full = sv.spec_kv_attention(q, cache, *idx)
    win = sv.spec_kv_attention(q, cache, *idx, window=200)
    assert torch.equal(sv.spec_kv_attention(q, cache, *idx, sinks=4), full)
    assert torch.equal(sv.spec_kv_attention(q, cache, *idx, window=200, sinks=0), win)
    assert torch.equal(sv.spec_kv_attention(q, cache, *idx, window=(1 << 31) - 1, sinks=4), full)
    assert torch.equal(sv.spec_kv_attention(q, cache, *idx, window=1, sinks=(1 << 31) - 1), full)
    assert not torch.equal(sv.spec_kv_attention(q, cache, *idx, window=200, sinks=4), win)
    for kw in (dict(sinks=-1), dict(window=200, sinks=1 << 31), dict(window=200, sinks=(1 << 32) + 4), dict(window=1 << 32)):
        with pytest.raises(sv.SpecError):
            sv.spec_kv_attention(q, cache, *idx, **kw)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_tokens_touch_the_rows_that_see_them(dtype):
    """A NaN key or value among the sinks makes every row NaN; one just behind them, beside them in their page, and one
    before the first row's window but in its page touch none."""
    import speculative_sampling_verification_spec_gb300 as sv
    B, T, S, window, sinks = 1, 3, 16, 33, 5
    for at, seen in ((4, [0, 1, 2]), (5, []), (15, []), (700 - 33, []), (700 - 32, [0]), (700 - 31, [0, 1])):
        for kind in ("k", "v"):
            s = Setup(540, B, T, 4, 2, 64, S, [700], [T], dtype)
            s.append(s.cache())
            s.ref_append()
            getattr(s, kind + "c")[s.table[0, at // S], 1, at % S, 7] = 0x7F
            evict(s, window, sinks)
            out, _ = sv.spec_kv_attention(s.dev(s.q), s.cache(), *s.idx(), window=window, sinks=sinks, return_lse=True)
            nan = torch.isnan(out).cpu().numpy()
            rows = np.array([t in seen for t in range(T)])
            assert np.array_equal(nan[0, :, 2:].any(axis=(1, 2)), rows), (at, kind)
            assert not nan[0, :, :2].any(), (at, kind)


@gpu
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f32", 128)])
@pytest.mark.parametrize("S", [16, 128])
def test_missing_pages(dtype, D, S):
    """A page of the sinks or of the window that is not the pool's is an error; one between is none."""
    for column, bad in ((0, True), (20 // S, True), (20 // S + 1, False), (600 // S - 1, False), (601 // S, True)):
        s = Setup(550, 2, 2, 4, 2, D, S, [700, 700], [2, 2], dtype)
        cache = s.cache()
        s.append(cache)
        s.table[0, column] = 1 << 20
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = run(s, 100, 20, cache=cache, status=status)
        assert status.item() == (8 if bad else 0), column
        assert torch.isnan(out[0, 0]).all().item() is bad and torch.isnan(lse[0, 0]).all().item() is bad, column
        assert torch.isfinite(out[1]).all(), column


@gpu
def test_graph_stream_and_strides():
    """Captured on a side stream and replayed with other contents; queries and outputs of another layout; each against
    the call made outright."""
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(560, 3, 4, 8, 2, 128, 16, [900, 30, 400], [4, 4, 2], "bf16")
    cache = s.cache()
    s.append(cache)
    q, idx = s.dev(s.q), s.idx()
    want, want_lse = sv.spec_kv_attention(q, cache, *idx, window=100, sinks=6, return_lse=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sv.spec_kv_attention(q, cache, *idx, window=100, sinks=6, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    qt = q.permute(1, 2, 0, 3).contiguous().permute(2, 0, 1, 3)
    out = torch.full((8, 3, 4, 128), 9.0, dtype=torch.bfloat16, device="cuda").permute(1, 2, 0, 3)
    sv.spec_kv_attention(qt, cache, *idx, window=100, sinks=6, out=out)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    lse = torch.zeros_like(want_lse)
    with torch.cuda.graph(graph):
        sv.spec_kv_attention(q, cache, *idx, window=100, sinks=6, out=out, lse=lse)
    for shift in (0, 3):
        idx[1].copy_(torch.tensor([900 - shift, 30, 400], dtype=torch.int32))
        graph.replay()
        w, wl = sv.spec_kv_attention(q, cache, *idx, window=100, sinks=6, return_lse=True)
        assert torch.equal(out, w) and torch.equal(lse, wl)
