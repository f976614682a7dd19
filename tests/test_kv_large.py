"""The kernel variants that only large calls select: several heads a query thread and several units a group in the append,
CTAs of 1024 threads and second passes over table and pool in holding and forking.

Appending: the bits of a large call equal those of one call for each sequence (which take one head a thread and one unit a
group, forms that other tests hold against the definition), and rows of it equal the definition's.  Pages: equal to the
restatement in numpy, round after round."""
import numpy as np
import pytest
import torch

import kv_ref
from test_kv_norm import EPS, normalise
from test_kv_pages import FULL, RANGE, Forks, Pool

gpu = pytest.mark.gpu
SMS = 152

# --------------------------------------------------------------------------
# append

APPEND = [
    # B, T, Hq, Hkv, D, S, dtype, rot, interleaved, norms ("q", "k", "qk", ""), weights a head
    (8, 2500, 32, 8, 128, 32, "bf16", 128, False, "qk", False),
    (8, 2500, 32, 8, 128, 32, "bf16", 128, False, "qk", True),
    (8, 2500, 32, 8, 128, 64, "bf16", 128, True, "q", True),
    (8, 2500, 32, 8, 128, 64, "bf16", 64, False, "k", True),
    (8, 2500, 32, 8, 128, 128, "bf16", 128, False, "", False),
    (9, 2300, 32, 4, 96, 32, "bf16", 96, False, "qk", True),        # six chunks a head: idle lanes
    (9, 2300, 32, 4, 80, 64, "bf16", 80, False, "k", False),        # five; queries pass as they are
    (9, 2300, 64, 4, 64, 16, "f32", 64, False, "qk", True),
    (6, 420, 32, 2, 128, 32, "bf16", 10, False, "", False),         # single pairs of channels, four heads a thread
    (6, 420, 32, 2, 128, 32, "bf16", 10, True, "k", True),          # with a norm of the keys alone
    (6, 420, 32, 2, 128, 16, "bf16", 10, False, "qk", True),        # a head of a query a warp
    (300, 17, 32, 8, 128, 16, "bf16", 128, False, "qk", True),      # short pieces of many sequences
]


def per_token(D, rot, norms):
    """Threads of a token's head."""
    chunks = D // 16 if rot % 16 == 0 else D // 2
    return 1 << (chunks - 1).bit_length() if norms and rot % 16 == 0 else chunks


def test_the_cases_are_large():
    """More than one head a query thread: from 4 * 4 * 152 * 2048 threads' work on (a head of a query is a warp's where
    single channels are normalised; the last case is of many groups instead)."""
    for B, T, Hq, Hkv, D, S, dtype, rot, inter, norms, per_head in APPEND[:-1]:
        assert Hq % 4 == 0 and B * T * Hq * per_token(D, rot, norms) >= 16 * SMS * 2048, (B, T, Hq, D)


@gpu
@pytest.mark.parametrize("i", range(len(APPEND)))
def test_large_appends(i):
    import speculative_sampling_verification_spec_gb300 as sv
    B, T, Hq, Hkv, D, S, dtype, rot, inter, norms, per_head = APPEND[i]
    g = torch.Generator(device="cuda").manual_seed(900 + i)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def values(H):
        return torch.randn(B, T, H, D, generator=g, device="cuda").mul_(2).to(dt)

    q, k, v = values(Hq), values(Hkv), values(Hkv)
    rng = np.random.default_rng(900 + i)
    seq = rng.integers(0, 3 * S, B).astype(np.int32)
    new = rng.integers(0, T + 1, B).astype(np.int32)
    new[0], new[1], seq[0] = T, 0, 0
    P = -(-(3 * S + T) // S)
    bad = B - 2                                  # a sequence that is out of range
    table = torch.from_numpy(rng.permutation(B * P).astype(np.int32).reshape(B, P)).cuda()
    at, n = torch.from_numpy(seq).cuda(), torch.from_numpy(new).cuda()
    at[bad] = P * S - int(new[bad]) + 1
    ang = np.arange(P * S)[:, None] * (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2)))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)
    w = {x: 1 + 0.3 * torch.randn(*((h, D) if per_head else (D,)), generator=g, device="cuda")
         for x, h in (("q", Hq), ("k", Hkv)) if x in norms}
    args = dict(cos_sin=torch.from_numpy(cs).cuda(), interleaved=inter, q_norm=w.get("q"), k_norm=w.get("k"), norm_eps=EPS)
    # pages hold earlier tokens, at scales below and above what the new ones need
    pools = [torch.randint(0, 0x70, (B * P, Hkv, S, D), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
    scales = [torch.randint(-9, -3, (B * P, Hkv), generator=g, device="cuda").float().exp2() for _ in range(2)]
    one, each = (sv.PagedKVCache(*[t.clone() for t in pools + scales]) for _ in range(2))
    status, other = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    out = sv.spec_kv_append(q, k, v, one, table, at, n, status=status, **args)
    for b in range(B):
        c = slice(b, b + 1)
        got = sv.spec_kv_append(q[c], k[c], v[c], each, table[c], at[c], n[c], status=other, **args)
        assert torch.equal(out[c].view(torch.uint8), got.view(torch.uint8)), b
    for x in ("k_codes", "v_codes"):
        assert torch.equal(getattr(one, x), getattr(each, x)), x
    for x in ("k_scale", "v_scale"):
        assert torch.equal(getattr(one, x), getattr(each, x)), x
    assert status.item() == other.item() == RANGE
    assert torch.isnan(out[bad]).all() and (out[1] == 0).all() and (out[0] != 0).any()
    # rows of queries against the definition
    for b in rng.choice([b for b in range(B) if b != bad and new[b]], 4):
        for t in rng.integers(0, new[b], 3):
            x = q[b, t].float().cpu().numpy()
            if "q" in norms:
                x = normalise(x, w["q"].cpu().numpy(), EPS)
            y = kv_ref.rotate(x, cs[seq[b] + t], rot, inter)
            y = kv_ref.bf16_round(y) if dtype == "bf16" else y
            assert np.array_equal(out[b, t].float().cpu().numpy(), y), (b, t)


# --------------------------------------------------------------------------
# pages

def words(B, P, N):
    """What decides between CTAs of 256 and of 1024 threads (more than 4096)."""
    return (B * P + N) // 32


HOLD = [
    # B, P, S, N, window, sinks, longest, T, more than 4096 words
    (150, 100, 16, 100001, 0, 0, 1500, 90, False),          # more than 65536 pages: a second pass over the pool
    (150, 130, 16, 70003, 400, 20, 2000, 40, False),        # wide rows, the next stretch under way
    (1200, 120, 16, 100000, 0, 0, 1700, 60, True),
    (1200, 128, 16, 300007, 200, 4, 2000, 33, True),        # more than 262144 pages
    (256, 1537, 16, 100000, 4000, 70, 24000, 17, True),     # wide rows
    (160, 700, 128, 120001, 0, 0, 80000, 9000, True),
    (100, 100, 16, 131072 + 31 - 10000, 0, 0, 1500, 90, False),     # the last size with few threads
    (100, 100, 16, 131072 + 32 - 10000, 0, 0, 1500, 90, True),      # and the first with many
    (100, 200, 16, 131072 + 31 - 20000, 500, 3, 3000, 90, False),
    (100, 200, 16, 131072 + 32 - 20000, 500, 3, 3000, 90, True),
]


def test_holds_and_forks_are_on_both_sides():
    for B, P, S, N, window, sinks, longest, T, many in HOLD:
        assert (words(B, P, N) > 4096) is many
    for B, P, S, N, many in FORK:
        assert (words(B, P, N) > 4096) is many


@gpu
@pytest.mark.parametrize("i", range(len(HOLD)))
def test_large_holds(i):
    B, P, S, N, window, sinks, longest, T, many = HOLD[i]
    g = np.random.default_rng(1700 + i)
    seq = g.integers(0, longest - T + 1, B)
    p = Pool(1700 + i, B, P, S, N, seq, window, sinks, shared=2)
    for step in range(3):
        assert p.hold(seq, g.integers(0, T + 1, B), window, sinks) == 0
        seq = np.where(g.random(B) < 0.2, 0, np.clip(seq + g.integers(-T, T + 1, B), 0, longest - T))
    assert p.hold(np.zeros(B), np.zeros(B), window, sinks) == 0
    assert (p.table == -1).all() and (p.refs == 0).all()


@gpu
@pytest.mark.parametrize("B,P", [(1200, 120), (300, 500)])
def test_large_hold_runs_out_and_has_bad_rows(B, P):
    p = Pool(1720, B, P, 16, B * 4 + 3, [40] * B)
    p.refs[7] += 1                                  # a count of the caller's own
    assert words(B, P, p.N) > 4096
    seq = [40] * B
    assert p.hold(seq, [40] * B) == FULL and (p.table[-1, 3:5] < 0).all()
    assert p.hold(seq, [0] * B) == 0                # released again
    p.table[5, 1], p.table[B - 1, P - 1] = p.N, 1 << 30
    seq[9] = P * 16 + 1
    before = p.table[9].copy()
    assert p.hold(seq, [0] * B) == RANGE
    assert p.table[5, 1] == p.N and p.table[B - 1, P - 1] == -1 and np.array_equal(p.table[9], before)


FORK = [
    # B, P, S, N, more than 4096 words
    (150, 100, 16, 100001, False),
    (150, 130, 16, 70003, False),
    (400, 100, 16, 100001, True),
    (1300, 128, 16, 280003, True),        # more than 262144 pages, the next stretch of every warp
    (250, 300, 16, 70001, True),
    (1100, 129, 16, 130001, True),        # wide rows, a second stretch a warp
]


@gpu
@pytest.mark.parametrize("i", range(len(FORK)))
def test_large_forks(i):
    B, P, S, N, many = FORK[i]
    g = np.random.default_rng(1740 + i)
    # a tenth of the rows long, so that the pool holds them
    lens = np.where(g.random(B) < 0.1, g.integers(0, P * S + 1, B), g.integers(0, 20 * S, B))
    p = Forks(1740 + i, B, P, S, N, lens, 1, 16, "head", shared=1)
    for step in range(2):
        stays = g.random(B) < 0.4
        stays[g.integers(B)] = True
        parents = np.where(stays, np.where(g.random(B) < 0.5, -1, np.arange(B)), g.choice(np.flatnonzero(stays), B))
        assert p.fork(parents) == 0
    p.seq[np.flatnonzero(stays)[0]] = P * S + 1     # a parent whose length is out of range
    parents = np.where(stays, -1, np.flatnonzero(stays)[0])
    before = p.table.copy()
    assert p.fork(parents) == RANGE and np.array_equal(p.table, before)
