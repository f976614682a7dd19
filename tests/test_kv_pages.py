"""Holding and forking pages of the paged cache: tables, counts, lengths, codes and scales equal to those of a restatement
in numpy, sequence by sequence."""
import os
import re

import numpy as np
import pytest
import torch

from conftest import ROOT

gpu = pytest.mark.gpu
RANGE, FULL = 8, 9


# --------------------------------------------------------------------------
# the definitions

def needed(S, L, n, window, sinks):
    first = max(0, L + 1 - window) if window else 0
    return [c for c in range(-(-(L + n) // S)) if (c + 1) * S > first or c * S < sinks]


def ref_hold(refs, table, seq, new, S, window=0, sinks=0):
    """In place; (free pages left, status)."""
    N, status = len(refs), 0
    want = {}
    for b in range(len(table)):
        L, n = int(seq[b]), int(new[b])
        if L < 0 or n < 0 or L + n > table.shape[1] * S:
            status = status or RANGE
            continue
        want[b] = needed(S, L, n, window, sinks)
        for c in set(range(table.shape[1])) - set(want[b]):
            if 0 <= table[b, c] < N:
                refs[table[b, c]] -= 1
            table[b, c] = -1
        if any(table[b, c] >= N for c in want[b]):
            status = status or RANGE
    free = list(np.flatnonzero(refs <= 0))
    for b, cols in want.items():
        for c in cols:
            if table[b, c] < 0:
                if free:
                    table[b, c] = free.pop(0)
                    refs[table[b, c]] = 1
                else:
                    status = status or FULL
    return len(free), status


def ref_fork(refs, table, seq, parents, S, pools):
    """In place; pools: the codes [N, H, S, D] and scales [N, H] of keys, then of values."""
    N, B, P = len(refs), len(table), table.shape[1]
    status, forks = 0, []
    for b in range(B):
        p = parents[b]
        if p in (-1, b):
            continue
        if not (0 <= p < B) or parents[p] not in (-1, p) or not (0 <= seq[p] <= P * S):
            status = status or RANGE
            continue
        forks.append((b, p))
    new = {}
    for b, p in forks:
        for c in range(P):
            if 0 <= table[b, c] < N:
                refs[table[b, c]] -= 1
        whole, rest = divmod(int(seq[p]), S)
        row = np.full(P, -1, np.int32)
        for c in range(whole):
            if 0 <= table[p, c] < N:
                row[c] = table[p, c]
                refs[row[c]] += 1
            elif table[p, c] >= N:
                status = status or RANGE
        copy = rest > 0 and 0 <= table[p, whole] < N
        if rest > 0 and not copy:
            status = status or RANGE
        new[b] = (row, whole, rest, table[p, whole] if copy else -1)
    free = list(np.flatnonzero(refs <= 0))
    for b, p in forks:
        row, whole, rest, old = new[b]
        if old >= 0:
            if free:
                page = free.pop(0)
                row[whole], refs[page] = page, 1
                for codes, scales in zip(pools[0::2], pools[1::2]):
                    codes[page, :, :rest] = codes[old, :, :rest]
                    scales[page] = scales[old]
            else:
                status = status or FULL
        seq[b], table[b] = seq[p], row
    return len(free), status


def dev(x):
    return torch.from_numpy(np.array(x)).cuda()


def same(got, want):
    assert np.array_equal(got.cpu().numpy(), want)


# --------------------------------------------------------------------------
# the boundary (CPU)

@pytest.fixture(scope="module")
def L():
    from speculative_sampling_verification_spec_gb300 import _build, kv_pages
    _build.build()
    return kv_pages._lib()


def test_header_library_and_binding_agree(L):
    from speculative_sampling_verification_spec_gb300 import binding, kv_pages
    text = open(os.path.join(ROOT, "include", "spec_kv_pages.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(spec_kv_[a-z_]+)\s*\(", text)))
    assert names == sorted(kv_pages.EXPORTED)
    for name in names:
        assert hasattr(L, name), name
    assert "free" in binding.spec_status_string(FULL)


GOOD = dict(num_pages=8, page_size=16, B=2, max_pages=4, refs=0x1000, page_table=0x2000, table_stride=4, free_pages=0,
            stream=0, status=0)
# pointers that are never read: every call below fails a check


def _pack(**over):
    from speculative_sampling_verification_spec_gb300 import kv_pages
    return kv_pages._PAGES.pack(*[over.get(k, v) for k, v in GOOD.items()])


def _cache(**over):
    from test_kv_cache import GOOD_CACHE
    from speculative_sampling_verification_spec_gb300 import kv_cache
    return kv_cache._CACHE.pack(*[over.get(k, v) for k, v in GOOD_CACHE.items()])


@pytest.mark.parametrize("over", [dict(num_pages=0), dict(page_size=8), dict(page_size=24), dict(B=-1), dict(max_pages=0),
                                  dict(refs=0), dict(refs=0x1002), dict(page_table=0), dict(page_table=0x2001),
                                  dict(table_stride=3), dict(table_stride=-4)], ids=str)
def test_both_refuse(L, over):
    assert L.spec_kv_hold(_pack(**over), 0x3000, None, 1, 0, 0) == 1
    assert L.spec_kv_fork(_pack(**over), _cache(num_pages=over.get("num_pages", 8)), 0x3000, 0x4000) == 1


def test_refusals_of_arguments_and_sizes(L):
    p = _pack()
    assert L.spec_kv_hold(None, 0x3000, None, 1, 0, 0) == 1
    assert L.spec_kv_hold(p, None, None, 1, 0, 0) == 1
    for bad in ((-1, 0, 0), (1, -1, 0), (1, 0, -1)):
        assert L.spec_kv_hold(p, 0x3000, None, *bad) == 1
    assert L.spec_kv_hold(_pack(max_pages=1 << 28, table_stride=1 << 28), 0x3000, None, 1, 0, 0) == 6    # positions
    assert L.spec_kv_hold(_pack(num_pages=1 << 30), 0x3000, None, 1, 0, 0) == 6                          # too many pages
    assert L.spec_kv_hold(_pack(B=1 << 20, max_pages=64, table_stride=64), 0x3000, None, 1, 0, 0) == 6   # and entries
    assert L.spec_kv_fork(p, None, 0x3000, 0x4000) == 1
    assert L.spec_kv_fork(p, _cache(), None, 0x4000) == 1
    assert L.spec_kv_fork(p, _cache(), 0x3000, None) == 1
    for over in (dict(num_pages=9), dict(page_size=32), dict(Hkv=0), dict(D=24), dict(D=272), dict(k_codes=0),
                 dict(v_codes=0x2008), dict(k_scale=0), dict(page_stride=1000), dict(token_stride=0), dict(head_stride=-16),
                 dict(scale_page_stride=0)):
        assert L.spec_kv_fork(p, _cache(**over), 0x3000, 0x4000) == 1, over


def test_host_tensors_are_refused(L):
    import speculative_sampling_verification_spec_gb300 as sv
    t, r, s = torch.full((2, 8), -1, dtype=torch.int32), torch.zeros(9, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.spec_kv_hold(r, t, s, page_size=16)
    with pytest.raises(ValueError):
        sv.spec_kv_fork(None, r, t, s, s)


# --------------------------------------------------------------------------
# hold

class Pool:
    """Sequences that hold pages of a shuffled pool, some of them shared; numpy and device copies."""

    def __init__(self, seed, B, P, S, N, lens, window=0, sinks=0, shared=0):
        g = np.random.default_rng(seed)
        self.g, self.S, self.N = g, S, N
        self.table, self.refs = np.full((B, P), -1, np.int32), np.zeros(N, np.int32)
        order = iter(g.permutation(N))
        for b, n in enumerate(lens):
            for c in needed(S, int(n), 0, window, sinks):
                if b and c < shared and self.table[b - 1, c] >= 0:
                    self.table[b, c] = self.table[b - 1, c]
                else:
                    self.table[b, c] = next(order)
                self.refs[self.table[b, c]] += 1

    def hold(self, seq, new, window=0, sinks=0, T=None, **kw):
        import speculative_sampling_verification_spec_gb300 as sv
        t, r = dev(self.table), dev(self.refs)
        free, status = torch.full((1,), -5, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        args = dict(page_size=self.S, window=window, sinks=sinks, free=free, status=status)
        seq, new = np.asarray(seq, np.int32), np.asarray(new, np.int32)
        if T is None:
            sv.spec_kv_hold(r, t, dev(seq), dev(new), **args, **kw)
        else:
            sv.spec_kv_hold(r, t, dev(seq), T=T, **args, **kw)
        t2, r2 = dev(self.table), dev(self.refs)      # without the number of free pages asked for
        sv.spec_kv_hold(r2, t2, dev(seq), dev(new), page_size=self.S, window=window, sinks=sinks)
        want = ref_hold(self.refs, self.table, seq, new, self.S, window, sinks)
        same(t, self.table)
        same(r, self.refs)
        same(t2, self.table)
        same(r2, self.refs)
        assert free.item() == want[0] and status.item() == want[1]
        return want[1]


HOLD = [
    # B, P, S, N, window, sinks, longest, T
    (1, 1, 16, 1, 0, 0, 16, 16),
    (1, 5, 16, 9, 0, 0, 50, 20),
    (7, 33, 16, 400, 0, 0, 400, 100),
    (5, 40, 32, 300, 100, 4, 1000, 17),
    (5, 40, 32, 300, 1, 33, 1000, 1),
    (33, 31, 64, 900, 333, 200, 1800, 100),
    (64, 257, 16, 20000, 1000, 4, 4000, 9),       # 8 CTAs
    (300, 64, 128, 30000, 0, 0, 8000, 150),
    (3, 3000, 16, 9001, 0, 0, 40000, 8000),
]


@gpu
@pytest.mark.parametrize("i", range(len(HOLD)))
def test_hold_equals_the_definition(i):
    """Rounds with growing, shrinking and emptied sequences, each checked as it leaves the one before."""
    B, P, S, N, window, sinks, longest, T = HOLD[i]
    g = np.random.default_rng(700 + i)
    seq = g.integers(0, longest - T + 1, B)
    p = Pool(700 + i, B, P, S, N, seq, window, sinks, shared=2)
    for step in range(4):
        assert p.hold(seq, g.integers(0, T + 1, B), window, sinks) == 0
        seq = np.where(g.random(B) < 0.2, 0, np.clip(seq + g.integers(-T, T + 1, B), 0, longest - T))
    assert p.hold(seq, np.full(B, T), window, sinks, T=T) == 0
    assert p.hold(np.zeros(B), np.zeros(B), window, sinks) == 0
    assert (p.table == -1).all() and (p.refs == 0).all()


@gpu
@pytest.mark.parametrize("big", [False, True])
def test_hold_when_pages_run_out(big):
    B, P, S = (40, 600, 16) if big else (5, 9, 16)
    p = Pool(720, B, P, S, B * 4 + 3, [40] * B)
    p.refs[7] += 1                                # a count of the caller's own
    full = p.hold([40] * B, [40] * B)
    assert full == FULL and (p.table[-1, 3:5] < 0).all()
    assert p.hold([40] * B, [0] * B) == 0         # released again
    assert p.hold([0] * B, [0] * B) == 0 and p.refs[7] == 1 and p.refs.sum() == 1


@gpu
def test_hold_device_errors_and_odd_entries():
    """Lengths out of range leave a row as it is; entries beyond the pool stay where they are needed and go where not;
    entries below -1 are none; counts below zero are free."""
    p = Pool(721, 6, 10, 16, 60, [50] * 6)
    p.table[0, 1], p.table[1, 8], p.table[2, 7], p.table[3, 9] = 60, 1 << 30, -9, -2
    free = np.flatnonzero(p.refs == 0)
    p.refs[free[0]] = -3
    assert p.hold([50, 50, 50, 160, 50, -1], [20, 20, 90, 1, 20, 5]) == RANGE
    assert p.table[0, 1] == 60 and p.table[1, 8] == -1 and p.table[3, 9] == -2
    p.table[0, 1] = -1
    assert p.hold([50, 50, 50, 50, (1 << 31) - 1, 50], [20, 20, 20, 20, (1 << 31) - 1, -1]) == RANGE


@gpu
def test_hold_strided_table_stream_graph_and_nothing():
    import speculative_sampling_verification_spec_gb300 as sv
    p = Pool(722, 4, 12, 16, 100, [30, 90, 0, 120])
    wide = np.full((4, 20), 77, np.int32)
    wide[:, 3:15] = p.table
    t, r, seq, new = dev(wide), dev(p.refs), dev(np.int32([30, 90, 0, 120])), dev(np.int32([10, 0, 40, 16]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_kv_hold(r, t[:, 3:15], seq, new, page_size=16)
    for lens in ([30, 90, 0, 120], [60, 0, 100, 16], [0, 0, 0, 1]):
        seq.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        ref_hold(p.refs, p.table, lens, [10, 0, 40, 16], 16)
        wide[:, 3:15] = p.table
        same(t, wide)
        same(r, p.refs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sv.spec_kv_hold(r, t[:, 3:15], seq, page_size=16, T=50, stream=side)
    side.synchronize()
    ref_hold(p.refs, p.table, lens, [50] * 4, 16)
    same(t[:, 3:15], p.table)
    # no sequences: only the free pages are counted
    free = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.spec_kv_hold(r, t[:0, 3:15], seq[:0], page_size=16, free=free)
    assert free.item() == int((p.refs <= 0).sum())
    # one row: its stride does not matter
    one = torch.full((1, 8), -1, dtype=torch.int32, device="cuda")
    r.zero_()
    sv.spec_kv_hold(r, one.as_strided((1, 8), (0, 1)), seq[:1], page_size=16, T=128 - lens[0])
    assert one.cpu().tolist() == [list(range(8))]


@gpu
def test_python_checks():
    import speculative_sampling_verification_spec_gb300 as sv
    t, r = torch.full((2, 8), -1, dtype=torch.int32, device="cuda"), torch.zeros(9, dtype=torch.int32, device="cuda")
    s = torch.zeros(2, dtype=torch.int32, device="cuda")
    for args, kw in (((r.cpu(), t, s), {}), ((r.long(), t, s), {}), ((r, t.long(), s), {}), ((r, t.cpu(), s), {}),
                     ((r, t, s.long()), {}), ((r, t, s[:1]), {}), ((r, t, s, s.cpu()), {}), ((r, t[:, ::2], s), {}),
                     ((r, t[0], s), {}), ((r[::2], t, s), {}), ((r, t, s), dict(free=s.long())),
                     ((r, t, s), dict(status=s.cpu()))):
        with pytest.raises(ValueError):
            sv.spec_kv_hold(*args, page_size=16, **kw)
    for kw in (dict(page_size=17), dict(page_size=16, T=-1), dict(page_size=16, window=-1), dict(page_size=16, sinks=-1),
               dict(page_size=16, T=(1 << 32) + 1), dict(page_size=16, window=1 << 31)):
        with pytest.raises(sv.SpecError):
            sv.spec_kv_hold(r, t, s, **kw)
    with pytest.raises(sv.SpecError):
        sv.spec_kv_hold(r, t[:1].expand(2, 8), s, page_size=16)
    cache = sv.PagedKVCache.empty(8, 16, 1, 16)
    with pytest.raises(ValueError):
        sv.spec_kv_fork(cache, r, t, s, s)           # nine counts for eight pages
    with pytest.raises(ValueError):
        sv.spec_kv_fork(cache, r[:8], t, s, s.long())


# --------------------------------------------------------------------------
# fork

class Forks(Pool):
    def __init__(self, seed, B, P, S, N, lens, Hkv, D, layout="head", **kw):
        super().__init__(seed, B, P, S, N, lens, **kw)
        g = self.g
        self.seq = np.asarray(lens, np.int32)
        self.codes = [g.integers(0, 256, (N, Hkv, S, D)).astype(np.uint8) for _ in range(2)]
        self.scales = [g.standard_normal((N, Hkv)).astype(np.float32) for _ in range(2)]
        self.layout = layout

    def cache(self):
        import speculative_sampling_verification_spec_gb300 as sv
        codes, scales = [dev(c) for c in self.codes], [dev(s) for s in self.scales]
        if self.layout == "token":        # [page, slot, head, channel] in memory
            codes = [c.transpose(1, 2).contiguous().transpose(1, 2) for c in codes]
        if self.layout == "both":         # keys and values side by side, padded
            N, H, S, D = codes[0].shape
            both = torch.zeros(N, H, S, 2 * D + 16, dtype=torch.uint8, device="cuda")
            both[..., :D], both[..., D + 16:] = codes[0], codes[1]
            codes = [both[..., :D], both[..., D + 16:]]
            scales = [torch.stack(scales)[i] for i in range(2)]
        return sv.PagedKVCache(*codes, *scales)

    def fork(self, parents, **kw):
        import speculative_sampling_verification_spec_gb300 as sv
        parents = np.asarray(parents, np.int32)
        cache, t, r, s = self.cache(), dev(self.table), dev(self.refs), dev(self.seq)
        free, status = torch.full((1,), -5, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        sv.spec_kv_fork(cache, r, t, s, dev(parents), free=free, status=status, **kw)
        pools = [self.codes[0], self.scales[0], self.codes[1], self.scales[1]]
        want = ref_fork(self.refs, self.table, self.seq, parents, self.S, pools)
        same(t, self.table)
        same(r, self.refs)
        same(s, self.seq)
        same(cache.k_codes.view(torch.uint8), self.codes[0])
        same(cache.v_codes.view(torch.uint8), self.codes[1])
        same(cache.k_scale, self.scales[0])
        same(cache.v_scale, self.scales[1])
        assert free.item() == want[0] and status.item() == want[1]
        return want[1]


FORK = [
    # B, P, S, N, Hkv, D, layout, lens
    (2, 1, 16, 3, 1, 16, "head", [1, 0]),
    (2, 2, 16, 5, 2, 64, "head", [16, 7]),                 # a whole page and nothing to copy
    (5, 9, 16, 60, 3, 80, "token", [0, 100, 144, 17, 31]),
    (6, 4, 128, 40, 2, 256, "both", [500, 127, 128, 129, 3, 0]),
    (40, 33, 32, 1500, 8, 128, "head", None),
    (70, 300, 16, 20000, 1, 48, "token", None),            # 8 CTAs
]


@gpu
@pytest.mark.parametrize("i", range(len(FORK)))
def test_fork_equals_the_definition(i):
    B, P, S, N, Hkv, D, layout, lens = FORK[i]
    g = np.random.default_rng(740 + i)
    p = Forks(740 + i, B, P, S, N, g.integers(0, P * S + 1, B) if lens is None else lens, Hkv, D, layout, shared=1)
    for step in range(3):
        stays = g.random(B) < 0.4
        stays[g.integers(B)] = True
        parents = np.where(stays, np.where(g.random(B) < 0.5, -1, np.arange(B)), g.choice(np.flatnonzero(stays), B))
        assert p.fork(parents) == 0
    counted = np.bincount(p.table[p.table >= 0], minlength=N)
    assert np.array_equal(counted, p.refs)


@gpu
def test_fork_errors():
    """Parents that are none, do not stay or have lengths out of range; pages that are gone or beyond the pool; no page
    left."""
    p = Forks(750, 8, 6, 16, 60, [40, 20, 70, 33, 5, 0, 96, 11], 2, 32)
    before = p.table.copy()
    assert p.fork([-1, 0, 1, 8, -2, -1, -1, 1 << 30]) == RANGE
    assert np.array_equal(p.table[2:], before[2:]) and not np.array_equal(p.table[1], before[1])
    p.seq[6] = 97
    assert p.fork([-1, -1, 6, -1, -1, -1, -1, -1]) == RANGE
    p.seq[6] = -1
    assert p.fork([-1, -1, 6, -1, -1, -1, -1, -1]) == RANGE
    p.seq[6] = 90
    p.table[6, 0], p.table[6, 1] = 1 << 20, -4
    assert p.fork([-1, -1, -1, 6, -1, -1, -1, -1]) == RANGE and p.table[3, 0] == -1 and p.table[3, 2] >= 0
    p.table[6, 0], p.table[6, 5] = -1, -1
    assert p.fork([-1, -1, -1, 6, -1, -1, -1, -1]) == RANGE
    p.table[6, 5] = 61
    assert p.fork([-1, -1, -1, 6, -1, -1, -1, -1]) == RANGE
    q = Forks(751, 4, 3, 16, 4, [20, 0, 0, 0], 1, 16)
    assert q.fork([-1, 0, 0, 0]) == FULL          # two free pages for three copies
    assert q.table[3, 0] == q.table[0, 0] and q.refs[q.table[0, 0]] == 4
    assert q.table[3, 1] == -1 and (q.table[:3, 1] >= 0).all()


@gpu
def test_fork_graph_and_stream():
    import speculative_sampling_verification_spec_gb300 as sv
    p = Forks(760, 4, 6, 16, 40, [40, 0, 77, 20], 2, 64)
    cache, t, r, s = p.cache(), dev(p.table), dev(p.refs), dev(p.seq)
    parents = dev(np.int32([-1, 0, -1, 2]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_kv_fork(cache, r, t, s, parents)
    pools = [p.codes[0], p.scales[0], p.codes[1], p.scales[1]]
    for par in ([-1, 0, -1, 2], [-1, 0, -1, 0], [2, 2, -1, 2]):
        parents.copy_(torch.tensor(par, dtype=torch.int32))
        graph.replay()
        ref_fork(p.refs, p.table, p.seq, par, 16, pools)
        same(t, p.table)
        same(r, p.refs)
        same(s, p.seq)
        same(cache.k_codes.view(torch.uint8), p.codes[0])
    side = torch.cuda.Stream()
    parents.fill_(-1)
    parents[0] = 2
    side.wait_stream(torch.cuda.current_stream())
    sv.spec_kv_fork(cache, r, t, s, parents, stream=side)
    side.synchronize()
    ref_fork(p.refs, p.table, p.seq, [2, -1, -1, -1], 16, pools)
    same(t, p.table)
    same(cache.v_codes.view(torch.uint8), p.codes[1])
