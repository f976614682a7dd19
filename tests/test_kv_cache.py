"""The paged 8-bit key/value cache: append and attention against their definitions (kv_ref.py).

Appending is defined value by value (each product and sum rounded to float32, codes to nearest even), so queries, codes
and scales have to be equal, bit for bit.  Attention is compared with float64 within a bound that follows from the
roundings (kv_ref.attention).
"""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import kv_ref
from conftest import ROOT

gpu = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


class Setup:
    """A pool with every sequence's pages in random order, filled with random tokens; slots that no sequence holds are
    NaN codes, so that anything read beyond the lengths shows."""

    def __init__(self, seed, B, T, Hq, Hkv, D, S, seq, new, dtype="f32", rot=0, interleaved=False, magnitude=1.0,
                 pow2=True, token_major=False, q_size=1.0):
        g = np.random.default_rng(seed)
        self.g, self.B, self.T, self.Hq, self.Hkv, self.D, self.S = g, B, T, Hq, Hkv, D, S
        self.dtype, self.rot, self.interleaved = dtype, rot, interleaved
        self.seq, self.new = np.asarray(seq, np.int32), np.asarray(new, np.int32)
        need = [max(1, -(-(int(s) + T) // S)) for s in seq]
        self.P = max(need) + 1
        N = sum(need) + 2
        order = g.permutation(N)
        self.table = np.full((B, self.P), N + 7, np.int32)    # unused columns hold no page
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        self.N = N
        self.kc, self.vc = np.full((N, Hkv, S, D), 0x7F, np.uint8), np.full((N, Hkv, S, D), 0xFF, np.uint8)
        self.ks, self.vs = np.zeros((N, Hkv), np.float32), np.zeros((N, Hkv), np.float32)
        for b in range(B):
            for i in range(-(-int(seq[b]) // S)):
                m = min(S, int(seq[b]) - i * S)
                pg = self.table[b, i]
                for codes, scales in ((self.kc, self.ks), (self.vc, self.vs)):
                    x = g.standard_normal((Hkv, m, D)) * magnitude * np.exp(g.standard_normal((Hkv, 1, 1)))
                    sc = kv_ref.scale_for(np.abs(x).max(axis=(1, 2)))
                    if not pow2:
                        sc = (np.abs(x).max(axis=(1, 2)) / 447.0).astype(np.float32)
                    scales[pg] = sc
                    codes[pg, :, :m] = kv_ref.encode(x / sc[:, None, None])
        self.q = self.values(B, T, Hq, D) * np.float32(q_size)
        if dtype == "bf16":
            self.q = kv_ref.bf16_round(self.q)
        self.k, self.v = self.values(B, T, Hkv, D), self.values(B, T, Hkv, D)
        ang = np.arange(self.P * S)[:, None] * (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2)))
        self.cs = np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)
        self.token_major = token_major

    def values(self, *shape):
        x = self.g.standard_normal(shape).astype(np.float32)
        return kv_ref.bf16_round(x) if self.dtype == "bf16" else x

    # ---- device side
    def dev(self, x):
        t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
        return t.to(DT[self.dtype]) if t.dtype == torch.float32 else t

    def cache(self):
        import speculative_sampling_verification_spec_gb300 as sv
        kc, vc = torch.from_numpy(self.kc).cuda(), torch.from_numpy(self.vc).cuda()
        if self.token_major:      # [page, slot, head, channel] in memory
            kc, vc = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (kc, vc))
        return sv.PagedKVCache(kc, vc, torch.from_numpy(self.ks).cuda(), torch.from_numpy(self.vs).cuda())

    def idx(self):
        return [torch.from_numpy(x).cuda() for x in (self.table, self.seq, self.new)]

    def append(self, cache, **kw):
        import speculative_sampling_verification_spec_gb300 as sv
        cs = torch.from_numpy(self.cs).cuda() if self.rot else None
        kw = dict(dict(cos_sin=cs, interleaved=self.interleaved), **kw)
        q, k, v = (kw.pop(n, None) for n in "qkv")
        return sv.spec_kv_append(self.dev(self.q) if q is None else q, self.dev(self.k) if k is None else k,
                                 self.dev(self.v) if v is None else v, cache, *self.idx(), **kw)

    def ref_append(self):
        return kv_ref.append(self.q, self.k, self.v, self.kc, self.vc, self.ks, self.vs, self.table, self.seq, self.new,
                             self.cs, self.rot, self.interleaved, self.dtype, self.S)

    def ref_attention(self, scale=None, window=0):
        return kv_ref.attention(self.q.astype(np.float64), self.kc, self.vc, self.ks, self.vs, self.table, self.seq,
                                self.new, self.S, 1 / math.sqrt(self.D) if scale is None else scale, window, self.dtype)


def assert_cache(cache, ref):
    """Codes equal as bytes (a NaN's sign aside) and scales equal, over the whole pool."""
    for name, got, want in (("k", cache.k_codes, ref.kc), ("v", cache.v_codes, ref.vc)):
        a, b = got.cpu().view(torch.uint8).numpy().copy(), want.copy()
        for x in (a, b):
            x[x == 0xFF] = 0x7F
        bad = np.argwhere(a != b)
        assert len(bad) == 0, (name, len(bad), bad[:4].tolist())
    assert np.array_equal(cache.k_scale.cpu().numpy(), ref.ks)
    assert np.array_equal(cache.v_scale.cpu().numpy(), ref.vs)


def assert_attention(got, lse, ref, where=""):
    out, rl, tol, tol_l = ref
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.all(np.isfinite(got)), where
    over = np.abs(got - out) > tol
    assert not over.any(), (where, int(over.sum()), float(np.max(np.abs(got - out) / np.maximum(tol, 1e-30))))
    empty = np.isinf(rl)
    assert np.array_equal(empty, np.isneginf(lse)), where
    assert np.all(got[empty] == 0), where
    assert np.all(np.abs(lse[~empty] - rl[~empty]) <= tol_l[~empty]), where


# --------------------------------------------------------------------------
# the reference itself (CPU)

def test_reference_codes_are_e4m3():
    """Codes round-trip, and encoding agrees with torch's float8_e4m3fn conversion on a dense set of values."""
    v = kv_ref.CODE_VALUES
    ok = ~np.isnan(v)
    back = kv_ref.encode(v[ok])
    assert np.array_equal(kv_ref.CODE_VALUES[back], v[ok])
    g = np.random.default_rng(0)
    x = np.concatenate([g.uniform(-448, 448, 20000), g.standard_normal(20000) * 2.0 ** g.integers(-14, 6, 20000),
                        (v[ok][:-1] + v[ok][1:]) / 2]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv_ref.CODE_VALUES[kv_ref.encode(x)], kv_ref.CODE_VALUES[want])


def test_reference_scales_are_tight():
    a = np.concatenate([np.float32([448, 447.9999, 449, 1e-30, 2e-44, 3e38, 0.0]),
                        np.random.default_rng(1).uniform(0, 10, 1000).astype(np.float32)])
    s = kv_ref.scale_for(a).astype(np.float64)
    assert np.all(a <= 448 * s)
    big = s > 2.0 ** -100
    assert np.all(a[big] > 448 * s[big] / 2)


# --------------------------------------------------------------------------
# the boundary (CPU)

def _declared():
    text = open(os.path.join(ROOT, "include", "spec_kv.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(spec_kv_[a-z_]+)\s*\(", text)))


@pytest.fixture(scope="module")
def L():
    from speculative_sampling_verification_spec_gb300 import _build, kv_cache
    _build.build()
    return kv_cache._lib()


def test_header_library_and_binding_agree(L):
    from speculative_sampling_verification_spec_gb300 import kv_cache
    assert _declared() == sorted(kv_cache.EXPORTED)
    for name in _declared():
        assert hasattr(L, name), name


GOOD_CACHE = dict(num_pages=8, page_size=16, Hkv=2, D=64, k_codes=0x1000, v_codes=0x2000, k_scale=0x3000, v_scale=0x4000,
                  page_stride=2048, head_stride=1024, token_stride=64, scale_page_stride=2, scale_head_stride=1)
GOOD = dict(B=2, T=3, Hq=4, dtype=0, max_pages=4, window=0, scale=0.125, rot_dim=0, rot_len=0, interleaved=0,
            page_table=0x5000, seq_lens=0x6000, new_lens=0x7000, table_stride=4, q1=768, q2=256, q3=64, k1=384, k2=128,
            k3=64, v1=384, v2=128, v3=64, o1=768, o2=256, o3=64, stream=0, status=0, workspace=0x10000,
            workspace_bytes=1 << 40)
# pointers that are never read: every call below fails a check, or has no sequences


def _pack(over):
    from speculative_sampling_verification_spec_gb300 import kv_cache
    c = [over.get(k, v) for k, v in GOOD_CACHE.items()]
    p = [over.get(k, v) for k, v in GOOD.items()]
    return kv_cache._CACHE.pack(*c), kv_cache._PARAMS.pack(*p)


BAD_BOTH = [dict(num_pages=0), dict(page_size=0), dict(page_size=8), dict(page_size=24), dict(page_size=256),
            dict(Hkv=0), dict(D=0), dict(D=24), dict(D=272), dict(k_codes=0), dict(v_codes=0x2008), dict(k_scale=0),
            dict(v_scale=0), dict(page_stride=-16), dict(token_stride=72), dict(head_stride=1000),
            dict(scale_page_stride=-1), dict(B=-1), dict(T=0), dict(Hq=0), dict(Hq=3), dict(dtype=2), dict(max_pages=0),
            dict(page_table=0), dict(seq_lens=0), dict(table_stride=-1), dict(q2=-1), dict(o3=-1),
            dict(token_stride=0), dict(head_stride=0), dict(page_stride=0), dict(scale_head_stride=0),
            dict(scale_page_stride=0), dict(o1=0), dict(o2=0), dict(o3=0)]


@pytest.mark.parametrize("over", BAD_BOTH + [dict(window=-1), dict(scale=math.inf), dict(scale=math.nan),
                                             dict(workspace=0), dict(workspace=0x10010), dict(workspace_bytes=64)], ids=str)
def test_attention_refuses(L, over):
    c, p = _pack(over)
    assert L.spec_kv_attention(0x8000, c, p, 0x9000, None) == 1


@pytest.mark.parametrize("over", BAD_BOTH + [dict(k1=-1), dict(v2=-1), dict(rot_dim=3, rot_len=9), dict(rot_dim=66, rot_len=9),
                                             dict(rot_dim=-2), dict(rot_dim=16, rot_len=0)], ids=str)
def test_append_refuses(L, over):
    c, p = _pack(over)
    assert L.spec_kv_append(0x8000, 0xA000, 0xB000, 0xC000, c, p, 0x9000) == 1


def test_refusals_of_pointers_and_sizes(L):
    c, p = _pack({})
    assert L.spec_kv_attention(None, c, p, 0x9000, None) == 1
    assert L.spec_kv_attention(0x8000, c, p, None, None) == 1
    assert L.spec_kv_attention(0x8000, None, p, 0x9000, None) == 1
    assert L.spec_kv_attention(0x8000, c, None, 0x9000, None) == 1
    assert L.spec_kv_append(0x8000, None, 0xB000, None, c, p, 0x9000) == 1
    assert L.spec_kv_append(0x8000, 0xA000, None, None, c, p, 0x9000) == 1
    assert L.spec_kv_append(None, 0xA000, 0xB000, None, c, p, 0x9000) == 1     # q_out without q
    assert L.spec_kv_append(0x8000, 0xA000, 0xB000, None, c, p, None) == 1     # q without q_out
    c2, p2 = _pack(dict(rot_dim=16, rot_len=9))
    assert L.spec_kv_append(0x8000, 0xA000, 0xB000, None, c2, p2, 0x9000) == 1     # rotation without a table
    assert L.spec_kv_append(0x8000, 0xA000, 0xB000, 0xC004, c2, p2, 0x9000) == 1   # an unaligned one
    c3, p3 = _pack(dict(B=0))
    assert L.spec_kv_append(0x8000, 0xA000, 0xB000, None, c3, p3, 0x9000) == 0     # nothing to do
    assert L.spec_kv_attention(0x8000, c3, p3, 0x9000, None) == 0
    for over in (dict(max_pages=1 << 28), dict(B=1 << 15, T=1 << 14, Hq=64)):      # beyond 32-bit counts
        c4, p4 = _pack(over)
        assert L.spec_kv_attention(0x8000, c4, p4, 0x9000, None) == 6


def test_workspace_size_is_host_only(L):
    def size(**over):
        c, p = _pack(over)
        return L.spec_kv_attention_workspace_size(c, p)
    assert size() > 0 and size(D=256) > size()
    assert size(max_pages=1) == size(max_pages=1 << 20)     # lengths do not matter
    assert size(T=0) == 0 and size(D=24) == 0 and size(dtype=5) == 0
    from speculative_sampling_verification_spec_gb300 import binding
    assert "cache" in binding.spec_status_string(8)


# --------------------------------------------------------------------------
# append

APPEND = [
    # B, T, Hq, Hkv, D, S, seq, new, dtype, rot, interleaved
    (1, 1, 8, 2, 128, 16, [0], [1], "bf16", 128, False),
    (1, 1, 8, 2, 128, 16, [15], [1], "bf16", 128, False),
    (1, 1, 4, 4, 64, 16, [16], [1], "f32", 64, True),
    (4, 5, 8, 2, 128, 16, [0, 14, 16, 31], [5, 5, 0, 3], "bf16", 128, False),
    (3, 9, 6, 3, 64, 32, [30, 7, 64], [9, 1, 9], "bf16", 32, True),
    (3, 9, 6, 3, 64, 32, [30, 7, 64], [9, 1, 9], "f32", 32, False),
    (2, 17, 2, 1, 80, 16, [3, 0], [17, 16], "f32", 80, False),        # rotated halves of 40: chunks of pairs cross nothing
    (2, 3, 4, 2, 48, 16, [3, 20], [3, 2], "bf16", 10, False),         # 10 of 48 channels: single pairs
    (2, 3, 4, 2, 48, 16, [3, 20], [3, 2], "f32", 10, True),
    (2, 70, 3, 3, 16, 16, [5, 0], [70, 33], "bf16", 0, False),        # no rotation
    (2, 300, 4, 2, 128, 128, [100, 0], [300, 256], "bf16", 128, False),
    (1, 200, 2, 1, 256, 128, [1], [200], "f32", 256, False),          # a unit larger than a CTA's registers
    (1, 129, 2, 2, 64, 64, [63], [129], "f32", 64, True),
]


@gpu
@pytest.mark.parametrize("i", range(len(APPEND)))
@pytest.mark.parametrize("token_major", [False, True])
def test_append_equals_the_definition(i, token_major):
    B, T, Hq, Hkv, D, S, seq, new, dtype, rot, inter = APPEND[i]
    s = Setup(100 + i, B, T, Hq, Hkv, D, S, seq, new, dtype, rot, inter, token_major=token_major)
    cache = s.cache()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(2):        # the second call writes the same again
        q = s.append(cache, status=status)
    want = s.ref_append()
    assert np.array_equal(q.float().cpu().numpy(), want)
    assert_cache(cache, s)
    assert status.item() == 0


@gpu
def test_append_rotation_against_64_bits():
    """The rotated queries against cos/sin in float64: products and sum of three roundings, and the angles' own."""
    s = Setup(7, 2, 9, 4, 2, 64, 16, [100, 3], [9, 9], "f32", 64)
    q = s.append(s.cache()).double().cpu().numpy()
    ang = (s.seq[:, None] + np.arange(9))[..., None] * 10000.0 ** (-np.arange(32) / 32)
    c, sn = np.cos(ang)[:, :, None], np.sin(ang)[:, :, None]
    x1, x2 = s.q[..., :32].astype(np.float64), s.q[..., 32:].astype(np.float64)
    want = np.concatenate([x1 * c - x2 * sn, x2 * c + x1 * sn], -1)
    tol = 4 * kv_ref.U * np.concatenate([np.abs(x1) + np.abs(x2)] * 2, -1)
    assert np.all(np.abs(q - want) <= tol)


@gpu
def test_append_strided_and_unaligned_inputs():
    """Heads of a fused projection (strides of its width), a slice that starts off a 16-byte boundary, a repeated head
    (stride 0) and reversed orders of the first three dimensions give the same codes as contiguous tensors."""
    for dtype, off in (("bf16", 0), ("bf16", 1), ("f32", 0), ("f32", 3)):
        s = Setup(20, 3, 5, 4, 2, 64, 16, [0, 13, 40], [5, 4, 5], dtype, 64)
        fused = torch.zeros(3, 5, 8 * 64 + 8, dtype=DT[dtype], device="cuda")
        q, k, v = (fused[..., off + a * 64:off + b * 64].view(3, 5, b - a, 64) if off == 0 else
                   fused[..., off + a * 64:off + b * 64].unflatten(-1, (b - a, 64)) for a, b in ((0, 4), (4, 6), (6, 8)))
        for d, x in ((q, s.q), (k, s.k), (v, s.v)):
            d.copy_(torch.from_numpy(x).cuda())
        cache = s.cache()
        out = torch.full((5, 4, 3, 64), 9.0, dtype=DT[dtype], device="cuda").permute(2, 0, 1, 3)
        got = s.append(cache, q=q, k=k, v=v, q_out=out)
        assert got is out
        want = s.ref_append()
        assert np.array_equal(got.float().cpu().numpy(), want)
        assert_cache(cache, s)
    s = Setup(21, 2, 3, 4, 2, 64, 16, [0, 13], [3, 3], "bf16", 64)
    s.k[:] = s.k[:, :, :1]
    cache = s.cache()
    s.append(cache, k=s.dev(s.k[:, :, :1]).expand(2, 3, 2, 64))
    s.ref_append()
    assert_cache(cache, s)


@gpu
def test_append_in_place_and_without_queries():
    s = Setup(22, 2, 3, 4, 2, 64, 16, [5, 16], [3, 2], "bf16", 64)
    cache, q = s.cache(), s.dev(s.q)
    assert s.append(cache, q=q, q_out=q) is q
    want = s.ref_append()
    assert np.array_equal(q.float().cpu().numpy(), want)
    import speculative_sampling_verification_spec_gb300 as sv
    t = Setup(22, 2, 3, 4, 2, 64, 16, [5, 16], [3, 2], "bf16", 64)
    c2 = t.cache()
    assert sv.spec_kv_append(None, t.dev(t.k), t.dev(t.v), c2, *t.idx(), cos_sin=torch.from_numpy(t.cs).cuda()) is None
    assert_cache(c2, s)


@gpu
@pytest.mark.parametrize("growth", [0.0, 0.01, 1.0, 3.0, 1000.0, 1e9])
def test_scale_of_a_partly_filled_page(growth):
    """New tokens `growth` times the stored ones: the scale stays or grows, the stored codes are rounded again."""
    s = Setup(23, 2, 2, 2, 2, 64, 32, [17, 30], [2, 2], "f32", 0)
    s.k *= np.float32(growth)
    s.v *= np.float32(growth)
    before = s.ks.copy()
    cache = s.cache()
    s.append(cache)
    s.ref_append()
    assert_cache(cache, s)
    pg = s.table[0, 0]
    assert np.all(s.ks[pg] >= before[pg])
    if growth >= 1000:
        assert np.all(s.ks[pg] > before[pg])
    if growth <= 0.01:
        assert np.array_equal(s.ks[pg], before[pg])


@gpu
def test_append_special_values():
    """Zeros, values at the edge of the codes, subnormals, the largest floats, NaN and infinities."""
    for fill in (0.0, 448.0, 448.00003, 1e-44, 1e-31, 3e38, -448.0):
        s = Setup(24, 1, 3, 2, 2, 32, 16, [0], [3], "f32", 0)
        s.k[:] = np.float32(fill)
        s.v *= np.float32(fill)
        cache = s.cache()
        s.append(cache)
        s.ref_append()
        assert_cache(cache, s)
    s = Setup(25, 2, 3, 2, 2, 32, 16, [0, 5], [3, 3], "f32", 32)
    s.k[0, 1, 0, 3], s.k[1, 0, 1, 7], s.v[0, 2, 1, 0], s.v[1, 1, 0, 31] = np.inf, np.nan, -np.inf, np.nan
    cache = s.cache()
    s.append(cache)
    s.ref_append()
    assert_cache(cache, s)
    assert np.isfinite(s.ks[s.table[0, 0]]).all()
    assert (kv_ref.CODE_VALUES[s.kc[s.table[0, 0], 0, 1]] != kv_ref.CODE_VALUES[s.kc[s.table[0, 0], 0, 1]]).sum() == 2


@gpu
def test_append_device_errors():
    """A bad page number skips that page, bad lengths skip the sequence; both are reported, nothing else changes."""
    base = dict(B=3, T=4, Hq=2, Hkv=2, D=64, S=16, seq=[5, 14, 3], new=[4, 4, 4], dtype="f32", rot=64)

    def run(change):
        s = Setup(26, **base)
        cache = s.cache()
        bad = Setup(26, **base)
        change(bad)
        import speculative_sampling_verification_spec_gb300 as sv
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        q = sv.spec_kv_append(bad.dev(bad.q), bad.dev(bad.k), bad.dev(bad.v), cache, *bad.idx(),
                              cos_sin=torch.from_numpy(bad.cs).cuda(), status=status)
        return s, cache, q.cpu().numpy(), status.item()

    for value in (-1, 10 ** 6):
        def page(t):
            t.table[1, 1] = value
        s, cache, q, st = run(page)
        assert st == 8
        kc, vc, ks, vs = s.kc.copy(), s.vc.copy(), s.ks.copy(), s.vs.copy()
        want = s.ref_append()
        pg = s.table[1, 1]
        s.kc[pg], s.vc[pg], s.ks[pg], s.vs[pg] = kc[pg], vc[pg], ks[pg], vs[pg]
        assert_cache(cache, s)
        assert np.array_equal(q, want)
    for field, value in (("seq", -1), ("seq", 1 << 30), ("new", 5), ("new", -1), ("seq", 2147483647)):
        def lens(t):
            getattr(t, field)[1] = value
        s, cache, q, st = run(lens)
        assert st == 8
        s.new[1] = 0
        want = s.ref_append()
        assert_cache(cache, s)
        assert np.isnan(q[1]).all() and np.array_equal(q[[0, 2]], want[[0, 2]])
    s = Setup(27, **base)     # positions beyond the table of angles
    s.cs = s.cs[:18]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = s.append(s.cache(), status=status)
    assert status.item() == 0 and torch.isfinite(q).all()
    s.cs = s.cs[:17]
    q = s.append(s.cache(), status=status)
    assert status.item() == 8 and torch.isnan(q[1]).all() and torch.isfinite(q[[0, 2]]).all()


# --------------------------------------------------------------------------
# attention

ATTEND = [
    # B, T, Hq, Hkv, D, S, seq, new, dtype, window
    (1, 1, 1, 1, 64, 16, [0], [1], "bf16", 0),
    (1, 1, 8, 2, 128, 16, [1], [1], "bf16", 0),
    (3, 5, 8, 2, 128, 16, [0, 127, 300], [5, 5, 2], "bf16", 0),
    (3, 5, 8, 2, 128, 64, [124, 128, 129], [5, 0, 5], "bf16", 0),
    (2, 9, 16, 2, 128, 32, [500, 250], [9, 4], "bf16", 0),            # 72 rows a key/value head
    (2, 4, 4, 4, 64, 32, [333, 70], [4, 1], "bf16", 0),               # one query head each
    (2, 3, 24, 1, 64, 128, [700, 0], [3, 3], "bf16", 0),              # one key/value head
    (2, 5, 12, 4, 128, 16, [300, 60], [5, 5], "bf16", 100),           # window
    (2, 5, 4, 2, 64, 16, [300, 0], [5, 5], "bf16", 1),                # a query sees itself alone
    (2, 5, 4, 2, 64, 16, [300, 128], [5, 5], "bf16", 128),
    (2, 150, 4, 2, 128, 64, [90, 0], [150, 130], "bf16", 0),          # part of a prompt
    (1, 140, 3, 1, 64, 16, [200], [140], "bf16", 33),
    (2, 3, 4, 2, 80, 16, [100, 31], [3, 3], "bf16", 0),               # other head sizes
    (2, 3, 4, 2, 256, 32, [140, 31], [3, 3], "bf16", 50),
    (2, 3, 4, 2, 16, 16, [100, 31], [3, 3], "f32", 0),
    (3, 5, 8, 2, 128, 16, [0, 127, 300], [5, 5, 2], "f32", 0),
    (2, 20, 3, 3, 64, 128, [200, 0], [20, 20], "f32", 64),
    (2, 3, 4, 2, 256, 32, [140, 31], [3, 3], "f32", 0),
]


@gpu
@pytest.mark.parametrize("i", range(len(ATTEND)))
@pytest.mark.parametrize("token_major", [False, True])
def test_attention_against_64_bits(i, token_major):
    """New tokens are stored first; slots no sequence holds are NaN and page numbers past the lengths are invalid."""
    import speculative_sampling_verification_spec_gb300 as sv
    B, T, Hq, Hkv, D, S, seq, new, dtype, window = ATTEND[i]
    s = Setup(200 + i, B, T, Hq, Hkv, D, S, seq, new, dtype, token_major=token_major)
    cache = s.cache()
    s.append(cache)
    s.ref_append()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = sv.spec_kv_attention(s.dev(s.q), cache, *s.idx(), window=window, return_lse=True, status=status)
    assert_attention(out, lse, s.ref_attention(window=window))
    assert status.item() == 0
    again = sv.spec_kv_attention(s.dev(s.q), cache, *s.idx(), window=window)
    assert torch.equal(out, again)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,seq,T,Hq,Hkv,window", [(16, 40000, 1, 4, 1, 0), (64, 20011, 5, 8, 2, 0), (128, 9000, 2, 2, 2, 5000)])
def test_attention_shared_by_many_ranges(dtype, S, seq, T, Hq, Hkv, window):
    """One long sequence beside short ones: its heads are cut into many ranges and joined; twice the same bits."""
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(31, 3, T, Hq, Hkv, 64, S, [seq, 3, 260], [T, T, T], dtype)
    cache = s.cache()
    s.append(cache)
    s.ref_append()
    out, lse = sv.spec_kv_attention(s.dev(s.q), cache, *s.idx(), window=window, return_lse=True)
    assert_attention(out, lse, s.ref_attention(window=window))
    for _ in range(3):
        o2, l2 = sv.spec_kv_attention(s.dev(s.q), cache, *s.idx(), window=window, return_lse=True)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_size,magnitude,pow2", [(30.0, 1.0, True), (1e-3, 1.0, True), (1.0, 1e-6, True), (1.0, 1e6, False),
                                                   (4.0, 1.0, False)])
def test_attention_of_peaked_flat_and_scaled_inputs(dtype, q_size, magnitude, pow2):
    """Scores from nearly one-hot to nearly equal; scales far from 1 and not powers of two, differing page by page."""
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(32, 2, 4, 6, 2, 128, 16, [517, 100], [4, 3], dtype, q_size=q_size / magnitude, magnitude=magnitude, pow2=pow2)
    s.k *= np.float32(magnitude)
    s.v *= np.float32(magnitude)
    if dtype == "bf16":
        s.k, s.v = kv_ref.bf16_round(s.k), kv_ref.bf16_round(s.v)
    cache = s.cache()
    s.append(cache)
    s.ref_append()
    assert_cache(cache, s)
    out, lse = sv.spec_kv_attention(s.dev(s.q), cache, *s.idx(), return_lse=True)
    assert_attention(out, lse, s.ref_attention())


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_rows_are_independent(dtype):
    """Rows of very different sizes in one call, and one row of NaN and infinities: the others are as without it."""
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(33, 2, 4, 4, 1, 64, 16, [300, 50], [4, 4], dtype)
    s.q *= np.exp2(np.arange(4) * 4 - 10).astype(np.float32)[None, :, None, None]
    cache = s.cache()
    s.append(cache)
    s.ref_append()
    out, lse = sv.spec_kv_attention(s.dev(s.q), cache, *s.idx(), return_lse=True)
    assert_attention(out, lse, s.ref_attention())
    bad = s.dev(s.q)
    bad[0, 1, 2, 5], bad[1, 3, 0, 0] = math.nan, math.inf
    o2, l2 = sv.spec_kv_attention(bad, cache, *s.idx(), return_lse=True)
    hit = torch.zeros(2, 4, 4, dtype=torch.bool, device="cuda")
    hit[0, 1, 2] = hit[1, 3, 0] = True
    assert torch.isnan(o2[hit]).all() and torch.isnan(l2[hit]).all()
    assert torch.equal(o2[~hit], out[~hit]) and torch.equal(l2[~hit], lse[~hit])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("window", [0, 40])
def test_attention_nan_tokens_touch_the_rows_that_see_them(dtype, what, window):
    """A NaN in the third of five new tokens, and one just outside the first query's window."""
    import speculative_sampling_verification_spec_gb300 as sv
    for at in (302, 260):
        s = Setup(34, 1, 5, 4, 2, 64, 16, [300], [5], dtype)
        cache = s.cache()
        s.append(cache)
        s.ref_append()
        ref = s.ref_attention(window=window)
        codes = cache.k_codes if what == "k" else cache.v_codes
        codes.view(torch.uint8)[int(s.table[0, at // 16]), 1, at % 16, 9] = 0x7F
        out, lse = sv.spec_kv_attention(s.dev(s.q), cache, *s.idx(), window=window, return_lse=True)
        sees = np.zeros((1, 5, 4), bool)
        for t in range(5):
            p = 300 + t
            sees[0, t, 2:] = at <= p and (window == 0 or at > p - window)
        o = out.float().cpu().numpy()
        assert np.isnan(o[..., 9][sees]).all()
        if what == "k":
            assert np.isnan(o[sees]).all() and torch.isnan(lse.cpu()[torch.from_numpy(sees)]).all()
        sel = ~sees
        assert np.isfinite(o[sel]).all()
        assert np.all(np.abs(o[sel] - ref[0][sel]) <= ref[2][sel])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_strides_streams_and_workspaces(dtype):
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(35, 3, 5, 8, 2, 128, 32, [50, 400, 0], [5, 3, 5], dtype)
    cache = s.cache()
    s.append(cache)
    s.ref_append()
    want = s.ref_attention(scale=0.05)
    q = s.dev(s.q)
    wide = torch.zeros(3, 5, 8 * 128 + 24, dtype=DT[dtype], device="cuda")
    for off in (0, 8, 1):
        qv = wide[..., off:off + 1024].unflatten(-1, (8, 128))
        qv.copy_(q)
        out = torch.full((8, 3, 5, 128 + off), 7.0, dtype=DT[dtype], device="cuda")[..., off:].permute(1, 2, 0, 3)
        lse = torch.empty(3, 5, 8, device="cuda")
        got = sv.spec_kv_attention(qv, cache, *s.idx(), scale=0.05, out=out, lse=lse)
        assert got[0] is out and got[1] is lse
        assert_attention(out, lse, want)
    n = sv.spec_kv_attention_workspace_size(cache, 3, 5, 8, DT[dtype])
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:65536] = 0      # the counters: calls leave them at zero, the rest needs no clearing
    for _ in range(2):
        out, lse = sv.spec_kv_attention(q, cache, *s.idx(), scale=0.05, return_lse=True, ws=ws)
        assert_attention(out, lse, want)
        assert not ws[:65536].any()
    with pytest.raises(sv.SpecError):
        sv.spec_kv_attention(q, cache, *s.idx(), ws=ws[:n - 256])
    # another stream than the current one, with the queries made there
    idx = s.idx()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        q2 = q * 1.0
    out2, lse2 = sv.spec_kv_attention(q2, cache, *idx, scale=0.05, return_lse=True, stream=side)
    side.synchronize()
    assert torch.equal(out2, out) and torch.equal(lse2, lse)


@gpu
def test_one_workspace_for_calls_of_many_shapes():
    """Shapes whose items are joined by their last CTA, by a kernel of its own, or not at all, in turn on one workspace;
    and more items than the workspace has standing counters for."""
    import speculative_sampling_verification_spec_gb300 as sv
    shapes = [(1, 1, 4, 1, [3000], "bf16"), (2, 40, 8, 2, [2000, 77], "bf16"), (1, 5, 8, 2, [5000], "f32"),
              (1, 20, 4, 1, [4000], "f32"), (3, 3, 4, 4, [10, 500, 0], "bf16"), (1, 1, 4, 1, [3000], "bf16")]
    runs = []
    for i, (B, T, Hq, Hkv, seq, dtype) in enumerate(shapes):
        s = Setup(60 + i, B, T, Hq, Hkv, 64, 16, seq, [T] * B, dtype)
        cache = s.cache()
        s.append(cache)
        s.ref_append()
        runs.append((s, cache, s.dev(s.q), s.idx(), s.ref_attention()))
    ws = torch.zeros(max(sv.spec_kv_attention_workspace_size(c, s.B, s.T, s.Hq, DT[s.dtype]) for s, c, *_ in runs),
                     dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for s, cache, q, idx, want in runs:
            out, lse = sv.spec_kv_attention(q, cache, *idx, return_lse=True, ws=ws)
            assert_attention(out, lse, want)
    # 4500 sequences x 4 heads: a few long ones are shared by ranges
    B = 4500
    seq = np.where(np.arange(B) % 900 == 0, 3000, np.arange(B) % 7)
    s = Setup(70, B, 1, 4, 4, 64, 16, seq, [1] * B, "bf16")
    cache = s.cache()
    s.append(cache)
    s.ref_append()
    want = s.ref_attention()
    for _ in range(2):
        out, lse = sv.spec_kv_attention(s.dev(s.q), cache, *s.idx(), return_lse=True)
        assert_attention(out, lse, want)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_device_errors(dtype):
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(36, 3, 4, 4, 2, 64, 16, [50, 90, 3], [4, 4, 4], dtype)
    cache = s.cache()
    s.append(cache)
    q = s.dev(s.q)
    out, lse = sv.spec_kv_attention(q, cache, *s.idx(), return_lse=True)
    for value in (-1, 1 << 30):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        table, seq, new = s.idx()
        table[1, 2] = value
        o, l = sv.spec_kv_attention(q, cache, table, seq, new, return_lse=True, status=status)
        assert status.item() == 8 and torch.isnan(o[1]).all() and torch.isnan(l[1]).all()
        assert torch.equal(o[[0, 2]], out[[0, 2]]) and torch.equal(l[[0, 2]], lse[[0, 2]])
    for which, value in ((1, -1), (1, 1 << 30), (2, 5), (2, -1), (1, 2147483647)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        idx = s.idx()
        idx[which][1] = value
        o, l = sv.spec_kv_attention(q, cache, *idx, return_lse=True, status=status)
        assert status.item() == 8 and torch.isnan(o[1]).all() and torch.isnan(l[1]).all()
        assert torch.equal(o[[0, 2]], out[[0, 2]]) and torch.equal(l[[0, 2]], lse[[0, 2]])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_beyond_32_bits(dtype):
    """A pool of more than 2^32 bytes of codes: the last pages' addresses need 64 bits."""
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(37, 2, 3, 2, 1, 128, 16, [40, 15], [3, 3], dtype, rot=128)
    N = (1 << 32) // (16 * 128) + 64
    shift = N - s.N
    codes = [torch.zeros(N, 1, 16, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(N, 1, device="cuda") for _ in range(2)]
    for t, x in zip(codes + scales, (s.kc, s.vc, s.ks, s.vs)):
        t[shift:] = torch.from_numpy(x).cuda()
    big = sv.PagedKVCache(*codes, *scales)
    small = s.cache()
    table, seq, new = s.idx()
    cs = torch.from_numpy(s.cs).cuda()
    q1 = sv.spec_kv_append(s.dev(s.q), s.dev(s.k), s.dev(s.v), small, table, seq, new, cos_sin=cs)
    q2 = sv.spec_kv_append(s.dev(s.q), s.dev(s.k), s.dev(s.v), big, table + shift, seq, new, cos_sin=cs)
    assert torch.equal(q1, q2)
    assert torch.equal(big.k_codes[shift:], small.k_codes) and torch.equal(big.v_codes[shift:], small.v_codes)
    assert torch.equal(big.k_scale[shift:], small.k_scale) and not big.k_codes[:shift].any()
    assert torch.equal(sv.spec_kv_attention(q1, small, table, seq, new),
                       sv.spec_kv_attention(q1, big, table + shift, seq, new))


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rounds_with_rejected_tokens(dtype):
    """Rounds as a speculative decoder runs them: append T tokens, attend, keep some, go on from the shorter length."""
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(38, 3, 5, 4, 2, 64, 16, [0, 30, 61], [5, 5, 5], dtype, rot=64)
    cols = 8
    s.N = 3 * cols
    s.table = s.g.permutation(s.N).reshape(3, cols).astype(np.int32)
    s.kc, s.vc = np.full((s.N, 2, 16, 64), 0x7F, np.uint8), np.full((s.N, 2, 16, 64), 0x7F, np.uint8)
    s.ks, s.vs = np.zeros((s.N, 2), np.float32), np.zeros((s.N, 2), np.float32)
    s.seq = np.zeros(3, np.int32)
    ang = np.arange(cols * 16)[:, None] * (10000.0 ** (-np.arange(32) / 32))
    s.cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    cache = s.cache()
    for r in range(12):
        s.k, s.v = s.values(3, 5, 2, 64) * np.float32(1 + r % 4), s.values(3, 5, 2, 64)
        s.k = kv_ref.bf16_round(s.k) if dtype == "bf16" else s.k
        s.q = s.values(3, 5, 4, 64)
        s.new = s.g.integers(1, 6, 3).astype(np.int32)
        raw = s.q
        got = s.append(cache)
        s.q = s.ref_append()
        assert np.array_equal(got.float().cpu().numpy(), s.q)
        assert_cache(cache, s)
        out, lse = sv.spec_kv_attention(got, cache, *s.idx(), return_lse=True)
        assert_attention(out, lse, s.ref_attention(), "round %d" % r)
        s.q = raw
        s.seq = s.seq + np.minimum(s.new, s.g.integers(1, 6, 3)).astype(np.int32)


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pad", [0, 16, 64])
def test_padded_pools(D, pad):
    """Token slots `pad` bytes apart beyond their channels: strides that a tensor map holds and strides that it does
    not (another kernel then) give the definition's results; so does a pool of one page and one head."""
    import speculative_sampling_verification_spec_gb300 as sv
    for B, Hkv, seq, new in ((2, 2, [37, 300], [3, 2]), (1, 1, [5], [3])):
        s = Setup(40, B, 3, 4, Hkv, D, 16, seq, new, "bf16", rot=D)
        if B == 1:      # one page
            keep = int(s.table[0, 0])
            s.kc, s.vc, s.ks, s.vs = (x[keep:keep + 1].copy() for x in (s.kc, s.vc, s.ks, s.vs))
            s.table, s.cs, s.N = np.zeros((1, 1), np.int32), s.cs[:16], 1
        codes = []
        for x in (s.kc, s.vc):
            wide = torch.full((s.N, Hkv, 16, D + pad), 0x7F, dtype=torch.uint8, device="cuda")
            wide[..., :D] = torch.from_numpy(x).cuda()
            codes.append(wide[..., :D])
        cache = sv.PagedKVCache(*codes, torch.from_numpy(s.ks).cuda(), torch.from_numpy(s.vs).cuda())
        q = s.append(cache)
        raw = s.q
        s.q = s.ref_append()
        assert np.array_equal(q.float().cpu().numpy(), s.q)
        assert_cache(cache, s)
        if pad:
            assert all((c._base if c._base is not None else c)[..., D:].eq(0x7F).all() for c in codes)
        out, lse = sv.spec_kv_attention(q, cache, *s.idx(), return_lse=True)
        assert_attention(out, lse, s.ref_attention())
        s.q = raw


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_calls_replay_from_a_graph(dtype):
    """Append and attention captured once and replayed with other lengths, queries and tokens in the same tensors give
    what direct calls give: lengths and page numbers are read on the device."""
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(41, 3, 4, 8, 2, 64, 16, [20, 400, 0], [4, 2, 3], dtype, rot=64)
    a, b = s.cache(), s.cache()
    table, seq, new = s.idx()
    cs = torch.from_numpy(s.cs).cuda()
    q, k, v = s.dev(s.q), s.dev(s.k), s.dev(s.v)

    def step(cache):
        r = sv.spec_kv_append(q, k, v, cache, table, seq, new, cos_sin=cs)
        return sv.spec_kv_attention(r, cache, table, seq, new, return_lse=True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a)             # makes the stream's workspace
        a = s.cache()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step(a)
    torch.cuda.current_stream().wait_stream(side)
    for seqs, news in (([20, 400, 0], [4, 2, 3]), ([22, 402, 3], [4, 4, 0]), ([24, 250, 3], [1, 4, 4])):
        seq.copy_(torch.tensor(seqs, dtype=torch.int32))
        new.copy_(torch.tensor(news, dtype=torch.int32))
        q.copy_(s.dev(s.values(3, 4, 8, 64)))
        k.copy_(s.dev(s.values(3, 4, 2, 64)))
        graph.replay()
        want = step(b)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(a.k_codes.view(torch.uint8), b.k_codes.view(torch.uint8))
        assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)


@gpu
def test_capture_on_a_fresh_stream():
    """A call captured on a stream that has no workspace yet: the graph's is its own, so a direct call on that stream,
    before and after a replay, finds cleared counters."""
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(42, 1, 1, 4, 1, 64, 16, [3000], [1], "bf16")
    cache = s.cache()
    s.append(cache)
    s.ref_append()
    want = s.ref_attention()
    q, idx = s.dev(s.q), s.idx()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    key = (torch.cuda.current_device(), side.cuda_stream)
    sv.kv_cache._ws_cache.pop(key, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = sv.spec_kv_attention(q, cache, *idx, return_lse=True)
    assert key not in sv.kv_cache._ws_cache
    for _ in range(2):
        with torch.cuda.stream(side):
            direct = sv.spec_kv_attention(q, cache, *idx, return_lse=True)
            graph.replay()
        side.synchronize()
        assert_attention(*direct, want)
        assert_attention(*got, want)


@gpu
def test_python_checks():
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(39, 2, 3, 4, 2, 64, 16, [5, 6], [3, 3], "bf16", 64)
    cache = s.cache()
    table, seq, new = s.idx()
    q, k, v = s.dev(s.q), s.dev(s.k), s.dev(s.v)
    cs = torch.from_numpy(s.cs).cuda()
    bad = [lambda: sv.spec_kv_append(q.float(), k, v, cache, table, seq, new),
           lambda: sv.spec_kv_append(q, k, v[:, :, :1], cache, table, seq, new),
           lambda: sv.spec_kv_append(q, k[..., :32], v[..., :32], cache, table, seq, new),
           lambda: sv.spec_kv_append(q, k.cpu(), v, cache, table, seq, new),
           lambda: sv.spec_kv_append(q, k, v.cpu(), cache, table, seq, new),
           lambda: sv.spec_kv_append(q, k, v, cache, table.long(), seq, new),
           lambda: sv.spec_kv_append(q, k, v, cache, table, seq.long(), new),
           lambda: sv.spec_kv_append(q, k, v, cache, table, seq, new[:1]),
           lambda: sv.spec_kv_append(q, k, v, cache, table, seq, new.cpu()),
           lambda: sv.spec_kv_append(q, k, v, cache, table, seq, new, cos_sin=cs.double()),
           lambda: sv.spec_kv_append(q, k, v, cache, table, seq, new, q_out=q.float()),
           lambda: sv.spec_kv_append(None, k, v, cache, table, seq, new, q_out=q),
           lambda: sv.spec_kv_append(q.half(), k.half(), v.half(), cache, table, seq, new),
           lambda: sv.spec_kv_attention(q[..., ::2], cache, table, seq, new),
           lambda: sv.spec_kv_attention(q[:, :, :, :32], cache, table, seq, new),
           lambda: sv.spec_kv_attention(q.cpu(), cache, table, seq, new),
           lambda: sv.spec_kv_attention(q, cache, table[:1], seq, new),
           lambda: sv.spec_kv_attention(q, cache, table, seq, new, lse=torch.empty(2, 3, 4, device="cuda").double()),
           lambda: sv.PagedKVCache(cache.k_codes, cache.v_codes[:1], cache.k_scale, cache.v_scale),
           lambda: sv.PagedKVCache(cache.k_codes.cpu(), cache.v_codes, cache.k_scale, cache.v_scale),
           lambda: sv.PagedKVCache(cache.k_codes, cache.v_codes, cache.k_scale.double(), cache.v_scale)]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            pytest.fail("call %d was accepted" % i)
    for f in (lambda: sv.spec_kv_attention(q[:, :, :3], cache, table, seq, new),      # 3 query heads over 2
              lambda: sv.spec_kv_attention(q, cache, table, seq, new, window=-1),
              lambda: sv.spec_kv_attention(q, cache, table, seq, new, scale=math.nan)):
        with pytest.raises(sv.SpecError):
            f()
    empty = sv.PagedKVCache.empty(4, 16, 2, 64)
    assert empty.nbytes() == 4 * 2 * 16 * 64 * 2 + 4 * 2 * 4 * 2
