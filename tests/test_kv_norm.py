"""Norms of queries and keys with the append: queries, codes and scales equal to the definition's, whose norm factor is the
nearest float to the one computed in float64."""
import math

import numpy as np
import pytest
import torch

import kv_ref
from test_kv_cache import L, Setup, _pack, assert_cache  # noqa: F401

gpu = pytest.mark.gpu
EPS = 1e-6


def normalise(x, w, eps):
    """x [..., H, D] float32, w [D] or [H, D]: (x r) w, each product rounded to float32."""
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        y = x.astype(np.float64)
        r = (1.0 / np.sqrt((y * y).mean(-1, keepdims=True) + np.float64(np.float32(eps)))).astype(np.float32)
        return (x * r) * w


def weights(g, *shape):
    return (1 + 0.3 * g.standard_normal(shape)).astype(np.float32)


def ref_append(s, qw, kw, eps=EPS):
    """Setup.ref_append on normalised queries and keys (rotation and rounding to the type come after)."""
    q, k = s.q, s.k
    s.q, s.k = (q if qw is None else normalise(q, qw, eps)), (k if kw is None else normalise(k, kw, eps))
    out = s.ref_append()
    s.q, s.k = q, k
    return out


def append(s, cache, qw, kw, eps=EPS, **kw2):
    dev = {n: None if w is None else torch.from_numpy(np.ascontiguousarray(w)).cuda()
           for n, w in (("q_norm", qw), ("k_norm", kw))}
    return s.append(cache, **dict(dev, norm_eps=eps, **kw2))


# --------------------------------------------------------------------------
# refusals (CPU)

def _norms(qw=0xD000, kw=0xE000, qh=0, kh=0, eps=EPS):
    from speculative_sampling_verification_spec_gb300 import kv_cache
    return kv_cache._NORMS.pack(qw, kw, qh, kh, eps)


@pytest.mark.parametrize("over", [dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(eps=1e-25),
                                  dict(eps=1.2e12), dict(qh=-1), dict(kh=-64), dict(qw=0xD002), dict(kw=0xE001)], ids=str)
def test_refuses(L, over):  # noqa: F811
    c, p = _pack({})
    assert L.spec_kv_append_norm(0x8000, 0xA000, 0xB000, 0xC000, _norms(**over), c, p, 0x9000) == 1


def test_refuses_as_append_does(L):  # noqa: F811
    c, p = _pack({})
    assert L.spec_kv_append_norm(None, 0xA000, 0xB000, None, _norms(), c, p, None) == 1        # query weights without queries
    for over in (dict(T=0), dict(D=24), dict(k1=-1), dict(rot_dim=3, rot_len=9)):
        assert L.spec_kv_append_norm(0x8000, 0xA000, 0xB000, 0xC000, _norms(), *_pack(over), 0x9000) == 1, over
    c, p = _pack(dict(B=0))
    assert L.spec_kv_append_norm(0x8000, 0xA000, 0xB000, None, _norms(), c, p, 0x9000) == 0    # nothing to do


@gpu
def test_python_checks():
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(600, 1, 2, 4, 2, 64, 16, [3], [2], "bf16")
    cache = s.cache()
    w = torch.ones(64, device="cuda")
    for bad in (w.double(), w[:63], torch.ones(4, 64, device="cuda"), torch.ones(64, 2, device="cuda")[:, 0], w.cpu()):
        with pytest.raises(ValueError):
            s.append(cache, k_norm=bad)
    with pytest.raises(ValueError):
        s.append(cache, q_norm=torch.ones(2, 64, device="cuda"))
    with pytest.raises(ValueError):
        sv.spec_kv_append(None, s.dev(s.k), s.dev(s.v), cache, *s.idx(), q_norm=w)
    with pytest.raises(sv.SpecError):
        s.append(cache, q_norm=w, norm_eps=0.0)


# --------------------------------------------------------------------------
# values

CASES = [
    # B, T, Hq, Hkv, D, S, seq, new, dtype, rot, interleaved
    (1, 1, 8, 2, 128, 16, [0], [1], "bf16", 128, False),
    (1, 1, 32, 8, 128, 16, [31], [1], "bf16", 128, False),
    (4, 5, 8, 2, 128, 16, [0, 14, 16, 31], [5, 5, 0, 3], "bf16", 128, False),
    (3, 9, 6, 3, 64, 32, [30, 7, 64], [9, 1, 9], "bf16", 32, True),
    (3, 9, 6, 3, 64, 32, [30, 7, 64], [9, 1, 9], "f32", 32, False),
    (2, 17, 2, 1, 80, 16, [3, 0], [17, 16], "f32", 80, False),        # five chunks a head: idle threads; halves of 40
    (2, 17, 6, 3, 96, 16, [3, 0], [17, 16], "bf16", 96, False),       # six
    (2, 17, 4, 2, 240, 16, [3, 0], [17, 16], "bf16", 240, True),      # fifteen
    (2, 3, 4, 2, 48, 16, [3, 20], [3, 2], "bf16", 10, False),         # 10 of 48 channels: single pairs
    (2, 3, 4, 2, 48, 16, [3, 20], [3, 2], "f32", 10, True),
    (2, 40, 3, 1, 176, 32, [3, 20], [40, 39], "bf16", 6, False),      # single pairs, more than a warp of them
    (2, 70, 3, 3, 16, 16, [5, 0], [70, 33], "bf16", 0, False),        # one chunk a head, no rotation
    (2, 300, 4, 2, 128, 128, [100, 0], [300, 256], "bf16", 128, False),
    (1, 200, 2, 1, 256, 128, [1], [200], "f32", 256, False),          # a unit larger than a CTA's registers
    (3, 700, 16, 4, 128, 64, [0, 50, 64], [700, 650, 3], "bf16", 128, False),     # several heads a query thread
]


@gpu
@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("per_head", [False, True])
def test_equals_the_definition(i, per_head):
    B, T, Hq, Hkv, D, S, seq, new, dtype, rot, inter = CASES[i]
    s = Setup(610 + i, B, T, Hq, Hkv, D, S, seq, new, dtype, rot, inter)
    qw, kw = (weights(s.g, Hq, D), weights(s.g, Hkv, D)) if per_head else (weights(s.g, D), weights(s.g, D))
    s.q *= np.float32(4)
    cache = s.cache()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(2):        # the second call writes the same again
        q = append(s, cache, qw, kw, status=status)
    want = ref_append(s, qw, kw)
    assert np.array_equal(q.float().cpu().numpy(), want)
    assert_cache(cache, s)
    assert status.item() == 0


@gpu
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64), ("bf16", 96), ("f32", 256)])
@pytest.mark.parametrize("off", [0, 1])
def test_one_side_strides_and_in_place(dtype, D, off):
    """Weights for the queries or the keys alone; inputs out of a fused projection, aligned or not; queries in place."""
    for qn, kn in ((True, False), (False, True), (True, True)):
        s = Setup(640, 3, 5, 4, 2, D, 16, [0, 13, 40], [5, 4, 5], dtype, D)
        fused = torch.zeros(3, 5, 8 * D + 8, dtype=s.dev(s.q).dtype, device="cuda")
        q, k, v = (fused[..., off + a * D:off + b * D].unflatten(-1, (b - a, D)) for a, b in ((0, 4), (4, 6), (6, 8)))
        for d, x in ((q, s.q), (k, s.k), (v, s.v)):
            d.copy_(torch.from_numpy(x).cuda())
        qw, kw = weights(s.g, D) if qn else None, weights(s.g, D) if kn else None
        cache = s.cache()
        assert append(s, cache, qw, kw, q=q, k=k, v=v, q_out=q) is q
        want = ref_append(s, qw, kw)
        assert np.array_equal(q.float().cpu().numpy(), want)
        assert_cache(cache, s)
    # weights that begin off a 16-byte boundary
    s = Setup(641, 2, 3, 4, 2, D, 16, [5, 16], [3, 2], dtype, D)
    buf = torch.zeros(2 * D + 3, device="cuda")
    qw, kw = weights(s.g, D), weights(s.g, D)
    buf[1:1 + D].copy_(torch.from_numpy(qw))
    buf[2 + D:2 + 2 * D].copy_(torch.from_numpy(kw))
    cache = s.cache()
    q = s.append(cache, q_norm=buf[1:1 + D], k_norm=buf[2 + D:2 + 2 * D])
    want = ref_append(s, qw, kw)
    assert np.array_equal(q.float().cpu().numpy(), want)
    assert_cache(cache, s)


@gpu
@pytest.mark.parametrize("dtype,D,rot", [("bf16", 128, 128), ("f32", 80, 80), ("bf16", 48, 10), ("f32", 256, 0)])
def test_sizes_of_heads(dtype, D, rot):
    """Heads of magnitudes from 2^-70 to 2^126, one of zeros, one with one large channel among small ones; eps from 2^-80
    to 2^40."""
    for eps in (2.0 ** -80, 1e-12, 1e-6, 1.0, 2.0 ** 40):
        s = Setup(650, 1, 24, 3, 3, D, 32, [0], [24], dtype, rot)
        size = np.exp2(np.linspace(-70, 123, 22)).astype(np.float32)[None, :, None, None]
        for x in (s.q, s.k):
            x[:, :22] *= size
            x[:, 22] = 0
            x[:, 23, :, 1:] *= np.float32(2.0 ** -30)
            if dtype == "bf16":
                x[:] = kv_ref.bf16_round(x)
            assert np.isfinite(x).all()
        qw, kw = weights(s.g, D), weights(s.g, D)
        cache = s.cache()
        q = append(s, cache, qw, kw, eps)
        want = ref_append(s, qw, kw, eps)
        assert np.array_equal(q.float().cpu().numpy(), want), eps
        assert_cache(cache, s)


@gpu
@pytest.mark.parametrize("dtype,D,rot", [("bf16", 128, 128), ("bf16", 48, 10), ("f32", 80, 0)])
def test_special_values(dtype, D, rot):
    """A head with a NaN is NaN; one with an infinity is zero but for that channel's NaN (and what it is rotated with)."""
    s = Setup(660, 2, 4, 4, 2, D, 16, [3, 14], [4, 4], dtype, rot)
    for x in (s.q, s.k):
        x[0, 1, 0, 5] = np.nan
        x[1, 2, 1, 7] = np.inf
        x[1, 3, 0, D - 1] = -np.inf
    qw, kw = weights(s.g, D), weights(s.g, D)
    cache = s.cache()
    q = append(s, cache, qw, kw).float().cpu().numpy()
    want = ref_append(s, qw, kw)
    assert np.isnan(want[0, 1, 0]).all() and np.isnan(want[1, 2, 1]).any() and np.isfinite(want[0, 0]).all()
    assert np.array_equal(q, want, equal_nan=True)
    assert_cache(cache, s)


@gpu
def test_norm_against_64_bits():
    """The normalised queries, not rotated, against float64: the factor's rounding and two products', 2^-24 each."""
    s = Setup(670, 2, 9, 4, 2, 128, 16, [100, 3], [9, 9], "f32")
    w = weights(s.g, 128)
    q = append(s, s.cache(), w, w).double().cpu().numpy()
    x = s.q.astype(np.float64)
    want = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(EPS))) * w
    assert np.all(np.abs(q - want) <= 3.01 * kv_ref.U * np.abs(want))


@gpu
def test_device_errors_and_empty_slots():
    """As without norms: slots past the new tokens are zero, a sequence out of range is left out and NaN."""
    for D, rot in ((64, 64), (48, 6)):
        s = Setup(680, 3, 3, 4, 2, D, 16, [5, 9, 7], [2, 3, 0], "bf16", rot)
        w = weights(s.g, D)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        s.seq[1] = 1 << 20
        q = append(s, s.cache(), w, w, status=status)
        assert status.item() == 8
        assert torch.isnan(q[1]).all() and (q[0, 2] == 0).all() and (q[2] == 0).all() and torch.isfinite(q[0]).all()


@gpu
def test_graph_and_stream():
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(690, 2, 4, 8, 2, 128, 16, [30, 5], [4, 3], "bf16", 128)
    w = torch.from_numpy(weights(s.g, 128)).cuda()
    cache, ref = s.cache(), s.cache()
    x, idx = [s.dev(t) for t in (s.q, s.k, s.v)], s.idx()
    args = dict(cos_sin=torch.from_numpy(s.cs).cuda(), q_norm=w, k_norm=w)
    want = sv.spec_kv_append(*x, ref, *idx, **args)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_kv_append(*x, cache, *idx, q_out=out, **args)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert torch.equal(cache.k_codes.view(torch.uint8), ref.k_codes.view(torch.uint8)) and torch.equal(cache.k_scale, ref.k_scale)
    side, other = torch.cuda.Stream(), s.cache()
    side.wait_stream(torch.cuda.current_stream())
    got = sv.spec_kv_append(*x, other, *idx, stream=side, **args)
    side.synchronize()
    assert torch.equal(got, want)
