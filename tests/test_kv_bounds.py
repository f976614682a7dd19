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


@gpu
@pytest.mark.parametrize("order", ["small first", "large first", "alternating"])
@pytest.mark.parametrize("large,small", [(60, -100), (20, -100), (120, -100), (120, 10)])
@pytest.mark.parametrize("B", [1, 304])         # one sequence cut into many ranges, or one range for each
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_value_scales_far_apart(order, large, small, B, dtype, D):
    """Half of the pages have value scales of 2^large, half of 2^small (what an append of zeros leaves): the tokens of
    both count in the sum of the weights."""
    import speculative_sampling_verification_spec_gb300 as sv
    g = torch.Generator(device="cuda").manual_seed(5)
    S, n = 16, 1024
    pages = n // S
    i = torch.arange(pages, device="cuda")
    big = {"small first": i >= pages // 2, "large first": i < pages // 2, "alternating": i % 2 == 0}[order]
    kc, vc = (torch.randn(pages, 1, S, D, generator=g, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    vs = torch.where(big, 2.0 ** large, 2.0 ** small).double().float()[:, None].contiguous()
    q = torch.randn(1, 1, 4, D, generator=g, device="cuda").expand(B, 1, 4, D).to(DT[dtype])
    table = i.to(torch.int32).expand(B, pages).contiguous()
    seq = torch.full((B,), n - 1, dtype=torch.int32, device="cuda")
    cache = sv.PagedKVCache(kc, vc, torch.ones_like(vs), vs)
    out, lse = sv.spec_kv_attention(q, cache, table, seq, scale=0.1, return_lse=True)
    k, v = kc.double().reshape(n, D), (vc.double() * vs.double()[:, :, None, None]).reshape(n, D)
    s = q[0, 0].double() @ k.T * 0.1
    w = torch.softmax(s, 1)
    tol = (2.0 ** -8 if dtype == "bf16" else 2.0 ** -15) * (w @ v.abs()) + 2.0 ** -9 * (w @ v).abs()
    assert ((out[:, 0].double() - w @ v).abs() <= tol).all()
    assert ((lse[:, 0].double() - torch.logsumexp(s, 1)).abs() <= 2.0 ** -11).all()


@gpu
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 80), ("f32", 64), ("f32", 256)])
@pytest.mark.parametrize("n", [3, 100, 9000])
@pytest.mark.parametrize("size", [1e20, 1e32])
def test_scores_far_below_zero(dtype, D, n, size):
    """Scores of -2 * size for one token and -4 * size and less for the others: all of the weight is the one's."""
    import speculative_sampling_verification_spec_gb300 as sv
    g = torch.Generator(device="cuda").manual_seed(6)
    S, pages = 16, -(-n // 16)
    k = torch.randint(4, 9, (pages, 1, S, D), generator=g, device="cuda").float()
    at = n // 3
    k[at // S, 0, at % S] = 2
    v = torch.randn(pages, 1, S, D, generator=g, device="cuda").to(torch.float8_e4m3fn)
    one = torch.ones(pages, 1, device="cuda")
    cache = sv.PagedKVCache(k.to(torch.float8_e4m3fn), v, one, one.clone())
    q = torch.zeros(1, 1, 2, D, device="cuda")
    q[..., 0] = -size
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    seq = torch.full((1,), n - 1, dtype=torch.int32, device="cuda")
    q = q.to(DT[dtype])
    out, lse = sv.spec_kv_attention(q, cache, table, seq, scale=1.0, return_lse=True)
    assert torch.equal(out[0, 0].float(), v[at // S, 0, at % S].float().expand(2, D))
    want = 2 * q[0, 0, 0, 0].double().item()
    assert (lse.double() / want - 1).abs().max().item() < 1e-6


@gpu
def test_far_joined_parts():
    """Parts whose largest scores are far apart: the lower ones add nothing, whatever their size."""
    import speculative_sampling_verification_spec_gb300 as sv
    n, S, D = 4096, 16, 64
    for dtype in ("bf16", "f32"):
        k = torch.zeros(n // S, 1, S, D, device="cuda")
        k.view(n, D)[:, 0] = torch.where(torch.arange(n, device="cuda") < n // 2, 448.0, -448.0)
        v = torch.ones(n // S, 1, S, D, device="cuda")
        v.view(n, D)[n // 2:] = 2.0
        one = torch.ones(n // S, 1, device="cuda")
        cache = sv.PagedKVCache(k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), one, one.clone())
        table = torch.arange(n // S, dtype=torch.int32, device="cuda")[None]
        seq = torch.full((1,), n - 1, dtype=torch.int32, device="cuda")
        for sign, want in ((1.0, 1.0), (-1.0, 2.0)):
            q = torch.zeros(1, 1, 2, D, device="cuda")
            q[..., 0] = sign * 2.0 ** 100
            out = sv.spec_kv_attention(q.to(DT[dtype]), cache, table, seq, scale=1.0)
            assert (out.float() == want).all()


class _OtherDevice:
    """Stands in for torch's notion of the current device: `index` until torch.cuda.device is entered."""

    def __init__(self, monkeypatch, kv_cache, index):
        self.now, self.entered = index, []
        monkeypatch.setattr(kv_cache, "_current_device", lambda: self.now)
        outer = self

        class Device:
            def __init__(self, i):
                self.i = i

            def __enter__(self):
                outer.entered.append(self.i)
                self.before, outer.now = outer.now, self.i

            def __exit__(self, *exc):
                outer.now = self.before

        monkeypatch.setattr(torch.cuda, "device", Device)


@gpu
def test_calls_run_on_the_caches_device(monkeypatch):
    """With another device current, a call makes the cache's current for its time (a launch goes to the current device,
    whatever the tensors' is); with the cache's current it leaves things as they are."""
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(310, 2, 3, 4, 2, 64, 16, [5, 100], [3, 2], "bf16")
    a, b = s.cache(), s.cache()
    idx, q, k, v = s.idx(), s.dev(s.q), s.dev(s.k), s.dev(s.v)
    sv.spec_kv_append(q, k, v, a, *idx)
    want = sv.spec_kv_attention(q, a, *idx, return_lse=True)
    here = a.device.index
    other = _OtherDevice(monkeypatch, sv.kv_cache, here + 1)
    sv.spec_kv_append(q, k, v, b, *idx)
    assert other.entered == [here] and other.now == here + 1
    got = sv.spec_kv_attention(q, b, *idx, return_lse=True)
    assert other.entered == [here, here] and other.now == here + 1
    assert torch.equal(a.k_codes.view(torch.uint8), b.k_codes.view(torch.uint8))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    other.now = here
    sv.spec_kv_attention(q, b, *idx)
    assert len(other.entered) == 2


@gpu
def test_streams_of_other_devices_are_refused():
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(311, 1, 1, 2, 2, 64, 16, [5], [1], "bf16")
    cache, idx, q, k = s.cache(), s.idx(), s.dev(s.q), s.dev(s.k)

    class Stream:
        device, cuda_stream = torch.device("cuda", cache.device.index + 1), 0

    with pytest.raises(ValueError):
        sv.spec_kv_append(q, k, k, cache, *idx, stream=Stream())
    with pytest.raises(ValueError):
        sv.spec_kv_attention(q, cache, *idx, stream=Stream())


@gpu
def test_workspaces_are_checked():
    """A workspace on the host, of another type or with gaps is refused before its address is used."""
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(312, 1, 1, 2, 2, 64, 16, [5], [1], "bf16")
    cache, idx, q = s.cache(), s.idx(), s.dev(s.q)
    n = sv.spec_kv_attention_workspace_size(cache, 1, 1, 2)
    good = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for ws in (good.cpu(), torch.zeros(n, device="cuda"), torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            sv.spec_kv_attention(q, cache, *idx, ws=ws)
    sv.spec_kv_attention(q, cache, *idx, ws=good)


def _long_call(seed, n=3000, B=1):
    import speculative_sampling_verification_spec_gb300 as sv
    s = Setup(seed, B, 1, 4, 1, 64, 16, [n] * B, [1] * B, "bf16")
    cache = s.cache()
    s.append(cache)
    s.ref_append()
    q, idx = s.dev(s.q), s.idx()
    return (lambda **kw: sv.spec_kv_attention(q, cache, *idx, return_lse=True, **kw)), s.ref_attention()


@gpu
def test_a_graph_has_a_workspace_of_its_own():
    """Whatever happens to the workspace that direct calls on the capturing stream use, before the capture too, is not
    the graph's concern: it may be replayed beside them."""
    import speculative_sampling_verification_spec_gb300 as sv
    call, want = _long_call(313, B=8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    key = (torch.cuda.current_device(), side.cuda_stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        assert_attention(*call(), want)
        with torch.cuda.graph(graph, stream=side):
            got = call()
        direct = sv.kv_cache._ws_cache[key]
        direct[:1 << 16] = 0x3F         # counters that no call leaves
        graph.replay()
        side.synchronize()
        assert_attention(*got, want)
        direct[:1 << 16] = 0
        assert_attention(*call(), want)
    side.synchronize()


@gpu
def test_overlapping_replays():
    """Two graphs of one stream, each of several calls of different sizes, replayed side by side on other streams with
    direct calls beside them."""
    import speculative_sampling_verification_spec_gb300 as sv
    calls = [_long_call(320 + i, n, B) for i, (n, B) in enumerate([(3000, 8), (9000, 1), (2000, 5), (500, 20)])]
    torch.cuda.synchronize()
    side, streams = torch.cuda.Stream(), [torch.cuda.Stream() for _ in range(2)]
    graphs, results = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            results.append([call() for call, _ in calls])
        graphs.append(g)
    key = (torch.cuda.current_device(), side.cuda_stream)
    assert key not in sv.kv_cache._ws_cache
    torch.cuda.synchronize()
    for _ in range(10):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                for _ in range(3):
                    g.replay()
        with torch.cuda.stream(side):
            direct = [call() for call, _ in calls]
        torch.cuda.synchronize()
        for res in results + [direct]:
            for r, (_, want) in zip(res, calls):
                assert_attention(*r, want)


@gpu
def test_capture_ids():
    import speculative_sampling_verification_spec_gb300 as sv
    L = sv.kv_cache._lib()
    side = torch.cuda.Stream()
    x = torch.zeros(4, device="cuda")
    ids = []
    assert L.spec_kv_capture_id(side.cuda_stream) == 0
    torch.cuda.synchronize()
    for _ in range(2):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
            x.add_(1)
            ids.append(L.spec_kv_capture_id(side.cuda_stream))
    assert ids[0] and ids[1] and ids[0] != ids[1]
    assert L.spec_kv_capture_id(side.cuda_stream) == 0
    torch.cuda.synchronize()


@gpu
def test_workspaces_after_a_timeout():
    """A call that gave up leaves counters behind; with the kept workspaces forgotten, calls are as on a fresh stream.
    (The counters are put there by the test: no wait runs out.)"""
    import speculative_sampling_verification_spec_gb300 as sv
    call, want = _long_call(314, B=8)
    assert_attention(*call(), want)
    key = (torch.cuda.current_device(), torch.cuda.current_stream().cuda_stream)
    sv.kv_cache._ws_cache[key][:1 << 16] = 0x3F
    sv.spec_kv_reset_workspaces()
    for _ in range(2):
        assert_attention(*call(), want)
