"""Attention with one strong token beside a long tail of small weights, against float64.

A token that carries most of the weight and has a small value, with the rest spread over thousands of tokens, is what
trained models do over long contexts.  The output is then the tail's, so each small weight has to keep its own relative
precision: the bounds below are relative to the weights and have no term in the number of tokens.  The sequences share
their pages and are as many as keep each (sequence, head) in one range of the kernel's list of tiles.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HKV, B, S = 8, 38, 128        # 304 (sequence, head) pairs


def make(n, T, G, D, m, sigma, strong_at, seed, vexp=-6):
    """Codes, scales, queries and lengths: the last query sees n tokens, of which the one at strong_at weighs about 1 - m
    and the others have scores of standard deviation sigma (in bits).  A score is k0 + k1 for queries of 8 and scale 1/8."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn(HKV, n, D, generator=g, device="cuda").to(torch.float8_e4m3fn)
    tail = (torch.randn(HKV, n, generator=g, device="cuda") * sigma * math.log(2)).to(torch.float8_e4m3fn)
    k[..., 0], k[..., 1] = tail, 0
    total = torch.logsumexp(tail.double(), 1)
    for h in range(HKV):
        s = total[h].item() + math.log((1 - m) / m)
        k[h, strong_at, 0], k[h, strong_at, 1] = math.floor(s), s - math.floor(s)
    v = (1 + 0.25 * torch.randn(HKV, n, D, generator=g, device="cuda")) * 64
    v[:, strong_at] = torch.randn(HKV, D, generator=g, device="cuda")
    v = v.to(torch.float8_e4m3fn)
    q = torch.zeros(B, T, HKV * G, D, device="cuda")
    q[..., :2] = 8.0
    q[:, :, 1::2, :2] = 7.5                       # rows of two sizes
    return k, v, q, 2.0 ** vexp


def paged(x):
    """[heads, n, D] -> pages of S tokens in a shuffled pool, and the table's row."""
    h, n, D = x.shape
    pages = -(-n // S)
    pad = torch.full((h, pages * S, D), 0x7F, dtype=torch.uint8, device="cuda")
    pad[:, :n] = x.view(torch.uint8)
    return pad.view(h, pages, S, D).transpose(0, 1).contiguous().view(torch.float8_e4m3fn)


def exact(k, v, q, vs, L, T, G, scale):
    """Outputs, their masses sum w |v| / sum w, and lse of one sequence, in float64: [T, HKV * G, ...]."""
    outs, masses, lses = [], [], []
    for t in range(T):
        e = L + t + 1
        for h in range(HKV):
            kk, vv = k[h, :e].double(), v[h, :e].double() * vs
            s = (q[0, t, h * G:(h + 1) * G].double() @ kk.T) * scale
            l = torch.logsumexp(s, 1)
            w = torch.exp(s - l[:, None])
            outs.append(w @ vv)
            masses.append(w @ vv.abs())
            lses.append(l)
    D = k.shape[-1]
    return (torch.cat(outs).view(T, HKV * G, D), torch.cat(masses).view(T, HKV * G, D), torch.cat(lses).view(T, HKV * G))


def check(n, T, G, D, m, sigma, dtype, strong_at, seed=0, vexp=-6):
    import speculative_sampling_verification_spec_gb300 as sv
    k, v, q, vs = make(n, T, G, D, m, sigma, strong_at, seed, vexp)
    L, pages = n - T, -(-n // S)
    kc, vc = paged(k), paged(v)
    cache = sv.PagedKVCache(kc, vc, torch.ones(pages, HKV, device="cuda"), torch.full((pages, HKV), vs, device="cuda"))
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, pages).contiguous()
    seq = torch.full((B,), L, dtype=torch.int32, device="cuda")
    out, lse = sv.spec_kv_attention(q.to(DT[dtype]), cache, table, seq, scale=0.125, return_lse=True)
    want, mass, l = exact(k, v, q, vs, L, T, G, 0.125)
    # bfloat16: the weights' own rounding and that of the scores and sums within 2^-8 of the mass, the output's 2^-9;
    # float32: a score is off by (D + 4) 2^-24 of at most 16, twice over, and a running sum by its few thousand steps
    tol = 2.0 ** -8 * mass + 2.0 ** -9 * want.abs() if dtype == "bf16" else 2.0 ** -10 * mass
    err = (out.double() - want[None]).abs()
    worst = (err / tol[None]).max().item()
    assert worst <= 1, (worst, (err / want.abs()[None].clamp(min=1e-30)).max().item())
    assert ((lse.double() - l[None]).abs() <= 2.0 ** -11).all()


@pytest.mark.parametrize("sigma", [0, 1])
@pytest.mark.parametrize("n,m", [(2048, 0.1), (8192, 0.25), (32768, 0.25), (131072, 0.5), (131072, 0.02)])
@pytest.mark.parametrize("D", [64, 128])
def test_small_weights_count(n, m, sigma, D):
    check(n, 1, 4, D, m, sigma, "bf16", strong_at=0)


@pytest.mark.parametrize("T,G", [(5, 4), (9, 4), (12, 4)])      # 20, 36 and 48 rows
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("strong_at", [3, 20000])
def test_small_weights_count_for_more_rows(T, G, D, strong_at):
    check(32768, T, G, D, 0.25, 1, "bf16", strong_at=strong_at, seed=1)


@pytest.mark.parametrize("n,m", [(8192, 0.25), (32768, 0.25)])
def test_small_weights_count_in_float32(n, m):
    check(n, 2, 4, 64, m, 1, "f32", strong_at=5)


@pytest.mark.parametrize("vexp", [-100, 100])
def test_denominators_of_values_far_from_one(vexp):
    """Values of scale 2^-100 or 2^100: the sum of the weights is in range whatever the values' scale."""
    check(32768, 1, 4, 128, 0.25, 1, "bf16", strong_at=0, seed=2, vexp=vexp)
