"""Measured cases of the paged key/value cache: `spec_kv_append` and `spec_kv_attention`.

A sequence's tokens live in pages of a pool shared by all sequences; keys and values are held in 8 bits (e4m3) with one
float32 scale for each page and key/value head.  `append` rotates the new tokens' queries and keys by position and stores
keys and values; `attend` computes the attention of the new tokens' queries over everything stored.  Each case is one call
of one operator.  In its plain form (`own` false) a call is elementary torch operations in 32 bits; otherwise it is the
framework's entry point.
"""
import math

import numpy as np
import torch

own = False

MAX_CODE = 448.0      # largest e4m3 value
MIN_EXP = -100        # scales are at least 2^-100


# --------------------------------------------------------------------------
# cases

def _append(name, B, T, length, hq, hkv, d, page, rot=None, interleaved=False, dtype="bf16", ragged=True):
    return dict(name=name, op="append", B=B, T=T, len=length, hq=hq, hkv=hkv, d=d, page=page,
                rot=d if rot is None else rot, interleaved=interleaved, dtype=dtype, ragged=ragged)


def _attend(name, B, T, length, hq, hkv, d, page, window=0, dtype="bf16", ragged=True):
    return dict(name=name, op="attend", B=B, T=T, len=length, hq=hq, hkv=hkv, d=d, page=page, window=window,
                dtype=dtype, ragged=ragged)


def listed():
    return [
        # one user, one new token: the call is all latency
        _append("append one token", 1, 1, 1000, 32, 8, 128, 16, ragged=False),
        # a round of verification: 32 sequences, 8 drafted tokens and the one before them, drafts of several lengths
        _append("append drafts", 32, 9, 8192, 32, 8, 128, 64),
        # odd sizes: a head per key/value head, half of each head rotated, neighbouring channels paired, float32
        _append("append f32 partial", 7, 5, 777, 12, 12, 64, 32, rot=32, interleaved=True, dtype="f32"),
        # prompts of up to 4096 tokens entering the cache
        _append("append prompts", 8, 4096, 0, 32, 8, 128, 128),
        # one user, one new token, a short context: latency again
        _attend("attend one token", 1, 1, 1000, 32, 8, 128, 16, ragged=False),
        # one user, 4 drafted tokens over a long context: the work has to be split along the sequence
        _attend("attend long drafts", 1, 5, 131072, 32, 8, 128, 64, ragged=False),
        # ordinary serving: 64 sequences of mixed lengths, one token each
        _attend("attend batch decode", 64, 1, 8192, 64, 8, 128, 16),
        # a round of verification at the longest drafts, mixed lengths up to 32768: the largest
        _attend("attend batch drafts", 32, 9, 32768, 32, 8, 128, 16),
        # as many key/value heads as query heads, 64 channels, a sliding window
        _attend("attend window", 16, 4, 4001, 16, 16, 64, 32, window=1024),
        # one key/value head for all query heads
        _attend("attend one kv head", 4, 5, 10007, 24, 1, 128, 64),
        # float32 model
        _attend("attend f32", 3, 2, 3001, 16, 4, 128, 32, dtype="f32"),
        # part of a prompt against what is cached: bound by the products
        _attend("attend prompt part", 2, 512, 8192, 32, 8, 128, 64, ragged=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = "f32" if rng.random() < 0.15 else "bf16"
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8, 12, 16])
    hq = hkv * rng.choice([1, 2, 3, 4, 4, 6, 8])
    while hq > 64:
        hq -= hkv
    page = rng.choice([16, 32, 64, 128])
    ragged = rng.random() < 0.8
    if rng.random() < 0.4:
        T = _log_int(rng, 1, 4096)
        most = (1 << 29) // (T * (2 * hq + 3 * hkv) * d * (4 if dtype == "f32" else 2))
        B = _log_int(rng, 1, max(1, min(128, most)))
        length = _log_int(rng, 1, 8192)
        rot = d if rng.random() < 0.7 else d // 2
        c = _append("", B, T, length, hq, hkv, d, page, rot, rng.random() < 0.3, dtype, ragged)
    else:
        T = rng.choice([1, 1, 2, 3, 4, 5, 5, 7, 9, 9, 16, 17])
        length = _log_int(rng, 1, 16384 if dtype == "f32" else 65536)
        if dtype == "bf16" and rng.random() < 0.15:
            T, length = _log_int(rng, 18, 512), min(length, 8192)
        # the cached bytes of a call stay under those of the largest listed case, and the products under those of the
        # prompt part (of a float32 call, which no 8-bit tensor arithmetic serves, under a share of them)
        products = (1 << 30) if dtype == "f32" else (1 << 35)
        most = min((1 << 29) // (length * hkv * d), products // (length * hq * d * T))
        B = _log_int(rng, 1, max(1, min(128, most)))
        window = _log_int(rng, 16, 4096) if rng.random() < 0.2 else 0
        c = _attend("", B, T, length, hq, hkv, d, page, window, dtype, ragged)
    del c["name"]
    return c


def _lengths(c):
    """(cached tokens, new tokens) of each sequence: fixed by the case, so that the work is too."""
    B, T, n = c["B"], c["T"], c["len"]
    if not c["ragged"]:
        return [n] * B, [T] * B
    seq, new = [], []
    for b in range(B):
        f = ((b * 7919 + 3) % B) / max(1, B - 1)
        seq.append(int(n // 4 + f * (n - n // 4)))
        g = ((b * 104729 + 1) % B) / max(1, B - 1)
        new.append(max(1, int(round(T - g * (T - 1) * 0.75))))
    if B >= 4:
        seq[B // 2] = 0          # a sequence that starts in this call
    if B >= 16:
        new[B // 3] = 0          # one with nothing new: its rows stay empty
    return seq, new


def work(case):
    c = case
    seq, new = _lengths(c)
    e = 4 if c["dtype"] == "f32" else 2
    tokens = sum(new)
    if c["op"] == "append":
        heads = (c["hq"] + 2 * c["hkv"]) * c["d"]
        nbytes = tokens * (heads * e + c["hq"] * c["d"] * e + 2 * c["hkv"] * c["d"] + c["rot"] * 4)
        return {"bytes": nbytes, "flops": tokens * (3 * (c["hq"] + c["hkv"]) * c["rot"] + 2 * c["hkv"] * c["d"] * 2)}
    nbytes = flops = 0
    for s, n in zip(seq, new):
        if n == 0:
            continue
        first = max(0, s + 1 - c["window"]) if c["window"] else 0
        nbytes += (s + n - first) * 2 * c["hkv"] * c["d"]
        nbytes += (-(-(s + n) // c["page"]) - first // c["page"]) * (2 * 4 * c["hkv"] + 4)
        for t in range(n):
            seen = min(s + t + 1, c["window"]) if c["window"] else s + t + 1
            flops += 4 * c["d"] * c["hq"] * seen
    nbytes += tokens * c["hq"] * c["d"] * e
    nbytes += c["B"] * c["T"] * c["hq"] * (c["d"] * e + 4)
    return {"bytes": nbytes, "flops": flops}


# --------------------------------------------------------------------------
# inputs

def _scale_of(amax):
    """The least power of two that brings amax into the range of the codes."""
    f, x = torch.frexp(amax)
    e = x - 9 + (f > 0.875).to(x.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    B, T, hq, hkv, d, S = c["B"], c["T"], c["hq"], c["hkv"], c["d"], c["page"]
    seq, new = _lengths(c)
    P = max(1, max(-(-(s + T) // S) for s in seq))        # width of the page table
    need = [max(1, -(-(s + T) // S)) for s in seq]
    N = sum(need) + 3                                     # pages of the pool, a few of them unused
    order = torch.randperm(N, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(B, P, dtype=torch.int32, device=dev)
    start = torch.tensor([0] + need[:-1], device=dev).cumsum(0)
    col = torch.arange(P, device=dev)
    at = (start[:, None] + col[None, :]).clamp(max=N - 1)
    used = col[None, :] < torch.tensor(need, device=dev)[:, None]
    table = torch.where(used, order[at], table)

    # keys: a few strong channels, as trained models have; values: plain
    strong = 1.0 + 4.0 * (torch.rand(hkv, 1, d, generator=g, device=dev) < 0.05).float()

    def pool(channel):
        codes = torch.empty(N, hkv, S, d, dtype=torch.float8_e4m3fn, device=dev)
        scales = torch.empty(N, hkv, dtype=torch.float32, device=dev)
        step = max(1, (1 << 27) // (hkv * S * d))
        for i in range(0, N, step):
            x = torch.randn(min(step, N - i), hkv, S, d, generator=g, device=dev) * channel
            s = _scale_of(x.abs().amax(dim=(2, 3)))
            scales[i:i + step] = s
            codes[i:i + step] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn)
        return codes, scales

    kc, ks = pool(strong)
    vc, vs = pool(1.0)
    st = dict(case=c, table=table, kc=kc, ks=ks, vc=vc, vs=vs,
              seq=torch.tensor(seq, dtype=torch.int32, device=dev), new=torch.tensor(new, dtype=torch.int32, device=dev))
    q = torch.randn(B, T, hq, d, generator=g, device=dev)
    if c["op"] == "append":
        st["q"] = q.to(dt)
        st["k"] = (torch.randn(B, T, hkv, d, generator=g, device=dev) * strong[None, :, 0] * 1.5).to(dt)
        st["v"] = (torch.randn(B, T, hkv, d, generator=g, device=dev) * 1.5).to(dt)
        half = c["rot"] // 2
        inv = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        ang = torch.arange(P * S, device=dev, dtype=torch.float64)[:, None] * inv
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()
    else:
        # scores of standard deviation about 1.5 (2 and more on the strong channels)
        st["q"] = (q * 1.5).to(dt)
    if own:
        import speculative_sampling_verification_spec_gb300 as sv
        st["sv"] = sv
        st["cache"] = sv.PagedKVCache(kc, vc, ks, vs)
    return st


# --------------------------------------------------------------------------
# one pass

def run(state):
    c = state["case"]
    if own:
        sv = state["sv"]
        if c["op"] == "append":
            q = sv.spec_kv_append(state["q"], state["k"], state["v"], state["cache"], state["table"], state["seq"],
                                  state["new"], cos_sin=state["cos_sin"], interleaved=c["interleaved"])
            return dict(q=q, kc=state["kc"], ks=state["ks"], vc=state["vc"], vs=state["vs"])
        out, lse = sv.spec_kv_attention(state["q"], state["cache"], state["table"], state["seq"], state["new"],
                                        window=c["window"], return_lse=True)
        return dict(out=out, lse=lse)
    return _plain_append(state) if c["op"] == "append" else _plain_attend(state)


def _rotate(x, cos_sin, pos, rot, interleaved):
    """x [B, T, H, d] in 32 bits, rotated at positions pos [B, T]."""
    half = rot // 2
    cs = cos_sin[pos.clamp(max=cos_sin.shape[0] - 1).long()][:, :, None, :]
    cos, sin = cs[..., :half], cs[..., half:]
    x1 = x[..., 0:rot:2] if interleaved else x[..., :half]
    x2 = x[..., 1:rot:2] if interleaved else x[..., half:rot]
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.stack([y1, y2], dim=-1).flatten(-2) if interleaved else torch.cat([y1, y2], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _store(x, codes, scales, page, slot, last, kept):
    """Write x [n, H, d] (32 bits) to slot [n] of page [n].  last [B], kept [B]: the page of each sequence's last stored
    token and how many of its slots stay beside new tokens (0: none, the page is full)."""
    N, H = scales.shape
    raw = codes.view(torch.uint8)
    fin = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)                 # [n, H]
    amax = torch.zeros(N, H, device=x.device).scatter_reduce_(0, page[:, None].expand(-1, H), fin, "amax")
    new = _scale_of(amax)
    touched = torch.zeros(N, 1, dtype=torch.bool, device=x.device).index_fill_(0, page, True)
    begun = torch.zeros(N, 1, dtype=torch.bool, device=x.device).index_put_((last,), (kept > 0)[:, None])
    new = torch.where(begun, torch.maximum(scales, new), new)
    new = torch.where(touched, new, scales)
    # earlier codes beside the new tokens, where the scale grew
    old = raw[last]
    again = (old.view(torch.float8_e4m3fn).float() * (scales[last] / new[last])[:, :, None, None])
    stays = torch.arange(codes.shape[2], device=x.device)[None, None, :, None] < kept[:, None, None, None]
    grew = (new[last] != scales[last])[:, :, None, None] & stays
    raw[last] = torch.where(grew, again.to(torch.float8_e4m3fn).view(torch.uint8), old)
    raw[page, :, slot] = (x / new[page][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scales.copy_(new)


def _plain_append(state):
    c = state["case"]
    T, S = c["T"], c["page"]
    seq, new = state["seq"].long(), state["new"].long()
    t = torch.arange(T, device=seq.device)
    pos = seq[:, None] + t[None, :]
    valid = (t[None, :] < new[:, None])
    q = _rotate(state["q"].float(), state["cos_sin"], pos, c["rot"], c["interleaved"]).to(state["q"].dtype)
    q = torch.where(valid[:, :, None, None], q, torch.zeros_like(q))
    k = _rotate(state["k"].float(), state["cos_sin"], pos, c["rot"], c["interleaved"])
    v = state["v"].float()
    table = state["table"].long()
    last = torch.gather(table, 1, ((seq - 1).clamp(min=0) // S)[:, None])[:, 0]
    row = valid.flatten().nonzero()[:, 0]
    page = torch.gather(table, 1, (pos // S).clamp(max=table.shape[1] - 1)).flatten()[row]
    args = (page, (pos % S).flatten()[row], last, seq % S)
    _store(k.flatten(0, 1)[row], state["kc"], state["ks"], *args)
    _store(v.flatten(0, 1)[row], state["vc"], state["vs"], *args)
    return dict(q=q, kc=state["kc"], ks=state["ks"], vc=state["vc"], vs=state["vs"])


def _gather(codes, scales, table):
    """The pages of each sequence, as values: [B, H, tokens, d] in 32 bits."""
    t = table.long()
    x = codes.view(torch.uint8)[t].view(torch.float8_e4m3fn).float() * scales[t][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attend(state):
    c = state["case"]
    B, T, hq, hkv, d, S = c["B"], c["T"], c["hq"], c["hkv"], c["d"], c["page"]
    G = hq // hkv
    seq, new = state["seq"].long(), state["new"].long()
    k = _gather(state["kc"], state["ks"], state["table"])
    q = state["q"].float().view(B, T, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, T * G, d)
    s = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    del k
    j = torch.arange(s.shape[-1], device=s.device)
    t = torch.arange(T, device=s.device)
    pos = seq[:, None] + t[None, :]                                                     # [B, T]
    see = (j[None, None, :] <= pos[:, :, None]) & (t[None, :] < new[:, None])[:, :, None]
    if c["window"]:
        see &= j[None, None, :] > pos[:, :, None] - c["window"]
    see = see[:, None, :, None, :].expand(B, 1, T, G, -1).reshape(B, 1, T * G, -1)
    s = torch.where(see, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m0)
    del s
    l = p.sum(-1, keepdim=True)
    v = _gather(state["vc"], state["vs"], state["table"])
    o = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    lse = torch.where(l > 0, m0 + torch.log(l), torch.full_like(l, -math.inf))
    o = o.view(B, hkv, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, hq, d).to(state["q"].dtype)
    return dict(out=o, lse=lse.view(B, hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, hq))


# --------------------------------------------------------------------------
# the definition in 64 bits, sequence by sequence

def _e4m3(x):
    """numpy float64 -> the nearest e4m3 value (ties to even), |x| <= 448."""
    a = np.abs(x)
    _, e = np.frexp(a)
    q = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.sign(x) * np.rint(a / q) * q


def exact(case, seed):
    c = dict(case)
    st = prepare(c, seed)
    seq, new = _lengths(c)
    return _exact_append(c, st, seq, new) if c["op"] == "append" else _exact_attend(c, st, seq, new)


def _exact_append(c, st, seq, new):
    if sum(new) * (c["hq"] + 2 * c["hkv"]) * c["d"] > 5e7:
        return None
    S, rot, half = c["page"], c["rot"], c["rot"] // 2
    cs = st["cos_sin"].double().cpu().numpy()
    table = st["table"].cpu().numpy()

    def host(n):
        return st[n].double().cpu().numpy()

    def rotated(x, p):
        y = x.copy()
        a = slice(0, rot, 2) if c["interleaved"] else slice(0, half)
        b = slice(1, rot, 2) if c["interleaved"] else slice(half, rot)
        co, si = cs[p, None, :half], cs[p, None, half:]
        y[..., a], y[..., b] = x[..., a] * co - x[..., b] * si, x[..., b] * co + x[..., a] * si
        return y

    q, k, v = host("q"), host("k"), host("v")
    out = np.zeros_like(q)
    kc, vc = st["kc"].float().cpu().numpy(), st["vc"].float().cpu().numpy()
    ks, vs = host("ks"), host("vs")
    for b in range(c["B"]):
        done = 0
        while done < new[b]:
            p = seq[b] + done
            n = min(new[b] - done, S - p % S)
            pos, ts, page, at = np.arange(p, p + n), slice(done, done + n), table[b, p // S], p % S
            out[b, ts] = rotated(q[b, ts], pos)
            for x, codes, scales in ((rotated(k[b, ts], pos), kc, ks), (v[b, ts], vc, vs)):
                f, e = np.frexp(np.abs(x).max(axis=(0, 2)))
                need = np.ldexp(1.0, np.maximum(e - 9 + (f > 0.875), MIN_EXP))
                if at:
                    need = np.maximum(need, scales[page])
                    codes[page, :, :at] = _e4m3(codes[page, :, :at] * (scales[page] / need)[:, None, None])
                scales[page] = need
                codes[page, :, at:at + n] = _e4m3(x / need[None, :, None]).transpose(1, 0, 2)
            done += n
    return dict(q=out, kc=kc.astype(np.float64), ks=ks, vc=vc.astype(np.float64), vs=vs)


def _exact_attend(c, st, seq, new):
    B, T, hq, hkv, d, S = c["B"], c["T"], c["hq"], c["hkv"], c["d"], c["page"]
    G = hq // hkv
    dev = st["q"].device
    out = torch.zeros(B, T, hq, d, dtype=torch.float64, device=dev)
    lse = torch.full((B, T, hq), -math.inf, dtype=torch.float64, device=dev)
    for b in range(B):
        n, end = new[b], seq[b] + new[b]
        if n == 0:
            continue
        pages = st["table"][b, :-(-end // S)].long()
        pos = seq[b] + torch.arange(n, device=dev)
        j = torch.arange(end, device=dev)
        hide = j[None, :] > pos[:, None]
        if c["window"]:
            hide |= j[None, :] <= pos[:, None] - c["window"]
        for h in range(hkv):
            k = (st["kc"].view(torch.uint8)[pages, h].view(torch.float8_e4m3fn).double()
                 * st["ks"][pages, h].double()[:, None, None]).flatten(0, 1)[:end]
            v = (st["vc"].view(torch.uint8)[pages, h].view(torch.float8_e4m3fn).double()
                 * st["vs"][pages, h].double()[:, None, None]).flatten(0, 1)[:end]
            q = st["q"][b, :n, h * G:(h + 1) * G].double()                              # [n, G, d]
            s = torch.einsum("tgd,jd->tgj", q, k) / math.sqrt(d)
            s.masked_fill_(hide[:, None, :], -math.inf)
            lse[b, :n, h * G:(h + 1) * G] = torch.logsumexp(s, -1)
            out[b, :n, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", torch.softmax(s, -1), v)
    return dict(out=out, lse=lse)
