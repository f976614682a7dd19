"""Measured cases of serving long streams over the paged key/value cache: norms with the append, attention with a window
and sinks, holding pages and forking sequences.

`append` normalises each head of the new tokens' queries and keys, rotates them by position and stores keys and values.
`attend` is the attention of the new tokens' queries over the last `window` tokens and the first `sinks` ones; pages in
between are gone.  `hold` gives every sequence the pages that its tokens need and releases the others, by a count of
holders for each page.  `fork` turns some sequences into copies of others: whole pages are shared, the last, partly filled
one is copied.  In its plain form (`own` false) a pass is elementary torch operations; otherwise it is the framework's
entry points.
"""
import math

import numpy as np
import torch

own = False

MAX_CODE = 448.0      # largest e4m3 value
MIN_EXP = -100        # scales are at least 2^-100
EPS = 1e-6


# --------------------------------------------------------------------------
# cases

def _append(name, B, T, length, hq, hkv, d, page, rot=None, interleaved=False, dtype="bf16", ragged=True):
    return dict(name=name, op="append", B=B, T=T, len=length, hq=hq, hkv=hkv, d=d, page=page,
                rot=d if rot is None else rot, interleaved=interleaved, dtype=dtype, ragged=ragged)


def _attend(name, B, T, length, window, sinks, hq, hkv, d, page, dtype="bf16", ragged=True):
    return dict(name=name, op="attend", B=B, T=T, len=length, window=window, sinks=sinks, hq=hq, hkv=hkv, d=d, page=page,
                dtype=dtype, ragged=ragged)


def _hold(name, B, T, length, page, window=0, sinks=0, ragged=True):
    return dict(name=name, op="hold", B=B, T=T, len=length, page=page, window=window, sinks=sinks, ragged=ragged)


def _fork(name, B, every, length, hkv, d, page, ragged=True):
    return dict(name=name, op="fork", B=B, every=every, len=length, hkv=hkv, d=d, page=page, ragged=ragged)


def listed():
    return [
        # one user, one new token: the call is all latency
        _append("append norm one token", 1, 1, 1000, 32, 8, 128, 16, ragged=False),
        # a round of verification in float32: odd sizes, half of each head rotated, neighbouring channels paired
        _append("append norm f32 drafts", 7, 5, 777, 12, 12, 64, 32, rot=32, interleaved=True, dtype="f32"),
        # prompts of up to 4096 tokens entering the cache
        _append("append norm prompts", 8, 4096, 0, 32, 8, 128, 128),
        # one user, one new token, a stream longer than its window: latency again
        _attend("sinks one token", 1, 1, 5000, 1024, 4, 32, 8, 128, 16, ragged=False),
        # a round of verification, 8 drafted tokens and the one before them, streams of up to 32768 tokens
        _attend("sinks batch drafts", 32, 9, 32768, 4096, 4, 32, 8, 128, 16),
        # ordinary serving: 128 streams of mixed lengths, one token each; the first 64 tokens (a system prompt's
        # beginning) stay visible.  The largest
        _attend("sinks batch decode", 128, 1, 65536, 4096, 64, 64, 8, 128, 64),
        # part of a prompt against what is cached
        _attend("sinks prompt part", 2, 512, 16384, 2048, 16, 32, 8, 128, 64, ragged=False),
        # float32 model, window and sinks that end inside pages
        _attend("sinks f32", 3, 2, 3001, 777, 100, 16, 4, 128, 32, dtype="f32"),
        # pages of a round: 8 drafted tokens and the one before them, then what verification left of them
        _hold("hold drafts", 32, 9, 8192, 64),
        # 256 streams in a pool of small pages, with what leaves the window
        _hold("hold streams", 256, 17, 131072, 16, window=8192, sinks=4),
        # one sequence becomes another's copy
        _fork("fork one", 8, 8, 1000, 8, 128, 16, ragged=False),
        # a search that goes on from every fourth sequence in three more copies
        _fork("fork beams", 512, 4, 4096, 8, 128, 128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "hold", "fork"])
    page = rng.choice([16, 32, 64, 128])
    ragged = rng.random() < 0.8
    if op == "hold":
        B = _log_int(rng, 1, 512)
        length = _log_int(rng, 1, min(131072, (1 << 25) * page // (16 * B)))
        window = _log_int(rng, 16, 16384) if rng.random() < 0.5 else 0
        c = _hold("", B, rng.choice([1, 2, 5, 9, 17, 100, 1000]), length, page, window,
                  rng.choice([0, 1, 4, 64, 200]) if window else 0, ragged)
    elif op == "fork":
        hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
        length = _log_int(rng, 1, 8192)
        most = (3 << 29) // (2 * hkv * d * (length + page))
        B = _log_int(rng, 2, max(2, min(512, most)))
        c = _fork("", B, rng.choice([2, 3, 4, 8]), length, hkv, d, page, ragged)
    else:
        dtype = "f32" if rng.random() < 0.15 else "bf16"
        hkv = rng.choice([1, 2, 4, 8, 8, 12, 16])
        hq = hkv * rng.choice([1, 2, 3, 4, 4, 6, 8])
        while hq > 64:
            hq -= hkv
        if op == "append":
            d = rng.choice([64, 80, 96, 128, 128, 128, 256])
            T = _log_int(rng, 1, 4096)
            most = (1 << 29) // (T * (2 * hq + 3 * hkv) * d * (4 if dtype == "f32" else 2))
            B = _log_int(rng, 1, max(1, min(128, most)))
            rot = d if rng.random() < 0.7 else d // 2
            c = _append("", B, T, _log_int(rng, 1, 8192), hq, hkv, d, page, rot, rng.random() < 0.3, dtype, ragged)
        else:
            d = rng.choice([64, 128, 128])
            T = rng.choice([1, 1, 2, 3, 4, 5, 5, 7, 9, 9, 16, 17])
            if dtype == "bf16" and rng.random() < 0.15:
                T = _log_int(rng, 18, 512)
            length = _log_int(rng, 1, 65536)
            window = _log_int(rng, 16, 16384 if dtype == "bf16" else 4096)
            sinks = rng.choice([1, 4, 4, 16, 64, 100, 300])
            seen = min(length, window + sinks) + T
            # the cached bytes of a call stay under those of the largest listed case, and the products under those of the
            # prompt part (of a float32 call, which no 8-bit tensor arithmetic serves, under a share of them)
            products = (1 << 30) if dtype == "f32" else (1 << 33)
            most = min((1 << 29) // (seen * hkv * d), products // (seen * hq * d * T))
            c = _attend("", _log_int(rng, 1, max(1, min(128, most))), T, length, window, sinks, hq, hkv, d, page, dtype,
                        ragged)
    del c["name"]
    return c


def _lengths(c):
    """(cached tokens, new tokens) of each sequence: fixed by the case, so that the work is too."""
    B, T, n = c["B"], c.get("T", 1), c["len"]
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


def _after(c):
    """hold: the tokens of each sequence when verification has dropped the rejected ones."""
    seq, new = _lengths(c)
    return [s + max(0, n - (b * 5) % (n + 1)) for b, (s, n) in enumerate(zip(seq, new))]


def _first_seen(c, s):
    """The first position that a query at s or later sees through the window."""
    return max(0, s + 1 - c["window"]) if c.get("window") else 0


def _pages_of(c, s, end):
    """Columns of the page table that a sequence holds: pages of sinks, pages from the window on."""
    S = c["page"]
    last = -(-end // S)
    keep = min(last, -(-c.get("sinks", 0) // S))
    return list(range(keep)) + list(range(max(keep, _first_seen(c, s) // S), last))


def _parents(c):
    """fork: every `every`th slot stays, the ones after it become its copies."""
    e = c["every"]
    return [-1 if b % e == 0 else b - b % e for b in range(c["B"])]


def work(case):
    c = case
    seq, new = _lengths(c)
    S = c["page"]
    if c["op"] == "hold":
        P = max(1, -(-(max(seq) + c["T"]) // S))
        N = _pool_pages(c)
        # both calls of a round read the table and the counts once
        return {"bytes": 2 * (4 * c["B"] * P + 4 * N), "flops": 0}
    if c["op"] == "fork":
        nbytes = 4 * _pool_pages(c)
        for b, p in enumerate(_parents(c)):
            if p >= 0:
                nbytes += 2 * (seq[p] % S) * 2 * c["hkv"] * c["d"] + 2 * 4 * -(-seq[p] // S) + 16 * c["hkv"]
        return {"bytes": nbytes, "flops": 0}
    e = 4 if c["dtype"] == "f32" else 2
    tokens = sum(new)
    if c["op"] == "append":
        heads = (c["hq"] + 2 * c["hkv"]) * c["d"]
        nbytes = tokens * (heads * e + c["hq"] * c["d"] * e + 2 * c["hkv"] * c["d"] + c["rot"] * 4)
        turned = (c["hq"] + c["hkv"])
        return {"bytes": nbytes, "flops": tokens * (turned * (3 * c["rot"] + 4 * c["d"]) + 2 * c["hkv"] * c["d"] * 2)}
    nbytes = flops = 0
    for s, n in zip(seq, new):
        if n == 0:
            continue
        first = _first_seen(c, s)
        kept = min(c["sinks"], first)          # sinks before the window
        nbytes += (s + n - first + kept) * 2 * c["hkv"] * c["d"]
        nbytes += len(_pages_of(c, s, s + n)) * (2 * 4 * c["hkv"] + 4)
        for t in range(n):
            lo = _first_seen(c, s + t)
            flops += 4 * c["d"] * c["hq"] * (s + t + 1 - lo + min(c["sinks"], lo))
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


def _held(c):
    """Columns that each sequence holds before the call."""
    seq, new = _lengths(c)
    if c["op"] == "fork":
        return [list(range(-(-s // c["page"]))) for s in seq]
    if c["op"] == "hold":
        return [_pages_of(c, s, s) for s in seq]
    return [_pages_of(c, s, s + c["T"]) for s in seq]


def _pool_pages(c):
    held = sum(len(x) for x in _held(c))
    if c["op"] == "hold":      # room for the round's tokens, and a tenth more
        return held + held // 10 + c["B"] * (-(-c["T"] // c["page"]) + 2) + 3
    if c["op"] == "fork":
        return held + c["B"] + 3
    return held + 3


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = torch.float32 if c.get("dtype") == "f32" else torch.bfloat16
    B, T, S = c["B"], c.get("T", 0), c["page"]
    seq, new = _lengths(c)
    P = max(1, max(-(-(s + T) // S) for s in seq))        # width of the page table
    held, N = _held(c), _pool_pages(c)
    order = torch.randperm(N, generator=g, device=dev).to(torch.int32)
    row = torch.tensor(np.repeat(np.arange(B), [len(x) for x in held]), device=dev)
    col = torch.tensor(np.concatenate([np.asarray(x, np.int64) for x in held]), device=dev)
    table = torch.full((B, P), -1, dtype=torch.int32, device=dev)
    table[row, col] = order[:len(col)]
    st = dict(case=c, table=table, seq=torch.tensor(seq, dtype=torch.int32, device=dev),
              new=torch.tensor(new, dtype=torch.int32, device=dev))
    if own:
        import speculative_sampling_verification_spec_gb300 as sv
        st["sv"] = sv
    if c["op"] in ("hold", "fork"):
        st["refs"] = torch.zeros(N, dtype=torch.int32, device=dev).index_fill_(0, table[row, col].long(), 1)
        st["free"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if c["op"] == "hold":
        st["after"] = torch.tensor(_after(c), dtype=torch.int32, device=dev)
        return st
    hkv, d = c["hkv"], c["d"]
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

    st["kc"], st["ks"] = pool(strong)
    st["vc"], st["vs"] = pool(1.0)
    if own:
        st["cache"] = sv.PagedKVCache(st["kc"], st["vc"], st["ks"], st["vs"])
    if c["op"] == "fork":
        st["parents"] = torch.tensor(_parents(c), dtype=torch.int32, device=dev)
        return st
    q = torch.randn(B, T, c["hq"], d, generator=g, device=dev)
    if c["op"] == "append":
        # heads as they come from the projection: of sizes of their own, which the norms take out
        def size(h):
            return torch.exp(torch.randn(B, T, h, 1, generator=g, device=dev))
        st["q"] = (q * size(c["hq"])).to(dt)
        st["k"] = (torch.randn(B, T, hkv, d, generator=g, device=dev) * size(hkv)).to(dt)
        st["v"] = (torch.randn(B, T, hkv, d, generator=g, device=dev) * 1.5).to(dt)
        st["q_norm"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=dev)
        st["k_norm"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=dev)) * strong[0, 0]
        half = c["rot"] // 2
        inv = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        ang = torch.arange(P * S, device=dev, dtype=torch.float64)[:, None] * inv
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()
    else:
        # scores of standard deviation about 1.5 (2 and more on the strong channels)
        st["q"] = (q * 1.5).to(dt)
    return st


# --------------------------------------------------------------------------
# one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state)
    return dict(append=_plain_append, attend=_plain_attend, hold=_plain_round, fork=_plain_fork)[op](state)


def _own(st):
    c, sv = st["case"], st["sv"]
    if c["op"] == "append":
        q = sv.spec_kv_append(st["q"], st["k"], st["v"], st["cache"], st["table"], st["seq"], st["new"],
                              cos_sin=st["cos_sin"], interleaved=c["interleaved"], q_norm=st["q_norm"],
                              k_norm=st["k_norm"], norm_eps=EPS)
        return dict(q=q, kc=st["kc"], ks=st["ks"], vc=st["vc"], vs=st["vs"])
    if c["op"] == "attend":
        out, lse = sv.spec_kv_attention(st["q"], st["cache"], st["table"], st["seq"], st["new"], window=c["window"],
                                        sinks=c["sinks"], return_lse=True)
        return dict(out=out, lse=lse)
    if c["op"] == "hold":
        args = dict(page_size=c["page"], window=c["window"], sinks=c["sinks"], free=st["free"])
        sv.spec_kv_hold(st["refs"], st["table"], st["seq"], st["new"], **args)
        sv.spec_kv_hold(st["refs"], st["table"], st["after"], **args)
        return dict(table=st["table"], refs=st["refs"], free=st["free"])
    sv.spec_kv_fork(st["cache"], st["refs"], st["table"], st["seq"], st["parents"], free=st["free"])
    return {n: st[n] for n in ("table", "refs", "free", "seq", "kc", "ks", "vc", "vs")}


def _norm(x, w):
    """x [..., d] in 32 bits: the mean of the squares in 64 bits (keys near the border between two scales go by it)."""
    r = torch.rsqrt(x.double().square().mean(-1, keepdim=True) + EPS).float()
    return (x * r) * w


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
    amax = torch.zeros(N, H, device=x.device).scatter_reduce_(0, page[:, None].expand(-1, H), x.abs().amax(-1), "amax")
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


def _plain_append(st):
    c = st["case"]
    T, S = c["T"], c["page"]
    seq, new = st["seq"].long(), st["new"].long()
    t = torch.arange(T, device=seq.device)
    pos = seq[:, None] + t[None, :]
    valid = (t[None, :] < new[:, None])
    q = _rotate(_norm(st["q"].float(), st["q_norm"]), st["cos_sin"], pos, c["rot"], c["interleaved"]).to(st["q"].dtype)
    q = torch.where(valid[:, :, None, None], q, torch.zeros_like(q))
    k = _rotate(_norm(st["k"].float(), st["k_norm"]), st["cos_sin"], pos, c["rot"], c["interleaved"])
    v = st["v"].float()
    table = st["table"].long()
    last = torch.gather(table, 1, ((seq - 1).clamp(min=0) // S)[:, None])[:, 0]
    row = valid.flatten().nonzero()[:, 0]
    page = torch.gather(table, 1, (pos // S).clamp(max=table.shape[1] - 1)).flatten()[row]
    args = (page, (pos % S).flatten()[row], last, seq % S)
    _store(k.flatten(0, 1)[row], st["kc"], st["ks"], *args)
    _store(v.flatten(0, 1)[row], st["vc"], st["vs"], *args)
    return dict(q=q, kc=st["kc"], ks=st["ks"], vc=st["vc"], vs=st["vs"])


def _gather(codes, scales, pages):
    """The pages [B, C] of each sequence, as values: [B, H, tokens, d] in 32 bits."""
    x = codes.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() * scales[pages][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attend(st):
    c = st["case"]
    B, T, hq, hkv, d, S, W, sinks = (c[n] for n in ("B", "T", "hq", "hkv", "d", "page", "window", "sinks"))
    G = hq // hkv
    seq, new = st["seq"].long(), st["new"].long()
    P = st["table"].shape[1]
    # columns of the table: the sinks' pages, then as many as the window can touch from its first page on
    ns = min(P, -(-sinks // S))
    start = ((seq + 1 - W).clamp(min=0) // S).clamp(min=ns)
    cols = torch.cat([torch.arange(ns, device=seq.device)[None, :].expand(B, -1),
                      start[:, None] + torch.arange(min(P, (W + T - 2) // S + 2), device=seq.device)[None, :]], dim=1)
    pages = torch.gather(st["table"].long(), 1, cols.clamp(max=P - 1)).clamp(min=0)
    j = (cols[:, :, None] * S + torch.arange(S, device=seq.device)).flatten(1)                  # [B, tokens]
    k = _gather(st["kc"], st["ks"], pages)
    q = st["q"].float().view(B, T, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, T * G, d)
    s = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    del k
    t = torch.arange(T, device=s.device)
    pos = seq[:, None] + t[None, :]                                                     # [B, T]
    see = (j[:, None, :] <= pos[:, :, None]) & ((j[:, None, :] > pos[:, :, None] - W) | (j[:, None, :] < sinks))
    see &= (t[None, :] < new[:, None])[:, :, None]
    see = see[:, None, :, None, :].expand(B, 1, T, G, -1).reshape(B, 1, T * G, -1)
    s = torch.where(see, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m0)
    del s
    l = p.sum(-1, keepdim=True)
    v = _gather(st["vc"], st["vs"], pages)
    o = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    lse = torch.where(l > 0, m0 + torch.log(l), torch.full_like(l, -math.inf))
    o = o.view(B, hkv, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, hq, d).to(st["q"].dtype)
    return dict(out=o, lse=lse.view(B, hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, hq))


def _count(refs, pages, keep, sign):
    """Adds sign to the count of pages[i] for every i that keep says."""
    N = refs.shape[0]
    at = torch.where(keep, pages, torch.full_like(pages, N)).flatten().long()
    more = torch.zeros(N + 1, dtype=refs.dtype, device=refs.device)
    refs.add_(more.scatter_add_(0, at, torch.full_like(at, sign, dtype=refs.dtype))[:N])


def _take(refs, need, free):
    """A page for every place that needs one: the lowest free ones in the places' order, -1 where there are no more.
    Counts them, and says how many are left."""
    N = refs.shape[0]
    is_free = refs <= 0
    among = torch.cumsum(is_free, 0)
    lowest = torch.full((N + 1,), -1, dtype=torch.int32, device=refs.device)
    lowest.scatter_(0, torch.where(is_free, among - 1, torch.full_like(among, N)),
                    torch.arange(N, dtype=torch.int32, device=refs.device))
    rank = torch.cumsum(need.flatten(), 0).view(need.shape) - 1
    got = need & (rank < among[-1])
    pages = torch.where(got, lowest[torch.where(got, rank, torch.zeros_like(rank))], torch.full_like(rank, -1, dtype=torch.int32))
    more = torch.zeros(N + 1, dtype=torch.bool, device=refs.device)
    more.index_fill_(0, torch.where(got, pages, torch.full_like(pages, N)).flatten().long(), True)
    refs.masked_fill_(more[:N], 1)
    free.copy_((among[-1] - got.sum()).to(torch.int32)[None])
    return pages


def _plain_hold(st, seq, new):
    c, table = st["case"], st["table"]
    S = c["page"]
    seq = seq.long()[:, None]
    end = seq + new.long()[:, None]
    col = torch.arange(table.shape[1], device=seq.device)[None, :]
    first = (seq + 1 - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(seq)
    want = (col * S < end) & ((col * S < c["sinks"]) | ((col + 1) * S > first))
    has = table >= 0
    _count(st["refs"], table, has & ~want, -1)
    pages = _take(st["refs"], want & ~has, st["free"])
    table.copy_(torch.where(want & has, table, pages))


def _plain_round(st):
    _plain_hold(st, st["seq"], st["new"])
    _plain_hold(st, st["after"], torch.zeros_like(st["after"]))
    return dict(table=st["table"], refs=st["refs"], free=st["free"])


def _plain_fork(st):
    c, table, refs = st["case"], st["table"], st["refs"]
    B, S = c["B"], c["page"]
    me = torch.arange(B, device=table.device)
    parents = st["parents"].long()
    child = (parents >= 0) & (parents != me)
    p = torch.where(child, parents, me)
    rows = table[p]
    length = st["seq"].long()[p]
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    whole = (col < (length // S)[:, None]) & (rows >= 0)
    partly = (col == (length // S)[:, None]) & (length % S > 0)[:, None] & (rows >= 0)
    _count(refs, table, child[:, None] & (table >= 0), -1)
    _count(refs, rows, child[:, None] & whole, 1)
    pages = _take(refs, child[:, None] & partly, st["free"])
    copies = (child[:, None] & partly & (pages >= 0)).nonzero()
    src, dst = rows[copies[:, 0], copies[:, 1]].long(), pages[copies[:, 0], copies[:, 1]].long()
    filled = torch.arange(S, device=table.device)[None, None, :, None] < (length % S)[copies[:, 0]][:, None, None, None]
    for codes, scales in ((st["kc"], st["ks"]), (st["vc"], st["vs"])):
        raw = codes.view(torch.uint8)
        raw[dst] = torch.where(filled, raw[src], raw[dst])
        scales[dst] = scales[src]
    table.copy_(torch.where(child[:, None], torch.where(whole, rows, pages), table))
    st["seq"].copy_(length)
    return {n: st[n] for n in ("table", "refs", "free", "seq", "kc", "ks", "vc", "vs")}


# --------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence

def exact(case, seed):
    c = dict(case)
    st = prepare(c, seed)
    seq, new = _lengths(c)
    return dict(append=_exact_append, attend=_exact_attend, hold=_exact_round, fork=_exact_fork)[c["op"]](c, st, seq, new)


def _e4m3(x):
    """numpy float64 -> the nearest e4m3 value (ties to even), |x| <= 448."""
    a = np.abs(x)
    _, e = np.frexp(a)
    q = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.sign(x) * np.rint(a / q) * q


def _exact_append(c, st, seq, new):
    if sum(new) * (c["hq"] + 2 * c["hkv"]) * c["d"] > 5e7:
        return None
    S, rot, half = c["page"], c["rot"], c["rot"] // 2
    cs = st["cos_sin"].double().cpu().numpy()
    table = st["table"].cpu().numpy()

    def host(n):
        return st[n].double().cpu().numpy()

    def turned(x, w, p):
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * w
        y = x.copy()
        a = slice(0, rot, 2) if c["interleaved"] else slice(0, half)
        b = slice(1, rot, 2) if c["interleaved"] else slice(half, rot)
        co, si = cs[p, None, :half], cs[p, None, half:]
        y[..., a], y[..., b] = x[..., a] * co - x[..., b] * si, x[..., b] * co + x[..., a] * si
        return y

    q, k, v, qw, kw = (host(n) for n in ("q", "k", "v", "q_norm", "k_norm"))
    out = np.zeros_like(q)
    kc, vc = st["kc"].float().cpu().numpy(), st["vc"].float().cpu().numpy()
    ks, vs = host("ks"), host("vs")
    for b in range(c["B"]):
        done = 0
        while done < new[b]:
            p = seq[b] + done
            n = min(new[b] - done, S - p % S)
            pos, ts, page, at = np.arange(p, p + n), slice(done, done + n), table[b, p // S], p % S
            out[b, ts] = turned(q[b, ts], qw, pos)
            for x, codes, scales in ((turned(k[b, ts], kw, pos), kc, ks), (v[b, ts], vc, vs)):
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
        cols = torch.tensor(_pages_of(c, seq[b], end), device=dev)
        pages = st["table"][b, cols].long()
        j = (cols[:, None] * S + torch.arange(S, device=dev)).flatten()
        pos = seq[b] + torch.arange(n, device=dev)
        hide = (j[None, :] > pos[:, None]) | ((j[None, :] <= pos[:, None] - c["window"]) & (j[None, :] >= c["sinks"]))
        for h in range(hkv):
            k = (st["kc"].view(torch.uint8)[pages, h].view(torch.float8_e4m3fn).double()
                 * st["ks"][pages, h].double()[:, None, None]).flatten(0, 1)
            v = (st["vc"].view(torch.uint8)[pages, h].view(torch.float8_e4m3fn).double()
                 * st["vs"][pages, h].double()[:, None, None]).flatten(0, 1)
            q = st["q"][b, :n, h * G:(h + 1) * G].double()                              # [n, G, d]
            s = torch.einsum("tgd,jd->tgj", q, k) / math.sqrt(d)
            s.masked_fill_(hide[:, None, :], -math.inf)
            lse[b, :n, h * G:(h + 1) * G] = torch.logsumexp(s, -1)
            out[b, :n, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", torch.softmax(s, -1), v)
    return dict(out=out, lse=lse)


def _exact_round(c, st, seq, new):
    table, refs = st["table"].cpu().numpy(), st["refs"].cpu().numpy()
    for lens, more in ((seq, new), (_after(c), [0] * c["B"])):
        want = np.zeros(table.shape, bool)
        for b in range(c["B"]):
            want[b, _pages_of(c, lens[b], lens[b] + more[b])] = True
        np.subtract.at(refs, table[~want & (table >= 0)], 1)
        table[~want] = -1
        missing = np.argwhere(table[want] < 0)[:, 0]
        spare = np.flatnonzero(refs <= 0)[:len(missing)]
        rows = table[want]
        rows[missing[:len(spare)]] = spare
        table[want] = rows
        refs[spare] = 1
    return dict(table=table, refs=refs, free=np.array([np.sum(refs <= 0)], np.int32))


def _exact_fork(c, st, seq, new):
    if st["kc"].numel() > 2e8:
        return None
    S = c["page"]
    table, refs = st["table"].cpu().numpy(), st["refs"].cpu().numpy()
    codes = [st[n].float().cpu().numpy() for n in ("kc", "vc")]
    scales = [st[n].double().cpu().numpy() for n in ("ks", "vs")]
    seq = list(seq)
    parents = _parents(c)
    forks = [b for b, p in enumerate(parents) if p >= 0]
    for b in forks:
        np.subtract.at(refs, table[b][table[b] >= 0], 1)
        p = parents[b]
        table[b] = -1
        table[b, :seq[p] // S] = table[p, :seq[p] // S]
        refs[table[b, :seq[p] // S]] += 1
        seq[b] = seq[p]
    spare = iter(np.flatnonzero(refs <= 0))
    for b in forks:
        full, rest = divmod(seq[b], S)
        if rest:
            new_page, old = next(spare), table[parents[b], full]
            table[b, full] = new_page
            refs[new_page] = 1
            for x, s in zip(codes, scales):
                x[new_page, :, :rest] = x[old, :, :rest]
                s[new_page] = s[old]
    return dict(table=table, refs=refs, free=np.array([np.sum(refs <= 0)], np.int32), seq=np.asarray(seq, np.int32),
                kc=codes[0].astype(np.float64), ks=scales[0], vc=codes[1].astype(np.float64), vs=scales[1])
