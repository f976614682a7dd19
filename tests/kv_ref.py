"""The paged key/value cache restated in numpy: storing in float32 and float64 as the definition says, attention in
float64, with bounds on how far a float32 evaluation may be off.  Test infrastructure; shares nothing with the library."""
import numpy as np

MAX_CODE, MIN_EXP = 448.0, -100

# the value of each e4m3 code: 1 sign, 4 exponent (bias 7), 3 mantissa bits; S.1111.111 is NaN
_c = np.arange(256)
_e, _m = (_c >> 3) & 15, _c & 7
CODE_VALUES = np.where(_e == 0, np.ldexp(_m / 8.0, -6), np.ldexp(1.0 + _m / 8.0, _e - 7)) * np.where(_c & 128, -1.0, 1.0)
CODE_VALUES[[0x7F, 0xFF]] = np.nan


def encode(x):
    """float64 values -> e4m3 codes, to nearest even; NaN and infinities -> 0x7f (sign ignored)."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    ok = np.isfinite(x)
    a0 = np.where(ok, a, 0.0)
    _, e = np.frexp(a0)
    e = np.maximum(e - 1, -6)
    n = np.rint(np.ldexp(a0, 3 - e))          # multiples of 2^(e-3)
    up = n >= 16                              # rounded into the next binade
    e, n = np.where(up, e + 1, e), np.where(up, 8, n)
    sub = n < 8                               # subnormal (e = -6)
    code = np.where(sub, n, ((e + 7) * 8 + (n - 8))).astype(np.int64)
    assert np.all(code[ok] <= 0x7E), "value beyond the codes"
    code = np.where(ok, code | (np.signbit(x) * 128), 0x7F)
    return code.astype(np.uint8)


def scale_for(amax):
    """The least power of two >= 2^-100 that brings amax within 448 of it."""
    f, e = np.frexp(np.asarray(amax, np.float64))
    return np.ldexp(1.0, np.where(amax > 0, np.maximum(e - 9 + (f > 0.875), MIN_EXP), MIN_EXP)).astype(np.float32)


def bf16_round(x):
    """float32 -> the nearest bfloat16 value, as float32 (NaN stays NaN)."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    r = ((b + np.uint32(0x7FFF) + ((b >> np.uint32(16)) & np.uint32(1))) & np.uint32(0xFFFF0000)).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r)


def rotate(x, cs, rot, interleaved):
    """x [..., H, D] float32, cs [..., rot] float32: each product and sum rounded to float32."""
    y = np.array(x, np.float32)
    h = rot // 2
    if rot:
        co, si = cs[..., None, :h], cs[..., None, h:]
        a = slice(0, rot, 2) if interleaved else slice(0, h)
        b = slice(1, rot, 2) if interleaved else slice(h, rot)
        x1, x2 = x[..., a], x[..., b]
        with np.errstate(invalid="ignore", over="ignore"):
            y[..., a] = x1 * co - x2 * si
            y[..., b] = x2 * co + x1 * si
    return y


def append(q, k, v, kc, vc, ks, vs, table, seq, new, cs, rot, interleaved, dtype, page_size):
    """Writes kc, vc [N, H, S, D] uint8 and ks, vs [N, H] float32 in place; returns the rotated queries (float32, rounded
    to dtype).  q, k, v [B, T, H, D] float32."""
    S = page_size
    out = np.zeros_like(q)
    for b in range(q.shape[0]):
        n, L = int(new[b]), int(seq[b])
        pos = L + np.arange(n)
        c = cs[pos] if rot else None
        if n == 0:
            continue
        y = rotate(q[b, :n], c, rot, interleaved)
        out[b, :n] = bf16_round(y) if dtype == "bf16" else y
        kr = rotate(k[b, :n], c, rot, interleaved)
        for x, codes, scales in ((kr, kc, ks), (v[b, :n], vc, vs)):
            done = 0
            while done < n:
                p = L + done
                m = min(n - done, S - p % S)
                pg, at = int(table[b, p // S]), p % S
                part = x[done:done + m].astype(np.float64)
                need = scale_for(np.where(np.isfinite(part), np.abs(part), 0).max(axis=(0, 2)))
                if at:
                    need = np.maximum(need, scales[pg])
                    for h in range(kc.shape[1]):
                        if need[h] != scales[pg, h]:
                            old = CODE_VALUES[codes[pg, h, :at]].astype(np.float32)
                            codes[pg, h, :at] = encode(old * np.float32(scales[pg, h] / need[h]))
                scales[pg] = need
                with np.errstate(invalid="ignore"):
                    codes[pg, :, at:at + m] = encode((part / need[None, :, None]).transpose(1, 0, 2))
                done += m
    return out


U = 2.0 ** -24       # half an ulp of float32


def attention(q, kc, vc, ks, vs, table, seq, new, page_size, scale, window=0, dtype="f32"):
    """q [B, T, Hq, D] float64 -> out, lse (float64), and tolerances of the same shapes.

    The tolerance of an output follows from rounding errors, with u = 2^-24:
      a score s_j = scale * sum_i q_i k_i, summed in float32 in any order, is off by at most (D + 4) u A with
      A = max_j |scale| sum_i |q_i k_ij|; evaluated in 2-power form it is multiplied and subtracted once more, which the
      4 covers with |s| <= A; exp2 itself adds a relative 2^-21; so a weight is off by the relative amount
      e = 2 ((D + 4) u A + 2^-21) (2: first-order bound with room, and the reference's own shift);
      sums of n weights, in any order, add n u.  Numerator and denominator are both off by this:
          |out - exact| <= 2 (e + n u) sum_j w_j |v_j| / sum_j w_j.
      bfloat16 queries: the weights reach the products in two 8-bit pieces of 4 significant bits each, a relative 2^-8
      of a weight, or 2^-17 of the largest weight where a piece is subnormal; the queries in two pieces as well, exact
      but for 2^-17 of the row's largest (of rows that share an exponent, the largest's, 2^4 times more at most: far
      inside the 2^-8 of the weights); and the output is rounded to 8 bits, 2^-8 |out| at most.
      lse: off by e + n u, and u |lse| a few times over."""
    B, T, Hq, D = q.shape
    Hkv, S = kc.shape[1], page_size
    G = Hq // Hkv
    out, lse = np.zeros((B, T, Hq, D)), np.full((B, T, Hq), -np.inf)
    tol, tol_lse = np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq))
    for b in range(B):
        n, L = int(new[b]), int(seq[b])
        if n == 0:
            continue
        end = L + n
        pages = table[b, :-(-end // S)].astype(np.int64)
        for h in range(Hkv):
            k = (CODE_VALUES[kc[pages, h]] * ks[pages, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:end]
            v = (CODE_VALUES[vc[pages, h]] * vs[pages, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:end]
            for t in range(n):
                p = L + t
                lo = max(0, p + 1 - window) if window else 0
                kk, vv = k[lo:p + 1], v[lo:p + 1]
                for g in range(G):
                    x = q[b, t, h * G + g]
                    s = scale * (kk @ x)
                    m = s.max()
                    w = np.exp(s - m)
                    l = w.sum()
                    i = (b, t, h * G + g)
                    out[i] = (w @ vv) / l
                    lse[i] = m + np.log(l)
                    A = abs(scale) * (np.abs(kk) @ np.abs(x)).max()
                    cnt = p + 1 - lo
                    e = 2 * ((D + 4) * U * A + 2.0 ** -21) + cnt * U
                    mass = (w @ np.abs(vv)) / l
                    tol[i] = 2 * e * mass
                    if dtype == "bf16":
                        dq = 2.0 ** -17 * abs(scale) * np.abs(x).max() * np.abs(kk).sum(axis=1).max()
                        e += 2 * dq
                        tol[i] = (2 * e + 2.0 ** -8) * mass + 2.0 ** -17 * np.abs(vv).sum(axis=0) / l \
                            + 2.0 ** -8 * np.abs(out[i])
                    tol_lse[i] = e + 4 * U * abs(lse[i])
    return out, lse, tol, tol_lse
