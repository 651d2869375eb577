"""Plain 64-bit references of the cache in 4 bits, the rotary positions and the
sampling, written from the definitions in include/dspark.h with numpy, and the
error bounds the tests allow."""
import numpy as np
import torch

EPS32 = torch.finfo(torch.float32).eps / 2     # unit roundoff of binary32, 2^-24
EPS16 = torch.finfo(torch.bfloat16).eps / 2    # of bfloat16, 2^-8
EPSH = torch.finfo(torch.float16).eps / 2      # of binary16, 2^-11

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the non-negative scales by their number: 4 bits of exponent, 3 of mantissa; the last one is NaN
SCALES = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)])
SCALES[127] = np.nan


def _nearest(x, table):
    """Number of the entry of an ascending table nearest to x >= 0, ties to the even number."""
    border = (table[:-1] + table[1:]) / 2
    low = np.searchsorted(border, x, side="left")          # borders below x
    high = np.searchsorted(border, x, side="right")        # and at x
    return np.where((low != high) & (low % 2 == 1), high, low)


def quantise(x, exp):
    """Codes [.., D / 2] and scales [.., D / 16] (uint8) of float64 x [.., D].
    Where a group holds a NaN only its scale is defined."""
    y = x.reshape(*x.shape[:-1], -1, 16) * 2.0 ** -exp
    top = np.abs(y).max(-1)
    bad = np.isnan(top)
    s = _nearest(np.minimum(np.where(bad, 0, top), 1e9) / 6, SCALES[:127]).astype(np.uint8)
    f = SCALES[s][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(f > 0, np.abs(y) / np.where(f > 0, f, 1), 0)
    code = _nearest(np.where(bad[..., None], 0, r), LEVELS) + 8 * np.signbit(y)
    code = code.astype(np.uint8).reshape(*x.shape[:-1], -1, 2)
    return code[..., 0] | code[..., 1] << 4, np.where(bad, 127, s).astype(np.uint8)


def values(codes, scales, exp):
    """What codes and scales stand for (float64)."""
    lev = np.concatenate([LEVELS, -LEVELS])
    x = np.stack([lev[codes & 15], lev[codes >> 4]], -1).reshape(*codes.shape[:-1], -1, 16)
    s = np.where(scales >= 128, -1, 1) * SCALES[scales & 127]
    return (x * (s * 2.0 ** exp)[..., None]).reshape(*codes.shape[:-1], -1)


def attention(q, K, V, table, kv_len, q_off, scale, bf16):
    """out, lse and the error allowed for each; K, V [pages, Hkv, P, D] the values
    of the cache, all float64.  Pages out of range are left out.

    A score: D products summed in binary32 by the tensor cores, which may cut where
    others round: d = 2 (D + 8) EPS32 scale sum |q_d k_d|; in bf16 calls q is rounded to
    2^-25 of its row's largest entry: scale 2^-25 max |q| sum |k_d| more.  A weight: 2 d + 2^-20
    (exponential, references, sum), and in bf16 calls EPSH for its rounding and 2^-32 of the largest
    weight where it is small.  An output: that times sum p |v|, and its own rounding."""
    N, Hq, D = q.shape
    Hkv, P = K.shape[1], K.shape[2]
    G = Hq // Hkv
    out, lse = np.zeros((N, Hq, D)), np.full((N, Hq), -np.inf)
    out_tol, lse_tol = np.zeros((N, Hq, D)), np.zeros((N, Hq))
    for b in range(len(kv_len)):
        n = q_off[b + 1] - q_off[b]
        for i in range(n):
            last = kv_len[b] - n + i
            if last < 0:
                continue
            pos = np.arange(last + 1)
            page, row = table[b, pos // P], pos % P
            ok = (page >= 0) & (page < K.shape[0])
            if not ok.any():
                continue
            page, row = page[ok], row[ok]
            for h in range(Hq):
                k, v = K[page, h // G, row], V[page, h // G, row]
                x, t = q[q_off[b] + i, h], q_off[b] + i
                with np.errstate(invalid="ignore"):
                    s = (k * x).sum(1) * scale
                    d = 2 * (D + 8) * EPS32 * scale * np.abs(k * x).sum(1).max()
                    if bf16:
                        d += scale * 2.0 ** -25 * np.abs(x).max() * np.abs(k).sum(1).max()
                    top = s.max()
                    w = np.exp(s - top)
                    p = w / w.sum()
                    out[t, h] = p @ v
                    lse[t, h] = top + np.log(w.sum())
                    rel = 2 * d + 2.0 ** -20 + (EPSH if bf16 else 0)
                    small = 2.0 ** -32 * np.abs(v).sum(0) / w.sum() if bf16 else 0
                    out_tol[t, h] = 1.01 * (rel * (p @ np.abs(v)) + small + (EPS16 if bf16 else 2 * EPS32) * np.abs(out[t, h])) + 1e-30
                    lse_tol[t, h] = 2 * d + 2.0 ** -20 + 4 * EPS32 * abs(lse[t, h])
    return out, lse, out_tol, lse_tol


def rope(x, positions, freq, mult, rotary, interleaved, eps):
    """x [T, heads, D] turned (float64), and the error allowed: the angle is off by
    2^-25 of a half turn and by the frequency's 2^-53 (pi 2^-25 + pos f 2^-52 radians), sine
    and cosine by 2 EPS32 each and by the multiplier's rounding, the two products and their sum by 2 EPS32,
    all relative to mult (|a| + |b|), and the result by its own rounding."""
    y, tol = x.copy(), np.zeros_like(x)
    r = rotary
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    angle = positions.astype(np.float64)[:, None] * freq[None]
    c, s = (np.cos(angle) * mult)[:, None], (np.sin(angle) * mult)[:, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    off = (np.pi * 2.0 ** -25 + 6 * EPS32 + angle * 2.0 ** -52)[:, None] * abs(mult) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    tol[..., a] = tol[..., b] = off
    return y, tol + eps * np.abs(y)


def sample(x, u, T, k, p, m):
    """(token, log-probability, distance of u to the nearest border of the draw, and
    of the top-p sum to its own) of one row x (float64)."""
    x = np.where(np.isfinite(x), x, -np.inf)
    V = len(x)
    top = x.max()
    if top == -np.inf:
        return -1, -np.inf, 1.0, 1.0
    if not (T > 0 and np.isfinite(T)):
        return int(np.argmax(x)), 0.0, 1.0, 1.0
    order = np.argsort(-x, kind="stable")
    with np.errstate(over="ignore", invalid="ignore"):
        w = np.exp((x[order] - top) / T)
    w[x[order] == -np.inf] = 0
    near = 1.0
    if k > 0:
        w[k:] = 0
    if p < 1:
        c = np.concatenate([[0.0], np.cumsum(w)])
        near = np.abs(c[1:] / c[-1] - p).min() if p > 0 else 1.0
        drop = c[:-1] >= p * c[-1]
        drop[0] = False
        w[drop] = 0
    if m > 0:
        w[x[order] < top + T * np.log(min(m, 1.0))] = 0
    full = np.zeros(V)
    full[order] = w
    c = np.cumsum(full)
    t = int(np.searchsorted(c, min(max(u, 0.0), 1 - 2.0 ** -24) * c[-1], side="right"))
    return t, float(np.log(full[t] / c[-1])), float(np.abs(c / c[-1] - u).min()), near
