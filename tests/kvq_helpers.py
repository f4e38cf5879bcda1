"""64-bit references of the 8-bit KV cache operators (numpy, no library code).

An e4m3 code is s.eeee.mmm: (-1)^s 2^(e - 7) (1 + m / 8), subnormals 2^-6 m / 8 at e = 0, NaN at
0x7f / 0xff.  Rounding goes to the nearest code, ties to the even one; a cache block of 64 rows
shares the smallest power of two s with amax <= 448 s.
"""
import math

import numpy as np

BLOCK = 64


def _table():
    t = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = (2.0 ** -6) * m / 8 if e == 0 else 2.0 ** (e - 7) * (1 + m / 8)
        t[c] = math.nan if (c & 127) == 127 else (-v if c & 128 else v)
    return t


TABLE = _table()
_POS = TABLE[:127]  # ascending, codes 0 .. 126


def decode(codes: np.ndarray) -> np.ndarray:
    return TABLE[codes]


def encode(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 code (|x| <= 448 (1 + 2^-5) or not finite: NaN)."""
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(a >= _POS[126], 126, c)
    c = np.where(np.signbit(x), c | 128, c)
    return np.where(np.isfinite(x), c, 127).astype(np.uint8)


def scale_of(amax: float) -> float:
    if not amax > 0:
        return 0.0
    e = math.frexp(amax)[1] - 10  # below the answer, then up
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** max(e, -126)


def append(codes, scale, x, start):
    """Rows x [n][D] (fp64; a row of None-like NaN pattern is ordinary data) into one head's
    codes [P][D] (uint8) and scale [blocks] (fp32) at row `start`, in place."""
    n, done = x.shape[0], 0
    while done < n:
        at = start + done
        b = at // BLOCK
        lo, hi = b * BLOCK, min((b + 1) * BLOCK, start + n)
        rows = x[done: done + hi - at]
        fin = np.abs(rows[np.isfinite(rows)])
        old = float(scale[b]) if at > lo else 0.0
        s = max(scale_of(float(fin.max()) if fin.size else 0.0), old)
        d = s if s > 0 else 1.0
        if at > lo and s > old > 0:
            codes[lo:at] = encode(decode(codes[lo:at]) * (old / d))
        codes[at:hi] = encode(rows / d)
        scale[b] = s
        done += hi - at


def values(codes, scale):
    """codes [..., P, D], scale [..., blocks] -> fp64 values (a scale of 0: zeros)."""
    s = np.repeat(scale.astype(np.float64), BLOCK, -1)[..., : codes.shape[-2], None]
    return np.where(s > 0, decode(codes) * s, 0.0)


def attention(q, k, v, tk, tv, seq, nodes, see, scale):
    """q [B][R][Hq][D]; k, v [B][Hkv][P][D] values; tk, tv [B][Hkv][R][D]; see [B][R][R] bool.
    Returns out, lse (NaN in rows past nodes), and for the error bounds sum p |v| and the
    largest sum |q||k| scale of a row's visible keys."""
    B, R, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out, lse = np.full(q.shape, np.nan), np.full(q.shape[:3], np.nan)
    mass, reach = np.full(q.shape, np.nan), np.zeros(q.shape[:3])
    for b in range(B):
        L, n = int(seq[b]), int(nodes[b])
        if n == 0:
            continue
        for h in range(Hkv):
            kk = np.concatenate((k[b, h, :L], tk[b, h, :n]))
            vv = np.concatenate((v[b, h, :L], tv[b, h, :n]))
            m = np.concatenate((np.ones((n, L), bool), see[b, :n, :n]), 1)
            for g in range(G):
                x = q[b, :n, h * G + g]
                s = np.where(m, x @ kk.T * scale, -np.inf)
                top = s.max(1, keepdims=True)
                p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
                z = p.sum(1, keepdims=True)
                p = np.divide(p, z, out=np.zeros_like(p), where=z > 0)
                out[b, :n, h * G + g] = p @ vv
                mass[b, :n, h * G + g] = p @ np.abs(vv)
                reach[b, :n, h * G + g] = np.where(m, np.abs(x) @ np.abs(kk).T * scale, 0).max(1)
                with np.errstate(divide="ignore"):
                    lse[b, :n, h * G + g] = top[:, 0] + np.log(z[:, 0])
    return out, lse, mass, reach


def rope(x, w, eps, pos, inv_freq, rot, interleaved):
    """One kind of heads x [..., H, D] at positions pos [...]: norm (w may be None), rotation."""
    y = x.copy()
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w
    t = (pos.astype(np.float64)[..., None] * inv_freq.astype(np.float64))[..., None, :]
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    ya, yb = y[..., a], y[..., b]
    res = y.copy()
    res[..., a], res[..., b] = ya * np.cos(t) - yb * np.sin(t), ya * np.sin(t) + yb * np.cos(t)
    bound = np.abs(y)
    bound[..., a] = bound[..., b] = np.abs(ya) + np.abs(yb)
    return res, bound
