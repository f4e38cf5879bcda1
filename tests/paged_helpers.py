"""64-bit references of the paged KV cache operators (numpy, no library code)."""
import math

import numpy as np
import torch

U32 = 2.0 ** -24  # half a step of fp32, relative


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def tables(rng, B, max_pages, extra=0):
    """Scattered pages: [B][max_pages] and [B][extra], and the pool's size."""
    n = B * (max_pages + extra) + 2
    order = rng.permutation(n)[: B * (max_pages + extra)].astype(np.int32)
    return order[: B * max_pages].reshape(B, max_pages), order[B * max_pages:].reshape(B, extra), n


def rows_of(pages, table, n):
    """The first n rows of the request with page list `table`: [H, n, ...] from pages [P, H, T, ...]."""
    T = pages.shape[2]
    return np.concatenate([pages[p] for p in table[: max(1, -(-n // T))]], 1)[:, :n]


def put_rows(pages, table, first, x):
    """x [H, n, ...] into rows first .. of a request, in place."""
    T = pages.shape[2]
    for i in range(x.shape[1]):
        pages[table[(first + i) // T], :, (first + i) % T] = x[:, i]


def trees(rng, B, R, back=6):
    """Parents before children; see [B][R][R] bool and the masks' words."""
    see = np.zeros((B, R, R), bool)
    for b in range(B):
        for i in range(R):
            if i:
                see[b, i] = see[b, i - rng.integers(1, min(i, back) + 1)]
            see[b, i, i] = True
    return see, words(see)


def words(see):
    B, R = see.shape[:2]
    m = np.zeros((B, R, (R + 63) // 64), np.uint64)
    for j in range(R):
        m[:, :, j // 64] |= see[:, :, j].astype(np.uint64) << np.uint64(j % 64)
    return torch.from_numpy(m.view(np.int64)).cuda()


def shape_scores(raw, dist, cap, window, slopes):
    """raw [n, hq, keys] (scaled), dist [n, keys] -> scores."""
    s = cap * np.tanh(raw / cap) if cap else raw.copy()
    if slopes is not None:
        s -= slopes[None, :, None] * dist[:, None]
    if window:
        s = np.where((dist < window)[:, None], s, -np.inf)
    return s


def score_error(size, s, bias, cap, adds):
    """How far an fp32 score may be off: `adds` roundings of the products' sum (their sizes `size`), a few of the
    cap's constants, the bias and the score itself, and of its exponential."""
    s = np.where(np.isfinite(s), np.abs(s), 0.0)
    return U32 * (adds * size + 8 * (cap or 0.0) + 4 * bias + 8 * s + 8)


def attention(q, k, v, tk, tv, see, L, n, scale, cap=0.0, window=0, slopes=None, adds=144):
    """One request: q [R, Hq, D]; k, v [H, L, D]; tk, tv [H, R, D] or None; see [R, R].  Returns out [n, Hq, D], lse
    [n, Hq] and bounds of their fp32 errors; adds: 9 for a sum of 128 products in fp32 by pairs, 144 where eight
    matrix instructions add 17 terms each to 24 bits."""
    H, G = k.shape[0], q.shape[1] // k.shape[0]
    if tk is not None:
        see = see[:n, :n]
        depth = np.maximum(see.sum(1) - 1, 0)
        k, v = np.concatenate((k, tk[:, :n]), 1), np.concatenate((v, tv[:, :n]), 1)
        dist = np.concatenate((L + depth[:, None] - np.arange(L), depth[:, None] - depth), 1)
        on = np.concatenate((np.ones((n, L), bool), see), 1)
    else:
        dist = np.broadcast_to(L - 1 - np.arange(L), (n, L))
        on = np.ones((n, L), bool)
    out, lse = np.zeros((n,) + q.shape[1:]), np.full((n, q.shape[1]), -np.inf)
    e_out, e_lse = np.zeros_like(out), np.zeros_like(lse)
    for h in range(H):
        hs = slice(h * G, (h + 1) * G)
        sl = None if slopes is None else slopes[hs]
        raw = np.einsum("ngd,kd->ngk", q[:n, hs], k[h]) * scale
        size = np.einsum("ngd,kd->ngk", np.abs(q[:n, hs]), np.abs(k[h])) * scale
        s = np.where(on[:, None], shape_scores(raw, dist, cap, window, sl), -np.inf)
        bias = np.abs(dist[:, None] * (0 if sl is None else sl[None, :, None]))
        e = score_error(size, s, bias, cap, adds)
        if not s.shape[-1]:
            continue
        top = s.max(-1, keepdims=True)
        p = np.where(np.isfinite(s), np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
        l = p.sum(-1, keepdims=True)
        p = p / np.where(l > 0, l, 1.0)
        with np.errstate(divide="ignore"):
            lse[:, hs] = (np.where(np.isfinite(top), top, 0.0) + np.log(l))[..., 0]
        o = np.einsum("ngk,kd->ngd", p, v[h])
        out[:, hs] = o
        e_out[:, hs] = np.einsum("ngk,kd->ngd", p * e, np.abs(v[h])) + (p * e).sum(-1)[..., None] * np.abs(o)
        e_out[:, hs] += 64 * U32 * np.einsum("ngk,kd->ngd", p, np.abs(v[h]))  # sums over keys, pieces and warps
        e_lse[:, hs] = (p * e).sum(-1) + 16 * U32 * (1 + np.abs(np.where(l > 0, lse[:, hs, None], 0.0))[..., 0])
    return out, lse, e_out, e_lse


def fp32_kinds(rows):
    """(adds, weights' relative error) of fp32 attention over so many rows of a KV head: up to four, sums of products
    by pairs.  Above, three tf32 products a product (12 of 2^-24), two steps of dims in two instructions of nine terms
    each, cut off at 24 bits, eight sums of those and one of the small products'; against V, 12 and three instructions'
    27, and one sum."""
    return (9, 0.0) if rows <= 4 else (12 + 18 + 8 + 1, 40 * U32)


def check_attention(out, lse, ref, bf16, p_error):
    """out bf16: half a step of the result more; p_error: what the weights may be off by, relative (2^-17 where they
    enter the product as two bf16 terms, 2^-9 as one, 0 in fp32), against the sum of p |v|."""
    o, z, e_o, e_z = ref
    tol = (1 + 2.0 ** -8 if bf16 else 1) * (e_o + p_error) + (2.0 ** -8 * np.abs(o) + 2.0 ** -133 if bf16 else 0)
    bad = ~(np.abs(out - o) <= tol)
    assert not bad.any(), (np.abs(out - o)[bad].max(), tol[bad].min(), np.argwhere(bad)[:4])
    assert np.array_equal(np.isfinite(lse), np.isfinite(z))
    f = np.isfinite(z)
    assert (np.abs(lse[f] - z[f]) <= e_z[f]).all(), (np.abs(lse[f] - z[f]).max(), e_z[f].min())


def weights(q, lse, k, L, scale, cap=0.0, window=0, slopes=None, adds=144):
    """Path rows q [n, Hq, D], lse [n, Hq], keys k [H, L, D] -> sums [H, L] and error bounds."""
    n, H = q.shape[0], k.shape[0]
    G = q.shape[1] // H
    dist = np.arange(L - n, L)[:, None] - np.arange(L)
    got, err = np.zeros((H, L)), np.zeros((H, L))
    for h in range(H):
        hs = slice(h * G, (h + 1) * G)
        sl = None if slopes is None else slopes[hs]
        raw = np.einsum("ngd,kd->ngk", q[:, hs], k[h]) * scale
        size = np.einsum("ngd,kd->ngk", np.abs(q[:, hs]), np.abs(k[h])) * scale
        s = np.where((dist >= 0)[:, None], shape_scores(raw, dist, cap, window, sl), -np.inf)
        z = lse[:, hs, None]
        p = np.where(np.isfinite(z) & np.isfinite(s), np.exp(s - np.where(np.isfinite(z), z, 0.0)), 0.0)
        bias = np.abs(dist[:, None] * (0 if sl is None else sl[None, :, None]))
        e = score_error(size, s, bias, cap, adds) + 8 * U32 * np.abs(np.where(np.isfinite(z), z, 0.0))
        got[h] = p.sum((0, 1))
        err[h] = (p * e).sum((0, 1)) + n * G * U32 * got[h]
    return got, err


def kept_rows(w, L, budget, sink, recent):
    """The rows of one head that stay, ascending; weights w [L]."""
    mid = np.arange(sink, L - recent)
    x = w[mid].astype(np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    nan = np.isnan(w[mid])
    order = np.lexsort((mid, nan, -x))  # heaviest first, NaN behind -inf, then the lower row
    keep = mid[order[: budget - sink - recent]]
    return np.sort(np.concatenate((np.arange(sink), keep, np.arange(L - recent, L))))
