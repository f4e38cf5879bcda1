"""GPU: tree attention over the 8-bit cache at the ends of its range: tiny V scales, V scales far
apart in one piece, query rows with a large element.

Bounds as derived in the other attention tests (u = 2^-24, per output element, A = sum p |v|), with
two terms of their own:
  query     an element of a row whose largest is m enters off by `dq` m at most, which moves a score
            by ds' = dq m scale sum |k|.  FAST on the head_dim 128 kernels: the row's largest in
            (224, 448], the second term in steps of 2^-13 or finer wherever the first is off by
            2^-10 or less: 2^-14 / 224 < 2^-21.  PRECISE: the largest in (28672, 57344], the last
            term in steps of 2^-16: 2^-17 / 28672 < 2^-31.  mma.sync: halves with the largest at or
            above 2^14, in steps of 2^-24: 2^-25 / 2^14 = 2^-39
  weight    P is stored as p vs / vref 2^c with c such that the row's largest p vs is at least 2^6
            there; its smallest step is 2^-24 (few rows, head_dim 128: 2^-19), half of which is 2^-31
            (2^-26) of the largest p vs = `top`: n keys of codes up to 448 are off by
            n 2^-31 448 top (n 2^-26 448 top) in all, whatever the other scales of the piece
"""
import math

import numpy as np
import pytest
import torch

import kvq_helpers as H
from eagle_speculative_decoding_tree_gb300 import binding as B
from test_gpu_kvq_attn import Case, bf16

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def settle(c):
    """The reference and the device tensors of a case whose contents were changed."""
    f = lambda t: t.double().numpy()
    vals = [H.TABLE[x] * np.repeat(s.astype(np.float64), 64, -1)[..., : x.shape[-2], None]
            for x, s in zip(c.codes, c.scale)]
    for v in vals:  # rows behind the prefix do not take part
        for b in range(v.shape[0]):
            v[b, :, c.seq[b]:] = 0.0
    c.vals = vals
    c.ref = H.attention(f(c.q), vals[0], vals[1], f(c.tk), f(c.tv), c.seq, c.nodes, c.see,
                        1 / math.sqrt(c.dims[4]))
    dev = [torch.from_numpy(x).cuda() for p in zip(c.codes, c.scale) for x in p]
    c.dev = [c.q.cuda(), *dev, c.tk.cuda(), c.tv.cuda(), *c.dev[7:]]
    return c


def weighted_top(c):
    """The largest p vs of each row, prefix keys, [B][R][Hq]."""
    Bn, R, Hq, Hkv, D, P = c.dims
    res, f = np.zeros((Bn, R, Hq)), lambda t: t.double().numpy()
    for b in range(Bn):
        L = int(c.seq[b])
        for hq in range(Hq if L else 0):
            h = hq // (Hq // Hkv)
            s = f(c.q)[b, :, hq] @ c.vals[0][b, h, :L].T / math.sqrt(D)
            vs = np.repeat(c.scale[1][b, h].astype(np.float64), 64)[:L]
            res[b, :, hq] = (np.exp(s - c.ref[1][b, :, hq][:, None]) * vs).max(1)
    return res


def check(c, d, few, dq=0.0, tiny=1e-37):
    Bn, R, Hq, Hkv, D, P = c.dims
    out, lse = c.run(d)
    ref, rl, mass, reach = c.ref
    o, ls = out.double().cpu().numpy(), lse.double().cpu().numpy()
    n = (c.seq + c.nodes)[:, None, None]
    f = lambda t: t.double().numpy()
    most = np.zeros((Bn, R, Hq))  # the largest sum |k| of a key, per head
    for b in range(Bn):
        for h in range(Hkv):
            k = np.abs(np.concatenate((c.vals[0][b, h, : c.seq[b]], f(c.tk)[b, h]))).sum(1).max()
            most[b, :, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)] = k
    ds = 2 * (D + 10) * U * reach + dq * np.abs(f(c.q)).max(-1) * most / math.sqrt(D)
    p_round = 2.0 ** -16 + (2.0 ** -21 if d.precision == B.EAGLE_ATTN_PRECISE else 2.0 ** -11)
    rel = (2 * ds + 2.0 ** -21 + p_round + 4 * U * n)[..., None]
    floor = (n * (2.0 ** -26 if few else 2.0 ** -31) * 448 * weighted_top(c))[..., None]
    tol = rel * mass + floor + (2.0 ** -8 if d.out_dtype == B.EAGLE_BF16 else 2.0 ** -24) * np.abs(ref) + tiny
    assert np.isfinite(o).all() and np.isfinite(ls).all()
    worst = (np.abs(o - ref) / tol).max()
    assert worst <= 1, worst
    lt = ds + 2 * U * n + 2.0 ** -21 + 2.0 ** -22 * np.abs(rl)
    assert (np.abs(ls - rl) <= lt).all(), (np.abs(ls - rl) / lt).max()


# (R, Hq, Hkv, D, engine): few rows, row tiles, mma.sync at both head sizes
KERNELS = [(1, 4, 1, 128, 0), (4, 8, 2, 128, 0), (8, 8, 2, 128, 0), (40, 8, 2, 128, 0), (61, 8, 2, 128, 0),
           (5, 4, 2, 64, 0), (40, 8, 2, 64, 0), (9, 8, 2, 128, 1)]
few_rows = lambda k: k[3] == 128 and k[4] == 0 and k[0] * (k[1] // k[2]) <= 32
name = lambda k: "R%d-%d:%dx%d-%d" % k


@pytest.mark.parametrize("splits", [1, 2, 0])
@pytest.mark.parametrize("vs", [-126, -118, -113, -64])
@pytest.mark.parametrize("kern", KERNELS, ids=name)
def test_tiny_v_scales_beside_a_tree(kern, vs, splits):
    """Prefix values down to the smallest that the writers store, and a tree of ordinary ones."""
    R, Hq, Hkv, D, engine = kern
    c = Case(51, 2, R, Hq, Hkv, D, 300, [300, 129])
    c.scale[1][:] = 2.0 ** vs
    settle(c)
    for precise in (False, True):
        check(c, c.desc(True, precise, splits, engine), few_rows(kern))


@pytest.mark.parametrize("vs", [-128, -130, -140])
@pytest.mark.parametrize("kern", KERNELS, ids=name)
def test_v_scales_below_the_normal_numbers(kern, vs):
    """Another writer's scales (any finite one is taken); 2^-149 is fp32's smallest step, and a row
    is rounded to it a few times."""
    R, Hq, Hkv, D, engine = kern
    c = Case(52, 1, R, Hq, Hkv, D, 200, [200])
    c.scale[1][:] = 2.0 ** vs
    c.tv = torch.zeros_like(c.tv)
    settle(c)
    for splits in (0, 1):
        check(c, c.desc(True, True, splits, engine), few_rows(kern), tiny=2.0 ** -146)


@pytest.mark.parametrize("first", [True, False], ids=["first", "last"])
@pytest.mark.parametrize("ratio", [14, 24, 32, 60, 90])
@pytest.mark.parametrize("kern", KERNELS, ids=name)
def test_the_heavy_keys_scale_is_far_below_another_one(kern, ratio, first):
    """One block of keys has all the weight and a V scale 2^-ratio of the others'; the heads of odd
    index look away from it, at the others."""
    R, Hq, Hkv, D, engine = kern
    L = 320
    c = Case(53, 1, R, Hq, Hkv, D, L, [L])
    g = np.random.default_rng(54)
    u = np.sign(g.normal(size=D))
    a = 2.0 if ratio <= 32 else (3.0 if ratio <= 60 else 4.0)  # weights apart by 2^(2 a sqrt(D) / ln 2)
    a *= 128 // D
    sign = np.where(np.arange(Hq) % 2 == 0, 1.0, -1.0) if Hq > 1 else np.ones(1)
    c.q = bf16(np.broadcast_to(u * sign[:, None], (1, R, Hq, D)).copy())
    rows = slice(0, 64) if first else slice(256, 320)
    k = np.broadcast_to(-a * u, (1, Hkv, L, D)).copy()
    k[:, :, rows] = a * u
    c.codes[0], c.scale[0][:] = H.encode(k), 1.0
    c.scale[1][:] = 1.0
    c.scale[1][:, :, 0 if first else 4] = 2.0 ** -ratio
    c.tk = bf16(np.zeros(c.tk.shape))                       # the tree's keys: in between, without values
    c.tv = torch.zeros_like(c.tv)
    settle(c)
    for splits in (1, 2):
        for precise in (False, True):
            check(c, c.desc(True, precise, splits, engine), few_rows(kern))


@pytest.mark.parametrize("kern", KERNELS, ids=name)
def test_scales_over_2_to_the_60_at_random(kern):
    R, Hq, Hkv, D, engine = kern
    c = Case(55, 2, R, Hq, Hkv, D, 1000, [1000, 700], q_size=6.0)
    c.scale[1][:] = 2.0 ** np.random.default_rng(56).integers(-60, 1, c.scale[1].shape)
    settle(c)
    for splits in (0, 1, 3):
        check(c, c.desc(True, True, splits, engine), few_rows(kern))


@pytest.mark.parametrize("size", [50, 2.0 ** 12, 2.0 ** 16])
@pytest.mark.parametrize("kern", KERNELS, ids=name)
def test_query_rows_with_a_large_element(kern, size):
    """One channel of every query row is `size` times the others and meets keys that have nothing in
    it: the scores come from the small elements."""
    R, Hq, Hkv, D, engine = kern
    c = Case(57, 2, R, Hq, Hkv, D, 200, [200, 65])
    c.q[..., 7] *= size
    c.q[:, :, 0, 7] = size
    c.codes[0][..., 7] = 0
    c.tk[..., 7] = 0.0
    settle(c)
    wide = D == 128 and engine == 0
    check(c, c.desc(True, True, 0, engine), few_rows(kern), dq=2.0 ** -31 if wide else 2.0 ** -39)
    check(c, c.desc(True, False, 0, engine), few_rows(kern), dq=2.0 ** -21 if wide else 2.0 ** -39)
