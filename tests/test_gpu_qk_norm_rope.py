"""GPU: head norms, rotation and layout in one pass against 64 bits.

Bound (u = 2^-24): the norm's sum of D squares, the root, the division and two products are off
by at most (D + 8) u of the value; sine and cosine by 2^-21 (the angle's reduction to [-1, 1]
half turns rounds once to fp32, pi u, and the functions 2 units); the rotation adds two more
roundings: (D + 8 + 4) u + 2^-21 of |a| + |b|, then the output's own 2^-8 or u.
"""
import numpy as np
import pytest
import torch

import kvq_helpers as H
from eagle_speculative_decoding_tree_gb300 import binding as B

pytestmark = pytest.mark.gpu
DT = {"bf16": (torch.bfloat16, B.EAGLE_BF16, 2.0 ** -8), "f32": (torch.float32, B.EAGLE_F32, 2.0 ** -24)}


def run(seed, Bn, R, Hq, Hkv, D, rot, inter, norm, dtype, pad=0, far=5000, nodes=None, size=1.0, eps=1e-6, zero_row=False):
    g = np.random.default_rng(seed)
    tdt, code, uo = DT[dtype]
    width = (Hq + 2 * Hkv) * D
    x = torch.from_numpy((size * g.normal(size=(Bn, R, width + pad))).astype(np.float32)).to(tdt)
    if zero_row:
        x[:, 0] = 0
    w = [torch.from_numpy((1 + 0.3 * g.normal(size=D)).astype(np.float32)).to(tdt) if norm[i] else None for i in (0, 1)]
    inv = (500000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)
    inv_t = torch.from_numpy(inv if rot else np.ones(1, np.float32)).cuda()
    pos = g.integers(0, far, (Bn, R)).astype(np.int32)
    pos[0, 0] = far - 1
    q = torch.full((Bn, R, Hq, D), 5.0, dtype=tdt, device="cuda")
    k = torch.full((Bn, Hkv, R, D), 5.0, dtype=tdt, device="cuda")
    v = k.clone()
    d = B.QkNormRopeDesc(Bn, R, Hq, Hkv, D, rot, width + pad if pad else 0, int(inter), eps, code)
    nn = None if nodes is None else torch.tensor(nodes, dtype=torch.int32, device="cuda")
    up = lambda t: None if t is None else t.cuda()
    B.eagle_qk_norm_rope(d, x.cuda(), up(w[0]), up(w[1]), inv_t, torch.from_numpy(pos).cuda(), q, k, v, n_nodes=nn)
    h = x[..., :width].double().numpy().reshape(Bn, R, Hq + 2 * Hkv, D)
    f = lambda t: None if t is None else t.double().numpy()
    rel = (D + 12) * 2.0 ** -24 + 2.0 ** -21
    for b in range(Bn):
        n = R if nodes is None else min(max(nodes[b], 0), R)
        for got, lo, hi, wt in ((q[b], 0, Hq, w[0]), (k[b].transpose(0, 1), Hq, Hq + Hkv, w[1])):
            ref, bound = H.rope(h[b, :, lo:hi], f(wt), eps, pos[b], inv, rot, inter)
            o = got.double().cpu().numpy()
            assert (np.abs(o - ref) <= rel * bound + uo * np.abs(ref) + 1e-37)[:n].all()
            assert (o[n:] == 5).all()
        vv = v[b].transpose(0, 1).double().cpu().numpy()
        assert np.array_equal(vv[:n], h[b, :n, Hq + Hkv:]) and (vv[n:] == 5).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Bn,R,Hq,Hkv,D,rot,inter,norm,pad", [
    (1, 1, 1, 1, 64, 64, False, (1, 1), 0),
    (1, 61, 32, 8, 128, 128, False, (1, 1), 0),
    (2, 7, 28, 4, 128, 128, True, (1, 1), 8),
    (3, 5, 5, 5, 64, 32, False, (0, 0), 64),
    (1, 130, 33, 1, 128, 64, True, (1, 0), 0),
    (2, 3, 71, 3, 64, 16, False, (0, 1), 0),
    (1, 4, 8, 2, 128, 0, False, (1, 1), 0),
    (1, 6, 8, 2, 128, 96, False, (1, 1), 0),
    (1, 6, 8, 2, 64, 48, True, (1, 1), 0),
])
def test_matches_64_bits(Bn, R, Hq, Hkv, D, rot, inter, norm, pad, dtype):
    run(1, Bn, R, Hq, Hkv, D, rot, inter, norm, dtype, pad)


@pytest.mark.parametrize("far", [2, 131072, 2 ** 24, 2 ** 31 - 1])
def test_far_positions(far):
    run(2, 1, 9, 4, 2, 128, 128, False, (1, 1), "f32", far=far)


@pytest.mark.parametrize("size,eps", [(1e-18, 0.0), (1e18, 1e-5), (1.0, 1.0)])
def test_sizes_and_eps(size, eps):
    run(3, 1, 5, 4, 2, 128, 128, False, (1, 1), "f32", size=size, eps=eps)


def test_zero_rows_and_missing_nodes():
    run(4, 1, 3, 4, 2, 128, 128, False, (1, 1), "bf16", zero_row=True)
    run(5, 4, 9, 8, 2, 128, 128, False, (1, 1), "bf16", nodes=[9, 0, 4, -1])


def test_captured():
    """A replayed call follows the positions in its buffer."""
    R, Hq, Hkv, D = 5, 4, 2, 64
    x = torch.randn(1, R, (Hq + 2 * Hkv) * D, device="cuda")
    inv = torch.ones(D // 2, device="cuda")
    pos = torch.zeros(1, R, dtype=torch.int32, device="cuda")
    outs = [torch.zeros(1, R, Hq, D, device="cuda")] + [torch.zeros(1, Hkv, R, D, device="cuda") for _ in range(2)]
    d = B.QkNormRopeDesc(1, R, Hq, Hkv, D, D, 0, 0, 1e-6, B.EAGLE_F32)
    B.eagle_qk_norm_rope(d, x, None, None, inv, pos, *outs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.eagle_qk_norm_rope(d, x, None, None, inv, pos, *outs)
    pos.fill_(3)
    g.replay()
    got = outs[0].clone()
    B.eagle_qk_norm_rope(d, x, None, None, inv, pos, *outs)
    assert torch.equal(got, outs[0]) and not torch.equal(got[0, :, 0], x[0, :, :D])
