"""GPU: writing, committing and reading the 8-bit KV cache, against the 64-bit reference.

Codes and scales are exact (a power-of-two scale makes the division exact), so every
comparison here is equality; a read value is code * scale rounded once.
"""
import numpy as np
import pytest
import torch

import kvq_helpers as H
from eagle_speculative_decoding_tree_gb300 import binding as B

pytestmark = pytest.mark.gpu

DT = {"bf16": (torch.bfloat16, B.EAGLE_BF16), "f32": (torch.float32, B.EAGLE_F32)}


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def rows_of(seed, shape, dtype):
    """Rows whose size changes from row to row, as the tensor and as fp64."""
    g = np.random.default_rng(seed)
    x = g.normal(size=shape) * 2.0 ** g.integers(-6, 7, shape[:-1] + (1,))
    t = torch.from_numpy(x.astype(np.float32)).to(DT[dtype][0]).cuda()
    return t, t.double().cpu().numpy()


def cache(seed, lead, P, D):
    """A cache with arbitrary content: finite codes, power-of-two scales."""
    g = np.random.default_rng(seed)
    codes = g.integers(0, 127, lead + (P, D)).astype(np.uint8) | (g.integers(0, 2, lead + (P, D)) * 128).astype(np.uint8)
    scale = (2.0 ** g.integers(-8, 3, lead + (-(-P // 64),))).astype(np.float32)
    return codes, scale


def same(got_codes, got_scale, codes, scale):
    assert np.array_equal(H.decode(got_codes.cpu().numpy()), H.decode(codes), equal_nan=True)
    assert np.array_equal(got_scale.cpu().numpy(), scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Bn,Hk,D,P,N,start,count", [
    (1, 1, 128, 64, 1, [0], None),
    (1, 2, 128, 64, 64, [0], None),
    (2, 3, 64, 200, 65, [0, 135], None),
    (3, 2, 128, 333, 130, [63, 64, 203], [130, 1, 130]),
    (4, 2, 64, 500, 129, [1, 127, 0, 371], [0, 2, 128, 129]),
    (2, 8, 128, 1021, 511, [510, 37], [511, 509]),
])
def test_write_matches_the_reference(Bn, Hk, D, P, N, start, count, dtype):
    ck, sk = cache(1, (Bn, Hk), P, D)
    cv, sv = cache(2, (Bn, Hk), P, D)
    k, kx = rows_of(3, (Bn, Hk, N, D), dtype)
    v, vx = rows_of(4, (Bn, Hk, N, D), dtype)
    dev = [torch.from_numpy(x.copy()).cuda() for x in (ck, sk, cv, sv)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = B.KvqDesc(Bn, Hk, D, P, N, DT[dtype][1])
    B.eagle_kvq_write(d, k, v, i32(start), None if count is None else i32(count), *dev, status)
    cnt = [N] * Bn if count is None else count
    for b in range(Bn):
        for h in range(Hk):
            H.append(ck[b, h], sk[b, h], kx[b, h, :cnt[b]], start[b])
            H.append(cv[b, h], sv[b, h], vx[b, h, :cnt[b]], start[b])
    same(dev[0], dev[1], ck, sk)
    same(dev[2], dev[3], cv, sv)
    assert int(status) == 0
    # read back: written rows and the ones around them
    for odt in ("bf16", "f32"):
        out = [torch.full((Bn, Hk, N, D), 7.0, dtype=DT[odt][0], device="cuda") for _ in range(2)]
        B.eagle_kvq_read(B.KvqDesc(Bn, Hk, D, P, N, DT[odt][1]), *dev, i32(start),
                         None if count is None else i32(count), *out, status)
        for o, c, s in ((out[0], ck, sk), (out[1], cv, sv)):
            val = H.values(c, s)
            for b in range(Bn):
                want = torch.from_numpy(val[b, :, start[b]:start[b] + cnt[b]]).to(DT[odt][0])
                assert torch.equal(o[b, :, :cnt[b]].cpu(), want)
                assert bool((o[b, :, cnt[b]:] == 7.0).all())


def test_spans_outside_the_cache_are_refused_on_the_device():
    Bn, P, N, D = 6, 100, 40, 64
    ck, sk = cache(5, (Bn, 1), P, D)
    k, kx = rows_of(6, (Bn, 1, N, D), "bf16")
    dev = [torch.from_numpy(x.copy()).cuda() for x in (ck, sk, ck, sk)]
    start, count = [-1, 61, 0, 2**31 - 1, 5, 60], [1, 40, 41, 40, -3, 40]
    d = B.KvqDesc(Bn, 1, D, P, N, B.EAGLE_BF16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.eagle_kvq_write(d, k, k, i32(start), i32(count), *dev, status)
    H.append(ck[5, 0], sk[5, 0], kx[5, 0], 60)
    same(dev[0], dev[1], ck, sk)
    assert int(status) == B.EAGLE_STATUS_CACHE_FULL
    out = torch.full((Bn, 1, N, D), 3.0, dtype=torch.bfloat16, device="cuda")
    status.zero_()
    B.eagle_kvq_read(d, *dev, i32(start), i32(count), out, out.clone(), status)
    assert bool((out[:5] == 3.0).all()) and int(status) == B.EAGLE_STATUS_CACHE_FULL
    B.eagle_kvq_write(d, k, k, i32(start), i32(count), *dev)  # status is optional


def test_special_values():
    """Zeros, values that are not finite, the largest and the smallest magnitudes."""
    D = 64
    x = np.zeros((1, 6, 64, D))
    x[0, 1, :, 0] = [np.nan if i % 3 == 0 else (np.inf if i % 3 == 1 else -np.inf) for i in range(64)]
    x[0, 1, :, 1] = 3.0
    x[0, 2] = 3.0e38
    x[0, 3] = 1e-41  # below the smallest scale's codes: zeros
    x[0, 4, :, :] = 2.0 ** -126 * 448
    x[0, 5, 0, :2] = [448.0, 449.0]
    t = torch.from_numpy(x.astype(np.float32)).cuda()
    dev = [torch.zeros(1, 6, 64, D, dtype=torch.uint8, device="cuda"), torch.zeros(1, 6, 1, device="cuda")]
    dev += [y.clone() for y in dev]
    d = B.KvqDesc(1, 6, D, 64, 64, B.EAGLE_F32)
    B.eagle_kvq_write(d, t, t, i32([0]), None, *dev)
    ck, sk = np.zeros((6, 64, D), np.uint8), np.zeros((6, 1), np.float32)
    for h in range(6):
        H.append(ck[h], sk[h], t[0, h].double().cpu().numpy(), 0)
    same(dev[0][0], dev[1][0], ck, sk)
    assert float(dev[1][0, 0]) == 0.0 and float(dev[1][0, 2]) == 2.0 ** 120
    out = torch.empty_like(t)
    B.eagle_kvq_read(d, *dev, i32([0]), None, out, out.clone())
    assert bool(out[0, 1, :, 0].isnan().all()) and bool((out[0, 1, :, 1] == 3.0).all())
    # any finite scale reads back; 0 marks zeros
    dev[1][0, 0] = 0.3
    dev[0][0, 0] = 0x38  # 1.0
    dev[0][0, 5] = 0x38
    dev[1][0, 5] = 0.0
    B.eagle_kvq_read(d, *dev, i32([0]), None, out, out.clone())
    assert bool((out[0, 0] == np.float32(0.3)).all()) and bool((out[0, 5] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,Bn,Hk,D,P,R,maxd", [(1, 1, 1, 64, 8, 1, 0), (3, 4, 2, 128, 200, 61, 7), (2, 3, 8, 64, 333, 128, 127)])
def test_commit_matches_the_reference(L, Bn, Hk, D, P, R, maxd, dtype):
    g = np.random.default_rng(7)
    ks = [cache(10 + l, (Bn, Hk), P, D) for l in range(L)]
    vs = [cache(20 + l, (Bn, Hk), P, D) for l in range(L)]
    tk, tv = [[rows_of(s + l, (Bn, Hk, R, D), dtype) for l in range(L)] for s in (30, 40)]
    n_acc = g.integers(0, min(maxd, R - 1) + 1, Bn)
    n_acc[0] = min(maxd, R - 1)
    path = np.full((Bn, maxd + 1), -1)
    for b in range(Bn):
        path[b, :n_acc[b] + 1] = np.sort(g.permutation(R)[:n_acc[b] + 1])
    seq = np.array([g.integers(0, P - n_acc[b]) for b in range(Bn)])
    if Bn > 2:
        seq[1] = 64 - (n_acc[1] + 1) // 2  # crosses a block
    up = lambda pairs, i: [torch.from_numpy(p[i].copy()).cuda() for p in pairs]
    dk, dks, dv, dvs = up(ks, 0), up(ks, 1), up(vs, 0), up(vs, 1)
    layers = B.KvqLayerPointers(dk, dks, dv, dvs, [t[0] for t in tk], [t[0] for t in tv])
    feat, tfeat = torch.zeros(Bn, P, 36, device="cuda"), torch.randn(Bn, R, 36, device="cuda")
    d = B.CommitDesc(L, Bn, Hk, D, R, P, maxd, DT[dtype][1], 36, B.EAGLE_F32)
    sl, pos = i32(seq), torch.zeros(Bn, maxd + 1, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.eagle_kvq_commit(d, layers, i32(n_acc), i32(path), sl, pos, feat, tfeat, status)
    for l in range(L):
        for b in range(Bn):
            nodes = path[b, :n_acc[b] + 1]
            for h in range(Hk):
                H.append(ks[l][0][b, h], ks[l][1][b, h], tk[l][1][b, h, nodes], int(seq[b]))
                H.append(vs[l][0][b, h], vs[l][1][b, h], tv[l][1][b, h, nodes], int(seq[b]))
        same(dk[l], dks[l], *ks[l])
        same(dv[l], dvs[l], *vs[l])
    assert np.array_equal(sl.cpu().numpy(), seq + n_acc + 1) and int(status) == 0
    m = np.arange(maxd + 1)
    assert np.array_equal(pos.cpu().numpy(), np.where(m <= n_acc[:, None], seq[:, None] + m, -1))
    for b in range(Bn):
        n = n_acc[b] + 1
        assert torch.equal(feat[b, seq[b]:seq[b] + n].cpu(), tfeat[b].cpu()[path[b, :n]])
        assert bool((feat[b, seq[b] + n:] == 0).all()) and bool((feat[b, :seq[b]] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_that_are_not_finite_are_committed_as_nan(dtype):
    """More rows than one round of a warp, some with NaN and infinities: the scale follows the
    finite values, the others read back as NaN."""
    L, Bn, Hk, D, P, R = 1, 1, 2, 128, 128, 40
    ck, sk = cache(55, (Bn, Hk), P, D)
    t, tx = rows_of(56, (Bn, Hk, R, D), dtype)
    for r, v in ((0, np.inf), (13, np.nan), (39, -np.inf)):
        t[0, 1, r, r] = v
        tx[0, 1, r, r] = v
    dev = [[torch.from_numpy(x.copy()).cuda()] for x in (ck, sk, ck, sk)]
    d = B.CommitDesc(L, Bn, Hk, D, R, P, R - 1, DT[dtype][1], 0, B.EAGLE_F32)
    B.eagle_kvq_commit(d, B.KvqLayerPointers(*dev, [t], [t]), i32([R - 1]), i32([np.arange(R)]), i32([50]),
                       torch.zeros(1, R, dtype=torch.int32, device="cuda"))
    for h in range(Hk):
        H.append(ck[0, h], sk[0, h], tx[0, h], 50)
    assert np.isnan(H.decode(ck)).sum() == 3
    same(dev[0][0], dev[1][0], ck, sk)
    same(dev[2][0], dev[3][0], ck, sk)


def test_commit_leaves_full_and_malformed_requests():
    Bn, Hk, D, P, R = 5, 2, 64, 70, 9
    ck, sk = cache(50, (Bn, Hk), P, D)
    t, tx = rows_of(51, (Bn, Hk, R, D), "f32")
    dev = [[torch.from_numpy(x.copy()).cuda()] for x in (ck, sk, ck, sk)]
    layers = B.KvqLayerPointers(*dev, [t], [t])
    seq = np.array([69, 68, 2**31 - 2, -1, 62])
    n_acc = np.array([1, 1, 1, 1, 3])
    path = np.array([[0, 1, -1, -1], [0, 2, -1, -1], [0, 1, -1, -1], [0, 1, -1, -1], [0, 9, 4, 4]])
    sl, pos = i32(seq), torch.zeros(Bn, 4, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = B.CommitDesc(1, Bn, Hk, D, R, P, 3, B.EAGLE_F32, 0, B.EAGLE_F32)
    B.eagle_kvq_commit(d, layers, i32(n_acc), i32(path), sl, pos, status=status)
    for h in range(Hk):
        H.append(ck[1, h], sk[1, h], tx[1, h, [0, 2]], 68)
        # node 9 is outside the tree: its row (63) is left as it was, the others land; block 0
        # takes row 62, block 1 rows 64 and 65 (the same node twice)
        H.append(ck[4, h], sk[4, h], tx[4, h, [0]], 62)
        H.append(ck[4, h], sk[4, h], tx[4, h, [4, 4]], 64)
    same(dev[0][0], dev[1][0], ck, sk)
    same(dev[2][0], dev[3][0], ck, sk)
    assert sl.cpu().tolist() == [69, 70, 2**31 - 2, -1, 66]
    assert int(status) == B.EAGLE_STATUS_CACHE_FULL | B.EAGLE_STATUS_BAD_TREE


def test_chunked_writes_equal_one_write_of_growing_blocks():
    """A prompt written in chunks that end inside blocks, by replaying one captured call that
    advances its own start: every block holds what the reference's appends give."""
    D, P, N = 128, 640, 90
    ck, sk = np.zeros((1, 2, P, D), np.uint8), np.zeros((1, 2, P // 64), np.float32)
    dev = [torch.from_numpy(x.copy()).cuda() for x in (ck, sk, ck, sk)]
    x, xx = rows_of(60, (1, 2, N, D), "bf16")
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = B.KvqDesc(1, 2, D, P, N, B.EAGLE_BF16)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.eagle_kvq_write(d, x, x, start, None, *dev)  # outside the capture once
        for t in dev:
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            B.eagle_kvq_write(d, x, x, start, None, *dev)
            start.add_(N)
    torch.cuda.synchronize()
    start.zero_()
    for i in range(7):
        g.replay()
        for h in range(2):
            H.append(ck[0, h], sk[0, h], xx[0, h], i * N)
    torch.cuda.synchronize()
    same(dev[0], dev[1], ck, sk)


def test_offsets_past_32_bits():
    """The last request of a cache whose codes take more than 2^32 bytes."""
    Bn, Hk, D, P, N = 34, 8, 128, 131072, 100
    kc = torch.zeros(Bn, Hk, P, D, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(Bn, Hk, P // 64, device="cuda")
    assert kc.numel() > 2 ** 32
    vc, sv = torch.zeros_like(kc), torch.zeros_like(sc)
    x, xx = rows_of(70, (Bn, Hk, N, D), "bf16")
    start, count = np.full(Bn, P - N), np.zeros(Bn, int)
    count[-1] = N
    d = B.KvqDesc(Bn, Hk, D, P, N, B.EAGLE_BF16)
    B.eagle_kvq_write(d, x, x, i32(start), i32(count), kc, sc, vc, sv)
    out = torch.zeros_like(x)
    B.eagle_kvq_read(d, kc, sc, vc, sv, i32(start), i32(count), torch.zeros_like(x), out)
    for h in range(Hk):
        c, s = np.zeros((P, D), np.uint8), np.zeros(P // 64, np.float32)
        H.append(c, s, xx[-1, h], P - N)
        same(vc[-1, h], sv[-1, h], c, s)
        assert torch.equal(out[-1, h].cpu(), torch.from_numpy(H.values(c, s)[P - N:]).bfloat16())
    assert int(kc[:-1].count_nonzero()) == 0 and bool((out[:-1] == 0).all())
