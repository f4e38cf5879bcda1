"""GPU: tree attention over the 8-bit cache against 64-bit attention over the cache's values.

Bounds (derived, u = 2^-24, per output element; A = sum p |v| of the row):
  score     the products are exact; D + 2 fp32 additions and multiplications of terms whose
            magnitudes sum to `reach` = sum |q||k| scale, each off by at most 2 u (a tensor core
            may truncate): ds = 2 (D + 8) u reach, and the exponent's own rounding 2 u reach
  weight    2 ds (numerator and sum) + the exponential and its offset, 2^-21
  P         rounded to a half: 2^-11 (FAST), twice: 2^-21 (PRECISE); the tree's part 2^-16
            and where it is below a half's normal range, by half of its smallest step, 2^-25:
            stored as p 2^11 vs / vref (vref the largest vs) that is 2^-36 vref of a code's
            weight, the row's reference is at most twice its largest weight, so the sum is at
            least 1/2, and a code at most 448: n 2^-35 448 vref.  (A dimension in which the
            heavy keys' values are tiny and the light ones' large sees nothing else.)  Few rows
            (R G <= 32, head_dim 128): 2^-17 (PRECISE), and steps of 2^-19 instead of 2^-24,
            n 2^-30 448 vref in the worst case; these tests hold them to the smaller bound
  sums      n additions of fp32 in each of the row sum and the output: 2 * 2 u n, n the keys
  output    2^-8 |out| for bf16, 2^-24 for fp32
  lse       ds + 2 u n + 2^-21 + 2^-22 |lse|
"""
import math

import numpy as np
import pytest
import torch

import kvq_helpers as H
from eagle_speculative_decoding_tree_gb300 import binding as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16()


def random_see(g, Bn, R):
    see = np.zeros((Bn, R, R), bool)
    for b in range(Bn):
        for i in range(R):
            if i:
                see[b, i] = see[b, int(g.integers(max(0, i - 6), i))]
            see[b, i, i] = True
    return see


def words(see):
    Bn, R, _ = see.shape
    W = -(-R // 64)
    m = np.zeros((Bn, R, W), np.uint64)
    for j in range(R):
        m[:, :, j // 64] |= see[:, :, j].astype(np.uint64) << np.uint64(j % 64)
    return torch.from_numpy(m.view(np.int64)).cuda()


class Case:
    def __init__(self, seed, Bn, R, Hq, Hkv, D, P, seq, nodes=None, q_size=1.0, scales=None, see=None):
        g = np.random.default_rng(seed)
        self.dims = (Bn, R, Hq, Hkv, D, P)
        self.seq, self.nodes = np.array(seq), np.full(Bn, R) if nodes is None else np.array(nodes)
        self.ragged = nodes is not None
        nb = -(-P // 64)
        mk = lambda *s: g.normal(size=s)
        self.codes = [H.encode(np.clip(mk(Bn, Hkv, P, D) * 100, -448, 448)) for _ in range(2)]
        if scales is None:  # what the writers produce: powers of two, changing from block to block
            self.scale = [(2.0 ** g.integers(-9, -5, (Bn, Hkv, nb))).astype(np.float32) for _ in range(2)]
        else:
            self.scale = [scales(g, (Bn, Hkv, nb)).astype(np.float32) for _ in range(2)]
        self.q, self.tk, self.tv = bf16(mk(Bn, R, Hq, D) * q_size), bf16(mk(Bn, Hkv, R, D)), bf16(mk(Bn, Hkv, R, D))
        self.see = random_see(g, Bn, R) if see is None else see
        vals = [H.values(c, s) for c, s in zip(self.codes, self.scale)]
        f = lambda t: t.double().numpy()
        self.ref = H.attention(f(self.q), vals[0], vals[1], f(self.tk), f(self.tv), self.seq, self.nodes, self.see,
                               1 / math.sqrt(D))
        # nothing behind a request's last row may matter
        for b in range(Bn):
            for c, s in zip(self.codes, self.scale):
                c[b, :, self.seq[b]:] = 0x7f
                s[b, :, -(-int(self.seq[b]) // 64):] = math.nan
            self.tk[b, :, self.nodes[b]:] = math.nan
            self.tv[b, :, self.nodes[b]:] = math.inf
            self.see[b, :, self.nodes[b]:] = True
        self.dev = [torch.from_numpy(x).cuda() for p in zip(self.codes, self.scale) for x in p]
        self.dev = [self.q.cuda(), *self.dev, self.tk.cuda(), self.tv.cuda(), i32(self.seq), words(self.see)]

    def desc(self, out_f32=False, precise=False, splits=0, engine=B.EAGLE_ENGINE_AUTO):
        Bn, R, Hq, Hkv, D, P = self.dims
        return B.AttnDesc(Bn, R, Hq, Hkv, D, P, 1 / math.sqrt(D), B.EAGLE_BF16, splits,
                          B.EAGLE_F32 if out_f32 else B.EAGLE_BF16,
                          B.EAGLE_ATTN_PRECISE if precise else B.EAGLE_ATTN_FAST, engine)

    def run(self, d, ws=None, lse=True):
        Bn, R, Hq, Hkv, D, P = self.dims
        out = torch.full((Bn, R, Hq, D), 9.0, dtype=torch.float32 if d.out_dtype == B.EAGLE_F32 else torch.bfloat16,
                         device="cuda")
        ls = torch.full((Bn, R, Hq), 9.0, device="cuda") if lse else None
        if ws is None:
            ws = torch.zeros(B.workspace_size(B.EAGLE_WS_TREE_ATTN_KVQ, d), dtype=torch.uint8, device="cuda")
        q, kc, ks, vc, vs, tk, tv, seq, mask = self.dev
        B.eagle_tree_attn_kvq(d, q, kc, ks, vc, vs, tk, tv, seq, mask, out, ls, ws,
                              n_nodes=i32(self.nodes) if self.ragged else None)
        torch.cuda.synchronize()
        assert int(ws[:4].view(torch.int32)) == 0
        return out, ls

    def check(self, d, p_round=None):
        Bn, R, Hq, Hkv, D, P = self.dims
        out, lse = self.run(d)
        ref, rl, mass, reach = self.ref
        o, ls = out.double().cpu().numpy(), lse.double().cpu().numpy()
        n = (self.seq + self.nodes)[:, None, None]
        ds = 2 * (D + 10) * U * reach
        if p_round is None:
            p_round = 2.0 ** -16 + (2.0 ** -21 if d.precision == B.EAGLE_ATTN_PRECISE else 2.0 ** -11)
        rel = (2 * ds + 2.0 ** -21 + p_round + 4 * U * n)[..., None]
        vmax = np.array([[max([float(x) for x in self.scale[1][b, h, : -(-int(self.seq[b]) // 64)]], default=0.0)
                          for h in range(Hkv)] for b in range(Bn)])
        floor = (n * 2.0 ** -35 * 448 * np.repeat(vmax, Hq // Hkv, 1)[:, None])[..., None]
        tol = rel * mass + floor + (2.0 ** -8 if d.out_dtype == B.EAGLE_BF16 else 2.0 ** -24) * np.abs(ref) + 1e-37
        for b in range(Bn):
            m = int(self.nodes[b])
            assert np.isfinite(o[b, :m]).all()
            worst = (np.abs(o[b, :m] - ref[b, :m]) / tol[b, :m]).max() if m else 0
            assert worst <= 1, worst
            fin = np.isfinite(rl[b, :m])
            assert np.array_equal(ls[b, :m][~fin], rl[b, :m][~fin])
            lt = (ds + 2 * U * n + 2.0 ** -21)[b, :m] + 2.0 ** -22 * np.abs(np.where(fin, rl[b, :m], 0))
            assert (np.abs(ls[b, :m][fin] - rl[b, :m][fin]) <= lt[fin]).all()
            assert (o[b, m:] == 9).all() and (ls[b, m:] == 9).all()


SHAPES = [
    # Bn, R, Hq, Hkv, D, P, seq
    (1, 1, 4, 1, 128, 64, [0]),
    (1, 1, 32, 8, 128, 777, [777]),
    (2, 1, 8, 8, 64, 130, [1, 129]),
    (5, 3, 8, 2, 128, 257, [63, 64, 65, 128, 257]),
    (2, 9, 28, 4, 128, 400, [127, 399]),       # seven query heads to a KV head
    (1, 8, 32, 8, 128, 2000, [1999]),          # a chain's rows: 32 of them
    (2, 61, 32, 8, 128, 900, [896, 517]),
    (1, 61, 8, 8, 128, 700, [700]),
    (1, 128, 16, 1, 128, 300, [290]),          # 2048 rows to a KV head, two mask words
    (2, 65, 6, 2, 64, 333, [0, 333]),
    (1, 100, 12, 4, 64, 1100, [1029]),
    (1, 33, 4, 1, 128, 520, [513]),            # one row block and a bit
    (1, 16, 2, 2, 128, 300, [260]),            # 16 rows to a KV head, and 17
    (1, 17, 2, 2, 128, 300, [260]),
    (2, 32, 3, 3, 128, 450, [450, 3]),         # 32 rows, as many tree keys
    (1, 1, 32, 1, 128, 3333, [3333]),          # 32 rows of one token
    (1, 2, 34, 2, 128, 200, [200]),            # 34 rows of two
    (1, 1, 4, 1, 128, 1, [1]),                 # a cache of one row, smaller than any tile
    (1, 61, 4, 1, 128, 70, [70]),
    (1, 61, 4, 1, 64, 3, [3]),
]


@pytest.mark.parametrize("precise,out_f32", [(False, False), (True, True), (False, True)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[:6])))
def test_matches_64_bits(shape, precise, out_f32):
    c = Case(1, *shape)
    c.check(c.desc(out_f32, precise))


@pytest.mark.parametrize("precise", [False, True])
@pytest.mark.parametrize("shape", [(2, 8, 8, 2, 128, 64, [0, 0]), (2, 61, 8, 2, 128, 64, [0, 0]),
                                   (1, 128, 4, 1, 128, 64, [0]), (2, 61, 8, 2, 64, 64, [0, 0])],
                         ids=lambda s: "-".join(map(str, s[:6])))
def test_tree_alone_is_precise(shape, precise):
    """No prefix: P with 22 bits or more whatever the precision asked for, and tree values (here
    over 2^-24 to 2^6, the smallest given up) as they are."""
    c = Case(7, *shape)
    g = np.random.default_rng(8)
    tv = c.tv.float() * torch.from_numpy(2.0 ** g.integers(-10, 5, c.tv.shape)).float()
    c.tv = torch.where(tv.abs() < 2.0 ** -24, 0.0, tv.clamp(-64, 64)).bfloat16()
    f = lambda t: t.double().numpy()
    none = np.zeros((*c.dims[:1], c.dims[3], c.dims[5], c.dims[4]))
    c.ref = H.attention(f(c.q), none, none, f(c.tk), f(c.tv), c.seq, c.nodes, c.see, 1 / math.sqrt(c.dims[4]))
    c.dev[6] = c.tv.cuda()
    c.check(c.desc(True, precise), p_round=2.0 ** -21)


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 64])
@pytest.mark.parametrize("shape", [(1, 5, 8, 2, 128, 1000, [1000]), (2, 61, 16, 4, 128, 1300, [1290, 70]),
                                   (1, 40, 8, 2, 64, 1000, [640])], ids=lambda s: "-".join(map(str, s[:6])))
def test_splits(shape, splits):
    c = Case(2, *shape)
    c.check(c.desc(True, True, splits))
    c.check(c.desc(False, False, splits, B.EAGLE_ENGINE_MMA_SYNC))


@pytest.mark.parametrize("shape,nodes", [((4, 61, 32, 8, 128, 700, [10, 700, 0, 333]), [61, 7, 1, 0]),
                                         ((3, 9, 8, 2, 128, 200, [10, 200, 128]), [0, 9, 4]),
                                         ((3, 70, 4, 4, 64, 200, [10, 200, 0]), [70, 64, 65])],
                         ids=["61", "9", "70"])
def test_trees_of_different_sizes(shape, nodes):
    c = Case(3, *shape, nodes=nodes)
    c.check(c.desc(False, False))
    c.check(c.desc(True, True, 2))


@pytest.mark.parametrize("R", [4, 61])
def test_rows_with_nothing_to_see(R):
    see = np.zeros((2, R, R), bool)
    see[:, 0, 0] = True
    see[:, R - 1, : R] = True
    c = Case(4, 2, R, 8, 2, 128, 300, [0, 200], see=see)
    c.check(c.desc(True, True))
    out, lse = c.run(c.desc(True, True))
    assert bool((out[0, 1:R - 1] == 0).all()) and bool((lse[0, 1:R - 1] == -math.inf).all())
    c.check(c.desc(False, False, 3))


@pytest.mark.parametrize("R", [2, 61])
@pytest.mark.parametrize("q_size", [1e-6, 30.0])
def test_flat_and_peaked_rows(q_size, R):
    c = Case(5, 1, R, 8, 2, 128, 800, [800], q_size=q_size)
    c.check(c.desc(True, True))
    c.check(c.desc(False, False))


@pytest.mark.parametrize("R", [3, 61])
def test_scales_of_any_kind(R):
    """Not powers of two, zero for some blocks, and block to block over 2^14."""
    def scales(g, shape):
        s = 0.004 * np.exp(g.normal(size=shape))
        s[g.random(shape) < 0.2] = 0.0
        s[g.random(shape) < 0.2] *= 2.0 ** -14
        return s
    c = Case(6, 2, R, 8, 2, 128, 1300, [1300, 640], scales=scales)
    c.check(c.desc(True, True))
    c.check(c.desc(False, False, 2))
    c = Case(7, 1, R, 8, 2, 128, 300, [300], scales=lambda g, s: np.zeros(s))
    c.check(c.desc(True, True))


@pytest.mark.parametrize("shape", [(1, 4, 32, 8, 128, 20000, [900]), (1, 61, 32, 8, 128, 20000, [1300]),
                                   (2, 40, 8, 2, 128, 20000, [127, 2100]), (1, 3, 4, 2, 64, 9000, [700])],
                         ids=lambda s: "-".join(map(str, s[:6])))
def test_capacity_far_above_the_lengths(shape):
    c = Case(13, *shape)
    c.check(c.desc(True, True))


@pytest.mark.parametrize("R", [1, 8, 61])
def test_growing_scores(R):
    """Keys whose scores rise from tile to tile move every row's reference, several times."""
    c = Case(14, 1, R, 8, 2, 128, 2000, [2000])
    kc, ks = c.codes[0], c.scale[0]
    for b in range(ks.shape[-1]):
        ks[..., b] = 2.0 ** (-9 + b // 3)
    vals = [H.values(x, s) for x, s in zip(c.codes, c.scale)]
    f = lambda t: t.double().numpy()
    c.ref = H.attention(f(c.q), vals[0], vals[1], f(c.tk), f(c.tv), c.seq, c.nodes, c.see, 1 / math.sqrt(128))
    c.dev[2] = torch.from_numpy(ks).cuda()
    c.check(c.desc(True, True))
    c.check(c.desc(False, False, 1))


@pytest.mark.parametrize("R", [4, 61])
def test_rows_that_are_not_finite_spoil_only_themselves(R):
    c = Case(15, 1, R, 8, 2, 128, 400, [390])
    good = c.run(c.desc(True, True))[0]
    q = c.dev[0].clone()
    q[0, 0, 1, 5] = math.inf
    q[0, R - 1, 6, 0] = math.nan
    c.dev[0] = q
    out, lse = c.run(c.desc(True, True))
    bad = torch.zeros(1, R, 8, dtype=torch.bool, device="cuda")
    bad[0, 0, 1] = bad[0, R - 1, 6] = True
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    assert torch.equal(out[~bad], good[~bad])


def test_repeats_are_identical_and_lse_is_optional():
    for shape in (SHAPES[5], SHAPES[6]):
        c = Case(8, *shape)
        d = c.desc(True, True)
        ws = torch.zeros(B.workspace_size(B.EAGLE_WS_TREE_ATTN_KVQ, d), dtype=torch.uint8, device="cuda")
        a, la = c.run(d, ws)
        for _ in range(3):
            b, _ = c.run(d, ws, lse=False)
            b2, l2 = c.run(d, ws)
            assert torch.equal(a, b) and torch.equal(a, b2) and torch.equal(la, l2)


def test_two_streams_and_a_captured_graph():
    """Two calls in flight on two streams (a workspace each), and both replayed from graphs."""
    cases = [Case(9, *SHAPES[6]), Case(10, *SHAPES[5])]
    want = [c.run(c.desc(True, True))[0] for c in cases]
    st = []
    for c in cases:
        d = c.desc(True, True)
        ws = torch.zeros(B.workspace_size(B.EAGLE_WS_TREE_ATTN_KVQ, d), dtype=torch.uint8, device="cuda")
        st.append((c, d, ws, torch.zeros_like(want[len(st)]), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def call(c, d, ws, out, s):
        q, kc, ks, vc, vs, tk, tv, seq, mask = c.dev
        B.eagle_tree_attn_kvq(d, q, kc, ks, vc, vs, tk, tv, seq, mask, out, None, ws, stream=s)

    for _ in range(20):
        for x in st:
            call(*x)
    torch.cuda.synchronize()
    for w, x in zip(want, st):
        assert torch.equal(w, x[3])
        x[3].zero_()
    graphs = []
    for x in st:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=x[4]):
            for _ in range(3):
                call(*x)
        graphs.append(g)
    for _ in range(5):
        for g, x in zip(graphs, st):
            with torch.cuda.stream(x[4]):
                g.replay()
    torch.cuda.synchronize()
    for w, x in zip(want, st):
        assert torch.equal(w, x[3])


def test_offsets_past_32_bits():
    """Only the last request of a cache of more than 2^32 bytes has a prefix."""
    Bn, Hkv, D, P, R, L = 34, 8, 128, 131072, 3, 1000
    g = np.random.default_rng(11)
    kc = torch.zeros(Bn, Hkv, P, D, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs = torch.zeros(Bn, Hkv, P // 64, device="cuda"), torch.zeros(Bn, Hkv, P // 64, device="cuda")
    small = Case(12, 1, R, 16, Hkv, D, 1024, [L])
    q0, kc0, ks0, vc0, vs0, tk0, tv0, _, mask0 = small.dev
    kc[-1, :, :1024], vc[-1, :, :1024] = kc0[0], vc0[0]
    ks[-1, :, :16], vs[-1, :, :16] = ks0[0], vs0[0]
    wide = lambda t: t.expand(Bn, *t.shape[1:]).contiguous()
    seq = np.zeros(Bn, int)
    seq[-1] = L
    d = B.AttnDesc(Bn, R, 16, Hkv, D, P, 1 / math.sqrt(D), B.EAGLE_BF16, 0, B.EAGLE_F32, B.EAGLE_ATTN_PRECISE)
    ws = torch.zeros(B.workspace_size(B.EAGLE_WS_TREE_ATTN_KVQ, d), dtype=torch.uint8, device="cuda")
    out = torch.zeros(Bn, R, 16, D, device="cuda")
    B.eagle_tree_attn_kvq(d, wide(q0), kc, ks, vc, vs, wide(tk0), wide(tv0), i32(seq), wide(mask0), out, None, ws)
    ref = small.ref[0][0]
    assert np.abs(out[-1].double().cpu().numpy() - ref).max() <= 1e-4 * np.abs(ref).max()
    none = H.attention(small.q.double().numpy(), np.zeros((1, Hkv, 1, D)), np.zeros((1, Hkv, 1, D)),
                       small.tk.double().numpy(), small.tv.double().numpy(), [0], [R], small.see, 1 / math.sqrt(D))[0]
    assert np.abs(out[0].double().cpu().numpy() - none[0]).max() <= 1e-4


def test_one_workspace_for_descriptors_in_turn():
    """Plans that merge in the kernel (counters) and plans that do not (partials where a plan's
    counters could be), over and over in the same workspace."""
    cases = [Case(31, 1, 61, 32, 8, 128, 900, [896]), Case(32, 6, 61, 16, 8, 128, 2000, [2000] * 6),
             Case(33, 1, 4, 8, 2, 128, 5000, [4999]), Case(34, 40, 2, 8, 8, 128, 600, [600] * 40),
             Case(35, 2, 9, 8, 2, 64, 700, [700, 64])]
    descs = [c.desc(False, False) for c in cases]
    want = [c.run(d)[0] for c, d in zip(cases, descs)]
    ws = torch.zeros(max(B.workspace_size(B.EAGLE_WS_TREE_ATTN_KVQ, d) for d in descs), dtype=torch.uint8, device="cuda")
    for i in [0, 1, 2, 3, 4, 0, 2, 1, 4, 0, 3, 2, 0]:
        assert torch.equal(cases[i].run(descs[i], ws=ws)[0], want[i])


def test_element_types_must_be_the_descriptor_s():
    c = Case(36, 1, 2, 2, 2, 64, 64, [10])
    d = c.desc(True)
    q, kc, ks, vc, vs, tk, tv, seq, mask = c.dev
    ws = torch.zeros(B.workspace_size(B.EAGLE_WS_TREE_ATTN_KVQ, d), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="out"):
        B.eagle_tree_attn_kvq(d, q, kc, ks, vc, vs, tk, tv, seq, mask, torch.empty_like(q), None, ws)
    w = B.KvqDesc(1, 2, 64, 64, 2, B.EAGLE_F32)
    with pytest.raises(ValueError, match="k has dtype"):
        B.eagle_kvq_write(w, tk, tv, seq, None, kc, ks, vc, vs)
    with pytest.raises(ValueError, match="k has dtype"):
        B.eagle_kvq_read(w, kc, ks, vc, vs, seq, None, tk, tv)
    with pytest.raises(ValueError, match="as many"):
        B.KvqLayerPointers([kc], [ks], [vc], [vs], [tk], [])
    lay = B.KvqLayerPointers([kc], [ks], [vc], [vs], [tk], [tv])
    one = i32([0])
    for layers, dt, msg in ((2, B.EAGLE_BF16, "2 layers"), (1, B.EAGLE_F32, "element type")):
        with pytest.raises(ValueError, match=msg):
            B.eagle_kvq_commit(B.CommitDesc(layers, 1, 2, 64, 2, 64, 0, dt, 0, dt), lay, one, one, seq, one)
    r = B.QkNormRopeDesc(1, 2, 2, 2, 64, 64, 0, 0, 1e-6, B.EAGLE_F32)
    with pytest.raises(ValueError, match="qkv has dtype"):
        B.eagle_qk_norm_rope(r, torch.zeros(2, 6 * 64, dtype=torch.bfloat16, device="cuda"), None, None,
                             torch.zeros(32, device="cuda"), i32([0, 0]), q, tk, tv)


@pytest.mark.parametrize("precise", [False, True])
@pytest.mark.parametrize("shape,nodes", [
    ((21, 61, 32, 8, 128, 1100, [0, 1, 127, 128, 129, 1100, 640, 3, 1000, 900, 0, 0, 77, 256, 1099, 512, 333, 64, 65, 800, 1]), None),
    ((20, 61, 32, 8, 128, 700, [700] * 20), [61, 1, 33, 32, 0, 16, 60, 5, 61, 61, 31, 40, 2, 61, 0, 0, 61, 33, 12, 50]),
    ((9, 100, 34, 17, 128, 400, [0, 0, 0, 400, 0, 0, 399, 0, 1]), [100, 0, 64, 65, 1, 0, 100, 3, 128 - 28]),
    ((3, 128, 64, 4, 128, 600, [600, 20, 0]), None),              # 2048 rows a group, eight row blocks
    ((160, 33, 8, 8, 128, 64, [i % 65 for i in range(160)]), None),  # one row tile a group, many short groups
    ((40, 40, 8, 2, 128, 2000, [2000] + [5] * 39), None),         # a long request among short ones
], ids=["lengths", "nodes", "empty", "blocks", "short", "one-long"])
def test_batches_of_many_groups(shape, nodes, precise):
    """More groups than fit on the SMs at once: pieces of every length, a combine launch."""
    c = Case(41, *shape, nodes=nodes)
    c.check(c.desc(precise, precise))


def test_batches_of_many_groups_repeat_exactly():
    c = Case(42, 24, 61, 16, 8, 128, 1500, list(range(100, 100 + 24 * 58, 58)), nodes=[61, 20, 33, 48] * 6)
    d = c.desc(False, False)
    ws = torch.zeros(B.workspace_size(B.EAGLE_WS_TREE_ATTN_KVQ, d), dtype=torch.uint8, device="cuda")
    first = c.run(d, ws=ws)[0]
    for _ in range(20):
        assert torch.equal(c.run(d, ws=ws)[0], first)
