"""GPU: the paged KV cache operators against 64-bit references (tolerances: paged_helpers)."""
import math

import numpy as np
import pytest
import torch

import paged_helpers as H
from eagle_speculative_decoding_tree_gb300 import binding as B

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"bf16": B.EAGLE_BF16, "f32": B.EAGLE_F32}


def rand(g, dt, *shape):
    return torch.randn(*shape, generator=g).to(dt).cuda()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def attn_case(seed, seq, R=1, Hq=8, Hkv=2, D=128, T=16, nodes=None, cap=0.0, window=0, slopes=False, dtype="bf16",
              out="bf16", precision=B.EAGLE_ATTN_PRECISE, engine=B.EAGLE_ENGINE_AUTO, tree=True, q_scale=1.0,
              extra_pages=1, poison=True):
    """Inputs of one call: rows behind seq_len, unused pages and rows of missing nodes hold NaN."""
    rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    dt, Bn = DT[dtype], len(seq)
    mp = max(1, -(-max(seq) // T)) + extra_pages
    table, _, n = H.tables(rng, Bn, mp)
    c = dict(seq=list(seq), nodes=nodes, cap=cap, window=window, T=T, Hkv=Hkv, D=D, R=R, table=table,
             scale=1 / math.sqrt(D))
    c["kp"], c["vp"] = (torch.full((n, Hkv, T, D), float("nan") if poison else 0.0).to(dt) for _ in range(2))
    for b, L in enumerate(seq):
        for j in range(-(-L // T)):
            m = min(T, L - j * T)
            for x in ("kp", "vp"):
                c[x][table[b, j], :, :m] = torch.randn(Hkv, m, D, generator=g).to(dt)
    c["kp"], c["vp"] = c["kp"].cuda(), c["vp"].cuda()
    c["q"] = rand(g, dt, Bn, R, Hq, D) * q_scale
    c["tk"], c["tv"] = (rand(g, dt, Bn, Hkv, R, D), rand(g, dt, Bn, Hkv, R, D)) if tree else (None, None)
    c["see"], c["mask"] = H.trees(rng, Bn, R)
    if nodes is not None and tree and poison:
        for b, m in enumerate(nodes):
            c["tk"][b, :, m:] = float("nan")
            c["tv"][b, :, m:] = float("nan")
    c["slopes"] = torch.exp2(-8 * torch.arange(1, Hq + 1) / Hq).cuda() if slopes else None
    c["desc"] = B.PagedAttnDesc(Bn, R, Hq, Hkv, D, T, n, mp, c["scale"], cap, window, CODE[dtype], CODE[out], precision,
                                engine)
    c["dtype"], c["outt"], c["precision"] = dtype, out, precision
    return c


def run_attn(c, ws=None, table=None, seq=None, st=None):
    Bn, R, Hq, D = c["q"].shape
    c["out"] = torch.full((Bn, R, Hq, D), 7.0, dtype=DT[c["outt"]], device="cuda")
    c["lse"] = torch.full((Bn, R, Hq), 7.0, device="cuda")
    st = status() if st is None else st
    ws = torch.zeros(B.workspace_size(B.EAGLE_WS_PAGED_ATTN, c["desc"]), dtype=torch.uint8, device="cuda") \
        if ws is None else ws
    tree = c["tk"] is not None
    B.eagle_paged_attn(c["desc"], c["q"], c["kp"], c["vp"], H.i32(c["table"] if table is None else table), c["tk"],
                       c["tv"], H.i32(c["seq"] if seq is None else seq), c["mask"] if tree else None, c["out"],
                       c["lse"], ws, n_nodes=None if c["nodes"] is None else H.i32(c["nodes"]), slopes=c["slopes"],
                       status=st)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32)) == 0
    return int(st), ws


def check_attn(c, only=None):
    q, kp, vp = H.f64(c["q"]), H.f64(c["kp"]), H.f64(c["vp"])
    out, lse = H.f64(c["out"]), H.f64(c["lse"])
    tk, tv = (H.f64(c["tk"]), H.f64(c["tv"])) if c["tk"] is not None else (None, None)
    sl = None if c["slopes"] is None else H.f64(c["slopes"])
    bf = c["outt"] == "bf16"
    adds, rel = H.fp32_kinds(c["R"] * c["q"].shape[2] // c["Hkv"])
    if c["dtype"] == "bf16":
        adds, rel = 144, 2.0 ** (-16 if c["precision"] == B.EAGLE_ATTN_PRECISE else -8)
    for b, L in enumerate(c["seq"]):
        n = c["R"] if c["nodes"] is None else c["nodes"][b]
        assert (out[b, n:] == 7.0).all() and (lse[b, n:] == 7.0).all()
        if n == 0 or (only is not None and b not in only):
            continue
        k, v = H.rows_of(kp, c["table"][b], L), H.rows_of(vp, c["table"][b], L)
        ref = H.attention(q[b], k, v, None if tk is None else tk[b], None if tv is None else tv[b], c["see"][b], L, n,
                          c["scale"], c["cap"], c["window"], sl, adds)
        mass = H.attention(q[b], k, np.abs(v), None if tk is None else tk[b], None if tv is None else np.abs(tv[b]),
                           c["see"][b], L, n, c["scale"], c["cap"], c["window"], sl)[0]
        H.check_attention(out[b, :n], lse[b, :n], ref, bf, rel * mass)


SHAPES = [
    dict(seq=[1]), dict(seq=[0]), dict(seq=[15, 16, 17]), dict(seq=[1000], Hq=32, Hkv=8),
    dict(seq=[700, 0, 1, 333, 128], T=64, Hq=4, Hkv=4), dict(seq=[129, 2000], T=128, Hq=28, Hkv=4),
    dict(seq=[511], Hq=16, Hkv=1, T=32), dict(seq=[300, 5], D=64, Hq=4, Hkv=4), dict(seq=[640, 77], D=64, T=32),
    dict(seq=[513, 100], R=8, T=64, Hq=32, Hkv=8), dict(seq=[90, 400], R=61, T=64), dict(seq=[37], R=128, Hq=4, Hkv=1),
    dict(seq=[250, 66, 0], R=9, nodes=[9, 4, 0]), dict(seq=[0, 19], R=65, nodes=[64, 65], Hq=2, Hkv=1),
    dict(seq=[100, 31], R=5, Hq=6, Hkv=2), dict(seq=[333], R=33, Hq=28, Hkv=4, T=32),
    dict(seq=[40] * 37, Hq=4, Hkv=2), dict(seq=[260, 3], R=17, D=64, Hq=8, Hkv=2, T=128, nodes=[17, 2]),
    dict(seq=[600, 1], R=3, Hq=64, Hkv=1, T=64), dict(seq=[4097], Hq=2, Hkv=1), dict(seq=[70, 20], R=2, Hq=130, Hkv=1),
    dict(seq=[300, 77], R=2, Hq=100, Hkv=1, T=64), dict(seq=[222], R=2, Hq=256, Hkv=2),
    dict(seq=[(37 * i) % 500 for i in range(41)], R=20, Hq=8, Hkv=2, T=64, nodes=[(7 * i) % 21 for i in range(41)]),
    dict(seq=[(53 * i) % 300 for i in range(70)], R=3, Hq=8, Hkv=2, D=64, nodes=[i % 4 for i in range(70)]),
    dict(seq=[900, 31, 1500], R=17, Hq=28, Hkv=4, D=64), dict(seq=[6000], Hq=16, Hkv=1, T=64), dict(seq=[9001, 0], R=2, Hq=16, Hkv=1), dict(seq=[7000], D=64, Hq=9, Hkv=1, R=3),
]
SCORES = [dict(), dict(cap=30.0), dict(cap=200.0), dict(window=50), dict(slopes=True), dict(cap=5.0, window=333, slopes=True),
          dict(window=1), dict(window=16, slopes=True)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_attention_shapes(i, dtype):
    kw = SHAPES[i]
    c = attn_case(100 + i, dtype=dtype, out=dtype if i % 3 else "f32", **kw)
    assert run_attn(c)[0] == 0
    check_attn(c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [1, 7, 61])
@pytest.mark.parametrize("j", range(len(SCORES)))
def test_attention_scores(j, R, dtype):
    c = attn_case(200 + j, [0, 47, 48, 777], R=R, Hq=8, Hkv=2, T=32, dtype=dtype, out="f32", q_scale=3.0, **SCORES[j])
    assert run_attn(c)[0] == 0
    check_attn(c)


@pytest.mark.parametrize("R,kw", [(1, {}), (5, dict(cap=20.0)), (3, dict(window=20, slopes=True)), (61, dict(window=100))])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_without_a_tree(R, kw, dtype):
    """The new tokens' K/V lies in the pages already; a request without a key gets zeros."""
    c = attn_case(300 + R, [0, 1, 200], R=R, tree=False, dtype=dtype, out="f32", **kw)
    assert run_attn(c)[0] == 0
    check_attn(c)
    assert (c["out"][0] == 0).all() and torch.isneginf(c["lse"][0]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_rows_without_a_key(dtype):
    c = attn_case(400, [0, 30, 0], R=6, dtype=dtype, out="f32", window=10)
    c["see"][0, 2] = False  # an empty row, a row that sees others but not itself
    c["see"][2, 4] = [True, True, False, False, False, False]
    c["mask"] = H.words(c["see"])
    assert run_attn(c)[0] == 0
    check_attn(c)
    assert (c["out"][0, 2] == 0).all() and torch.isneginf(c["lse"][0, 2]).all()


@pytest.mark.parametrize("R", [1, 61])
def test_attention_fast_precision(R):
    c = attn_case(410, [500, 64], R=R, precision=B.EAGLE_ATTN_FAST, out="f32")
    assert run_attn(c)[0] == 0
    check_attn(c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [1, 61])
def test_attention_pages_before_the_window_are_not_read(dtype, R):
    """Table entries of pages that no row sees may be anything."""
    c = attn_case(420, [300], R=R, window=100, dtype=dtype, out="f32")
    table = c["table"].copy()
    table[0, : (300 - 100) // 16] = -5
    table[0, 19:] = 1 << 30
    assert run_attn(c, table=table)[0] == 0
    check_attn(c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [1, 61])
def test_attention_flags_bad_pages(dtype, R):
    """A page outside the pool: flagged, page 0 is read in its place, the other requests are right."""
    c = attn_case(430, [100, 90, 120], R=R, dtype=dtype, out="f32", poison=False)
    for bad in (-1, c["kp"].shape[0], 2 ** 31 - 1):
        table = c["table"].copy()
        table[1, 2] = bad
        assert run_attn(c, table=table)[0] == B.EAGLE_STATUS_BAD_PAGE
        check_attn(c, only=(0, 2))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [1, 61])
def test_attention_without_rows(R, dtype):
    """Requests without nodes: nothing is written."""
    c = attn_case(435, [100, 0, 50], R=R, nodes=[0, 0, 0], dtype=dtype, out="f32")
    assert run_attn(c)[0] == 0
    assert (c["out"] == 7).all() and (c["lse"] == 7).all()


@pytest.mark.parametrize("R", [1, 61])
def test_attention_optional_arguments(R):
    """No lse, no status: the same output."""
    c = attn_case(436, [333, 20], R=R)
    ws = run_attn(c)[1]
    want = c["out"].clone()
    B.eagle_paged_attn(c["desc"], c["q"], c["kp"], c["vp"], H.i32(c["table"]), c["tk"], c["tv"], H.i32(c["seq"]),
                       c["mask"], c["out"].zero_(), None, ws)
    assert torch.equal(c["out"], want)


@pytest.mark.parametrize("R,Hkv", [(1, 8), (61, 8), (1, 1)])
def test_attention_on_two_streams(R, Hkv):
    """Calls on two streams with workspaces of their own, back to back: the same bits as alone."""
    cases = [attn_case(437 + i, [2000, 700], R=R, Hq=32, Hkv=Hkv, T=64) for i in range(2)]
    want, args = [], []
    for c in cases:
        ws = run_attn(c)[1]
        want.append(c["out"].clone())
        args.append((H.i32(c["table"]), H.i32(c["seq"]), ws))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for c, (table, seq, ws), st in zip(cases, args, streams):
            B.eagle_paged_attn(c["desc"], c["q"], c["kp"], c["vp"], table, c["tk"], c["tv"], seq, c["mask"], c["out"],
                               c["lse"], ws, st)
    torch.cuda.synchronize()
    for c, w, a in zip(cases, want, args):
        assert torch.equal(c["out"], w) and int(a[2][:4].view(torch.int32)) == 0


def test_attention_clamps_lengths():
    """seq_len past the table's rows counts as all of them, below 0 as none."""
    c = attn_case(440, [64, 0], extra_pages=0)
    run_attn(c, seq=[1000, -3])
    check_attn(c)


def test_attention_one_workspace_many_descriptors_and_graphs():
    """Descriptors in turn over one workspace, then each captured and replayed twice: the same bits."""
    cases = [attn_case(450 + i, **SHAPES[i]) for i in (3, 4, 9, 10, 16)]
    size = max(B.workspace_size(B.EAGLE_WS_PAGED_ATTN, c["desc"]) for c in cases)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    first = []
    for c in cases:
        assert run_attn(c, ws)[0] == 0
        check_attn(c)
        first.append((c["out"].clone(), c["lse"].clone()))
    side = torch.cuda.Stream()
    for c, (o, z) in zip(cases, first):
        seq, table = H.i32(c["seq"]), H.i32(c["table"])
        nodes = None if c["nodes"] is None else H.i32(c["nodes"])
        call = lambda: B.eagle_paged_attn(c["desc"], c["q"], c["kp"], c["vp"], table, c["tk"], c["tv"], seq, c["mask"],
                                          c["out"], c["lse"], ws, n_nodes=nodes, slopes=c["slopes"])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                call()
                call()
            c["out"].fill_(3)
            graph.replay()
            graph.replay()
        side.synchronize()
        assert torch.equal(c["out"], o) and torch.equal(c["lse"], z)


# ------------------------------------------------------------------------------- writers
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Bn,Hkv,D,T,N,spans", [
    (1, 8, 128, 64, 300, [(0, 300)]), (3, 2, 64, 16, 40, [(5, 40), (0, 0), (16, 33)]), (2, 3, 128, 32, 1, [(31, 1), (32, 1)]),
    (4, 1, 64, 128, 257, [(0, 257), (127, 2), (1, 128), (300, 84)])])
def test_write(Bn, Hkv, D, T, N, spans, dtype):
    rng, g = np.random.default_rng(N), torch.Generator().manual_seed(N)
    mp = -(-384 // T)
    table, _, n = H.tables(rng, Bn, mp)
    k, v = (rand(g, DT[dtype], Bn, Hkv, N, D) for _ in range(2))
    kp, vp = (rand(g, DT[dtype], n, Hkv, T, D) for _ in range(2))
    want = [H.f64(kp), H.f64(vp)]
    for b, (s, m) in enumerate(spans):
        for w, x in zip(want, (k, v)):
            H.put_rows(w, table[b], s, H.f64(x)[b, :, :m])
    d = B.PagedDesc(Bn, Hkv, D, T, n, mp, N, CODE[dtype])
    st = status()
    B.eagle_paged_write(d, k, v, H.i32(table), H.i32([s for s, _ in spans]), H.i32([m for _, m in spans]), kp, vp, st)
    assert int(st) == 0 and np.array_equal(H.f64(kp), want[0]) and np.array_equal(H.f64(vp), want[1])


def test_write_leaves_what_does_not_fit():
    """Spans past the table, negative ones, counts past N: untouched and flagged; count NULL; a bad page."""
    rng, g = np.random.default_rng(0), torch.Generator().manual_seed(0)
    table, _, n = H.tables(rng, 5, 2)
    k, v = (rand(g, torch.bfloat16, 5, 2, 8, 64) for _ in range(2))
    kp, vp = (rand(g, torch.bfloat16, n, 2, 16, 64) for _ in range(2))
    d = B.PagedDesc(5, 2, 64, 16, n, 2, 8, B.EAGLE_BF16)
    want = H.f64(kp)
    H.put_rows(want, table[1], 24, H.f64(k)[1])
    st = status()
    B.eagle_paged_write(d, k, v, H.i32(table), H.i32([25, 24, -1, 0, 2 ** 31 - 1]), H.i32([8, 8, 3, 9, 8]), kp, vp, st)
    assert int(st) == B.EAGLE_STATUS_CACHE_FULL and np.array_equal(H.f64(kp), want)
    st.zero_()
    for b in range(5):
        H.put_rows(want, table[b], 16, H.f64(k)[b])
    B.eagle_paged_write(d, k, v, H.i32(table), H.i32([16] * 5), None, kp, vp, st)
    assert int(st) == 0 and np.array_equal(H.f64(kp), want)
    bad = table.copy()
    bad[2, 1], bad[3, 0] = n, -1
    B.eagle_paged_write(d, k, v, H.i32(bad), H.i32([12] * 5), None, kp, vp, st)
    for b in range(5):
        for i in range(8):
            if 0 <= bad[b, (12 + i) // 16] < n:
                H.put_rows(want, bad[b], 12 + i, H.f64(k)[b, :, i: i + 1])
    assert int(st) == B.EAGLE_STATUS_BAD_PAGE and np.array_equal(H.f64(kp), want)


@pytest.mark.parametrize("dtype,feat", [("bf16", 40), ("f32", 0), ("bf16", 33)])
def test_commit(dtype, feat):
    L, Bn, Hkv, D, T, R, maxd = 3, 5, 3, 64, 16, 20, 6
    rng, g = np.random.default_rng(feat), torch.Generator().manual_seed(feat)
    mp = 4
    table, _, n = H.tables(rng, Bn, mp)
    kp, vp = ([rand(g, DT[dtype], n, Hkv, T, D) for _ in range(L)] for _ in range(2))
    tk, tv = ([rand(g, DT[dtype], Bn, Hkv, R, D) for _ in range(L)] for _ in range(2))
    fp, tf = rand(g, torch.bfloat16, n, T, max(1, feat)), rand(g, torch.bfloat16, Bn, R, max(1, feat))
    seq, n_acc = np.array([0, 15, 60, 30, 58]), np.array([6, 2, 4, 0, 5])  # the third does not fit
    path = np.full((Bn, maxd + 1), -1)
    for b in range(Bn):
        path[b, : n_acc[b] + 1] = np.sort(rng.permutation(R)[: n_acc[b] + 1])
    d = B.PagedCommitDesc(L, Bn, Hkv, D, T, n, mp, R, maxd, CODE[dtype], feat, B.EAGLE_BF16)
    want = [[H.f64(x) for x in xs] for xs in (kp, vp)]
    wf, pos = H.f64(fp), np.full((Bn, maxd + 1), -1)
    for step in range(2):  # the second behind the first
        fits = seq + n_acc + 1 <= mp * T
        pos[:] = -1
        for b in np.nonzero(fits)[0]:
            nodes = path[b, : n_acc[b] + 1]
            for w, t in zip(want, (tk, tv)):
                for l in range(L):
                    H.put_rows(w[l], table[b], int(seq[b]), H.f64(t[l])[b][:, nodes])
            H.put_rows(wf[:, None], table[b], int(seq[b]), H.f64(tf)[b, nodes][None])
            pos[b, : len(nodes)] = seq[b] + np.arange(len(nodes))
        if step == 0:
            dev_seq, ws, cp, st = H.i32(seq), torch.zeros(64, dtype=torch.uint8, device="cuda"), H.i32(pos * 0), status()
        B.eagle_paged_commit(d, B.LayerPointers(kp, vp, tk, tv), H.i32(table), H.i32(n_acc), H.i32(path), dev_seq, cp, ws,
                             fp if feat else None, tf if feat else None, st)
        seq = np.where(fits, seq + n_acc + 1, seq)
        assert int(st) == B.EAGLE_STATUS_CACHE_FULL and not ws.any()
        assert np.array_equal(dev_seq.cpu().numpy(), seq) and np.array_equal(cp.cpu().numpy(), pos)
        for got, w in zip((kp, vp), want):
            for l in range(L):
                assert np.array_equal(H.f64(got[l]), w[l])
        if feat:
            assert np.array_equal(H.f64(fp), wf)


def test_commit_flags_bad_paths_and_pages():
    rng, g = np.random.default_rng(1), torch.Generator().manual_seed(1)
    table, _, n = H.tables(rng, 3, 2)
    kp, vp = ([rand(g, torch.bfloat16, n, 1, 16, 64)] for _ in range(2))
    tk, tv = ([rand(g, torch.bfloat16, 3, 1, 4, 64)] for _ in range(2))
    d = B.PagedCommitDesc(1, 3, 1, 64, 16, n, 2, 4, 2, B.EAGLE_BF16, 0, B.EAGLE_BF16)
    want = H.f64(kp[0])
    path = np.array([[0, 4, 2], [0, 1, 2], [0, 3, -1]])
    bad = table.copy()
    bad[1, 1] = -7
    seq = H.i32([3, 14, -1])
    for b, rows in ((0, (0, 2)), (1, (0, 1))):
        for m in rows:
            H.put_rows(want, table[b], [3, 14][b] + m, H.f64(tk[0])[b][:, path[b, m]][:, None])
    st, ws = status(), torch.zeros(16, dtype=torch.uint8, device="cuda")
    B.eagle_paged_commit(d, B.LayerPointers(kp, vp, tk, tv), H.i32(bad), H.i32([2, 2, 1]), H.i32(path), seq, None, ws,
                         status=st)
    assert int(st) == B.EAGLE_STATUS_BAD_TREE | B.EAGLE_STATUS_BAD_PAGE | B.EAGLE_STATUS_CACHE_FULL
    assert np.array_equal(H.f64(kp[0]), want) and seq.tolist() == [6, 17, -1]


# ------------------------------------------------------------------------------- weights
def weights_case(seed, seq, n_acc, R, Hq, Hkv, D, T, dtype, cap=0.0, window=0, slopes=False, maxd=None, q_scale=1.0):
    c = attn_case(seed, seq, R, Hq, Hkv, D, T, dtype=dtype, cap=cap, window=window, slopes=slopes, q_scale=q_scale)
    rng = np.random.default_rng(seed)
    Bn, maxd = len(seq), max(n_acc) if maxd is None else maxd
    path = np.full((Bn, maxd + 1), -1)
    for b in range(Bn):
        path[b, : n_acc[b] + 1] = np.sort(rng.permutation(R)[: n_acc[b] + 1])
    n = c["kp"].shape[0]
    c["lse"] = torch.from_numpy(rng.normal(6, 1, (Bn, R, Hq)).astype(np.float32)).cuda()
    c["prior"] = torch.from_numpy(rng.exponential(1, (n, Hkv, T)).astype(np.float32)).cuda()
    c["wdesc"] = B.PagedWeightsDesc(Bn, R, Hq, Hkv, D, T, n, c["table"].shape[1], maxd, c["scale"], cap, window, CODE[dtype])
    c["n_acc"], c["path"] = np.array(n_acc), path
    return c


def run_weights(c, prior, out, path=True, st=None):
    st = status() if st is None else st
    B.eagle_paged_weights(c["wdesc"], c["q"], c["lse"], c["kp"], H.i32(c["table"]), H.i32(c["seq"]),
                          H.i32(c["n_acc"]) if path else None, H.i32(c["path"]) if path else None, prior, out,
                          slopes=c["slopes"], status=st)
    torch.cuda.synchronize()
    return int(st)


def check_weights(c, prior, before, got, only=None):
    q, kp, z = H.f64(c["q"]), H.f64(c["kp"]), H.f64(c["lse"])
    sl = None if c["slopes"] is None else H.f64(c["slopes"])
    want, tol = before.copy(), np.zeros_like(before)
    for b, L in enumerate(c["seq"]):
        if only is not None and b not in only:
            continue
        nodes = c["path"][b, : c["n_acc"][b] + 1]
        n = len(nodes)
        w, e = H.weights(q[b, nodes], z[b, nodes], H.rows_of(kp, c["table"][b], L), L, c["scale"], c["cap"], c["window"],
                         sl, 9 if c["dtype"] == "f32" else 144)
        if prior is not None:
            w[:, : L - n] += H.rows_of(prior, c["table"][b], L)[:, : L - n]
        H.put_rows(want, c["table"][b], 0, w)
        H.put_rows(tol, c["table"][b], 0, e + 2 * H.U32 * np.abs(w))
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) - tol).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seq,n_acc,R,Hq,Hkv,D,T,kw", [
    ([1], [0], 1, 4, 1, 128, 16, {}), ([1000, 77], [0, 0], 1, 32, 8, 128, 64, {}),
    ([300, 9, 64], [7, 8, 0], 61, 8, 2, 128, 16, {}), ([129, 2000], [3, 5], 20, 4, 4, 64, 32, dict(cap=20.0)),
    ([200, 333], [1, 6], 9, 28, 4, 128, 128, dict(window=40)), ([500], [8], 30, 16, 1, 64, 64, dict(slopes=True)),
    ([260, 70], [4, 11], 12, 6, 2, 128, 32, dict(cap=4.0, window=100, slopes=True, q_scale=3.0)),
    ([150], [127], 128, 4, 1, 128, 16, {}), ([90] * 33, [2] * 33, 5, 2, 1, 64, 16, {})])
def test_weights(seq, n_acc, R, Hq, Hkv, D, T, kw, dtype):
    c = weights_case(sum(seq), seq, n_acc, R, Hq, Hkv, D, T, dtype, **kw)
    before = torch.full_like(c["prior"], -5.0)
    out = before.clone()
    assert run_weights(c, c["prior"], out) == 0
    check_weights(c, H.f64(c["prior"]), H.f64(before), H.f64(out))
    again = c["prior"].clone()  # in place, and without a prior
    assert run_weights(c, again, again) == 0
    check_weights(c, H.f64(c["prior"]), H.f64(c["prior"]), H.f64(again))
    assert run_weights(c, None, out) == 0
    check_weights(c, None, H.f64(before), H.f64(out))


def test_weights_rows_in_order_and_rows_without_keys():
    c = weights_case(5, [100, 40], [6, 6], 7, 8, 2, 128, 16, "bf16")
    c["lse"][1, 3] = -math.inf  # such a row gave nothing
    c["path"][:] = np.arange(7)
    out = torch.zeros_like(c["prior"])
    assert run_weights(c, None, out, path=False) == 0
    check_weights(c, None, 0 * H.f64(out), H.f64(out))


def test_weights_of_the_attention_sum_to_the_rows():
    """Attention, commit, weights: every accepted row's weights add up to one a query head."""
    Bn, R, Hq, Hkv, D, T, maxd = 2, 12, 8, 2, 128, 16, 4
    c = attn_case(6, [200, 35], R, Hq, Hkv, D, T, extra_pages=2, cap=10.0, slopes=True)
    run_attn(c)
    n_acc, path = np.array([4, 2]), np.full((2, maxd + 1), -1)
    for b in range(2):  # a root-to-leaf path
        i = max(range(R), key=lambda r: min(c["see"][b, r].sum(), n_acc[b] + 1))
        nodes = np.nonzero(c["see"][b, i])[0][: n_acc[b] + 1]
        n_acc[b] = len(nodes) - 1
        path[b, : len(nodes)] = nodes
    n, mp = c["kp"].shape[0], c["table"].shape[1]
    seq, table = H.i32(c["seq"]), H.i32(c["table"])
    d = B.PagedCommitDesc(1, Bn, Hkv, D, T, n, mp, R, maxd, B.EAGLE_BF16, 0, B.EAGLE_BF16)
    B.eagle_paged_commit(d, B.LayerPointers([c["kp"]], [c["vp"]], [c["tk"]], [c["tv"]]), table, H.i32(n_acc), H.i32(path),
                         seq, None, torch.zeros(16, dtype=torch.uint8, device="cuda"))
    wd = B.PagedWeightsDesc(Bn, R, Hq, Hkv, D, T, n, mp, maxd, c["scale"], 10.0, 0, B.EAGLE_BF16)
    w = torch.zeros(n, Hkv, T, device="cuda")
    B.eagle_paged_weights(wd, c["q"], c["lse"], c["kp"], table, seq, H.i32(n_acc), H.i32(path), None, w, slopes=c["slopes"])
    for b in range(Bn):
        got = H.rows_of(H.f64(w), c["table"][b], int(seq[b])).sum(1)
        assert np.allclose(got, (n_acc[b] + 1) * Hq / Hkv, rtol=1e-4)


def test_weights_flags():
    c = weights_case(8, [50, 60, 3, 40], [2, 2, 3, 1], 6, 4, 2, 64, 16, "bf16", maxd=3)
    c["path"][0, 1] = 6        # no such row
    c["n_acc"][1] = 4          # past max_depth
    before = torch.full_like(c["prior"], -5.0)
    out = before.clone()
    assert run_weights(c, c["prior"], out) == B.EAGLE_STATUS_BAD_TREE | B.EAGLE_STATUS_CACHE_FULL
    check_weights(c, H.f64(c["prior"]), H.f64(before), H.f64(out), only=(3,))


# ------------------------------------------------------------------------------- eviction
def evict_case(seed, L, seq, Hkv, D, T, limit, budget, sink, recent, dtype="bf16", room=20):
    rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    Bn, mp, sp = len(seq), -(-(max(seq) + room) // T), -(-budget // T)
    table, spare, n = H.tables(rng, Bn, mp, sp)
    c = dict(seq=np.array(seq), table=table, spare=spare, args=(budget, sink, recent), limit=limit)
    c["kp"], c["vp"] = ([rand(g, DT[dtype], n, Hkv, T, D) for _ in range(L)] for _ in range(2))
    c["w"] = [torch.exp(2 * torch.randn(n, Hkv, T, generator=g)).cuda() for _ in range(L)]
    c["desc"] = B.PagedEvictDesc(L, Bn, Hkv, D, T, n, mp, limit, budget, sink, recent, CODE[dtype])
    c["kept0"] = np.full((L, Bn, Hkv, budget), -9)
    return c


def evict_reference(c):
    """What the call leaves: pages, weights, kept, table, spare, seq (numpy)."""
    k, v, w = ([H.f64(x) for x in c[n]] for n in ("kp", "vp", "w"))
    wf = [x.cpu().numpy() for x in c["w"]]
    kept, table, spare, seq = c["kept0"].copy(), c["table"].copy(), c["spare"].copy(), c["seq"].copy()
    budget = c["args"][0]
    for b, n in enumerate(c["seq"]):
        if n <= c["limit"]:
            continue
        for l in range(len(k)):
            rows = [H.rows_of(x[l], c["table"][b], n) for x in (k, v, w)]
            ranks = H.rows_of(wf[l], c["table"][b], n)
            for h in range(ranks.shape[0]):
                r = H.kept_rows(ranks[h], n, *c["args"])
                kept[l, b, h] = r
                for x, old in zip((k, v, w), rows):
                    H.put_rows(x[l][:, h: h + 1], c["spare"][b], 0, old[h: h + 1, r])
        m = spare.shape[1]
        table[b, :m], spare[b] = c["spare"][b], c["table"][b, :m]
        seq[b] = budget
    return k, v, w, kept, table, spare, seq


def run_evict(c, ws=None):
    c["dev"] = [H.i32(c[x]) for x in ("table", "spare", "seq", "kept0")]
    ws = torch.zeros(B.workspace_size(B.EAGLE_WS_PAGED_EVICT, c["desc"]), dtype=torch.uint8, device="cuda") if ws is None else ws
    st = status()
    B.eagle_paged_evict(c["desc"], B.PagedLayerPointers(c["kp"], c["vp"], c["w"]), *c["dev"], ws, st)
    torch.cuda.synchronize()
    assert not ws.any()
    return int(st)


def check_evict(c, ref):
    k, v, w, kept, table, spare, seq = ref
    for got, want in zip(c["dev"], (table, spare, seq, kept)):
        assert np.array_equal(got.cpu().numpy(), want)
    for got, want in ((c["kp"], k), (c["vp"], v), (c["w"], w)):
        for x, y in zip(got, want):
            assert np.array_equal(H.f64(x), y, equal_nan=True)


@pytest.mark.parametrize("kw", [
    dict(L=2, seq=[500], Hkv=2, D=128, T=16, limit=300, budget=200, sink=4, recent=32),
    dict(L=3, seq=[100, 101, 700, 40], Hkv=3, D=64, T=64, limit=100, budget=100, sink=0, recent=0),
    dict(L=1, seq=[2000], Hkv=1, D=64, T=128, limit=1, budget=1, sink=0, recent=0),
    dict(L=1, seq=[300, 90], Hkv=4, D=128, T=32, limit=80, budget=33, sink=3, recent=30),
    dict(L=2, seq=[1000], Hkv=2, D=64, T=16, limit=999, budget=999, sink=1, recent=7, dtype="f32"),
    dict(L=1, seq=[40000], Hkv=2, D=64, T=64, limit=30000, budget=25001, sink=4, recent=256),
    dict(L=1, seq=[77], Hkv=1, D=128, T=16, limit=64, budget=64, sink=64, recent=0),
    dict(L=128, seq=[50, 9], Hkv=1, D=64, T=16, limit=20, budget=8, sink=2, recent=2)])
def test_evict(kw):
    c = evict_case(11, **kw)
    ref = evict_reference(c)
    assert run_evict(c) == 0
    check_evict(c, ref)


@pytest.mark.parametrize("kind", ["equal", "few", "zeros", "nan", "negative", "inf"])
@pytest.mark.parametrize("n", [700, 30000])
def test_evict_ties_and_odd_weights(kind, n):
    c = evict_case(12, 1, [n], 2, 64, 64, 600, 600, 4, 16)
    g = torch.Generator().manual_seed(3)
    w = c["w"][0]
    if kind == "equal":
        w.fill_(0.25)
    elif kind == "few":
        w.copy_(torch.randint(0, 3, w.shape, generator=g).float())
    elif kind == "zeros":
        w.copy_(torch.where(torch.rand(w.shape, generator=g) < 0.5, 0.0, -0.0))
    elif kind == "nan":
        w[torch.rand(w.shape, generator=g).cuda() < 0.6] = float("nan")
    elif kind == "negative":
        w.neg_()
    else:
        w[torch.rand(w.shape, generator=g).cuda() < 0.3] = float("inf")
        w[torch.rand(w.shape, generator=g).cuda() < 0.3] = -float("inf")
    ref = evict_reference(c)
    assert run_evict(c) == 0
    check_evict(c, ref)


def test_evict_twice_and_a_shared_prefix():
    """The pages given up are the next spare ones; a page that another request reads keeps its rows."""
    c = evict_case(13, 2, [200, 150], 2, 64, 16, 100, 64, 4, 8)
    c["table"][1, :3] = c["table"][0, :3]  # a common prefix
    ws = None
    for step in range(3):
        ref = evict_reference(c)
        ws = torch.zeros(B.workspace_size(B.EAGLE_WS_PAGED_EVICT, c["desc"]), dtype=torch.uint8, device="cuda") if ws is None else ws
        if step == 0:
            c["seq"][1] = 90  # not over: its shared pages must stay
            ref = evict_reference(c)
        assert run_evict(c, ws) == 0
        check_evict(c, ref)
        c["table"], c["spare"], c["seq"] = (t.cpu().numpy().astype(np.int64) for t in c["dev"][:3])
        c["seq"] = c["seq"] + np.array([45, 0])  # rows written since


def test_evict_flags():
    """Lengths past the table and spare pages outside the pool: left as they are."""
    c = evict_case(14, 1, [100, 100, 100], 2, 64, 16, 50, 40, 2, 4)
    good = evict_reference(c)
    c["seq"][0] = 1000
    c["spare"][1, 1] = -2
    before = [H.f64(x[0]) for x in (c["kp"], c["vp"], c["w"])]
    table, spare, seq, kept = c["table"].copy(), c["spare"].copy(), c["seq"].copy(), c["kept0"].copy()
    assert run_evict(c) == B.EAGLE_STATUS_CACHE_FULL | B.EAGLE_STATUS_BAD_PAGE
    got = [x.cpu().numpy() for x in c["dev"]]
    for x, y, want in zip(got[:2], (table, spare), good[4:6]):
        assert np.array_equal(x[:2], y[:2]) and np.array_equal(x[2], want[2])
    assert got[2].tolist() == [1000, 100, 40] and (got[3][:, :2] == -9).all()
    assert np.array_equal(got[3][:, 2], good[3][:, 2])
    pages = spare[2]
    for x, y, want in zip((c["kp"], c["vp"], c["w"]), before, good[:3]):
        new = H.f64(x[0])
        assert np.array_equal(new[pages], want[0][pages])
        rest = np.setdiff1d(np.arange(len(new)), pages)
        assert np.array_equal(new[rest], y[rest])


@pytest.mark.parametrize("R,G,Hkv,extra", [(8, 4, 8, 1), (8, 4, 8, 5000), (5, 4, 4, 1), (2, 16, 1, 1), (3, 7, 4, 5000)])
def test_attention_of_chains_in_every_kernel(R, G, Hkv, extra):
    """17 to 32 rows a KV head: short tables, long ones and the MMA_SYNC engine take different kernels."""
    for engine in (B.EAGLE_ENGINE_AUTO, B.EAGLE_ENGINE_MMA_SYNC):
        c = attn_case(500 + R, [1300, 2, 400], R=R, Hq=G * Hkv, Hkv=Hkv, T=16, engine=engine, extra_pages=extra, out="f32")
        c["see"] = np.broadcast_to(np.tril(np.ones((R, R), bool)), c["see"].shape).copy()
        c["mask"] = H.words(c["see"])
        assert run_attn(c)[0] == 0
        check_attn(c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,Hq,Hkv", [(8, 32, 8), (1, 16, 2), (4, 16, 4)])
def test_attention_joins_of_many_partials(R, Hq, Hkv, dtype):
    """One request over all CTAs, behind a table too long for the tree kernel: its CTAs share the join."""
    c = attn_case(600 + R, [5003], R=R, Hq=Hq, Hkv=Hkv, T=16, extra_pages=4500, dtype=dtype, out="f32", cap=40.0)
    first = None
    for _ in range(2):
        assert run_attn(c)[0] == 0
        first = c["out"].clone() if first is None else first
        assert torch.equal(c["out"], first)
    check_attn(c)
