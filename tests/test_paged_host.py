"""The paged KV cache entry points without a GPU: bad descriptors, pointers and workspaces are refused on the host,
with the documented codes."""
import ctypes

import pytest

from eagle_speculative_decoding_tree_gb300 import binding as B
from eagle_speculative_decoding_tree_gb300 import build as build_mod

A = 0x100000  # an aligned fake device address: every call below fails validation before it matters
INV, UNS, ALI, WS = B.EAGLE_ERR_INVALID_ARG, B.EAGLE_ERR_UNSUPPORTED, B.EAGLE_ERR_ALIGNMENT, B.EAGLE_ERR_WORKSPACE
TOP = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


GEOM = dict(batch=2, n_kv_heads=2, head_dim=64, page_size=16, n_pages=40, max_pages=8, dtype=1)
SCORE = dict(n_q_heads=4, rows=4, scale=0.1, softcap=0.0, window=0)
BAD_GEOM = [(dict(batch=0), INV), (dict(n_kv_heads=0), INV), (dict(n_pages=0), INV), (dict(max_pages=-1), INV),
            (dict(page_size=0), INV), (dict(head_dim=0), INV), (dict(head_dim=96), UNS), (dict(page_size=48), UNS),
            (dict(page_size=256), UNS), (dict(batch=65536), UNS), (dict(n_kv_heads=1025, n_q_heads=1025), UNS),
            (dict(max_pages=TOP), UNS), (dict(n_pages=TOP), UNS), (dict(dtype=2), UNS)]
BAD_SCORE = [(dict(rows=0), INV), (dict(rows=129), UNS), (dict(n_q_heads=5), UNS), (dict(n_q_heads=0), INV),
             (dict(scale=0.0), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
             (dict(softcap=-1.0), INV), (dict(softcap=float("nan")), INV), (dict(softcap=float("inf")), INV),
             (dict(window=-1), INV), (dict(batch=40000), UNS)]


def desc(cls, **kw):
    names = {n for n, _ in cls._fields_}
    return cls(**{k: v for k, v in kw.items() if k in names})


def args(n, **at):
    """n fake pointers; at: index -> value."""
    p = [A] * n
    for i, v in at.items():
        p[int(i[1:])] = v
    return p


def call(fn, d, n, ws_bytes=None, **at):
    p = args(n, **at)
    return fn(ctypes.byref(d) if d is not None else None, *p, *([] if ws_bytes is None else [ws_bytes]), None)


def write(lib, at={}, **kw):
    return call(lib.eagle_paged_write, desc(B.PagedDesc, **{**GEOM, "rows": 4, **kw}), 8, **at)


def attn(lib, at={}, ws_bytes=1 << 40, **kw):
    d = desc(B.PagedAttnDesc, **{**GEOM, **SCORE, "out_dtype": 1, "precision": 0, "engine": 0, **kw})
    return call(lib.eagle_paged_attn, d, 14, ws_bytes, **at)


def weights(lib, at={}, **kw):
    return call(lib.eagle_paged_weights, desc(B.PagedWeightsDesc, **{**GEOM, **SCORE, "max_depth": 3, **kw}), 11, **at)


def layers(n=2, bad=None, value=None):
    a = [A] * n
    if bad is not None:
        a[bad] = value
    return (ctypes.c_void_p * n)(*a)


def commit(lib, at={}, ws_bytes=16, arrays=None, **kw):
    d = desc(B.PagedCommitDesc, **{**GEOM, "layers": 2, "rows": 4, "max_depth": 3, "feat_dim": 0, "feat_dtype": 1, **kw})
    arrays = arrays or [layers() for _ in range(4)]
    p = args(9, **at)  # table, n_acc, path, seq_len, commit_pos, feat_pages, tree_feat, status, ws
    return lib.eagle_paged_commit(ctypes.byref(d), *arrays, *p, ws_bytes, None)


EVICT = dict(layers=2, limit=64, budget=32, sink=2, recent=8)


def evict(lib, at={}, ws_bytes=1 << 20, arrays=None, **kw):
    d = desc(B.PagedEvictDesc, **{**GEOM, **EVICT, **kw})
    arrays = arrays or [layers() for _ in range(3)]
    p = args(6, **at)  # table, spare, seq_len, kept, status, ws
    return lib.eagle_paged_evict(ctypes.byref(d), *arrays, *p, ws_bytes, None)


@pytest.mark.parametrize("kw,code", BAD_GEOM)
def test_geometry(lib, kw, code):
    for fn in (write, attn, weights, commit, evict):
        assert fn(lib, **kw) == code, fn.__name__


@pytest.mark.parametrize("kw,code", BAD_SCORE)
def test_scores(lib, kw, code):
    assert attn(lib, **kw) == code and weights(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(precision=2), INV), (dict(engine=2), INV), (dict(out_dtype=3), UNS), (dict(dtype=0, out_dtype=1), UNS),
    (dict(rows=128, n_q_heads=1 << 14), UNS), (dict(batch=30000, max_pages=1 << 20), UNS)])
def test_attn_descriptor(lib, kw, code):
    assert attn(lib, **kw) == code
    d = desc(B.PagedAttnDesc, **{**GEOM, **SCORE, "out_dtype": 1, "precision": 0, "engine": 0, **kw})
    assert B.workspace_size(B.EAGLE_WS_PAGED_ATTN, d) == 0


def test_attn_pointers_and_workspace(lib):
    d = desc(B.PagedAttnDesc, **{**GEOM, **SCORE, "out_dtype": 1, "precision": 0, "engine": 0})
    need = B.workspace_size(B.EAGLE_WS_PAGED_ATTN, d)
    assert need > 256
    # q, k, v, table, tree_k, tree_v, seq_len, n_nodes, anc_mask, slopes, out, lse, status, ws
    for i in (0, 1, 2, 3, 6, 10):
        assert attn(lib, {f"p{i}": None}) == INV
    for i in (4, 5, 8):  # the tree's three belong together
        assert attn(lib, {f"p{i}": None}) == INV
    for i in (0, 1, 2, 4, 5, 10, 13):
        assert attn(lib, {f"p{i}": A + 8}) == ALI
    for i in (3, 6, 7, 9, 11, 12):
        assert attn(lib, {f"p{i}": A + 2}) == ALI
    assert attn(lib, {"p8": A + 4}) == ALI
    assert attn(lib, {"p13": None}) == WS and attn(lib, ws_bytes=need - 1) == WS


def test_write_refuses(lib):
    assert write(lib, rows=0) == INV and write(lib, rows=1 << 30) == UNS
    for i in (0, 1, 2, 3, 5, 6):
        assert write(lib, {f"p{i}": None}) == INV
    for i in (0, 1, 5, 6):
        assert write(lib, {f"p{i}": A + 8}) == ALI
    for i in (2, 3, 4, 7):
        assert write(lib, {f"p{i}": A + 2}) == ALI
    assert lib.eagle_paged_write(None, *([A] * 8), None) == INV


def test_weights_refuses(lib):
    # q, lse, k, table, seq_len, n_acc, path, slopes, prior, weights, status
    assert weights(lib, batch=30000, max_pages=1 << 20) == UNS  # units counted in 32 bits
    assert weights(lib, max_depth=-1) == INV and weights(lib, max_depth=128) == UNS
    for i in (0, 1, 2, 3, 4, 5, 6, 9):
        assert weights(lib, {f"p{i}": None}) == INV
    for i in (0, 2, 8, 9):
        assert weights(lib, {f"p{i}": A + 8}) == ALI
    for i in (1, 3, 4, 5, 6, 7, 10):
        assert weights(lib, {f"p{i}": A + 2}) == ALI


def test_commit_refuses(lib):
    assert commit(lib, layers=0) == INV and commit(lib, layers=129) == UNS and commit(lib, rows=129) == UNS
    assert commit(lib, max_depth=-1) == INV and commit(lib, max_depth=128) == UNS and commit(lib, feat_dim=-1) == INV
    assert commit(lib, feat_dim=8, feat_dtype=2) == UNS
    assert commit(lib, batch=65535, n_kv_heads=1024, layers=3, max_depth=127, n_pages=40) == UNS  # CTAs counted in 32 bits
    for k in range(4):
        arr = [layers() for _ in range(4)]
        arr[k] = layers(2, 1, None)
        assert commit(lib, arrays=arr) == INV
        arr[k] = layers(2, 1, A + 8)
        assert commit(lib, arrays=arr) == ALI
    for i in (0, 1, 2, 3):
        assert commit(lib, {f"p{i}": None}) == INV
        assert commit(lib, {f"p{i}": A + 2}) == ALI
    assert commit(lib, {"p5": None}, feat_dim=8) == INV and commit(lib, {"p6": A + 8}, feat_dim=8) == ALI
    assert commit(lib, {"p8": None}) == WS and commit(lib, ws_bytes=15) == WS


def test_evict_refuses(lib):
    for kw in (dict(layers=0), dict(budget=0), dict(sink=-1), dict(recent=-1), dict(limit=31), dict(sink=25),
               dict(budget=129, limit=200)):
        assert evict(lib, **kw) == INV
    assert evict(lib, layers=129) == UNS and evict(lib, batch=60000, n_kv_heads=1000) == UNS
    for k in range(3):
        arr = [layers() for _ in range(3)]
        arr[k] = layers(2, 0, None)
        assert evict(lib, arrays=arr) == INV
        arr[k] = layers(2, 0, A + 4)
        assert evict(lib, arrays=arr) == ALI
    for i in (0, 1, 2, 3):
        assert evict(lib, {f"p{i}": None}) == INV
        assert evict(lib, {f"p{i}": A + 2}) == ALI
    assert evict(lib, {"p5": None}) == WS and evict(lib, ws_bytes=15) == WS
    assert B.workspace_size(B.EAGLE_WS_PAGED_EVICT, desc(B.PagedEvictDesc, **{**GEOM, **EVICT})) >= 2 * 8 + 4
