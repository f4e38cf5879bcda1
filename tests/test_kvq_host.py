"""The 8-bit KV cache operators without a GPU: their references pinned, the refusals of the
entry points, workspace sizes, and the binding's argument checks."""
import ctypes
import math

import numpy as np
import pytest
import torch

import kvq_helpers as H
from eagle_speculative_decoding_tree_gb300 import binding as B
from eagle_speculative_decoding_tree_gb300 import build as build_mod

A = 0x100000  # an aligned fake device address: every call below fails validation before it matters


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


# ------------------------------------------------------------------ references
def test_decode_and_encode_against_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(H.TABLE, ref, equal_nan=True)
    g = np.random.default_rng(0)
    x = np.concatenate((g.normal(size=4000) * 2.0 ** g.integers(-12, 8, 4000), ref[:127], -ref[:127],
                        (ref[:126] + ref[1:127]) / 2, np.array([448.0, -448.0, 0.0, -0.0])))
    x = x[np.abs(x) <= 448].astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(H.encode(x.astype(np.float64)), want)
    assert (H.encode(np.array([np.inf, -np.inf, np.nan])) == 127).all()


@pytest.mark.parametrize("amax,s", [(0.0, 0.0), (448.0, 1.0), (448.5, 2.0), (224.0, 0.5), (224.01, 1.0), (1.0, 2.0 ** -8),
                                    (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7), (3e38, 2.0 ** 120),
                                    (1e-40, 2.0 ** -126)])
def test_scale_is_the_smallest_power_of_two(amax, s):
    assert H.scale_of(amax) == s


def test_append_keeps_or_moves_the_rows_before():
    codes, scale = np.zeros((130, 16), np.uint8), np.zeros(3, np.float32)
    g = np.random.default_rng(1)
    a, b = g.normal(size=(70, 16)), 100 * g.normal(size=(40, 16))
    H.append(codes, scale, a, 0)
    before = H.values(codes, scale)[:70]
    assert np.abs(before - a).max() <= 2.0 ** -4 * np.abs(a).max()
    H.append(codes, scale, b, 70)
    after = H.values(codes, scale)
    assert scale[1] >= np.abs(b).max() / 448
    assert np.array_equal(after[:64], before[:64])
    # moved rows: a value the new scale holds as a normal is unchanged
    big = np.abs(before[64:70]) >= scale[1] * 2.0 ** -6
    assert np.array_equal(after[64:70][big], before[64:70][big])
    assert np.abs(after[64:70] - before[64:70]).max() <= scale[1] * 2.0 ** -10


# ------------------------------------------------------------------ refusals
def _attn(**kw):
    d = dict(batch=1, rows=61, n_q_heads=32, n_kv_heads=8, head_dim=128, max_seq=8256, scale=0.088, dtype=1,
             num_splits=0, out_dtype=1, precision=0)
    d.update(kw)
    return B.AttnDesc(**d)


def _call_attn(lib, d, ws_bytes=1 << 40, **kw):
    names = ("q", "k8", "ks", "v8", "vs", "tk", "tv", "seq", "nodes", "mask", "out", "lse", "ws")
    p = [kw.get(n, A) for n in names]
    return lib.eagle_tree_attn_kvq(ctypes.byref(d), *p, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=96), B.EAGLE_ERR_UNSUPPORTED), (dict(rows=129), B.EAGLE_ERR_UNSUPPORTED),
    (dict(dtype=0, out_dtype=0), B.EAGLE_ERR_UNSUPPORTED), (dict(n_q_heads=12), B.EAGLE_ERR_UNSUPPORTED),
    (dict(batch=40, max_seq=1 << 23), B.EAGLE_ERR_UNSUPPORTED), (dict(fault_test=1), B.EAGLE_ERR_UNSUPPORTED),
    (dict(engine=3), B.EAGLE_ERR_INVALID_ARG), (dict(rows=0), B.EAGLE_ERR_INVALID_ARG),
    (dict(precision=2), B.EAGLE_ERR_INVALID_ARG), (dict(scale=math.inf), B.EAGLE_ERR_INVALID_ARG),
])
def test_attn_refuses_descriptors(lib, kw, code):
    d = _attn(**kw)
    assert _call_attn(lib, d) == code
    assert B.workspace_size(B.EAGLE_WS_TREE_ATTN_KVQ, d) == 0


def test_attn_refuses_pointers_and_workspace(lib):
    d = _attn()
    for n in ("q", "k8", "ks", "v8", "vs", "tk", "tv", "seq", "mask", "out"):
        assert _call_attn(lib, d, **{n: None}) == B.EAGLE_ERR_INVALID_ARG, n
    for n, off in (("q", 8), ("k8", 4), ("v8", 8), ("tk", 2), ("out", 8), ("ws", 8), ("ks", 2), ("mask", 4), ("lse", 2),
                   ("nodes", 1), ("seq", 2)):
        assert _call_attn(lib, d, **{n: A + off}) == B.EAGLE_ERR_ALIGNMENT, n
    need = B.workspace_size(B.EAGLE_WS_TREE_ATTN_KVQ, d)
    assert need > 256
    assert _call_attn(lib, d, ws_bytes=need - 1) == B.EAGLE_ERR_WORKSPACE
    assert _call_attn(lib, d, ws=None) == B.EAGLE_ERR_WORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), B.EAGLE_ERR_INVALID_ARG), (dict(rows=0), B.EAGLE_ERR_INVALID_ARG),
    (dict(head_dim=0), B.EAGLE_ERR_INVALID_ARG), (dict(head_dim=80), B.EAGLE_ERR_UNSUPPORTED),
    (dict(dtype=2), B.EAGLE_ERR_UNSUPPORTED), (dict(batch=9000), B.EAGLE_ERR_UNSUPPORTED),
])
def test_write_and_read_refuse_descriptors(lib, kw, code):
    d = dict(batch=1, n_kv_heads=8, head_dim=128, max_seq=512, rows=64, dtype=1)
    d.update(kw)
    d = B.KvqDesc(**d)
    for fn in (lib.eagle_kvq_write, lib.eagle_kvq_read):
        assert fn(ctypes.byref(d), *([A] * 9), None) == code


def test_write_and_read_refuse_pointers(lib):
    d = B.KvqDesc(1, 8, 128, 512, 64, 1)
    for fn, names in ((lib.eagle_kvq_write, "k v start count k8 ks v8 vs status"),
                      (lib.eagle_kvq_read, "k8 ks v8 vs start count k v status")):
        names = names.split()
        for i, n in enumerate(names):
            p = [A] * 9
            if n not in ("count", "status"):
                p[i] = None
                assert fn(ctypes.byref(d), *p, None) == B.EAGLE_ERR_INVALID_ARG, n
            p[i] = A + (8 if n in ("k", "v", "k8", "v8") else 2)
            assert fn(ctypes.byref(d), *p, None) == B.EAGLE_ERR_ALIGNMENT, n
        assert fn(None, *([A] * 9), None) == B.EAGLE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=96), B.EAGLE_ERR_UNSUPPORTED), (dict(layers=129), B.EAGLE_ERR_UNSUPPORTED),
    (dict(rows=200), B.EAGLE_ERR_UNSUPPORTED), (dict(max_depth=128), B.EAGLE_ERR_UNSUPPORTED),
    (dict(layers=0), B.EAGLE_ERR_INVALID_ARG), (dict(feat_dim=8), B.EAGLE_ERR_INVALID_ARG),
    (dict(batch=9000), B.EAGLE_ERR_UNSUPPORTED),
])
def test_commit_refuses_descriptors(lib, kw, code):
    d = dict(layers=2, batch=1, n_kv_heads=8, head_dim=128, rows=61, max_seq=512, max_depth=7, dtype=1, feat_dim=0,
             feat_dtype=1)
    d.update(kw)
    d = B.CommitDesc(**d)
    arr = (ctypes.c_void_p * 128)(*([A] * 128))
    assert lib.eagle_kvq_commit(ctypes.byref(d), *([arr] * 6), A, A, A, A, None, None, A, None) == code


def test_commit_refuses_layer_pointers(lib):
    d = B.CommitDesc(2, 1, 8, 128, 61, 512, 7, 1, 0, 1)
    good = (ctypes.c_void_p * 2)(A, A)
    for i in range(6):
        for bad, code in ((None, B.EAGLE_ERR_INVALID_ARG), (A + 2, B.EAGLE_ERR_ALIGNMENT)):
            p = [good] * 6
            p[i] = (ctypes.c_void_p * 2)(A, bad)
            assert lib.eagle_kvq_commit(ctypes.byref(d), *p, A, A, A, A, None, None, A, None) == code
        p = [good] * 6
        p[i] = None
        assert lib.eagle_kvq_commit(ctypes.byref(d), *p, A, A, A, A, None, None, A, None) == B.EAGLE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(rot_dim=-16), B.EAGLE_ERR_INVALID_ARG), (dict(rot_dim=24), B.EAGLE_ERR_UNSUPPORTED),
    (dict(rot_dim=144), B.EAGLE_ERR_INVALID_ARG), (dict(head_dim=96), B.EAGLE_ERR_UNSUPPORTED),
    (dict(row_stride=6136), B.EAGLE_ERR_INVALID_ARG), (dict(row_stride=6148), B.EAGLE_ERR_ALIGNMENT),
    (dict(eps=-1.0), B.EAGLE_ERR_INVALID_ARG), (dict(eps=math.nan), B.EAGLE_ERR_INVALID_ARG),
    (dict(interleaved=2), B.EAGLE_ERR_INVALID_ARG), (dict(batch=70000), B.EAGLE_ERR_UNSUPPORTED),
    (dict(dtype=3), B.EAGLE_ERR_UNSUPPORTED), (dict(rows=0), B.EAGLE_ERR_INVALID_ARG),
])
def test_norm_rope_refuses_descriptors(lib, kw, code):
    d = dict(batch=1, rows=61, n_q_heads=32, n_kv_heads=8, head_dim=128, rot_dim=128, row_stride=0, interleaved=0,
             eps=1e-6, dtype=1)
    d.update(kw)
    d = B.QkNormRopeDesc(**d)
    assert lib.eagle_qk_norm_rope(ctypes.byref(d), *([A] * 9), None) == code


def test_norm_rope_refuses_pointers(lib):
    d = B.QkNormRopeDesc(1, 61, 32, 8, 128, 128, 0, 0, 1e-6, 1)
    for i, n in enumerate("qkv wq wk inv_freq pos nodes q k v".split()):
        p = [A] * 9
        if n not in ("wq", "wk", "nodes"):
            p[i] = None
            assert lib.eagle_qk_norm_rope(ctypes.byref(d), *p, None) == B.EAGLE_ERR_INVALID_ARG, n
        p[i] = A + 2
        assert lib.eagle_qk_norm_rope(ctypes.byref(d), *p, None) == B.EAGLE_ERR_ALIGNMENT, n


def test_binding_refuses_host_tensors(lib):
    d = B.KvqDesc(1, 1, 64, 64, 1, 0)
    k = torch.zeros(1, 1, 1, 64)
    with pytest.raises(ValueError, match="CUDA"):
        B.eagle_kvq_write(d, k, k, torch.zeros(1, dtype=torch.int32), None, torch.zeros(64, 64, dtype=torch.uint8),
                          torch.zeros(1), torch.zeros(64, 64, dtype=torch.uint8), torch.zeros(1))


def test_workspace_counters_have_one_place():
    """Descriptors that share a workspace: the first partial comes behind every counter."""
    sizes = [B.workspace_size(B.EAGLE_WS_TREE_ATTN_KVQ, _attn(batch=b, rows=r, max_seq=p, num_splits=1))
             for b, r, p in ((1, 61, 512), (2, 61, 512), (1, 61, 64))]
    part = 2 * 8 * 256 * (128 * 4 + 8)  # the tree and one piece, eight heads of 256 rows
    head = sizes[0] - part
    assert sizes[1] - head == 2 * part and sizes[2] == sizes[0] and head % 256 == 0
    assert head >= 256 + 8 * 148
