"""The 8-bit KV cache entry points without a GPU: sizes behind their 32-bit arithmetic and misaligned
index arrays are refused on the host, with the documented codes."""
import ctypes

import pytest

from eagle_speculative_decoding_tree_gb300 import binding as B
from eagle_speculative_decoding_tree_gb300 import build as build_mod

A = 0x100000  # an aligned fake device address: every call below fails validation before it matters
TOP = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


@pytest.mark.parametrize("kw", [dict(max_seq=TOP), dict(max_seq=TOP - 62), dict(batch=4096, n_kv_heads=15, rows=1 << 20),
                                dict(batch=8191, n_kv_heads=8, rows=TOP)])
def test_write_and_read_refuse_sizes(lib, kw):
    d = B.KvqDesc(**{**dict(batch=1, n_kv_heads=1, head_dim=64, max_seq=512, rows=64, dtype=1), **kw})
    for fn in (lib.eagle_kvq_write, lib.eagle_kvq_read):
        assert fn(ctypes.byref(d), *([A] * 9), None) == B.EAGLE_ERR_UNSUPPORTED


@pytest.mark.parametrize("max_seq", [TOP, TOP - 126])
def test_attn_refuses_sizes(lib, max_seq):
    d = B.AttnDesc(batch=1, rows=1, n_q_heads=1, n_kv_heads=1, head_dim=64, max_seq=max_seq, scale=0.1, dtype=1,
                   num_splits=0, out_dtype=1, precision=0)
    assert lib.eagle_tree_attn_kvq(ctypes.byref(d), *([A] * 13), 1 << 40, None) == B.EAGLE_ERR_UNSUPPORTED
    assert B.workspace_size(B.EAGLE_WS_TREE_ATTN_KVQ, d) == 0


def _commit(lib, d, **kw):
    arr = (ctypes.c_void_p * d.layers)(*([A] * d.layers))
    p = [kw.get(n, A) for n in ("n_acc", "path", "seq_len", "commit_pos")]
    return lib.eagle_kvq_commit(ctypes.byref(d), *([arr] * 6), *p, None, None, kw.get("status", A), None)


@pytest.mark.parametrize("max_seq", [TOP, TOP - 62])
def test_commit_refuses_sizes(lib, max_seq):
    assert _commit(lib, B.CommitDesc(1, 1, 1, 64, 61, max_seq, 7, 1, 0, 1)) == B.EAGLE_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["n_acc", "path", "seq_len", "commit_pos", "status"])
def test_commit_refuses_misaligned_index_arrays(lib, name):
    for off in (1, 2):
        assert _commit(lib, B.CommitDesc(1, 1, 1, 64, 61, 512, 7, 1, 0, 1), **{name: A + off}) == B.EAGLE_ERR_ALIGNMENT


def test_norm_rope_refuses_sizes(lib):
    d = B.QkNormRopeDesc(batch=60000, rows=1 << 20, n_q_heads=1, n_kv_heads=1, head_dim=64, rot_dim=64, row_stride=0,
                         interleaved=0, eps=1e-6, dtype=1)
    assert lib.eagle_qk_norm_rope(ctypes.byref(d), *([A] * 9), None) == B.EAGLE_ERR_UNSUPPORTED
