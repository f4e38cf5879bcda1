"""GPU: what an 8-bit cache holds where a block has no finite value but zeros, or a scale of 0.

A row's value is its code's times its block's scale, whatever the scale: a NaN code is NaN under
a scale of 0 too, every other code is 0 there.  The reference below is that product, written
apart from the other tests' one.
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


def read(D, P, dev, start, n, odt):
    """Rows start .. start + n - 1 of the K cache of one request, by the library."""
    Hk = dev[0].shape[1]
    out = [torch.full((1, Hk, n, D), 7.0, dtype=DT[odt][0], device="cuda") for _ in range(2)]
    B.eagle_kvq_read(B.KvqDesc(1, Hk, D, P, n, DT[odt][1]), *dev, i32([start]), None, *out)
    assert torch.equal(out[0].isnan(), out[1].isnan()) and torch.equal(out[0].nan_to_num(), out[1].nan_to_num())
    return out[0][0].double().cpu().numpy()


def put(how, D, P, dev, x, start, dtype):
    """Rows x [Hk][n][D] behind `start` of K and V: one write, or a commit of as many tree rows."""
    n = x.shape[1]
    t = torch.from_numpy(x.astype(np.float32)).to(DT[dtype][0]).cuda()[None].contiguous()
    if how == "write":
        B.eagle_kvq_write(B.KvqDesc(1, x.shape[0], D, P, n, DT[dtype][1]), t, t, i32([start]), None, *dev)
    else:
        d = B.CommitDesc(1, 1, x.shape[0], D, n, P, n - 1, DT[dtype][1], 0, B.EAGLE_F32)
        B.eagle_kvq_commit(d, B.KvqLayerPointers(*[[y] for y in dev], [t], [t]), i32([n - 1]), i32([np.arange(n)]),
                           i32([start]), torch.zeros(1, n, dtype=torch.int32, device="cuda"))


def values(dev):
    """fp64 code * scale of every K row."""
    c, s = dev[0][0].cpu().numpy(), dev[1][0].double().cpu().numpy()
    return H.TABLE[c] * np.repeat(s, 64, -1)[:, : c.shape[1], None]


def same(got, want):
    return np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


@pytest.mark.parametrize("odt", ["bf16", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("how", ["write", "commit"])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_without_a_finite_value_read_back_as_nan(D, how, dtype, odt):
    """Rows of NaN and of infinities, beside zeros only, in blocks that nothing else is in."""
    P, n = 192, 40
    dev = [torch.zeros(1, 2, P, D, dtype=torch.uint8, device="cuda"), torch.zeros(1, 2, 3, device="cuda")]
    dev += [y.clone() for y in dev]
    x = np.zeros((2, n, D))
    x[0, 3], x[0, 7, ::2], x[0, 39, 5] = np.nan, np.inf, -np.inf
    x[1, 0] = np.nan
    put(how, D, P, dev, x, 64, dtype)
    want = np.where(np.isfinite(x), 0.0, np.nan)
    assert same(values(dev)[:, 64:64 + n], want)
    assert same(read(D, P, dev, 64, n, odt), want)
    # rows behind them give the block a scale: the others stay what they are
    y = np.full((2, 5, D), 3.0)
    put(how, D, P, dev, y, 64 + n, dtype)
    assert same(read(D, P, dev, 64, n + 5, odt), np.concatenate((want, y), 1))


@pytest.mark.parametrize("how", ["write", "commit"])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_under_a_scale_of_zero_stay_zeros_when_it_grows(D, how):
    """A cache whose block has a scale of 0 and codes that are not 0 (another writer's): zeros, also
    behind an append that gives the block a scale; NaN codes stay NaN."""
    P = 128
    g = np.random.default_rng(3)
    codes = g.integers(0, 126, (1, 3, P, D)).astype(np.uint8)
    codes[0, 2, 4] = 0x7f
    dev = [torch.from_numpy(codes.copy()).cuda(), torch.zeros(1, 3, 2, device="cuda")]
    dev += [y.clone() for y in dev]
    want = np.zeros((3, 10, D))
    want[2, 4] = np.nan
    assert same(read(D, P, dev, 0, 10, "f32"), want)
    y = np.full((3, 6, D), 3.0)
    y[1] = 0.0  # no scale for this head
    put(how, D, P, dev, y, 10, "bf16")
    got = read(D, P, dev, 0, 16, "f32")
    assert same(got, np.concatenate((want, y), 1))
    assert same(values(dev)[:, :16], got)
