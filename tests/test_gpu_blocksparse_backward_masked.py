"""What the block-sparse gradients must not take from masked places.

The bounds of a query block end anywhere on a grid of 64 keys, the kernels' tiles hold 128: values
of keys outside the bounds lie in the same tiles, and at the end of a row those of the next sequence.
Whatever they hold, infinities and NaN among them, the gradients are those of a run in which they
hold zeros, bit for bit: no sum may take them in, with a weight of 0 either.  The same goes for the rows
of query blocks whose bounds are empty.
"""

import numpy as np
import pytest
import torch

from tests.test_gpu_blocksparse_backward import DEV, Case, check

pytestmark = pytest.mark.gpu
BAD = [float("nan"), float("inf"), -float("inf")]


@pytest.fixture(scope="module")
def sba():
    import __graft_entry__

    __graft_entry__.build()
    import selected_block_attention_gb300 as m

    return m


def _fill(x, where, seed):
    """Non-finite values at the tokens `where` [B, T] of x."""
    n = int(where.sum())
    rng = np.random.default_rng(seed)
    bad = torch.tensor(rng.choice(BAD, (n, *x.shape[2:])), dtype=x.dtype, device=DEV)
    x[torch.from_numpy(where).to(DEV)] = bad


def _same(c, sba, tensors, where):
    """The call's gradients with zeros and with non-finite values at `where` of the tensors."""
    at = torch.from_numpy(where).to(DEV)
    for x in tensors:
        x[at] = 0
    want = [x.clone() for x in c.call(sba)]
    sba.check_error()
    ref = c.reference()
    for i, name in enumerate(("dq", "dk", "dv")):
        check(want[i], ref[i], ref[3 + i], name)
    for seed, x in enumerate(tensors):
        _fill(x, where, seed)
    got = c.call(sba)
    sba.check_error()
    for name, a, b in zip(("dq", "dk", "dv"), got, want):
        assert torch.isfinite(a).all(), f"{name}: {int((~torch.isfinite(a)).sum())} values are not finite"
        assert torch.equal(a, b), name
    return want


def _odd_bounds(D, Hq, Hkv, seed):
    """Three rows of 512 tokens over bounds of 64 keys, most of them odd in number.  Of the second row no
    query block reaches keys 0 .. 63 and 448 .. 511, of the third one's not the first 64."""
    T = 512
    lo = np.array([[[0, 0, 0, 5]], [[1, 1, 1, 2]], [[1, 2, 3, 3]]])
    up = np.array([[[2, 4, 6, 8]], [[2, 4, 6, 7]], [[2, 3, 6, 8]]])
    none = np.full_like(lo, T // 64), np.zeros_like(up)
    seg = np.zeros((3, T), np.int32)
    seg[1, :64], seg[1, 448:], seg[2, :64] = -1, -1, -1
    c = Case(B=3, T=T, Hq=Hq, Hkv=Hkv, D=D, kb=64, seg=seg, seed=seed, bounds=(lo, up, *none))
    return c.forward(), seg < 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [(4, 2), (3, 1)])
def test_keys_outside_the_bounds(sba, D, heads):
    """Also where the last step of a row's last query block reaches into the next row."""
    c, outside = _odd_bounds(D, *heads, seed=200 + D)
    want = _same(c, sba, (c.w.k, c.w.v), outside)
    at = torch.from_numpy(outside).to(DEV)
    for x in want[1:]:
        assert torch.count_nonzero(x[at]).item() == 0


def test_keys_outside_the_bounds_with_heads_in_parts(sba):
    c, outside = _odd_bounds(64, 8, 1, seed=210)
    # parts: an fp32 dK and dV for each of them in the workspace
    assert sba.blocksparse_attn_bwd_workspace_size(3, 512, 8, 1, 64) > 2 * 3 * 512 * 64 * 4
    _same(c, sba, (c.w.k, c.w.v), outside)


@pytest.mark.parametrize("heads", [(4, 2), (8, 1)])
def test_query_blocks_without_keys(sba, heads):
    """A block of padding whose bounds are empty: nothing of its rows is taken."""
    T = 512
    seg = np.zeros((2, T), np.int32)
    seg[0, 128:256], seg[1, 256:] = -1, -1
    c = Case(B=2, T=T, Hq=heads[0], Hkv=heads[1], D=64, kb=64, seg=seg, seed=220).forward()
    assert (c.bounds[0] >= c.bounds[1])[[0, 1, 1], 0, [1, 2, 3]].all()
    want = [x.clone() for x in c.call(sba)]
    for seed, x in enumerate((c.w.q, c.out, c.lse, c.do)):
        _fill(x, seg < 0, seed)
    got = c.call(sba)
    sba.check_error()
    for name, a, b in zip(("dq", "dk", "dv"), got, want):
        assert torch.isfinite(b).all() and torch.equal(a, b), name
