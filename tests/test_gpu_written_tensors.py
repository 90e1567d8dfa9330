"""Tensors that a training call writes for the caller are seen as changed by autograd.

The calls build no graph.  A tensor that autograd saved and that a call then writes, as the rotation in
place does, must end the backward pass of that graph with an error, as torch's own in-place functions do,
and not give gradients of values that are no longer there.
"""

import pytest
import torch

from tests.test_gpu_blocksparse_backward import DEV, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sba():
    import __graft_entry__

    __graft_entry__.build()
    import selected_block_attention_gb300 as m

    return m


def test_rotation_in_place(sba):
    cos, sin = sba.rotary_tables(8, 32, device=DEV)
    q, k = torch.randn((1, 8, 2, 64), device=DEV), torch.randn((1, 8, 1, 64), device=DEV)
    was = [x._version for x in (q, k, cos, sin)]
    weight = torch.ones((), device=DEV, requires_grad=True)
    loss = (q * weight).sum()  # saves q
    sba.rotary_embed(q, k, cos, sin, q_out=q)
    assert [x._version for x in (q, k, cos, sin)] == [was[0] + 1, *was[1:]]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    sba.rotary_embed(q, k, cos, sin, q_out=q, k_out=k)
    assert (q._version, k._version) == (was[0] + 2, was[1] + 1)


def test_views_share_their_version(sba):
    """Slices of one projection's output, turned where they lie."""
    x = torch.randn((1, 8, 192), device=DEV)
    q, k = x[..., :128].unflatten(-1, (2, 64)), x[..., 128:].unflatten(-1, (1, 64))
    was = x._version
    sba.rotary_embed(q, k, *sba.rotary_tables(8, 64, device=DEV), q_out=q, k_out=k)
    assert x._version == was + 2


def test_given_tables_and_gradients(sba):
    cos, sin = (torch.empty((5, 16), device=DEV) for _ in range(2))
    was = cos._version, sin._version
    sba.rotary_tables(5, 32, cos=cos, sin=sin)
    assert (cos._version, sin._version) == (was[0] + 1, was[1] + 1)
    c = Case(T=128, Hq=2, Hkv=1, seed=300).forward()
    made = [torch.empty_like(x) for x in (c.w.q, c.w.k, c.w.v)]
    was = [x._version for x in made]
    inputs = (c.w.q, c.w.k, c.w.v, c.out, c.lse, c.do)
    old = [x._version for x in inputs]
    c.call(sba, dq=made[0], dk=made[1], dv=made[2])
    sba.check_error()
    assert [x._version for x in made] == [n + 1 for n in was] and [x._version for x in inputs] == old


def test_refused_calls_and_inference_tensors(sba):
    """A call that is refused changes nothing; tensors of inference mode have no version."""
    cos, sin = sba.rotary_tables(8, 32, device=DEV)
    q = torch.randn((1, 8, 2, 64), device=DEV)
    was = q._version
    with pytest.raises(sba.SBAError):
        sba.rotary_embed(q, None, cos[:4].contiguous(), sin[:4].contiguous(), q_out=q)
    assert q._version == was
    with torch.inference_mode():
        x = torch.ones((1, 8, 2, 64), device=DEV)
    sba.rotary_embed(x, None, cos, sin, q_out=x)
    want, _ = sba.rotary_embed(torch.ones((1, 8, 2, 64), device=DEV), None, cos, sin)
    assert torch.equal(x.clone(), want)
    sba.check_error()
