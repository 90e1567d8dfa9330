"""GPU parity: rotary tables and the rotation of queries and keys vs the fp64 oracle, and a training
step made of them and the block-sparse attention.

Tolerances.  Tables: the fraction of a turn comes out of 64-bit fixed point; as a float it is off
by half a step of 2^-24 relative, so the angle by at most pi 2^-24, and sincospif and the product
with the amplitude add at most 2 + 1 steps of 2^-23 of the largest value: 2^-20 amplitude covers all.
Rotation: two products and a sum in fp32 (3 half steps of 2^-24 of |x0| + |x1| times the amplitude,
below 2^-22), then one rounding to the output's type: half a step, 2^-8 of the value in bf16 and
2^-24 in fp32.
"""

import numpy as np
import pytest
import torch

import oracle
from tests._parity import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def sba():
    import __graft_entry__

    __graft_entry__.build()
    import selected_block_attention_gb300 as m

    return m


@pytest.mark.parametrize("length,rot", [(1, 16), (2, 128), (777, 48), (1000, 80), (5000, 256), (33, 112)])
@pytest.mark.parametrize("kw", [dict(), dict(base=5e5, amplitude=0.5), dict(base=1.0),
                                dict(factor=4.0), dict(base=3e4, factor=8.0, original_length=2048, amplitude=1.2),
                                dict(factor=2.0, original_length=500, slow=0.0, fast=1.5)])
def test_tables(sba, length, rot, kw):
    got = sba.rotary_tables(length, rot, device=DEV, **kw)
    ref = oracle.rotary_tables(length, rot, **kw)
    for g, r in zip(got, ref):
        assert g.shape == (length, rot // 2) and g.dtype == torch.float32 and g.is_contiguous()
        assert np.abs(to_np(g) - r).max() <= 2.0 ** -20 * kw.get("amplitude", 1.0)


def test_tables_of_far_positions(sba):
    """Positions around 2^22, where an fp32 angle has steps of half a radian; the oracle's own fp64
    angle is off by 2^22 2^-53 there."""
    n = 1 << 22
    cos, sin = sba.rotary_tables(n, 16, device=DEV)
    f = oracle.rotary_frequencies(16)
    pos = np.r_[np.arange(n - 500, n), np.arange(0, n, 9973)]
    at = torch.from_numpy(pos).to(DEV)
    for g, fn in ((cos, np.cos), (sin, np.sin)):
        assert np.abs(to_np(g[at]) - fn(pos[:, None] * f)).max() <= 2.0 ** -20
    # a small angle keeps its relative precision: the slowest pair at position 1
    slow = sba.rotary_tables(2, 256, base=1e9, device=DEV)[1][1, -1].item()
    assert abs(slow / (1e9 ** (-254 / 256)) - 1) <= 2.0 ** -21


def test_tables_into_given_tensors_and_none(sba):
    cos, sin = torch.full((2, 9, 8), float("nan"), device=DEV)
    out = sba.rotary_tables(9, 16, cos=cos, sin=sin)
    assert out[0] is cos and out[1] is sin
    assert all(torch.equal(a, b) for a, b in zip(out, sba.rotary_tables(9, 16, device=torch.device(DEV))))
    assert sba.rotary_tables(0, 16, device=DEV)[0].shape == (0, 8)


def _inputs(shape_q, Hkv, dtype, seed, sliced):
    g = torch.Generator(device=DEV).manual_seed(seed)
    *lead, Hq, D = shape_q
    x = torch.randn((*lead, (Hq + 2 * Hkv) * D), generator=g, device=DEV).to(dtype)
    q, k = x[..., :Hq * D].unflatten(-1, (Hq, D)), x[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    return (q, k) if sliced else (q.contiguous(), k.contiguous())


def _check(got, x, cos, sin, pos, **kw):
    ref = oracle.rotary_embed(to_np(x), to_np(cos), to_np(sin), pos, **kw)
    step = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24
    amp = max(1.0, float(cos.abs().max()))
    # |x0| + |x1| of each pair, by rotating magnitudes with c = s = 1
    one = np.ones((1, cos.shape[1]))
    rot = 2 * cos.shape[1]
    both = np.abs(to_np(x))
    pair = np.abs(oracle.rotary_embed(both, one, one, np.zeros(x.shape[:-2], int), interleaved=kw.get("interleaved", False)))
    pair = np.maximum(pair, np.abs(oracle.rotary_embed(both, one, -one, np.zeros(x.shape[:-2], int), interleaved=kw.get("interleaved", False))))
    pair[..., rot:] = 0
    off = np.abs(to_np(got) - ref)
    assert (off <= step * np.abs(ref) + (1 + step) * 2.0 ** -22 * amp * pair).all(), off.max()
    same = torch.equal(got[..., rot:], x[..., rot:])
    assert same, "dimensions behind rot_dim changed"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (128, 96), (80, 32), (256, 256), (16, 16)])
def test_rotation(sba, D, rot, dtype, inverse, interleaved):
    B, T, Hq, Hkv = 2, 37, 5, 2
    q, k = _inputs((B, T, Hq, D), Hkv, dtype, D + rot, sliced=True)
    cos, sin = sba.rotary_tables(400, rot, amplitude=1.25, device=DEV)
    pos = np.random.default_rng(D).integers(-3, 400, (B, T))
    kw = dict(interleaved=interleaved, inverse=inverse)
    got = sba.rotary_embed(q, k, cos, sin, positions=torch.from_numpy(pos.astype(np.int32)).to(DEV), **kw)
    sba.check_error()
    for g, x in zip(got, (q, k)):
        assert g.shape == x.shape and g.is_contiguous()
        _check(g, x, cos, sin, pos, **kw)
        # padding passes through bit for bit
        off = torch.from_numpy(pos < 0).to(DEV)
        assert torch.equal(g[off], x[off])


@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 1), (3, 1, 8, 1), (1, 257, 1, 4), (2, 128, 33, 3)])
def test_positions_in_the_row(sba, B, T, Hq, Hkv):
    q, k = _inputs((B, T, Hq, 64), Hkv, torch.bfloat16, T, sliced=False)
    cos, sin = sba.rotary_tables(T, 64, device=DEV)
    got = sba.rotary_embed(q, k, cos, sin)
    pos = np.broadcast_to(np.arange(T), (B, T))
    for g, x in zip(got, (q, k)):
        _check(g, x, cos, sin, pos)


def test_packed_tokens_queries_alone_and_empty_calls(sba):
    q, k = _inputs((301, 6, 128), 2, torch.bfloat16, 3, sliced=True)
    cos, sin = sba.rotary_tables(64, 128, device=DEV)
    pos = np.r_[np.arange(60), np.arange(64), np.arange(50), np.arange(64), np.arange(63)]
    at = torch.from_numpy(pos.astype(np.int32)).to(DEV)
    both = sba.rotary_embed(q, k, cos, sin, positions=at)
    _check(both[0], q, cos, sin, pos)
    _check(both[1], k, cos, sin, pos)
    alone, none = sba.rotary_embed(q, None, cos, sin, positions=at)
    assert none is None and torch.equal(alone, both[0])
    empty = sba.rotary_embed(q[:0], k[:0], cos, sin, positions=at[:0])
    assert empty[0].shape == (0, 6, 128) and empty[1].shape == (0, 2, 128)
    sba.check_error()


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_in_a_projections_output(sba, interleaved):
    """q and k turned where they lie; the values between and behind them stay."""
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn((2, 50, 8 * 64), generator=g, device=DEV).to(torch.bfloat16)
    was = x.clone()
    q, k = x[..., :256].unflatten(-1, (4, 64)), x[..., 320:448].unflatten(-1, (2, 64))
    cos, sin = sba.rotary_tables(50, 32, device=DEV)
    want = sba.rotary_embed(q.clone(), k.clone(), cos, sin, interleaved=interleaved)
    got = sba.rotary_embed(q, k, cos, sin, interleaved=interleaved, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(x[..., 256:320], was[..., 256:320]) and torch.equal(x[..., 448:], was[..., 448:])
    back = sba.rotary_embed(*sba.rotary_embed(q.float(), k.float(), cos, sin), cos, sin, inverse=True)
    assert (back[0] - q.float()).abs().max() <= 2.0 ** -20 * q.abs().max()


def test_infinities_and_nan_stay_in_their_pair(sba):
    x = torch.ones((1, 4, 1, 64), device=DEV)
    x[0, 1, 0, 3], x[0, 2, 0, 40], x[0, 3, 0, 60] = float("nan"), float("inf"), float("nan")
    cos, sin = sba.rotary_tables(4, 32, device=DEV)
    y, _ = sba.rotary_embed(x, None, cos, sin)
    bad = [(t, d) for t, d in (~y[0, :, 0].isfinite()).nonzero().tolist()]
    assert bad == [[1, 3], [1, 19], [2, 40], [3, 60]] or bad == [(1, 3), (1, 19), (2, 40), (3, 60)]


def test_positions_outside_the_tables(sba):
    q = torch.ones((1, 3, 1, 16), device=DEV)
    cos, sin = sba.rotary_tables(5, 16, device=DEV)
    sba.check_error()
    y, _ = sba.rotary_embed(q, None, cos, sin, positions=torch.tensor([[4, 5, 1 << 30]], dtype=torch.int32, device=DEV))
    with pytest.raises(sba.SBAError) as e:
        sba.check_error()
    assert e.value.code == -5 and "rotary_embed" in str(e.value)
    assert torch.equal(y[0, 1:], q[0, 1:])
    sba.check_error()


def test_tables_feed_the_paged_append(sba):
    """The same tables, positions and layout in both calls give the same keys and queries."""
    for interleaved in (False, True):
        q, k = _inputs((1, 70, 4, 64), 2, torch.bfloat16, 9, sliced=True)
        cos, sin = sba.rotary_tables(128, 48, factor=4.0, original_length=64, device=DEV)
        pages = [torch.zeros((2, 2, 128, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        table, lens = torch.tensor([[1]], dtype=torch.int32, device=DEV), torch.tensor([70], dtype=torch.int32, device=DEV)
        qo = sba.paged_kv_append(k, k, *pages, table, lens, q=q, cos=cos, sin=sin, interleaved=interleaved)
        mine = sba.rotary_embed(q, k, cos, sin, interleaved=interleaved)
        sba.check_error()
        for a, b in ((qo, mine[0]), (pages[0][1, :, :70].transpose(0, 1)[None], mine[1])):
            # the same formula: at most the two last places of the fp32 sum between them
            assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.abs().max()
            assert (a != b).float().mean() < 0.01


def test_a_training_step(sba):
    """Tables, rotation, bounds, attention, its gradients, rotation back, twice through one captured
    graph, against autograd of the whole in fp64.

    The chain rounds to bf16 after the rotation (2^-8 of the rotated values, so logits of standard
    deviation 1 move by about 2^-8 sqrt(2 / 3) of it each and P with them), after the attention, in P
    and dS, after the gradients and after the rotation back: six independent roundings of at most
    2^-8 / sqrt(3) relative, and the two on the logits count by |logit|, up to 4: together below
    2^-8 sqrt((6 + 2 * 16) / 3) = 1.4e-2 in the Frobenius norm.
    """
    B, T, Hq, Hkv, D, rot, left = 2, 384, 4, 2, 64, 48, 150
    G = Hq // Hkv
    cos, sin = sba.rotary_tables(T, rot, base=2e4, factor=2.0, original_length=200, device=DEV)
    qkv = torch.empty((B, T, (Hq + 2 * Hkv) * D), dtype=torch.bfloat16, device=DEV)
    d_out = torch.empty((B, T, Hq, D), dtype=torch.bfloat16, device=DEV)
    seg = np.zeros((B, T), np.int32)
    seg[0, 100:], seg[0, 290:], seg[1, 370:] = 1, 2, -1
    at = np.broadcast_to(np.arange(T, dtype=np.int32), (B, T)).copy()
    start = np.where(seg == 2, 290, np.where(seg == 1, 100, 0))
    inner = np.where(seg < 0, -1, at - start).astype(np.int32)
    seg_d, at_d, inner_d = (torch.from_numpy(x).to(DEV) for x in (seg, at, inner))

    def parts(x):
        return (x[..., :Hq * D].unflatten(-1, (Hq, D)), x[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D)),
                x[..., (Hq + Hkv) * D:].unflatten(-1, (Hkv, D)))

    def step():
        q, k, v = parts(qkv)
        q, k = sba.rotary_embed(q, k, cos, sin, positions=inner_d)
        v = v.contiguous()
        ints = (at_d, seg_d, at_d, seg_d)
        bounds = sba.sparse_mask_bounds(*ints, 128, 64, causal=True, window_left=left, window_right=0)
        mask = dict(causal=True, window_left=left, window_right=0)
        out, lse = sba.blocksparse_attn_fwd(q, k, v, *ints, *bounds, 128, 64, **mask)
        dq, dk, dv = sba.blocksparse_attn_bwd(q, k, v, out, lse, d_out, *ints, *bounds, 128, 64, **mask)
        sba.rotary_embed(dq, dk, cos, sin, positions=inner_d, inverse=True, q_out=dq, k_out=dk)
        return out, dq, dk, dv

    def fill(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        qkv.copy_(torch.randn(qkv.shape, generator=g, device=DEV))
        d_out.copy_(torch.randn(d_out.shape, generator=g, device=DEV))

    def reference():
        x = qkv.double().cpu().requires_grad_()
        q, k, v = parts(x)

        def turn(y):
            c, s = (z.double().cpu()[torch.from_numpy(np.maximum(inner, 0)).long()][:, :, None] for z in (cos, sin))
            pad = torch.from_numpy(inner < 0)[..., None, None]
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            return torch.where(pad, y, torch.cat((a * c - b * s, b * c + a * s, y[..., rot:]), -1))

        q, k = turn(q).transpose(1, 2), turn(k).transpose(1, 2).repeat_interleave(G, 1)
        v = v.transpose(1, 2).repeat_interleave(G, 1)
        sg, p = torch.from_numpy(seg), torch.arange(T)
        see = (sg[:, :, None] == sg[:, None]) & (sg[:, :, None] >= 0)
        see &= ((p[:, None] - p >= 0) & (p[:, None] - p <= left))[None]
        # a window that is no multiple of the block: the bounds leave out a key block that begins
        # left of the first query's window
        lo, up = (torch.from_numpy(np.repeat(np.asarray(x)[:, 0], 128, axis=1))[:, :, None]
                  for x in oracle.sparse_mask_bounds(at, seg, at, seg, 128, 64, causal=True, window_left=left, window_right=0)[:2])
        see &= (p // 64 >= lo) & (p // 64 < up)
        some = see.any(-1)[:, None, :, None]
        s = (q @ k.transpose(-1, -2) / D ** 0.5).masked_fill(~see[:, None], float("-inf"))
        w = torch.where(some, torch.softmax(torch.where(some, s, torch.zeros_like(s)), -1), torch.zeros_like(s))
        out = (w @ v).transpose(1, 2)
        out.backward(d_out.double().cpu())
        return (out.detach(), *parts(x.grad))

    fill(1)
    step()  # outside the capture: the library finds its per-device state
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (2, 3):
        fill(seed)
        graph.replay()
        sba.check_error()
        for name, a, b in zip(("out", "dq", "dk", "dv"), got, reference()):
            rel = np.linalg.norm(to_np(a) - b.numpy()) / np.linalg.norm(b.numpy())
            assert rel <= 1.4e-2, (seed, name, rel)
            assert torch.count_nonzero(a[1, 370:]).item() == 0
