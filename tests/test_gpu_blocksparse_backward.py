"""GPU parity: gradients of block-sparse attention (dq, dk, dv) vs the fp64 oracle.

out and lse are computed here in fp64 and rounded to what the forward leaves (bf16, fp32), so the
backward is tested by itself.  Keys of blocks in [lower_full, upper_full) count without a token test,
as the entry points define them: bounds hold one full range for a query block, which takes in the
blocks between two full ones (a document that goes on behind padding).

Tolerances.  A rounding to bf16 is off by at most half a step, 2^-8 of the value.  The kernel
rounds P and dS once each before their products and the outputs at the end, so with M the sums of
magnitudes (oracle, ``magnitudes``), in which |dS| counts both terms of P (dP - Delta):
    |dv - ref| <= 2^-8 sum P |dO| + 2^-8 |ref|,      |dq - ref|, |dk - ref| <= 2^-8 M + 2^-8 |ref|,
beside the fp32 part: exponents of magnitude below 64 in steps of 2^-23 (relative error of P below
2^-16, with the approximate 2^x 2^-22 more), sums of up to 2^13 / 16 products in steps of 2^-23
(2^-14 of M).  2^-13 M covers those.  Each element is held to that bound, and the whole to 5e-3 in
the Frobenius norm: independent roundings of relative size 2^-8 / sqrt(3) at most, twice in a row,
are 3.2e-3.
"""

import numpy as np
import pytest
import torch

import oracle
from selected_block_attention_gb300 import workloads
from tests._parity import assert_attention_close, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = 2.0 ** -8
REL_FRO = 5e-3


@pytest.fixture(scope="module")
def sba():
    import __graft_entry__

    __graft_entry__.build()
    import selected_block_attention_gb300 as m

    return m


class Case:
    """Inputs of a call on the GPU and the arrays the oracle takes."""

    def __init__(self, B=1, T=512, Hq=4, Hkv=2, D=128, kb=128, doc=150, pad=20, causal=True, left=-1, right=-1,
                 scale=None, seed=0, seg=None, pos=None, bounds=None):
        self.w = workloads.blocksparse(device=DEV, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, mean_doc=doc, pad_tail=pad,
                                       window=(left, right), seed=seed)
        m = self.w.mask
        self.seg = m.q_segment_ids.cpu().numpy() if seg is None else np.asarray(seg, np.int32)
        self.pos = m.q_positions.cpu().numpy() if pos is None else np.asarray(pos, np.int32)
        self.kb, self.scale = kb, scale
        self.mask = dict(causal=causal, window_left=left, window_right=right)
        self.ints = (self.pos, self.seg, self.pos, self.seg)
        self.bounds = bounds or oracle.sparse_mask_bounds(*self.ints, 128, kb, **self.mask)
        g = torch.Generator(device=DEV).manual_seed(seed + 99)
        self.do = torch.randn(self.w.q.shape, generator=g, device=DEV).to(torch.bfloat16)
        to = lambda a: torch.from_numpy(np.array(a, np.int32)).to(DEV)  # noqa: E731
        self.dev_ints = [to(x) for x in self.ints]
        self.dev_bounds = [to(x) for x in self.bounds]

    def forward(self):
        """out and lse as the forward leaves them."""
        q, k, v = (to_np(x) for x in (self.w.q, self.w.k, self.w.v))
        B, T, Hq, D = q.shape
        G = Hq // k.shape[2]
        scale = self.scale or D ** -0.5
        left, right = self.mask["window_left"], self.mask["window_right"]
        out, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
        for b in range(B):
            for n in range(T // 128):
                lo, up, lf, uf = (int(np.asarray(x)[b, 0, n]) for x in self.bounds)
                t, key = np.arange(n * 128, n * 128 + 128), np.arange(lo * self.kb, up * self.kb)
                gap = self.pos[b, t][:, None].astype(np.int64) - self.pos[b, key]
                see = (self.seg[b, t][:, None] == self.seg[b, key]) & (self.seg[b, t] != -1)[:, None]
                see &= (gap >= 0) | (not self.mask["causal"])
                see &= (gap <= left) | (left < 0)
                see &= (-gap <= right) | (right < 0)
                see |= (key // self.kb >= lf) & (key // self.kb < uf)
                some = see.any(-1)
                for h in range(Hq) if key.size else ():
                    s = np.where(see, scale * q[b, t, h] @ k[b, key, h // G].T, -np.inf)
                    top = np.where(some, s.max(-1), 0.0)
                    e = np.exp(s - top[:, None])
                    total = np.where(some, e.sum(-1), 1.0)
                    out[b, t, h] = e @ v[b, key, h // G] / total[:, None]
                    lse[b, t, h] = np.where(some, top + np.log(total), -np.inf)
        self.out, self.lse = torch.from_numpy(out).to(DEV, torch.bfloat16), torch.from_numpy(lse).to(DEV, torch.float32)
        return self

    def call(self, sba, **kw):
        return sba.blocksparse_attn_bwd(self.w.q, self.w.k, self.w.v, self.out, self.lse, self.do, *self.dev_ints,
                                        *self.dev_bounds, 128, self.kb, softmax_scale=self.scale, **self.mask, **kw)

    def reference(self, **kw):
        return oracle.blocksparse_attention_backward(
            to_np(self.w.q), to_np(self.w.k), to_np(self.w.v), to_np(self.out), to_np(self.lse), to_np(self.do),
            *self.ints, *self.bounds[:2], 128, self.kb, softmax_scale=self.scale, magnitudes=True, **self.mask,
            lower_full=self.bounds[2], upper_full=self.bounds[3], **kw)


def check(got, ref, big, what):
    got = to_np(got) if isinstance(got, torch.Tensor) else got
    assert np.isfinite(got).all(), f"{what}: non-finite gradient"
    off = np.abs(got - ref)
    bar = (HALF + 2.0 ** -13) * big + HALF * np.abs(ref) + 1e-30
    worst = np.unravel_index(np.argmax(off - bar), off.shape)
    assert (off <= bar).all(), f"{what}{list(worst)}: {got[worst]} for {ref[worst]}, bound {bar[worst]:.3g}"
    norm = np.linalg.norm(ref)
    rel = np.linalg.norm(got - ref) / norm if norm else np.linalg.norm(got)
    assert rel <= REL_FRO, f"{what}: relative Frobenius error {rel:.3g}"


def check_all(sba, c):
    got = c.call(sba)
    sba.check_error()
    ref = c.reference()
    for i, name in enumerate(("dq", "dk", "dv")):
        check(got[i], ref[i], ref[3 + i], name)
    return got


def test_one_tile(sba):
    check_all(sba, Case(T=128, Hq=1, Hkv=1, doc=1000, pad=0, seed=1).forward())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kb", [64, 128])
@pytest.mark.parametrize("heads", [(4, 2), (3, 1), (5, 5)])
def test_documents(sba, D, kb, heads):
    check_all(sba, Case(B=2, T=640, Hq=heads[0], Hkv=heads[1], D=D, kb=kb, seed=10 + D + kb).forward())


@pytest.mark.parametrize("kb", [64, 128])
@pytest.mark.parametrize("mask", [dict(left=100, right=0), dict(causal=False, left=130, right=70), dict(causal=False),
                                  dict(causal=False, right=40), dict(causal=False, left=33), dict(left=0, right=0),
                                  dict(left=-1, right=5)])
def test_windows(sba, mask, kb):
    check_all(sba, Case(T=640, Hq=2, Hkv=1, kb=kb, doc=400, seed=40, **mask).forward())


@pytest.mark.parametrize("kb,D", [(64, 64), (128, 128)])
def test_unsorted_segments_and_positions(sba, kb, D):
    """Blocks whose positions are not consecutive or whose segments are not runs take the test of
    each pair; padding lies anywhere."""
    rng = np.random.default_rng(kb)
    B, T = 2, 512
    seg = np.sort(rng.integers(0, 4, (B, T)), axis=1)
    seg[:, 256:] = rng.integers(0, 3, (B, 256))
    seg[rng.random((B, T)) < 0.05] = -1
    pos = np.broadcast_to(np.arange(T), (B, T)).copy()
    pos[:, 128:384] = rng.permuted(pos[:, 128:384], axis=1)
    check_all(sba, Case(B=B, T=T, D=D, kb=kb, seg=seg, pos=pos, left=90, seed=50).forward())


def test_nothing_in_view(sba):
    """A row of padding only, a padded query block, and keys that no row sees: zeros, also where d_out
    and out hold large numbers."""
    B, T = 3, 512
    seg = np.zeros((B, T), np.int32)
    seg[0] = -1
    seg[1, 128:256] = -1
    seg[2, 300:] = -1
    c = Case(B=B, T=T, seg=seg, left=60, seed=60)
    c.do[0] *= 1e4
    c.forward()
    dq, dk, dv = check_all(sba, c)
    off = torch.from_numpy(seg == -1).to(DEV)
    for x in (dq, dk, dv):
        assert torch.count_nonzero(x[off]).item() == 0


def test_bounds_rule_what_is_visited(sba):
    """Bounds narrower than the mask leave keys out (of one 64-key block too), full ranges need no
    token test: both as the forward takes them."""
    B, T, kb = 1, 512, 64
    lo, up = np.array([[[0, 1, 3, 5]]]), np.array([[[2, 2, 6, 8]]])
    lf, uf = np.array([[[1, 8, 4, 5]]]), np.array([[[2, 0, 5, 7]]])
    c = Case(B=B, T=T, kb=kb, doc=60, pad=9, causal=True, seed=70, bounds=(lo, up, lf, uf))
    c.forward()
    out, lse = sba.blocksparse_attn_fwd(c.w.q, c.w.k, c.w.v, *c.dev_ints, *c.dev_bounds, 128, kb, causal=True)
    assert_attention_close(to_np(out), to_np(c.out), to_np(lse), to_np(c.lse), what="forward over the same bounds")
    check_all(sba, c)


@pytest.mark.parametrize("scale", [0.02, 0.6])
def test_scales(sba, scale):
    check_all(sba, Case(T=384, Hq=2, Hkv=1, doc=300, scale=scale, seed=80).forward())


def test_difference_quotients(sba):
    """The gradients against central differences of the forward oracle along random directions.
    g = bf16(gradient): its rounding errors are independent, so <g, u> is off by about
    2^-8 |g| |u| / sqrt(n) sqrt(3), and the roundings of P and dS by as much again; 12 of those."""
    c = Case(T=256, Hq=2, Hkv=1, D=64, kb=64, doc=120, left=100, seed=90).forward()
    got = [to_np(x) for x in c.call(sba)]
    sba.check_error()
    x = [to_np(t) for t in (c.w.q, c.w.k, c.w.v)]
    rng = np.random.default_rng(3)
    loss = lambda *y: (oracle.blocksparse_attention(*y, *c.ints, *c.bounds[:2], 128, 64, **c.mask)[0] * to_np(c.do)).sum()  # noqa: E731
    for i in range(3):
        u = rng.choice([-1.0, 1.0], x[i].shape)
        y, z = list(x), list(x)
        y[i], z[i] = x[i] + 1e-4 * u, x[i] - 1e-4 * u
        ref = (loss(*y) - loss(*z)) / 2e-4
        sigma = 2.0 ** -8 / 3 ** 0.5 * np.linalg.norm(got[i])
        assert abs((got[i] * u).sum() - ref) <= 12 * sigma, (i, (got[i] * u).sum(), ref, sigma)


def test_same_from_run_to_run_and_on_another_stream(sba):
    c = Case(B=2, T=1024, Hq=8, Hkv=2, left=300, seed=100).forward()
    first = [x.clone() for x in c.call(sba)]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, c.call(sba)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = c.call(sba)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, got))
    sba.check_error()


def test_given_outputs_and_workspace(sba):
    c = Case(T=256, seed=110).forward()
    want = c.call(sba)
    made = [torch.full_like(x, float("nan")) for x in want]
    need = sba.blocksparse_attn_bwd_workspace_size(1, 256, 4, 2, 128)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
    got = c.call(sba, dq=made[0], dk=made[1], dv=made[2], workspace=ws)
    sba.check_error()
    assert all(a is b for a, b in zip(got, made)) and all(torch.equal(a, b) for a, b in zip(got, want))
    assert (ws[need:] == 255).all()
    with pytest.raises(sba.SBAError):
        c.call(sba, workspace=ws[:need - 256])
    with pytest.raises(sba.SBAError):
        c.call(sba, dk=made[1], dv=made[1])
    with pytest.raises(sba.SBAError):
        c.call(sba, dq=c.w.q)


def test_captured_and_replayed(sba):
    """A captured call on new contents (another mask and bounds among them), and two captured calls with
    workspaces of their own replayed on two streams at once."""
    a, b = Case(T=640, left=100, seed=120).forward(), Case(T=640, left=100, doc=50, seed=121).forward()
    want = [[x.clone() for x in c.call(sba)] for c in (a, b)]
    graphs, outs = [], []
    cases = [Case(T=640, left=100, seed=120).forward() for _ in range(2)]
    for c in cases:
        c.call(sba)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.call(sba))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(x, y) for x, y in zip(o, want[0]))
    c = cases[0]
    for name in ("q", "k", "v"):
        getattr(c.w, name).copy_(getattr(b.w, name))
    for x, y in zip([c.out, c.lse, c.do, *c.dev_ints, *c.dev_bounds], [b.out, b.lse, b.do, *b.dev_ints, *b.dev_bounds]):
        x.copy_(y)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs[0], want[1]))
    sba.check_error()


def test_many_items_a_block(sba):
    """More items than blocks that run at once, in both kernels, of very different lengths (empty ones
    among them)."""
    rng = np.random.default_rng(7)
    B, T = 4, 1536
    seg = np.zeros((B, T), np.int64)
    seg[1] = np.arange(T) // 40
    seg[2, 200:1300] = -1
    seg[3] = np.sort(rng.integers(0, 6, T))
    check_all(sba, Case(B=B, T=T, Hq=8, Hkv=4, D=64, kb=64, seg=seg, seed=130).forward())


@pytest.mark.parametrize("D,seen", [(64, 512), (128, 128), (128, 256)])
def test_runs_of_unseen_key_tiles(sba, D, seen):
    """More key tiles than blocks on the GPU, and after every few that queries see many that none does:
    a block takes several of those behind one with sums still to store."""
    B, T, Hq = 2, 4096, 8
    seg = np.full((B, T), -1, np.int64)
    for t in range(0, T, 1024):
        seg[:, t:t + seen] = t
    check_all(sba, Case(B=B, T=T, Hq=Hq, Hkv=Hq, D=D, seg=seg, seed=140).forward())


@pytest.mark.parametrize("B,T,Hq,Hkv,D", [(1, 1024, 8, 1, 128), (1, 1536, 12, 2, 64), (2, 1024, 5, 1, 64)])
def test_heads_in_parts(sba, B, T, Hq, Hkv, D):
    """Few key tiles and KV heads: a KV head's query heads are divided among items and their sums merged
    (also for key tiles that no query sees)."""
    assert sba.blocksparse_attn_bwd_workspace_size(B, T, Hq, Hkv, D) > 8 * B * T * Hkv * D
    seg = np.zeros((B, T), np.int64)
    seg[:, 500:800] = -1
    seg[:, 800:] = 1
    check_all(sba, Case(B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, seg=seg, seed=135).forward())


def test_heads_in_parts_captured_and_at_once(sba):
    """The form with a merge, the same results eager, from a graph, and on two streams at once."""
    c = Case(T=1024, Hq=8, Hkv=1, D=64, seed=136).forward()
    want = [x.clone() for x in c.call(sba)]
    for _ in range(2):
        c.call(sba)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = c.call(sba)
    streams = [torch.cuda.Stream() for _ in range(2)]
    made = []
    torch.cuda.synchronize()
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                made.append(c.call(sba))
        g.replay()
    torch.cuda.synchronize()
    for got in (out, *made):
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    sba.check_error()


def test_full_size_sampled(sba):
    """4 x 16384 tokens, 32 heads over 8, window (1024, 0): the forward's own out and lse, dq on sampled
    tokens, dk and dv of whole key tiles from all rows that see them."""
    c = Case(B=4, T=16384, Hq=32, Hkv=8, doc=2048, pad=300, left=1024, right=0, seed=workloads.SEED_BASE + 4)
    c.out, c.lse = sba.blocksparse_attn_fwd(c.w.q, c.w.k, c.w.v, *c.dev_ints, *c.dev_bounds, 128, 128, **c.mask)
    got = c.call(sba)
    sba.check_error()
    q, k, v, out, lse, do = (to_np(x) for x in (c.w.q, c.w.k, c.w.v, c.out, c.lse, c.do))
    rng = np.random.default_rng(5)

    def sub(b, t0, t1, hkv):
        """Oracle on the rows t0 .. t1 of one KV head."""
        e = slice(0, t1)
        hs = slice(4 * hkv, 4 * hkv + 4)
        pick = lambda x, s: x[b:b + 1, e, s]  # noqa: E731
        ints = [x[b:b + 1, e] for x in c.ints]
        bnd = [np.asarray(x)[b:b + 1] for x in c.bounds]
        return oracle.blocksparse_attention_backward(
            pick(q, hs), pick(k, slice(hkv, hkv + 1)), pick(v, slice(hkv, hkv + 1)), pick(out, hs), lse[b:b + 1, e, hs],
            pick(do, hs), *ints, *bnd[:2], 128, 128, rows=[(0, t) for t in range(t0, t1)], magnitudes=True,
            lower_full=bnd[2], upper_full=bnd[3], **c.mask)

    for b, kt in ((0, 3), (1, 77), (2, 100), (3, 127), (3, 125)):
        hkv = int(rng.integers(0, 8))
        t0, t1 = kt * 128, min(16384, kt * 128 + 128 + 1025)
        ref = sub(b, t0, t1, hkv)
        ks = slice(kt * 128, kt * 128 + 128)
        for i, name in ((1, "dk"), (2, "dv")):
            check(to_np(got[i][b, ks, hkv]), ref[i][0, ks, 0], ref[3 + i][0, ks, 0], f"{name} tile {kt}")
        check(to_np(got[0][b, t0:t0 + 128, 4 * hkv:4 * hkv + 4]), ref[0][0, t0:t0 + 128], ref[3][0, t0:t0 + 128], f"dq block {kt}")


def test_a_wait_that_runs_out_is_reported(sba):
    c = Case(T=1024, seed=140).forward()
    want = [x.clone() for x in c.call(sba)]
    sba.check_error()
    sba.set_wait_timeout_cycles(100)
    try:
        c.call(sba)
        with pytest.raises(sba.SBAError) as e:
            sba.check_error()
    finally:
        sba.set_wait_timeout_cycles(0)
    assert e.value.code == -4 and "[blocksparse_attn_bwd d" in str(e.value), str(e.value)
    assert all(torch.equal(a, b) for a, b in zip(want, c.call(sba)))
    sba.check_error()
