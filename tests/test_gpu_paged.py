"""GPU parity of the paged-cache operators (append, attention over pages, selected-block
decode) against the fp64 oracle, at the sizes and masks where they can go wrong.

Tolerances, from the roundings on the way (half a step each: bf16 2^-8, fp16 2^-11, fp32
2^-24 of the value).  With A = sum p |v| / sum p: the probabilities are rounded once before
their products (fp16 over an e4m3 cache, bf16 over a bf16 one), which moves the output by
at most 2^-11 A or 2^-8 A; logits are fp32 sums of D products, off by at most D 2^-24 times
the sum of their magnitudes, which for the unit-normal inputs here (below 0.1 D after the
1 / sqrt(D) scale, a few units with larger keys) is below 2^-13 and moves the output by
2^-12 A; the output is rounded to bf16.  LSE: the same 2^-13 and a few fp32 roundings of
its own value.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def sba():
    import __graft_entry__

    __graft_entry__.build()
    import selected_block_attention_gb300 as m

    return m


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


class Cache:
    """Pools whose unowned slots and pages hold NaN, and tables whose unused entries are no
    page numbers."""

    def __init__(self, lens, Hkv, D, P, f8, seed, extra=2, joint=False, amp=0.5):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        lens = np.asarray(lens)
        used = -(-lens // P)
        pages = int(used.sum()) + extra
        W = max(1, int(used.max()))
        rng = np.random.default_rng(seed)
        order = rng.permutation(pages)
        table = np.full((len(lens), W), -7, dtype=np.int32)
        at = 0
        for b, u in enumerate(used):
            table[b, :u] = order[at:at + u]
            at += u
        dt = F8 if f8 else torch.bfloat16
        both = torch.zeros((pages, 2, Hkv, P, D), dtype=dt, device=DEV)
        self.k, self.v = (both[:, 0], both[:, 1]) if joint else (both[:, 0].contiguous(), both[:, 1].contiguous())
        self.ks = self.vs = None
        if f8:
            self.ks, self.vs = (torch.empty((pages, Hkv), device=DEV) for _ in range(2))
        for n, t in (("ks", self.k), ("vs", self.v)):
            x = torch.randn((pages, Hkv, P, D), generator=g, device=DEV)
            if f8:
                s = torch.exp2(torch.round(torch.randn((pages, Hkv), generator=g, device=DEV) * amp) - 7)
                setattr(self, n, s)
                t.copy_((x * 60).to(F8))
            else:
                t.copy_(x.to(torch.bfloat16))
        self.table = torch.from_numpy(table).to(DEV)
        self.lens = torch.from_numpy(lens.astype(np.int32)).to(DEV)
        self.P, self.D, self.Hkv, self.f8 = P, D, Hkv, f8
        own = torch.zeros((pages, P), dtype=torch.bool, device=DEV)
        for b, n in enumerate(lens):
            for j in range(used[b]):
                own[table[b, j], :min(P, n - j * P)] = True
        self.own = own
        for t in (self.k, self.v):
            x = t.view(torch.uint8) if f8 else t
            x.masked_fill_(~own[:, None, :, None], 0x7F if f8 else float("nan"))
        if f8:
            gone = ~own.any(1)
            self.ks[gone] = float("nan")
            self.vs[gone] = float("nan")

    def kw(self):
        return dict(k_scales=self.ks, v_scales=self.vs)

    def pool(self):
        return self.k, self.v, self.table, self.lens

    def host(self):
        return dict(k=np64(self.k.float()), v=np64(self.v.float()), ks=np64(self.ks), vs=np64(self.vs))

    def q(self, shape, seed):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def close(got, got_lse, ref, ref_lse, mag, f8, what="", lse_abs=2.0 ** -12):
    got, gl = np64(got).reshape(ref.shape), np64(got_lse).reshape(ref_lse.shape)
    none = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(gl), none), f"{what}: empty rows differ"
    assert (got[none] == 0).all(), f"{what}: empty rows must be zero"
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 if f8 else 2.0 ** -8) * mag + 2.0 ** -12 * mag + 1e-30
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} outside, worst {(np.abs(got - ref) / tol)[bad][:4]}"
    off = np.abs(gl[~none] - ref_lse[~none])
    assert (off <= lse_abs + 2.0 ** -21 * np.abs(ref_lse[~none])).all(), f"{what}: LSE off by {off.max()}"


# ------------------------------------------------------------------ attention
def check_attention(sba, c, n, Hq, seed, what="", **kw):
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q = c.q((int(cu[-1]), Hq, c.D), seed)
    out, lse = sba.paged_attention_fwd(q, *c.pool(), **c.kw(), cu_seqlens=torch.from_numpy(cu).to(DEV), **kw)
    sba.check_error()
    hk = {k: (np64(v) if isinstance(v, torch.Tensor) else v) for k, v in kw.items()}
    ref, rl, mag = oracle.paged_attention(np64(q), c.host(), c.table.cpu().numpy(), c.lens.cpu().numpy(), cu, **hk)
    close(out, lse, ref, rl, mag, c.f8, what)
    if len(set(n)) == 1 and n[0] > 0:  # the same rows without offsets
        q4 = q.view(len(n), n[0], Hq, c.D)
        o2, l2 = sba.paged_attention_fwd(q4 if n[0] > 1 else q, *c.pool(), **c.kw(), **kw)
        sba.check_error()
        close(o2, l2, ref, rl, mag, c.f8, what + " fixed")
    return out, lse


LENS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 0, 127, 129, 300, 1000]


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("G", [1, 4, 9, 16])
def test_one_token(sba, f8, D, P, G):
    c = Cache(LENS, 2, D, P, f8, 100 + P + D + G, joint=(G == 4))
    check_attention(sba, c, [1] * len(LENS), 2 * G, 7, what=f"f8={f8} D={D} P={P} G={G}")


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("left,right,cap,sinks", [(-1, 0, 0.0, 0), (0, 0, 0.0, 0), (100, 0, 0.0, 0), (100, 3, 2.0, 3),
                                                  (-1, 5, 50.0, 16), (511, -1, 0.0, 1), (31, 0, 5.0, 16), (20, 0, 0.0, 4)])
def test_windows_caps_sinks(sba, f8, left, right, cap, sinks):
    """Several tokens a row, counts from 0 to 21, some rows shorter than their tokens."""
    lens = [5, 40, 513, 0, 700, 1500, 64, 2, 33, 250]
    n = [5, 1, 7, 1, 21, 8, 0, 4, 33, 2]
    for P, D in ((16, 128), (64, 64)):
        c = Cache(lens, 2, D, P, f8, 300 + P)
        g = torch.Generator(device=DEV)
        g.manual_seed(4)
        bias = torch.randn((8, sinks), generator=g, device=DEV) if sinks else None
        check_attention(sba, c, n, 8, 8, what=f"{left} {right} {cap} {sinks} P={P}", window_left=left,
                        window_right=right, logits_soft_cap=cap, sink_bias=bias)
        if sinks:  # one bias for all heads
            check_attention(sba, c, n, 8, 9, what="shared bias", window_left=left, window_right=right,
                            logits_soft_cap=cap, sink_bias=bias[0].contiguous())


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("D,G", [(128, 4), (64, 3), (128, 20)])
def test_chunks(sba, f8, D, G):
    """Many tokens a row: whole prompts, chunks after a prefix, counts that fill no tile."""
    lens, n = [130, 700, 257, 40], [130, 200, 129, 1]
    c = Cache(lens, 2, D, 32, f8, 400 + G)
    check_attention(sba, c, n, 2 * G, 10, what="chunks", window_right=0)
    check_attention(sba, c, n, 2 * G, 10, what="chunks window", window_left=90, window_right=0)
    check_attention(sba, c, n, 2 * G, 10, what="chunks open")


@pytest.mark.parametrize("D", [64, 128])
def test_equal_chunks(sba, D):
    c = Cache([512, 300, 1000], 1, D, 64, True, 410)
    check_attention(sba, c, [256] * 3, 4, 11, what="equal chunks", window_right=0)
    check_attention(sba, c, [256] * 3, 4, 11, what="equal chunks cap", window_right=0, logits_soft_cap=9.0,
                    window_left=200)


@pytest.mark.parametrize("f8,P", [(True, 16), (True, 64), (True, 128), (False, 16), (False, 64)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("left,right,cap", [(-1, 0, 0.0), (70, 0, 0.0), (-1, 2, 7.0), (0, 0, 0.0)])
def test_many_rows(sba, f8, P, D, left, right, cap):
    """The kernel for many rows: rows without a sequence and without tokens, rows shorter
    than their tokens, one token among many, a group of 256 rows filled to one row."""
    lens, n = [0, 300, 64, 515, 40, 128, 1], [3, 129, 0, 1, 65, 128, 2]
    c = Cache(lens, 2, D, P, f8, 415 + P)
    check_attention(sba, c, n, 6, 24, what="many rows", window_left=left, window_right=right, logits_soft_cap=cap)


def test_many_rows_of_many_sequences(sba):
    """More batch rows than warps look at one by one, runs that hold several items."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 150, 100)
    n = np.minimum(rng.integers(0, 90, 100), np.maximum(lens, 1))
    c = Cache(lens, 1, 128, 32, True, 416)
    check_attention(sba, c, list(n), 4, 25, what="many sequences", window_right=0)


def test_many_rows_of_one_long_sequence(sba):
    """One item row cut into as many runs as there are."""
    c = Cache([20000], 1, 128, 64, True, 417)
    q = c.q((1, 40, 4, 128), 26)
    out, lse = sba.paged_attention_fwd(q, *c.pool(), **c.kw(), window_right=0)
    few, few_lse = sba.paged_attention_fwd(q[:, -1].contiguous(), *c.pool(), **c.kw())
    sba.check_error()
    ref, rl, mag = oracle.paged_attention(np64(q[:, -1]), c.host(), c.table.cpu().numpy(), [20000], [0, 1])
    close(out[:, -1], lse[:, -1], ref, rl, mag, True, "last token among 40")
    close(few, few_lse, ref, rl, mag, True, "last token alone")
    ref, rl, mag = oracle.paged_attention(np64(q[0, :1]), c.host(), c.table.cpu().numpy(), [20000 - 39], [0, 1])
    close(out[:, 0], lse[:, 0], ref, rl, mag, True, "first token")


@pytest.mark.parametrize("P", [16, 64])
def test_many_rows_scales_far_apart(sba, P):
    """As test_scales_far_apart, in the kernel for many rows."""
    c = Cache([200, 333], 2, 128, P, True, 418)
    rng = np.random.default_rng(8)
    shape = tuple(c.ks.shape)
    c.vs = torch.from_numpy((2.0 ** rng.integers(-60, 60, shape) * 1.37).astype(np.float32)).to(DEV)
    check_attention(sba, c, [60, 150], 8, 27, what="value scales", window_right=0)
    zero = torch.from_numpy(rng.random(shape[0]) < 0.5).to(DEV)
    c.k.view(torch.uint8)[zero] = 0
    c.v.view(torch.uint8)[zero] = 0
    c.ks[zero] = 2.0 ** -126
    c.vs = torch.where(zero[:, None], torch.full_like(c.vs, 2.0 ** -126), torch.full_like(c.vs, 0.02))
    check_attention(sba, c, [60, 150], 8, 27, what="zero pages", window_right=0)


def test_many_rows_give_pages_back_and_leave_rows_alone(sba):
    lens, left, n = [900, 400], 60, 100
    c = Cache(lens, 1, 128, 16, True, 419)
    for b, L in enumerate(lens):
        c.table[b, :max(0, L - n - left) // 16] = -1
    q = c.q((2 * n + 5, 4, 128), 28)
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device=DEV)
    out, lse = torch.full_like(q, 3.0), torch.full((2 * n + 5, 4), 5.0, device=DEV)
    sba.paged_attention_fwd(q, *c.pool(), **c.kw(), cu_seqlens=cu, window_left=left, window_right=0, out=out, lse=lse)
    sba.check_error()
    ref, rl, mag = oracle.paged_attention(np64(q)[:2 * n], c.host(), c.table.clamp(min=0).cpu().numpy(), lens,
                                          [0, n, 2 * n], window_left=left, window_right=0)
    close(out[:2 * n], lse[:2 * n], ref, rl, mag, True, "window pages")
    assert (out[2 * n:] == 3).all() and (lse[2 * n:] == 5).all()
    bad = c.table.clone()
    bad[0, -1] = c.k.shape[0]
    sba.paged_attention_fwd(q, c.k, c.v, bad, c.lens, **c.kw(), cu_seqlens=cu, window_left=left, window_right=0)
    with pytest.raises(sba.SBAError) as e:
        sba.check_error()
    assert e.value.code == -5 and "out of range" in str(e.value)


def test_caps_at_both_ends(sba):
    """A huge cap is none; a tiny one leaves the mean of the values (fp32 throughout)."""
    c = Cache([900, 77], 2, 128, 64, True, 420)
    q = c.q((2, 8, 128), 12)
    free = sba.paged_attention_fwd(q, *c.pool(), **c.kw())
    huge = sba.paged_attention_fwd(q, *c.pool(), **c.kw(), logits_soft_cap=1e20)
    sba.check_error()
    assert (free[0].double() - huge[0].double()).abs().max() <= 2.0 ** -7 * free[0].double().abs().max()
    assert (free[1] - huge[1]).abs().max() < 2.0 ** -12
    check_attention(sba, c, [1, 1], 8, 12, what="tiny cap", logits_soft_cap=1e-3)
    for cap in (256.0, 300.0):  # either side of where the formula changes
        check_attention(sba, c, [1, 1], 8, 12, what=f"cap {cap}", logits_soft_cap=cap)


def test_scales_far_apart(sba):
    """Value and key scales 2^-60 .. 2^60 apart from page to page (pages of 16, so a tile
    can hold two of them), all-zero pages with the smallest scale, scales that are no powers
    of two."""
    lens = [200, 64, 333]
    c = Cache(lens, 2, 128, 16, True, 430)
    rng = np.random.default_rng(6)
    shape = tuple(c.ks.shape)
    c.vs = torch.from_numpy((2.0 ** rng.integers(-60, 60, shape) * 1.37).astype(np.float32)).to(DEV)
    check_attention(sba, c, [1, 3, 2], 8, 13, what="value scales")
    c.ks = torch.from_numpy((2.0 ** rng.integers(-40, -6, shape) * 1.1).astype(np.float32)).to(DEV)
    check_attention(sba, c, [1, 3, 2], 8, 13, what="key scales")
    zero = torch.from_numpy(rng.random(shape[0]) < 0.5).to(DEV)
    c.k.view(torch.uint8)[zero] = 0
    c.v.view(torch.uint8)[zero] = 0
    c.ks[zero] = 2.0 ** -126
    c.vs = torch.where(zero[:, None], torch.full_like(c.vs, 2.0 ** -126), torch.full_like(c.vs, 0.02))
    check_attention(sba, c, [1, 3, 2], 8, 13, what="zero pages")


@pytest.mark.parametrize("size", [1e-20, 1e-6, 300.0, 1e5])
def test_large_and_small_queries(sba, size):
    """Queries outside fp16's range: they are scaled by powers of two on their way."""
    c = Cache([150, 40], 2, 128, 64, True, 440)
    c.ks.mul_(1.0 / max(size, 1.0))  # logits stay moderate
    q = (c.q((2, 8, 128), 14).float() * size).to(torch.bfloat16)
    out, lse = sba.paged_attention_fwd(q, *c.pool(), **c.kw())
    sba.check_error()
    ref, rl, mag = oracle.paged_attention(np64(q), c.host(), c.table.cpu().numpy(), c.lens.cpu().numpy(), [0, 1, 2])
    close(out, lse, ref, rl, mag, True, f"q of {size}")


@pytest.mark.parametrize("f8", [True, False])
def test_nan_in_own_values_reaches_only_its_row(sba, f8):
    c = Cache([70, 90], 1, 128, 32, f8, 450)
    pg = int(c.table[0, 1])
    (c.v.view(torch.uint8) if f8 else c.v)[pg, 0, 3] = 0x7F if f8 else float("nan")
    out, _ = sba.paged_attention_fwd(c.q((2, 4, 128), 15), *c.pool(), **c.kw())
    sba.check_error()
    assert out[0].isnan().all() and out[1].isfinite().all()
    q = c.q((2, 4, 128), 15)
    q[1, 2, 5] = float("nan")
    out, lse = sba.paged_attention_fwd(q, *c.pool(), **c.kw())
    sba.check_error()
    assert out[1, 2].isnan().all() and lse[1, 2].isnan() and out[1, [0, 1, 3]].isfinite().all()


def test_pages_left_of_the_window_may_be_given_back(sba):
    lens, left = [1000, 517, 90], 100
    for sinks in (0, 4):
        c = Cache(lens, 2, 128, 16, True, 460)
        for b, n in enumerate(lens):
            first = max(0, n - 3 - left) // 16  # page of the oldest visible key
            c.table[b, (1 if sinks else 0):first] = -1
        bias = torch.zeros((8, sinks), device=DEV) if sinks else None
        q = c.q((3, 3, 8, 128), 16)
        out, lse = sba.paged_attention_fwd(q, *c.pool(), **c.kw(), window_left=left, window_right=0, sink_bias=bias)
        sba.check_error()
        full = c.table.clamp(min=0).cpu().numpy()
        ref, rl, mag = oracle.paged_attention(np64(q).reshape(9, 8, 128), c.host(), full, lens, [0, 3, 6, 9],
                                              window_left=left, window_right=0, sink_bias=np64(bias))
        close(out, lse, ref, rl, mag, True, "window pages")


def test_rows_behind_the_last_sequence_stay(sba):
    c = Cache([70, 33], 2, 64, 32, True, 470)
    q = c.q((9, 4, 64), 17)
    cu = torch.tensor([0, 2, 5], dtype=torch.int32, device=DEV)
    out, lse = torch.full_like(q, 3.0), torch.full((9, 4), 5.0, device=DEV)
    sba.paged_attention_fwd(q, *c.pool(), **c.kw(), cu_seqlens=cu, out=out, lse=lse)
    sba.check_error()
    assert (out[5:] == 3).all() and (lse[5:] == 5).all() and not (out[:5] == 3).all(-1).any()


def test_bad_input_is_reported(sba):
    """Kernels check page numbers, lengths and offsets before they use them."""
    c = Cache([70, 33], 2, 64, 32, True, 480)
    q = c.q((2, 4, 64), 18)
    for change in ("page", "negative", "length", "offsets"):
        d = dict(table=c.table.clone(), lens=c.lens.clone(), cu=None)
        if change == "page":
            d["table"][0, 1] = c.k.shape[0]
        elif change == "negative":
            d["table"][1, 0] = -1
        elif change == "length":
            d["lens"][1] = 32 * d["table"].shape[1] + 1
        else:
            d["cu"] = torch.tensor([0, 2, 1], dtype=torch.int32, device=DEV)
        out, _ = sba.paged_attention_fwd(q, c.k, c.v, d["table"], d["lens"], **c.kw(), cu_seqlens=d["cu"])
        with pytest.raises(sba.SBAError) as e:
            sba.check_error()
        assert e.value.code == -5 and "paged attention" in str(e.value)
        kv = c.q((2, 2, 64), 19)
        k2, v2 = c.k.clone(), c.v.clone()
        sba.paged_kv_append(kv, kv, k2, v2, d["table"], d["lens"], k_scales=c.ks.clone(), v_scales=c.vs.clone(),
                            cu_seqlens=d["cu"])
        if change in ("length", "offsets"):  # the new tokens lie in other pages
            with pytest.raises(sba.SBAError) as e:
                sba.check_error()
            assert e.value.code == -5 and "append" in str(e.value)
    idx = torch.tensor([[[0, 1]] * 2] * 2, dtype=torch.int32, device=DEV)
    bad = c.table.clone()
    bad[0, 1] = c.k.shape[0]
    sba.nsa_select_paged_fwd(q, c.k, c.v, bad, c.lens, idx, 2, 32, **c.kw())
    with pytest.raises(sba.SBAError):
        sba.check_error()
    sba.check_error()


@pytest.mark.parametrize("B", [1, 130, 700])
def test_batches(sba, B):
    """More rows than threads in a block; runs that hold many short rows; one row cut into
    as many runs as there are."""
    rng = np.random.default_rng(B)
    lens = [9000] if B == 1 else rng.integers(0, 90, B)
    c = Cache(lens, 2, 64, 16, True, 490 + B)
    n = rng.integers(0, 3, B) if B > 1 else [1]
    check_attention(sba, c, list(n), 4, 20, what=f"B={B}")


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("B,n,G,D", [(5, 1, 4, 128), (300, 1, 4, 128), (5, 3, 3, 64), (130, 3, 9, 64), (300, 1, 16, 128)])
def test_equal_token_counts(sba, f8, B, n, G, D):
    """Few and many rows with as many tokens each: the kernel whose clusters share an item
    and the one whose runs are cut, with windows, caps and sinks."""
    rng = np.random.default_rng(B + n)
    c = Cache(rng.integers(0, 400, B), 2, D, 32, f8, 496 + B + G)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    bias = torch.randn((2 * G, 5), generator=g, device=DEV)
    for kw in (dict(window_right=0), dict(window_left=60, window_right=0, logits_soft_cap=4.0, sink_bias=bias),
               dict(window_left=33, window_right=2, sink_bias=bias[0].contiguous()), dict(logits_soft_cap=400.0)):
        check_attention(sba, c, [n] * B, 2 * G, 28, what=f"B={B} n={n} {list(kw)}", **kw)


@pytest.mark.parametrize("long", [5000, 30000])
def test_results_repeat(sba, long):
    c = Cache([long, 17, 900, 3333], 4, 128, 64, True, 495)
    q = c.q((4, 16, 128), 21)
    a, la = sba.paged_attention_fwd(q, *c.pool(), **c.kw())
    for _ in range(20):
        b, lb = sba.paged_attention_fwd(q, *c.pool(), **c.kw())
        assert torch.equal(a, b) and torch.equal(la, lb)
    q = c.q((4, 50, 16, 128), 21)
    a, la = sba.paged_attention_fwd(q, *c.pool(), **c.kw(), window_right=0)
    for _ in range(20):
        b, lb = sba.paged_attention_fwd(q, *c.pool(), **c.kw(), window_right=0)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_pool_beyond_32_bit_offsets(sba):
    """The row's pages are the last of pools of more than 2^32 bytes."""
    pages, P, Hkv, D = 70000, 64, 8, 128
    k = torch.empty((pages, Hkv, P, D), dtype=F8, device=DEV)
    v = torch.empty_like(k)
    assert k.numel() > 1 << 32
    small = Cache([200, 130], Hkv, D, P, True, 500)
    m = small.k.shape[0]
    for big, t in ((k, small.k), (v, small.v)):
        big[-m:].copy_(t)
    ks, vs = (torch.zeros((pages, Hkv), device=DEV) for _ in range(2))
    ks[-m:], vs[-m:] = small.ks, small.vs
    table = torch.where(small.table >= 0, small.table + (pages - m), small.table)
    q = small.q((2, 32, D), 22)
    a = sba.paged_attention_fwd(q, *small.pool(), **small.kw())
    b = sba.paged_attention_fwd(q, k, v, table, small.lens, k_scales=ks, v_scales=vs)
    idx = torch.tensor([2, 0, 1, 2], dtype=torch.int32, device=DEV).expand(2, Hkv, 4).contiguous()
    s = sba.nsa_select_paged_fwd(q, *small.pool(), idx, 4, 64, **small.kw())
    t = sba.nsa_select_paged_fwd(q, k, v, table, small.lens, idx, 4, 64, k_scales=ks, v_scales=vs)
    kv = small.q((2, Hkv, D), 23)
    sba.paged_kv_append(kv, kv, k, v, table, small.lens, k_scales=ks, v_scales=vs)
    sba.paged_kv_append(kv, kv, *small.pool(), **small.kw())
    sba.check_error()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(s[0], t[0])
    assert torch.equal(k[-m:].view(torch.uint8), small.k.view(torch.uint8))
    assert torch.equal(ks[-m:][small.own.any(1)], small.ks[small.own.any(1)])


# ------------------------------------------------------------------ selection
@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("D,P,bs,G,S", [(128, 64, 64, 16, 16), (64, 16, 32, 1, 5), (128, 128, 32, 4, 32),
                                        (64, 32, 128, 9, 1), (128, 16, 64, 8, 7)])
@pytest.mark.parametrize("Q", [1, 3])
def test_selection(sba, f8, D, P, bs, G, S, Q):
    """Ids out of range, after the token, negative and twice; counts from 0 past S; rows
    shorter than a block, than their tokens, and empty."""
    lens = [1, 31, 64, 65, 400, 0, 2, 1300]
    c = Cache(lens, 2, D, P, f8, 600 + P + G)
    rng = np.random.default_rng(S)
    B, NB = len(lens), -(-1300 // bs)
    idx = rng.integers(-2, NB + 2, (B, Q, 2, S))
    idx[:, :, 0, 0] = np.maximum(np.array(lens)[:, None] - 1, 0) // bs
    idx[rng.random(idx.shape) < 0.2] = 0
    cnt = rng.integers(0, S + 2, (B, Q, 2))
    ti = torch.from_numpy(idx.astype(np.int32)).to(DEV)
    tc = torch.from_numpy(cnt.astype(np.int32)).to(DEV)
    q = c.q((B, Q, 2 * G, D), 30)
    gate = torch.sigmoid(c.q((B, Q, 2 * G), 31).float()).to(torch.bfloat16)
    for counts, causal, g in ((tc, True, None), (S, True, gate), (tc, False, gate), (0, True, None)):
        args = (q, ti, counts, g)
        if Q == 1:  # the form without a token dimension
            args = (q[:, 0].contiguous(), ti[:, 0].contiguous(),
                    counts[:, 0].contiguous() if isinstance(counts, torch.Tensor) else counts,
                    None if g is None else g[:, 0].contiguous())
        out, lse = sba.nsa_select_paged_fwd(args[0], *c.pool(), args[1], args[2], bs, **c.kw(), causal=causal,
                                            g_slc=args[3])
        sba.check_error()
        ref, rl, mag = oracle.nsa_select_paged(np64(q), c.host(), c.table.cpu().numpy(), lens, idx,
                                               cnt if counts is tc else counts, bs, causal=causal, g_slc=np64(g))
        close(out, lse, ref, rl, mag, f8, f"selection {causal} {g is not None}")


def test_selection_of_every_block_is_attention(sba):
    c = Cache([500, 64, 129], 2, 128, 64, True, 650)
    q = c.q((3, 16, 128), 32)
    idx = torch.arange(8, dtype=torch.int32, device=DEV).flip(0).expand(3, 2, 8).contiguous()
    a = sba.nsa_select_paged_fwd(q, *c.pool(), idx, 8, 64, **c.kw())
    b = sba.paged_attention_fwd(q, *c.pool(), **c.kw())
    sba.check_error()
    assert (a[1] - b[1]).abs().max() < 2.0 ** -16
    # both lie within the fp16 rounding of their probabilities and one bf16 rounding
    assert ((a[0].double() - b[0].double()).abs() <= 2.0 ** -7 * b[0].double().abs() + 2.0 ** -8).all()


# ------------------------------------------------------------------ append
def angles(n, rot, base=10000.0):
    pos = torch.arange(n, dtype=torch.float64, device=DEV)[:, None]
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    return (pos * f).cos().float(), (pos * f).sin().float()


def check_append(sba, c, n, Hq, rot, interleaved, seed, fixed=None, size=1.0):
    """The call's tokens from slices of one array; everything the call must not touch stays
    bit for bit.  Values: fp32 rotation (three roundings of products and a sum), then one
    rounding to the cache's type; e4m3 subnormals have steps of 2^-9 of the scale."""
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    N, H, D = int(cu[-1]), c.Hkv, c.D
    both = (c.q((N + 2, (Hq + 2 * H) * D), seed).float() * size).to(torch.bfloat16)
    if fixed:
        both = both[:N]
    T = both.shape[0]
    q = both[:, :Hq * D].view(T, Hq, D)
    k = both[:, Hq * D:(Hq + H) * D].view(T, H, D)
    v = both[:, (Hq + H) * D:].view(T, H, D)
    cos, sin = angles(int(c.lens.max()) + 1, rot) if rot else (None, None)
    host = c.host()
    raw = [t.clone() for t in (c.k, c.v)]
    q_out = torch.full((T, Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)
    shape = (lambda t: t.unflatten(0, (len(n), fixed)) if fixed > 1 else t) if fixed else (lambda t: t)
    got = sba.paged_kv_append(shape(k), shape(v), *c.pool(), **c.kw(),
                              cu_seqlens=None if fixed else torch.from_numpy(cu).to(DEV), q=shape(q), cos=cos,
                              sin=sin, interleaved=interleaved, q_out=shape(q_out))
    sba.check_error()
    assert got.data_ptr() == q_out.data_ptr()
    table, lens = c.table.cpu().numpy(), c.lens.cpu().numpy()
    ref = {m: None if x is None else x.copy() for m, x in host.items()}
    oracle.paged_kv_append(ref, np64(k), np64(v), table, lens, cu, cos=np64(cos), sin=np64(sin), interleaved=interleaved)
    new = torch.zeros_like(c.own)
    pairs = np.zeros((N, H, D))
    for b in range(len(n)):
        for t in range(int(cu[b]), int(cu[b + 1])):
            p = int(lens[b]) - int(cu[b + 1]) + t
            if p < 0:
                assert (q_out[t] == 9).all()
                continue
            new[table[b, p // c.P], p % c.P] = True
            want = oracle.paged.rotate(np64(q[t]), p, np64(cos), np64(sin), interleaved)
            x = np.abs(np64(q[t]))
            off = np.abs(np64(q_out[t]) - want)
            assert (off <= 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * x.max()).all()
    assert (q_out[N:] == 9).all()
    after = c.host()
    for name, was in (("k", raw[0]), ("v", raw[1])):
        have = after[name]
        fresh = np.broadcast_to(new.cpu().numpy()[:, None, :, None], have.shape)
        slop = 2.0 ** -22 * float(np.abs(np64(k if name == "k" else v)).max()) if rot and name == "k" else 0.0
        if c.f8:
            s, r = after[name + "s"], ref[name + "s"]
            used = c.own.any(1).cpu().numpy()
            assert np.array_equal(s[used], r[used]), f"{name} scales"
            S = np.broadcast_to(r[:, :, None, None], have.shape)
            if not rot or name == "v":
                assert np.array_equal(have[used], ref[name][used], equal_nan=True), f"{name} codes"
            a, b = (have * S)[fresh], (ref[name] * S)[fresh]
            # two roundings of nearly the same number: a step apart where it lies between
            assert (np.abs(a - b) <= np.where(slop > 0, 2.0 ** -3 * np.abs(b) + 2.0 ** -9 * S[fresh], 0) + 1e-45).all()
            assert (a != b).mean() < 1e-3
        else:
            a, b = have[fresh], ref[name][fresh]
            assert (np.abs(a - b) <= 2.0 ** -8 * np.abs(b) + slop).all()
            keep = ~new[:, None, :, None].expand(was.shape)
            assert torch.equal((c.k if name == "k" else c.v)[keep].view(torch.int16), was[keep].view(torch.int16))


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("D,P,rot,interleaved", [(128, 64, 128, False), (64, 16, 64, True), (128, 128, 32, False),
                                                 (64, 32, 16, True), (128, 16, 0, False), (64, 128, 64, False)])
def test_append_ragged(sba, f8, D, P, rot, interleaved):
    """New tokens that begin a page, continue one, cross several; none; more than the row is
    long; token rows behind the last sequence."""
    lens = [1, 16, 130, 300, 17, 0, 64, 65, 3, 500]
    n = [1, 16, 5, 300, 2, 0, 1, 33, 6, 257]
    c = Cache(lens, 3, D, P, f8, 700 + P, joint=(P == 32))
    check_append(sba, c, n, 5, rot, interleaved, 40)


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("Q", [1, 2, 4, 5, 8, 9, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_append_fixed(sba, f8, Q, D):
    lens = [Q, Q + 15, Q + 16, 200, 64 + Q // 2, 128, 0, max(1, Q - 1)]
    c = Cache(lens, 2, D, 16 if Q == 5 else 64, f8, 720 + Q)
    check_append(sba, c, [Q] * len(lens), 4, D, False, 41, fixed=Q)


@pytest.mark.parametrize("B", [33, 700, 1500])
def test_append_many_ragged_rows(sba, B):
    """The row of a page is searched among the offsets, 32 at a time."""
    rng = np.random.default_rng(B)
    n = rng.integers(0, 4, B)
    c = Cache(rng.integers(0, 40, B) + n, 1, 64, 16, True, 735)
    check_append(sba, c, n, 1, 0, False, 46)


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("D,P,B", [(128, 16, 150), (128, 64, 150), (64, 32, 150), (64, 16, 600), (128, 16, 600)])
def test_append_long_rows_among_short(sba, f8, D, P, B):
    """Few tokens on average: pages with few and with many, first, last and in between, are
    different kernels' work; rows without tokens and rows shorter than theirs."""
    rng = np.random.default_rng(D + P)
    n = rng.integers(0, 3, B)
    n[[3, 40, 77, 120, B - 1]] = 512 // D + 1, 2 * P, P + 1, 3 * P - 1, 37
    n[60:70] = np.arange(10)
    lens = rng.integers(0, 40, B) + n
    lens[[9, 120, 65]] = 0, P + 2, 1
    c = Cache(lens, 2, D, P, f8, 736 + P)
    check_append(sba, c, n, 3, D, False, 49)


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("fixed", [None, 11])
def test_append_many_rows_of_several_tokens(sba, f8, fixed):
    """More rows than a block counts, more tokens than the kernel for few takes."""
    rng = np.random.default_rng(31)
    n = np.full(300, fixed) if fixed else rng.integers(0, 30, 300)
    c = Cache(rng.integers(0, 40, 300) + n, 1, 64, 16, f8, 745)
    check_append(sba, c, n, 1, 64, False, 50, fixed=fixed)


@pytest.mark.parametrize("n", [[1, 2, 0, 3], [40, 2, 0, 33], [1] * 200 + [50], [9] * 300])
def test_token_rows_ahead_of_the_first_sequence(sba, n):
    """Offsets that begin past 0: the token rows before belong to nobody either."""
    rng = np.random.default_rng(len(n))
    lens = rng.integers(0, 40, len(n)) + np.array(n)
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(DEV)
    res = []
    for ahead in (0, 70):
        c = Cache(lens, 2, 64, 16, True, 746)
        kv, q = c.q((sum(n), 2, 64), 51), c.q((sum(n), 8, 64), 52)
        pad = lambda t: torch.cat([torch.full((ahead, *t.shape[1:]), 7.0, dtype=t.dtype, device=DEV), t])
        sba.paged_kv_append(pad(kv), pad(kv), *c.pool(), **c.kw(), cu_seqlens=cu + ahead)
        out, lse = (torch.full((ahead + sum(n), 8, *d), 5.0, dtype=t, device=DEV) for d, t in (((64,), torch.bfloat16), ((), torch.float32)))
        sba.paged_attention_fwd(pad(q), *c.pool(), **c.kw(), cu_seqlens=cu + ahead, window_right=0, out=out, lse=lse)
        sba.check_error()
        assert (out[:ahead] == 5).all() and (lse[:ahead] == 5).all()
        # the token count may choose another kernel, so its results are held to the oracle's
        ref, rl, mag = oracle.paged_attention(np64(q), c.host(), c.table.cpu().numpy(), lens, cu.cpu().numpy(), window_right=0)
        close(out[ahead:], lse[ahead:], ref, rl, mag, True, f"ahead {ahead}")
        res.append((c.k.view(torch.uint8), c.v.view(torch.uint8), c.ks[c.own.any(1)]))
    assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("size", [1e-3, 40.0, 1e30])
def test_append_grows_and_keeps_scales(sba, size):
    """Tokens much larger (codes in the page move to the new scale), much smaller (it
    stays)."""
    c = Cache([20, 77, 130, 64], 2, 128, 64, True, 740)
    check_append(sba, c, [1, 1, 1, 1], 4, 0, False, 42, fixed=1, size=size)
    c = Cache([20, 77, 130, 70], 2, 64, 32, True, 741)
    check_append(sba, c, [3, 9, 1, 40], 4, 0, False, 43, size=size)


def test_append_special_values(sba):
    """Infinities become +-448 of a scale that the finite values set, NaN stays NaN, a page
    of zeros gets the smallest scale."""
    c = Cache([3, 2], 1, 64, 16, True, 750)
    k = torch.zeros((5, 1, 64), dtype=torch.bfloat16, device=DEV)
    k[0, 0, 0], k[1, 0, 1], k[2, 0, 2], k[2, 0, 3] = float("inf"), float("-inf"), float("nan"), 3.0
    cu = torch.tensor([0, 3, 5], dtype=torch.int32, device=DEV)
    sba.paged_kv_append(k, k, *c.pool(), **c.kw(), cu_seqlens=cu)
    sba.check_error()
    pg = c.table[:, 0].long()
    assert c.ks[pg, 0].tolist() == [2.0 ** -7, 2.0 ** -126]
    x = c.k[pg[0], 0].float()
    assert x[0, 0] == 448 and x[1, 1] == -448 and x[2, 2].isnan() and x[2, 3] == 3 * 128
    assert (c.k[pg[1], 0, :2].float() == 0).all()


def test_append_rotates_in_place(sba):
    c = Cache([30, 50], 2, 128, 32, True, 760)
    cos, sin = angles(64, 128)
    q, kv = c.q((2, 8, 128), 44), c.q((2, 2, 128), 45)
    want = sba.paged_kv_append(kv, kv, *c.pool(), **c.kw(), q=q, cos=cos, sin=sin)
    got = sba.paged_kv_append(kv, kv, *c.pool(), **c.kw(), q=q, cos=cos, sin=sin, q_out=q)
    sba.check_error()
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)


def test_waits_of_the_many_row_kernel_run_out(sba):
    """With a limit far below a wait's normal time the launch returns, is reported with its
    place, and the next launch on the same context is right: nothing hangs, every wait and
    drain is bounded."""
    c = Cache([700, 300], 2, 128, 64, True, 780)
    q = c.q((2, 200, 8, 128), 47)
    want = sba.paged_attention_fwd(q, *c.pool(), **c.kw(), window_right=0)
    sba.check_error()
    try:
        sba.set_wait_timeout_cycles(100)
        sba.paged_attention_fwd(q, *c.pool(), **c.kw(), window_right=0)
        with pytest.raises(sba.SBAError) as e:
            sba.check_error()
        assert e.value.code == -4 and "paged attention chunk role" in str(e.value)
    finally:
        sba.set_wait_timeout_cycles(0)
    got = sba.paged_attention_fwd(q, *c.pool(), **c.kw(), window_right=0)
    sba.check_error()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ as they are used
@pytest.mark.parametrize("f8", [True, False])
def test_prompt_then_decode(sba, f8):
    """A prompt in two chunks, then tokens one by one through one captured graph: append,
    attention, selection.  Every step against the oracle on the cache as it stands."""
    B, H, G, D, P, steps = 3, 2, 4, 128, 16, 20
    room = 200
    c = Cache([room] * B, H, D, P, f8, 800)
    (c.k.view(torch.uint8) if f8 else c.k).fill_(0x7F if f8 else float("nan"))
    (c.v.view(torch.uint8) if f8 else c.v).fill_(0x7F if f8 else float("nan"))
    cos, sin = angles(room, D)
    have = np.zeros(B, dtype=int)
    for n in ([50, 0, 77], [13, 90, 32]):
        cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        have = have + np.array(n)
        c.lens.copy_(torch.from_numpy(have.astype(np.int32)))
        tcu = torch.from_numpy(cu).to(DEV)
        q, k, v = c.q((cu[-1], H * G, D), 50), c.q((cu[-1], H, D), 51), c.q((cu[-1], H, D), 52)
        qr = sba.paged_kv_append(k, v, *c.pool(), **c.kw(), cu_seqlens=tcu, q=q, cos=cos, sin=sin)
        out, lse = sba.paged_attention_fwd(qr, *c.pool(), **c.kw(), cu_seqlens=tcu, window_right=0)
        sba.check_error()
        ref, rl, mag = oracle.paged_attention(np64(qr), c.host(), c.table.cpu().numpy(), have, cu, window_right=0)
        close(out, lse, ref, rl, mag, f8, "prompt")

    qs, ks, vs = (torch.empty((B, h, D), dtype=torch.bfloat16, device=DEV) for h in (H * G, H, H))
    idx = torch.empty((B, H, 3), dtype=torch.int32, device=DEV)
    ws = torch.empty(sba.paged_attention_workspace_size(B, B, H * G, H, D), dtype=torch.uint8, device=DEV)
    qr, out, sel = (torch.empty_like(qs) for _ in range(3))
    lse, sel_lse = (torch.empty((B, H * G), device=DEV) for _ in range(2))

    def step():
        sba.paged_kv_append(ks, vs, *c.pool(), **c.kw(), q=qs, cos=cos, sin=sin, q_out=qr)
        sba.paged_attention_fwd(qr, *c.pool(), **c.kw(), out=out, lse=lse, workspace=ws)
        sba.nsa_select_paged_fwd(qr, *c.pool(), idx, 3, 32, **c.kw(), out=sel, lse=sel_lse)

    def load(t):
        for i, x in enumerate((qs, ks, vs)):
            x.copy_(c.q(x.shape, 900 + 10 * t + i) * (1 + t % 5))
        c.lens.copy_(torch.from_numpy(have.astype(np.int32)))
        idx.copy_(torch.stack([torch.as_tensor([(n - 1) // 32, 0, t % ((n - 1) // 32 + 1)]) for n in have])
                  [:, None].expand(B, H, 3))

    graph = None
    for t in range(steps):
        have = have + 1
        load(t)
        if t == 1:
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                step()
        graph.replay() if graph else step()
        sba.check_error()
        host, table = c.host(), c.table.cpu().numpy()
        ref, rl, mag = oracle.paged_attention(np64(qr), host, table, have, np.arange(B + 1))
        close(out, lse, ref, rl, mag, f8, f"step {t}")
        ref, rl, mag = oracle.nsa_select_paged(np64(qr)[:, None], host, table, have, idx.cpu().numpy()[:, None], 3, 32)
        close(sel, sel_lse, ref[:, 0], rl[:, 0], mag[:, 0], f8, f"selection {t}")


def test_two_streams(sba):
    """Calls that overlap, each with its own workspace, give what they give alone."""
    cs = [Cache([30000, 900, 17], 4, 128, 64, True, 820 + i) for i in range(2)]
    qs = [c.q((3, 16, 128), 60 + i) for i, c in enumerate(cs)]
    alone = [sba.paged_attention_fwd(q, *c.pool(), **c.kw()) for c, q in zip(cs, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(sba.paged_attention_workspace_size(3, 3, 16, 4, 128), dtype=torch.uint8, device=DEV) for _ in range(2)]
    got = [None, None]
    for _ in range(30):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = sba.paged_attention_fwd(qs[i], *cs[i].pool(), **cs[i].kw(), workspace=ws[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i][0], alone[i][0]) and torch.equal(got[i][1], alone[i][1])


def test_workspace_needs_no_initialisation_and_may_be_shared_in_order(sba):
    c = Cache([30000, 900, 17], 4, 128, 64, True, 830)
    q = c.q((3, 16, 128), 61)
    ws = torch.full((sba.paged_attention_workspace_size(3, 3, 16, 4, 128),), 0xFF, dtype=torch.uint8, device=DEV)
    want = sba.paged_attention_fwd(q, *c.pool(), **c.kw())
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sba.paged_attention_fwd(q, *c.pool(), **c.kw(), workspace=ws, window_left=(-1, 200)[i]))
        graphs.append(g)
    for _ in range(5):
        for g in graphs:
            g.replay()
    sba.check_error()
    assert torch.equal(outs[0][0], want[0])
    win = sba.paged_attention_fwd(q, *c.pool(), **c.kw(), window_left=200)
    assert torch.equal(outs[1][0], win[0])
