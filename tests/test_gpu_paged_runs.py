"""GPU parity of the many-row kernel of paged attention where a CTA's run holds more items
than the kernel has slots for them: long runs, items without keys between them.  Tolerances
as in test_gpu_paged.py."""

import numpy as np
import pytest
import torch

from tests._paged_line import SLOTS, runs, waits_for_itself
from tests.test_gpu_paged import DEV, Cache, close, np64, sba  # noqa: F401 (sba is a fixture)

pytestmark = pytest.mark.gpu


def plain64(q, c, cu, left=-1, right=-1):
    """Attention of a whole batch in 64 bits on the GPU: (out, lse, sum of p |v|)."""
    lens, G = c.lens.tolist(), q.shape[1] // c.Hkv
    out, mag = (torch.zeros(q.shape, dtype=torch.float64, device=DEV) for _ in range(2))
    lse = torch.full(q.shape[:2], -torch.inf, dtype=torch.float64, device=DEV)
    for b, L in enumerate(lens):
        t0, t1 = int(cu[b]), int(cu[b + 1])
        if t0 == t1 or L == 0:
            continue
        pages = c.table[b, :-(-L // c.P)].long()
        pos = torch.arange(L - (t1 - t0), L, device=DEV).repeat_interleave(G)[:, None]
        key = torch.arange(L, device=DEV)
        see = torch.ones((pos.shape[0], L), dtype=torch.bool, device=DEV)
        if left >= 0:
            see &= key >= pos - left
        if right >= 0:
            see &= key <= pos + right
        for h in range(c.Hkv):
            k, v = (p[pages, h].double() * (1.0 if s is None else s[pages, h].double()[:, None, None])
                    for p, s in ((c.k, c.ks), (c.v, c.vs)))
            k, v = (x.reshape(-1, c.D)[:L] for x in (k, v))
            hs = slice(h * G, (h + 1) * G)
            s = (q[t0:t1, hs].double().reshape(-1, c.D) @ k.T) * c.D ** -0.5
            s = torch.where(see, s, -torch.inf)
            m = s.amax(1, keepdim=True)
            some = torch.isfinite(m[:, 0])
            p = torch.where(see, (s - m.clamp(min=-1e300)).exp(), 0.0)
            l = p.sum(1, keepdim=True)
            for x, y in ((out, p @ v), (mag, p @ v.abs())):
                x[t0:t1, hs] = torch.where(some[:, None], y / l, 0.0).view(t1 - t0, G, c.D)
            lse[t0:t1, hs] = torch.where(some, m[:, 0] + l[:, 0].log(), -torch.inf).view(t1 - t0, G)
    return np64(out), np64(lse), np64(mag)


def check(sba, c, n, G, what, left=-1, right=-1):
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    assert int(cu[-1]) * G > 96 * len(n)  # of the many-row kernel, whatever the cache
    q = c.q((int(cu[-1]), c.Hkv * G, c.D), 70)
    out, lse = sba.paged_attention_fwd(q, *c.pool(), **c.kw(), cu_seqlens=torch.from_numpy(cu).to(DEV),
                                       window_left=left, window_right=right)
    sba.check_error()
    close(out, lse, *plain64(q, c, cu, left, right), c.f8, what)


def most(parts, empty):
    return max(sum(t > 0 or empty for t in p) for p in parts)


@pytest.mark.parametrize("f8,P", [(True, 16), (True, 64), (False, 16), (False, 128)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("left", [-1, 100])
def test_runs_of_more_items_than_slots(sba, f8, P, D, left):  # noqa: F811
    """Dozens of ragged rows, some slots of the batch empty with and without tokens, in the
    middle and at the end."""
    rng = np.random.default_rng(1)
    B = 48
    lens, n = rng.integers(100, 900, B), rng.integers(20, 150, B)
    lens[[5, 6, 20, 33, 47]] = 0
    n[[20, 33]] = 1
    n[[5, 6, 47]] = 130, 64, 200
    parts = runs(lens, n, 4, 8, left, 0)
    assert most(parts, False) > SLOTS
    if left < 0:
        assert any(waits_for_itself(p, True) for p in parts)
    c = Cache(lens, 8, D, P, f8, 900 + P + D)
    check(sba, c, n, 4, "long runs", left, 0)


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("lens,n,right", [([8192, 8192, 0, 8192, 8192], [512, 512, 1, 512, 512], -1),
                                          ([100, 8192], [4000, 512], 0)])
def test_items_without_keys_among_long_ones(sba, f8, lens, n, right):  # noqa: F811
    """A slot without a sequence between long rows; a row much shorter than its tokens, whose
    first groups see nothing."""
    parts = runs(lens, n, 4, 8, -1, right)
    assert any(waits_for_itself(p, True) for p in parts)
    c = Cache(lens, 8, 128, 64, f8, 910)
    check(sba, c, n, 4, "items without keys", -1, right)


@pytest.mark.parametrize("f8,P", [(True, 16), (True, 64), (False, 32)])
def test_drafts_with_empty_slots(sba, f8, P):  # noqa: F811
    """Drafts of grouped heads: every eleventh slot of the batch holds no sequence."""
    B = 60
    rng = np.random.default_rng(7)
    lens, n = rng.integers(8, 6000, B), rng.integers(6, 13, B)
    lens[5::11], n[5::11] = 0, 1
    parts = runs(lens, n, 16, 8, -1, 0)
    assert most(parts, True) > SLOTS
    c = Cache(lens, 8, 128, P, f8, 920)
    check(sba, c, n, 16, "drafts", -1, 0)


def test_only_items_without_keys(sba):  # noqa: F811
    """Nothing but slots without a sequence, and rows of which no token has a position."""
    c = Cache([0, 0, 1, 0], 2, 64, 16, True, 930)
    check(sba, c, [300, 64, 260, 1], 8, "nothing", -1, 0)
