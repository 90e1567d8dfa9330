"""GPU parity of paged attention where slots that no query sees lie beside visible ones:
they may hold anything, and pages without a visible key may be given back.  Tolerances as in
test_gpu_paged.py."""

import pytest
import torch

from tests.test_gpu_paged import DEV, Cache, check_attention, sba  # noqa: F401 (sba is a fixture)

pytestmark = pytest.mark.gpu

# first key of the first query's window
STARTS = [0, 1, 5, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 79, 95, 100, 127, 130, 200]


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("sinks", [0, 1, 4, 16])
@pytest.mark.parametrize("left,n", [(20, 1), (70, 3)])
def test_between_the_sinks_and_the_window(sba, f8, D, P, sinks, left, n):  # noqa: F811
    """Every slot from the sinks to the window holds NaN, pages that lie there wholly are gone
    from the table, and page 0 of the pool, which a reader of such an entry might fall back
    to, is all NaN.  Both kernels: with and without offsets."""
    lens = [lo + left + n for lo in STARTS] + [n]
    c = Cache(lens, 2, D, P, f8, 1000 + P + D)
    nan = 0x7F if f8 else float("nan")
    for pool in ("k", "v"):  # a page ahead of the others
        t = getattr(c, pool)
        grown = torch.empty((t.shape[0] + 1, *t.shape[1:]), dtype=t.dtype, device=DEV)
        grown[1:] = t
        raw = grown.view(torch.uint8) if f8 else grown
        raw[0] = nan
        setattr(c, pool, grown)
        if f8:
            s = getattr(c, pool + "s")
            setattr(c, pool + "s", torch.cat([torch.full_like(s[:1], float("nan")), s]))
    c.table += 1
    for b, lo in enumerate(STARTS):
        for key in range(sinks, lo):
            j, off = divmod(key, P)
            for t in (c.k, c.v):
                (t.view(torch.uint8) if f8 else t)[int(c.table[b, j]), :, off] = nan
    for b, lo in enumerate(STARTS):
        c.table[b, -(-sinks // P):lo // P] = -1
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    bias = torch.randn((8, sinks), generator=g, device=DEV) if sinks else None
    check_attention(sba, c, [n] * len(lens), 8, 71, what=f"sinks {sinks}", window_left=left, window_right=0, sink_bias=bias)
