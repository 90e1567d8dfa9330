"""What an append must not touch, bit for bit: codes and scales of pages that get no token,
slots that get none, and the codes that a page holds already (moved where its scale grows).
Keys are rotated here, so the written slots' own values are test_gpu_paged.py's matter."""

import numpy as np
import pytest
import torch

import oracle
from tests.test_gpu_paged import DEV, F8, Cache, angles, np64, sba  # noqa: F401 (sba is a fixture)

pytestmark = pytest.mark.gpu


def raw(t):
    return t.view(torch.uint8) if t.dtype == F8 else t.view(torch.int16)


def check_rest(sba, c, n, rot, size, fixed=None):
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    N, D = int(cu[-1]), c.D
    k, v = ((c.q((N, c.Hkv, D), 80 + i).float() * size).to(torch.bfloat16) for i in range(2))
    cos, sin = angles(int(c.lens.max()) + 1, rot)
    before = [t.clone() for t in (c.k, c.v)]
    scales = [t.clone() for t in (c.ks, c.vs)] if c.f8 else None
    table, lens = c.table.cpu().numpy(), c.lens.cpu().numpy()
    new = torch.zeros_like(c.own)                 # slots written
    held = torch.zeros_like(c.own)                # slots of those pages held already
    for b in range(len(n)):
        for p in range(max(0, int(lens[b]) - int(n[b])), int(lens[b])):
            new[table[b, p // c.P], p % c.P] = True
        first = max(0, int(lens[b]) - int(n[b]))
        if n[b] and first < lens[b]:
            held[table[b, first // c.P], :first % c.P] = True
    if fixed:
        k, v = (t.view(len(n), fixed, c.Hkv, D) for t in (k, v))
    sba.paged_kv_append(k, v, *c.pool(), **c.kw(), cu_seqlens=None if fixed else torch.from_numpy(cu).to(DEV),
                        cos=cos, sin=sin)
    sba.check_error()
    touched = new.any(1)
    for i, t in enumerate((c.k, c.v)):
        keep = ~new[:, None, :, None].expand(t.shape)
        if not c.f8:
            assert torch.equal(raw(t)[keep], raw(before[i])[keep])
            continue
        s, was = (c.ks, c.vs)[i], scales[i]
        assert torch.equal(s[~touched].view(torch.int32), was[~touched].view(torch.int32)), "scales of other pages"
        grown = (s != was)[:, :, None, None] & held[:, None, :, None] & touched[:, None, None, None]
        grown = grown.expand(t.shape)
        rest = keep & ~grown
        assert torch.equal(raw(t)[rest], raw(before[i])[rest]), "codes that stay"
        old = np64(before[i].float())
        ratio = np64(was / s)[:, :, None, None]
        g = grown.cpu().numpy()
        want = oracle.paged.round_e4m3(np.where(g, old * ratio, 0.0))
        assert np.array_equal(np64(t.float())[g], want[g]), "codes that moved"
        if size > 10:
            assert g.any()  # else nothing grew and the case shows nothing


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("D,P,rot", [(128, 64, 128), (64, 16, 32), (128, 16, 64), (64, 128, 64)])
@pytest.mark.parametrize("size", [0.01, 1.0, 40.0])
def test_append_leaves_the_rest(sba, f8, D, P, rot, size):  # noqa: F811
    """Ragged rows that begin, continue and cross pages, beside pages of nobody."""
    lens = [1, 16, 130, 300, 17, 0, 64, 65, 3, 500, 200]
    n = [1, 16, 5, 250, 2, 0, 1, 33, 6, 257, 0]
    c = Cache(lens, 3, D, P, f8, 1300 + P, extra=5, joint=(P == 64))
    check_rest(sba, c, n, rot, size)


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("Q,D", [(1, 128), (3, 64), (8, 128), (40, 128)])
@pytest.mark.parametrize("size", [0.01, 40.0])
def test_append_of_equal_counts_leaves_the_rest(sba, f8, Q, D, size):  # noqa: F811
    lens = [Q, Q + 15, Q + 16, 200, 64 + Q // 2, 128, Q + 1, 99 + Q]
    c = Cache(lens, 2, D, 32, f8, 1320 + Q, extra=5)
    check_rest(sba, c, [Q] * len(lens), D, size, fixed=Q)


def test_append_of_few_tokens_to_many_rows_leaves_the_rest(sba):  # noqa: F811
    """Both kernels of a ragged call, runs found by search."""
    rng = np.random.default_rng(5)
    n = rng.integers(0, 4, 600)
    n[[7, 300, 599]] = 40, 21, 9
    c = Cache(rng.integers(0, 60, 600) + n, 2, 64, 16, True, 1340, extra=9)
    check_rest(sba, c, n, 64, 40.0)
