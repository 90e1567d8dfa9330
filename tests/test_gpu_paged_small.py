"""GPU parity of paged attention where logits all but vanish: small queries, pages of zeros
with the smallest scale, masked keys among them.  Tolerances as in test_gpu_paged.py."""

import numpy as np
import pytest
import torch

import oracle
from tests.test_gpu_paged import DEV, Cache, close, np64, sba  # noqa: F401 (sba is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,G", [(64, 4), (128, 4)])
@pytest.mark.parametrize("P", [16, 64, 128])
@pytest.mark.parametrize("size", [2.0 ** -9, 1e-20, 1e-37])
@pytest.mark.parametrize("left", [-1, 90])
def test_small_queries_over_zero_pages(sba, D, G, P, size, left):  # noqa: F811
    """Pages of zero keys, whose scale is the smallest, under a causal diagonal and a window's
    edge, in the kernel for many rows: the factor of their logits is far below fp32's range."""
    lens, n = [130, 700, 64], [130, 200, 64]
    c = Cache(lens, 2, D, P, True, 1100 + P)
    zero = torch.from_numpy(np.random.default_rng(9).random(c.ks.shape[0]) < 0.5).to(DEV)
    zero[c.table[0, 0].item()] = zero[c.table[1, -1].item()] = True
    own = c.own & zero[:, None]
    c.k.view(torch.uint8).masked_fill_(own[:, None, :, None], 0)
    c.ks[zero & c.own.any(1)] = 2.0 ** -126
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    assert int(cu[-1]) * G > 96 * len(n)  # of the many-row kernel
    q = (c.q((int(cu[-1]), 2 * G, D), 72).float() * size).to(torch.bfloat16)
    out, lse = sba.paged_attention_fwd(q, *c.pool(), **c.kw(), cu_seqlens=torch.from_numpy(cu).to(DEV),
                                       window_left=left, window_right=0)
    sba.check_error()
    ref, rl, mag = oracle.paged_attention(np64(q), c.host(), c.table.cpu().numpy(), lens, cu, window_left=left,
                                          window_right=0)
    close(out, lse, ref, rl, mag, True, f"q of {size}")
