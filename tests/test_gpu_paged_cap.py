"""Accuracy of the soft cap near zero, on the GPU: a row of one key has its logit as LSE."""

import numpy as np
import pytest
import torch

from tests.test_gpu_paged import DEV, Cache, np64, sba  # noqa: F401 (sba is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [0.5, 5.0, 50.0, 200.0, 256.0, 300.0, 3e4])
@pytest.mark.parametrize("mixed", [False, True])
def test_capped_logits_keep_their_relative_error(sba, f8, D, cap, mixed):  # noqa: F811
    """Query and key are single elements, so <q, k> is one exact product.  What follows: the
    scale, the quotient with the cap, log2(e) cap and its way back, seven roundings of 2^-24;
    and a series (next term below 2^-22), or 1 - 2 / (1 + e) with an exponential of 2^-22, a
    reciprocal of 2^-23 and a sum: 1.15 * 2^-22 against tanh >= 0.124, below 2^-18.7.  Together
    less than 2^-18 of the value.  `mixed`: rows far from zero beside the near ones."""
    x = torch.cat([torch.logspace(-6, -0.8, 24), torch.logspace(-0.5, 1, 8) if mixed else torch.empty(0)]) * cap
    x = torch.cat([x, -x]).to(torch.bfloat16)
    B = x.numel()
    c = Cache([1] * B, 2, D, 16, f8, 1200)
    page = c.table[:, 0].long()
    one = torch.zeros((B, 2, D), device=DEV)
    one[..., 5] = 1.0
    c.k[page, :, 0] = (one * (128 if f8 else 1)).to(c.k.dtype)
    if f8:
        c.ks[page] = 2.0 ** -7
    q = torch.zeros((B, 8, D), dtype=torch.bfloat16, device=DEV)
    q[..., 5] = x.to(DEV)[:, None]
    want = cap * np.tanh(np64(x) / cap)[:, None]
    cu = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    for kw in ({}, dict(cu_seqlens=cu)):
        _, lse = sba.paged_attention_fwd(q, *c.pool(), **c.kw(), softmax_scale=1.0, logits_soft_cap=cap, **kw)
        sba.check_error()
        off = np.abs(np64(lse) - want) / np.abs(want)
        assert off.max() <= 2.0 ** -18, f"{off.max()} at {np64(x)[off.max(1).argmax()]}"
