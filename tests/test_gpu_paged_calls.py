"""Calls of the paged entry points that a server makes and no other test does: many heads a
KV head, batches in which nobody has a token, one captured call of many rows for batches that
change, rows as long as their table.  Tolerances as in test_gpu_paged.py."""

import numpy as np
import pytest
import torch

from tests.test_gpu_paged import DEV, Cache, check_attention, close, np64, sba  # noqa: F401 (sba is a fixture)
from tests.test_gpu_paged_runs import plain64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [32, 71, 128, 300])
def test_many_heads_of_one_kv_head(sba, f8, D, G):  # noqa: F811
    """One token a row: groups of 16 heads of a few rows, and with more than 96 heads the
    kernel for many rows, whose items a token's heads may not fill or may pass."""
    lens = [1, 64, 700, 0, 130]
    c = Cache(lens, 1, D, 64, f8, 1400 + G)
    check_attention(sba, c, [1] * 5, G, 90, what=f"G={G}", window_right=0)
    check_attention(sba, c, [2, 1, 3, 1, 0], G, 91, what=f"G={G} ragged", window_left=50, window_right=0)
    bias = c.q((G, 3), 92).float()
    check_attention(sba, c, [1] * 5, G, 93, what=f"G={G} sinks", window_left=60, window_right=0, sink_bias=bias)


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("N", [3, 700])
def test_nobody_has_a_token(sba, f8, N):  # noqa: F811
    """All token rows belong to nobody: nothing is read or written."""
    c = Cache([40, 0, 7], 2, 64, 16, f8, 1410)
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)
    before = [t.clone() for t in (c.k, c.v)]
    q, kv = c.q((N, 8, 64), 94), c.q((N, 2, 64), 95)
    out, lse = torch.full_like(q, 3.0), torch.full((N, 8), 5.0, device=DEV)
    for at in (0, N):
        sba.paged_attention_fwd(q, *c.pool(), **c.kw(), cu_seqlens=cu + at, out=out, lse=lse)
        qo = sba.paged_kv_append(kv, kv, *c.pool(), **c.kw(), cu_seqlens=cu + at, q=q, q_out=torch.full_like(q, 3.0))
        sba.check_error()
        assert (out == 3).all() and (lse == 5).all() and (qo == 3).all()
        for t, b in zip((c.k, c.v), before):
            assert torch.equal(t.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("f8,P", [(True, 16), (True, 64), (False, 32)])
def test_captured_chunks_of_changing_batches(sba, f8, P):  # noqa: F811
    """One captured call of many rows: lengths and offsets change between its replays, slots
    empty themselves and fill again."""
    rng = np.random.default_rng(3)
    B, N, G, room = 24, 2400, 4, 1200
    c = Cache([room] * B, 8, 128, P, f8, 1420)
    q = c.q((N, 8 * G, 128), 96)
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    out, lse = torch.empty_like(q), torch.empty((N, 8 * G), device=DEV)
    ws = torch.empty(sba.paged_attention_workspace_size(B, N, 8 * G, 8, 128), dtype=torch.uint8, device=DEV)
    assert N * G > 96 * B

    def call():
        sba.paged_attention_fwd(q, *c.pool(), **c.kw(), cu_seqlens=cu, window_right=0, out=out, lse=lse, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for turn in range(5):
        lens, n = rng.integers(1, room, B), rng.integers(0, 200, B)
        gone = rng.random(B) < (0.0, 0.2, 0.5, 0.9, 1.0)[turn]
        lens[gone] = 0
        n[gone] = np.minimum(n[gone], rng.integers(0, 3, int(gone.sum())))
        off = np.minimum(np.concatenate([[0], np.cumsum(n)]), N).astype(np.int32)
        c.lens.copy_(torch.from_numpy(lens.astype(np.int32)))
        cu.copy_(torch.from_numpy(off))
        out.fill_(3.0)
        lse.fill_(5.0)
        graph.replay()
        sba.check_error()
        e = int(off[-1])
        assert (out[e:] == 3).all() and (lse[e:] == 5).all()
        ref, rl, mag = plain64(q[:e], c, off, -1, 0)
        close(out[:e], lse[:e], ref, rl, mag, f8, f"turn {turn}")


@pytest.mark.parametrize("n", [1, 70])
def test_rows_as_long_as_their_table(sba, n):  # noqa: F811
    c = Cache([256, 256], 2, 128, 128, True, 1430)
    assert c.table.shape[1] * c.P == 256
    check_attention(sba, c, [n, n], 8, 97, what="full tables", window_right=0)
