"""Refusals of the paged-cache entry points: the C ABI's checks come before any launch, and
the Python binding's before the library (no GPU)."""

import ctypes

import pytest
import torch

FAKE = 0x10000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from selected_block_attention_gb300 import _build
    import selected_block_attention_gb300 as sba

    _build.build()
    return sba.load_library()


POOL = dict(k_pages=FAKE, v_pages=FAKE, k_scales=FAKE, v_scales=FAKE, page_stride=2 * 64 * 128, num_pages=4,
            page_size=64, page_table=FAKE, table_width=8, seq_lens=FAKE)


def append(lib, **kw):
    a = dict(k=FAKE, ks=256, v=FAKE, vs=256, q=FAKE, qs=1024, qo=FAKE, qos=1024, cos=FAKE, sin=FAKE, rot=128,
             max_pos=512, inter=0, **POOL, cu=None, B=3, Q=2, N=6, Hq=8, Hkv=2, D=128, dt=2, stream=None)
    a.update(kw)
    return lib.sba_paged_kv_append(*a.values())


def attend(lib, **kw):
    need = lib.sba_paged_attention_workspace_size(128)
    a = dict(q=FAKE, qs=1024, **POOL, cu=None, B=3, Q=2, N=6, Hq=8, Hkv=2, D=128, dt=2, scale=0.0, left=-1, right=-1,
             cap=0.0, bias=None, sinks=0, per_head=0, out=FAKE, lse=None, ws=FAKE, ws_bytes=need, stream=None)
    a.update(kw)
    return lib.sba_paged_attention_fwd(*a.values())


def select(lib, **kw):
    a = dict(q=FAKE, qs=1024, **POOL, B=3, Q=2, Hq=8, Hkv=2, D=128, dt=2, idx=FAKE, cnt=None, n=4, S=4, bs=64,
             causal=1, scale=0.0, gate=None, out=FAKE, lse=None, stream=None)
    a.update(kw)
    return lib.sba_nsa_select_paged_fwd(*a.values())


COMMON = [(dict(k_pages=None), -1, b"null"), (dict(page_table=None), -1, b"null"), (dict(seq_lens=None), -1, b"null"),
          (dict(k_scales=None), -1, b"scales"), (dict(dt=0), -1, b"scales"), (dict(dt=1), -1, b"dtype"),
          (dict(D=96), -2, b"D must"), (dict(page_size=48), -2, b"page_size"), (dict(page_size=256), -2, b"page_size"),
          (dict(page_stride=2 * 64 * 128 - 16), -1, b"page_stride"),
          (dict(page_stride=2 * 64 * 128 + 8), -1, b"page_stride"), (dict(v_pages=FAKE + 8), -1, b"aligned"),
          (dict(num_pages=0), -1, b"positive"), (dict(table_width=1 << 25), -2, b"table_width"),
          (dict(B=0), -1, b"positive"), (dict(Q=0), -1, b"")]


@pytest.mark.parametrize("change,code,text", COMMON)
def test_cache_arguments(lib, change, code, text):
    for call in (append, attend, select):
        assert call(lib, **change) == code, call.__name__
        assert text in lib.sba_last_error()


@pytest.mark.parametrize("change,code", [
    (dict(k=None), -1), (dict(q=None), -1), (dict(qo=None), -1), (dict(N=7), -1), (dict(ks=128), -1), (dict(vs=260), -1),
    (dict(qos=1000), -1), (dict(k=FAKE + 2), -1), (dict(cos=None), -1), (dict(rot=24), -1), (dict(rot=144), -1),
    (dict(rot=0), -1), (dict(max_pos=0), -1), (dict(sin=FAKE + 4), -1), (dict(Hq=0), -1), (dict(Hq=1 << 17, qs=1 << 24, qos=1 << 24), -2)])
def test_append_arguments(lib, change, code):
    assert append(lib, **change) == code


@pytest.mark.parametrize("change,code", [
    (dict(q=None), -1), (dict(out=None), -1), (dict(N=5), -1), (dict(Hq=7), -1), (dict(left=-2), -1), (dict(right=-2), -1),
    (dict(sinks=2), -1), (dict(bias=FAKE, sinks=17), -2), (dict(cap=float("inf")), -1), (dict(scale=float("nan")), -1),
    (dict(ws=None), -1), (dict(ws_bytes=16), -1), (dict(ws=FAKE + 8), -1), (dict(qs=1004), -1), (dict(out=FAKE + 4), -1)])
def test_attention_arguments(lib, change, code):
    assert attend(lib, **change) == code


@pytest.mark.parametrize("change,code", [
    (dict(idx=None), -1), (dict(S=0), -1), (dict(S=33), -2), (dict(bs=48), -2), (dict(bs=16), -2), (dict(n=-1), -1),
    (dict(Hq=34, qs=34 * 128), -2), (dict(Hq=9), -1), (dict(out=None), -1), (dict(q=FAKE + 8), -1), (dict(scale=float("inf")), -1)])
def test_selection_arguments(lib, change, code):
    assert select(lib, **change) == code


def test_workspace_size(lib):
    a, b = (lib.sba_paged_attention_workspace_size(d) for d in (64, 128))
    assert 0 < a < b < 16 << 20
    assert lib.sba_paged_attention_workspace_size(96) == 0


def test_binding_refuses_host_tensors():
    import selected_block_attention_gb300 as sba

    k = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)
    t, n = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    x = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    for call in (lambda: sba.paged_kv_append(x, x, k, k, t, n), lambda: sba.paged_attention_fwd(x, k, k, t, n),
                 lambda: sba.nsa_select_paged_fwd(x, k, k, t, n, t.view(1, 1, 2), 2, 32)):
        with pytest.raises(ValueError):
            call()
