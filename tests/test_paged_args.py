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


class Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_pages", "v_pages", "k_scales", "v_scales", "page_table", "seq_lens",
                                               "cu")] + [("page_stride", ctypes.c_longlong)]
    _fields_ += [(n, ctypes.c_int) for n in ("num_pages", "page_size", "Hkv", "D", "dt", "table_width", "B", "Q", "N")]


def struct(name, pointers, longs, rest):
    p, ll = ctypes.c_void_p, ctypes.c_longlong
    fields = [("cache", Cache)] + [(n, p) for n in pointers] + [(n, ll) for n in longs]
    fields += [(n, ctypes.c_float if n in ("scale", "cap") else ctypes.c_int) for n in rest]
    return type(name, (ctypes.Structure,), {"_fields_": fields})


APPEND = struct("Append", ("k", "v", "q", "qo", "cos", "sin"), ("ks", "vs", "qs", "qos"), ("Hq", "rot", "max_pos", "inter"))
ATTEND = struct("Attend", ("q", "bias", "out", "lse", "ws"), ("ws_bytes", "qs"),
                ("Hq", "scale", "left", "right", "cap", "sinks", "per_head"))
SELECT = struct("Select", ("q", "idx", "cnt", "gate", "out", "lse"), ("qs",),
                ("Hq", "n", "S", "bs", "causal", "scale"))
OUT = 0x20000
POOL = dict(k_pages=FAKE, v_pages=FAKE + 4 * 2 * 64 * 128, k_scales=FAKE, v_scales=FAKE, page_table=FAKE, seq_lens=FAKE, cu=None,
            page_stride=2 * 64 * 128, num_pages=4, page_size=64, Hkv=2, D=128, dt=2, table_width=8, B=3, Q=2, N=6)


def call(fn, kind, defaults, change):
    own = [n for n, _ in kind._fields_]
    cache = Cache(**{**POOL, **{n: v for n, v in change.items() if n in POOL}})
    args = kind(cache=cache, **{**defaults, **{n: v for n, v in change.items() if n in own}})
    return fn(ctypes.addressof(args), None)


def append(lib, **kw):
    d = dict(k=0x30000, ks=256, v=0x40000, vs=256, q=FAKE, qs=1024, qo=FAKE, qos=1024, cos=FAKE, sin=FAKE, rot=128,
             max_pos=512, inter=0, Hq=8)
    return call(lib.sba_paged_kv_append, APPEND, d, kw)


def attend(lib, **kw):
    d = dict(q=FAKE, qs=1024, Hq=8, scale=0.0, left=-1, right=-1, cap=0.0, bias=None, sinks=0, per_head=0, out=OUT,
             lse=None, ws=FAKE, ws_bytes=lib.sba_paged_attention_workspace_size(3, 6, 8, 2, 128))
    return call(lib.sba_paged_attention_fwd, ATTEND, d, kw)


def select(lib, **kw):
    d = dict(q=FAKE, qs=1024, Hq=8, idx=FAKE, cnt=None, n=4, S=4, bs=64, causal=1, scale=0.0, gate=None, out=OUT,
             lse=None)
    return call(lib.sba_nsa_select_paged_fwd, SELECT, d, kw)


COMMON = [(dict(k_pages=None), -1, b"null"), (dict(page_table=None), -1, b"null"), (dict(seq_lens=None), -1, b"null"),
          (dict(k_scales=None), -1, b"scales"), (dict(dt=0), -1, b"scales"), (dict(dt=1), -1, b"dtype"),
          (dict(D=96), -2, b"D must"), (dict(page_size=48), -2, b"page_size"), (dict(page_size=256), -2, b"page_size"),
          (dict(page_stride=2 * 64 * 128 - 16), -1, b"page_stride"),
          (dict(page_stride=2 * 64 * 128 + 8), -1, b"page_stride"), (dict(v_pages=FAKE + 8), -1, b"aligned"),
          (dict(num_pages=0), -1, b"positive"), (dict(table_width=1 << 25), -2, b"table_width"),
          (dict(B=0), -1, b"positive"), (dict(Q=0), -1, b"")]


@pytest.mark.parametrize("change,code,text", COMMON)
def test_cache_arguments(lib, change, code, text):
    for entry in (append, attend, select):
        assert entry(lib, **change) == code, entry.__name__
        assert text in lib.sba_last_error()


@pytest.mark.parametrize("change,code", [
    (dict(k=None), -1), (dict(q=None), -1), (dict(qo=None), -1), (dict(N=7), -1), (dict(ks=128), -1), (dict(vs=260), -1),
    (dict(qos=1000), -1), (dict(k=FAKE + 2), -1), (dict(cos=None), -1), (dict(rot=24), -1), (dict(rot=144), -1),
    (dict(rot=0), -1), (dict(max_pos=0), -1), (dict(sin=FAKE + 4), -1), (dict(Hq=0), -1), (dict(Hq=1 << 17, qs=1 << 24, qos=1 << 24), -2),
    (dict(qs=2048), -1), (dict(qo=0x30000), -1), (dict(qo=0x40000), -1), (dict(v_pages=FAKE), -1),
    (dict(v_pages=FAKE + 2 * 64 * 128), -1), (dict(v_pages=FAKE + 64, page_stride=4 * 64 * 128), -1),
    (dict(v_pages=FAKE + 3 * 64 * 128, page_stride=4 * 64 * 128), -1)])
def test_append_arguments(lib, change, code):
    assert append(lib, **change) == code


@pytest.mark.parametrize("change,code", [
    (dict(q=None), -1), (dict(out=None), -1), (dict(N=5), -1), (dict(Hq=7), -1), (dict(left=-2), -1), (dict(right=-2), -1),
    (dict(sinks=2), -1), (dict(bias=FAKE, sinks=17), -2), (dict(cap=float("inf")), -1), (dict(scale=float("nan")), -1),
    (dict(ws=None), -1), (dict(ws_bytes=16), -1), (dict(ws=FAKE + 8), -1), (dict(qs=1004), -1), (dict(out=FAKE + 4), -1), (dict(out=FAKE), -1)])
def test_attention_arguments(lib, change, code):
    assert attend(lib, **change) == code


@pytest.mark.parametrize("change,code", [
    (dict(idx=None), -1), (dict(S=0), -1), (dict(S=33), -2), (dict(bs=48), -2), (dict(bs=16), -2), (dict(n=-1), -1),
    (dict(Hq=34, qs=34 * 128), -2), (dict(Hq=9), -1), (dict(out=None), -1), (dict(q=FAKE + 8), -1), (dict(scale=float("inf")), -1),
    (dict(out=FAKE), -1), (dict(cu=FAKE), -1)])
def test_selection_arguments(lib, change, code):
    assert select(lib, **change) == code


def test_workspace_size(lib):
    size = lib.sba_paged_attention_workspace_size
    few, many = size(64, 64, 32, 8, 128), size(4, 2048, 32, 8, 128)
    assert 0 < size(64, 64, 32, 8, 64) < few < many < 64 << 20
    assert few == size(2, 8, 32, 8, 128) and many == size(2, 9, 32, 8, 128)  # over 16 rows a KV head
    for bad in ((0, 1, 8, 8, 128), (1, 0, 8, 8, 128), (1, 1, 8, 8, 96), (1, 1, 9, 8, 128), (1, 1, 4, 8, 128)):
        assert size(*bad) == 0


def test_binding_refuses_host_tensors(lib):
    import selected_block_attention_gb300 as sba

    k = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)
    t, n = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    x = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    for call in (lambda: sba.paged_kv_append(x, x, k, k, t, n), lambda: sba.paged_attention_fwd(x, k, k, t, n),
                 lambda: sba.nsa_select_paged_fwd(x, k, k, t, n, t.view(1, 1, 2), 2, 32)):
        with pytest.raises(ValueError):
            call()
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()
    with pytest.raises(TypeError, match="misses the argument 'seq_lens'"):
        sba.paged_attention_fwd(x, k, k, t)
    with pytest.raises(TypeError, match="unexpected argument 'scale'"):
        sba.paged_attention_fwd(x, k, k, t, n, scale=1.0)
    with pytest.raises(TypeError, match="second argument 'q'"):
        sba.paged_attention_fwd(x, k, k, t, n, q=x)
    with pytest.raises(TypeError, match="at most 6 positional"):
        sba.paged_kv_append(x, x, k, k, t, n, None)
    with pytest.raises(TypeError, match="k_pages must be a tensor"):
        sba.paged_attention_fwd(x, None, k, t, n)
    assert "page_table" in sba.paged_kv_append.__doc__
