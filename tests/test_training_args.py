"""What the block-sparse gradients and the rotary calls refuse, before anything is launched (no GPU)."""

import ctypes as c
import os
import shutil

import pytest
import torch

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")

INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def sba():
    from selected_block_attention_gb300 import _build
    import selected_block_attention_gb300 as m

    _build.build()
    return m


def _at(n):
    return c.c_void_p(n)


GRAD = ["q", "k", "v", "out", "lse", "d_out", "q_pos", "q_seg", "kv_pos", "kv_seg", "lower", "upper", "lower_full",
        "upper_full", "B", "T", "Hq", "Hkv", "D", "q_block", "kv_block", "causal", "left", "right", "pad", "scale", "dq",
        "dk", "dv", "workspace", "bytes", "stream"]


def _grad(sba, **kw):
    lib = sba.load_library()
    a = {n: _at((i + 1) << 32) for i, n in enumerate(GRAD)}
    a.update(B=1, T=256, Hq=4, Hkv=2, D=128, q_block=128, kv_block=64, causal=1, left=-1, right=-1, pad=-1, scale=0.0,
             bytes=lib.sba_blocksparse_attn_bwd_workspace_size(1, 256, 4, 2, 128), stream=None)
    a.update(kw)
    return lib.sba_blocksparse_attn_bwd(*[a[n] for n in GRAD]), lib.sba_last_error().decode()


@pytest.mark.parametrize("kw,code,says", [
    *[({n: None}, INVALID, "null") for n in GRAD[:14] + ["dq", "dk", "dv"]],
    *[({n: _at(0x900000000008)}, INVALID, "aligned") for n in ("q", "k", "v", "out", "lse", "d_out", "dq", "dk", "dv")],
    (dict(B=0), INVALID, "size"), (dict(Hkv=3), INVALID, "head"), (dict(left=-2), INVALID, "window"),
    (dict(scale=float("nan")), INVALID, "finite"), (dict(workspace=None), INVALID, "workspace"),
    (dict(workspace=_at(0x900000000080)), INVALID, "workspace"), (dict(bytes=1000), INVALID, "workspace"),
    (dict(q_block=64), UNSUPPORTED, "q_block"), (dict(kv_block=32), UNSUPPORTED, "kv_block"),
    (dict(T=200), UNSUPPORTED, "T must"), (dict(D=96), UNSUPPORTED, "D must"),
    (dict(T=1 << 20, Hq=2048), UNSUPPORTED, "2^31"),
    (dict(dq=_at(1 << 32)), INVALID, "overlap"),                      # on q
    (dict(dk=_at((2 << 32) + 16)), INVALID, "overlap"),               # inside k
    (dict(dk=_at(0x900000000000), dv=_at(0x900000000100)), INVALID, "overlap"),
    (dict(workspace=_at(6 << 32)), INVALID, "overlap"),               # on d_out
    (dict(dv=_at((8 << 32) - 16)), INVALID, "overlap"),               # into q_seg
    (dict(dq=_at((14 << 32) - 0x1fff0)), INVALID, "overlap"),         # into upper_full
])
def test_gradients(sba, kw, code, says):
    got, text = _grad(sba, **kw)
    assert got == code and says in text, text


def test_gradient_workspace(sba):
    size = sba.blocksparse_attn_bwd_workspace_size
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    rows = lambda B, T, Hq: 2 * up(B * T * Hq * 4) + up(B * T // 128 * 16) + 2 * up(B * T // 32 * 16) + 256  # noqa: E731
    assert size(2, 1024, 6, 3, 128) == rows(2, 1024, 6)
    # 32 key tiles of one KV head: its 8 query heads in parts of 1, so that there are 152 items
    assert size(1, 4096, 8, 1, 64) == rows(1, 4096, 8) + 8 * 2 * 4096 * 64 * 4
    assert size(1, 200, 4, 2, 128) == size(0, 128, 4, 2, 128) == size(1, 128, 0, 1, 128) == size(1, 1 << 20, 2048, 1, 64) == 0
    assert size(1, 128, 4, 3, 128) == size(1, 128, 4, 2, 96) == 0


def _tables(sba, length=8, rot=32, base=1e4, factor=1.0, original=0, slow=1.0, fast=32.0, amplitude=1.0,
            cos=_at(1 << 32), sin=_at(2 << 32)):
    lib = sba.load_library()
    return lib.sba_rotary_tables(length, rot, base, factor, original, slow, fast, amplitude, cos, sin, None), \
        lib.sba_last_error().decode()


@pytest.mark.parametrize("kw,says", [
    (dict(length=-1), "length"), (dict(rot=0), "rot_dim"), (dict(rot=24), "rot_dim"), (dict(rot=272), "rot_dim"),
    (dict(base=0.5), "base"), (dict(base=float("inf")), "base"), (dict(factor=0.9), "factor"),
    (dict(factor=float("nan")), "factor"), (dict(original=-1), "original"), (dict(original=5, slow=3.0, fast=3.0), "slow"),
    (dict(original=5, slow=-1.0), "slow"), (dict(original=5, fast=float("nan")), "slow"),
    (dict(amplitude=float("inf")), "amplitude"), (dict(amplitude=1e300), "amplitude"), (dict(cos=None), "null"),
    (dict(sin=_at(0x200000004)), "aligned"), (dict(sin=_at((1 << 32) + 64)), "overlap")])
def test_tables(sba, kw, says):
    code, text = _tables(sba, **kw)
    assert code == INVALID and says in text, text


def test_empty_calls_launch_nothing(sba):
    assert _tables(sba, length=0, cos=None, sin=None)[0] == 0
    assert _embed(sba, T=0)[0] == 0
    assert _embed(sba, B=0, q=None, q_out=None)[0] == 0


class Embed(c.Structure):
    _fields_ = [(n, c.c_void_p) for n in ("q", "k", "q_out", "k_out", "positions", "cos", "sin")] + \
        [(n, c.c_longlong) for n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")] + \
        [(n, c.c_int) for n in ("B", "T", "Hq", "Hkv", "D", "dtype", "rot_dim", "max_pos", "interleaved", "inverse")]


def _embed(sba, **kw):
    lib = sba.load_library()
    a = Embed(q=1 << 32, k=2 << 32, q_out=3 << 32, k_out=4 << 32, positions=None, cos=6 << 32, sin=7 << 32, q_stride=256,
              k_stride=128, q_out_stride=256, k_out_stride=128, B=2, T=10, Hq=4, Hkv=2, D=64, dtype=0, rot_dim=32,
              max_pos=10, interleaved=0, inverse=0)
    for n, v in kw.items():
        setattr(a, n, v)
    return lib.sba_rotary_embed(c.byref(a), None), lib.sba_last_error().decode()


@pytest.mark.parametrize("kw,code,says", [
    (dict(q=None), INVALID, "null"), (dict(q_out=None), INVALID, "null"), (dict(cos=None), INVALID, "null"),
    (dict(k=None), INVALID, "together"), (dict(k_out=None), INVALID, "together"), (dict(Hq=0), INVALID, "head"),
    (dict(Hkv=0), INVALID, "head"), (dict(T=-1), INVALID, "size"), (dict(dtype=2), INVALID, "dtype"),
    (dict(rot_dim=8), INVALID, "rot_dim"), (dict(rot_dim=24), INVALID, "rot_dim"), (dict(rot_dim=80), INVALID, "rot_dim"),
    (dict(D=72), UNSUPPORTED, "D must"), (dict(D=272), UNSUPPORTED, "D must"), (dict(max_pos=0), INVALID, "position"),
    (dict(B=1 << 16, T=1 << 15), UNSUPPORTED, "2^31"), (dict(q=(1 << 32) + 8), INVALID, "aligned"),
    (dict(q_stride=255), INVALID, "stride"), (dict(q_stride=260), INVALID, "stride"), (dict(k_out_stride=64), INVALID, "stride"),
    (dict(q_out=1 << 32, q_out_stride=512), INVALID, "q_out"), (dict(q_out=(1 << 32) + 16), INVALID, "q_out"),
    (dict(k_out=(2 << 32) + 16), INVALID, "k_out"), (dict(q_out=2 << 32), INVALID, "overlap"),
    (dict(k_out=(1 << 32) + 1024), INVALID, "overlap"), (dict(k_out=(3 << 32) + 1024), INVALID, "overlap"),
    (dict(cos=(3 << 32) + 1024), INVALID, "overlap"), (dict(sin=4 << 32), INVALID, "overlap"),
    (dict(positions=(4 << 32) + 64), INVALID, "overlap"),
    # parts of one projection's output: q_out would reach into k
    (dict(k=(1 << 32) + 256, q_stride=512, k_stride=512, q_out=(1 << 32), q_out_stride=512), INVALID, "overlap")])
def test_rotation(sba, kw, code, says):
    got, text = _embed(sba, **kw)
    assert got == code and says in text, text


def test_tensors_off_the_gpu_and_of_other_types(sba):
    x = torch.zeros((1, 128, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros((1, 128), dtype=torch.int32)
    b = torch.zeros((1, 1, 1), dtype=torch.int32)
    with pytest.raises(ValueError):
        sba.blocksparse_attn_bwd(x, x, x, x, torch.zeros((1, 128, 2)), x, i, i, i, i, b, b, b, b, 128, 64)
    with pytest.raises(ValueError):
        sba.rotary_embed(x, x, torch.zeros((128, 32)), torch.zeros((128, 32)))
    with pytest.raises(ValueError):
        sba.rotary_tables(8, 32, device="cpu")
    with pytest.raises(ValueError):
        sba.rotary_tables(8, 32, cos=torch.zeros((8, 16)), sin=torch.zeros((8, 16)))
    with pytest.raises(ValueError):
        sba.rotary_tables(8, 32, cos=torch.zeros((8, 16)))
    with pytest.raises(TypeError):
        sba.rotary_tables(8)
    with pytest.raises(TypeError):
        sba.rotary_tables(8, 32, device=3)
    with pytest.raises(TypeError):
        sba.rotary_embed([1], None, 1, 2)
    with pytest.raises(TypeError):
        sba.rotary_embed(x, None)
