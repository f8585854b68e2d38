"""The block-scaled 8-bit entry points refuse bad arguments on the host, before any CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch

from lut_dequant_gemv_b200 import binding as B
from lut_dequant_gemv_b200 import build as build_mod


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


@pytest.mark.parametrize("kw,msg", [
    (dict(x_type=B.SQZ_TYPE_F32), "x_type"),
    (dict(x_type=7), "x_type"),
    (dict(format=2), "format"),
    (dict(block_rows=64), "block_rows"),
    (dict(batch=-1), "negative"),
    (dict(rows=-1), "negative"),
    (dict(cols=-5), "negative"),
    (dict(x=None), "NULL"),
    (dict(q=None), "NULL"),
    (dict(scale=None), "NULL"),
    (dict(ldx=299), "ldx"),
    (dict(ldq=288), "ldq"),
    (dict(ld_scale=2), "ld_scale"),
    (dict(q=0x2008), "16-byte"),
    (dict(ldq=305), "multiple"),
    (dict(x=0x1001), "aligned"),
    (dict(scale=0x3002), "aligned"),
])
def test_quantize_refuses(lib, kw, msg):
    a = dict(x=0x1000, x_type=B.SQZ_TYPE_F16, batch=1, rows=4, cols=300, ldx=300, block_rows=1, format=0, q=0x2000,
             ldq=304, scale=0x3000, ld_scale=3)
    a.update(kw)
    st = lib.sqz_fp8_quantize(a["x"], a["x_type"], a["batch"], a["rows"], a["cols"], a["ldx"], a["block_rows"],
                              a["format"], a["q"], a["ldq"], a["scale"], a["ld_scale"], None)
    assert st == B.SQZ_ERR_INVALID_ARG and msg in B.sqz_last_error()


def test_quantize_refuses_more_row_blocks_than_a_grid_has(lib):
    st = lib.sqz_fp8_quantize(0x1000, B.SQZ_TYPE_F16, 70000, 1, 16, 16, 128, 0, 0x2000, 16, 0x3000, 1, None)
    assert st == B.SQZ_ERR_UNSUPPORTED


def test_empty_calls_do_nothing(lib):
    assert lib.sqz_fp8_quantize(None, B.SQZ_TYPE_F16, 1, 0, 5, 5, 1, 0, None, 16, None, 1, None) == B.SQZ_OK
    m = B.sqz_fp8_matrix(None, 0, None, 0, 0)
    assert lib.sqz_fp8_gemm(ctypes.byref(m), ctypes.byref(m), 0, 0, 128, None, 0, 0, None) == B.SQZ_OK


@pytest.mark.parametrize("kw,msg", [
    (dict(m=-1), "negative"),
    (dict(n=-1), "negative"),
    (dict(k=-1), "negative"),
    (dict(y_type=3), "y_type"),
    (dict(y=None), "y is NULL"),
    (dict(ldy=63), "ldy"),
    (dict(y=0x5001), "aligned"),
    (dict(a=dict(q=None)), "a: codes or scales"),
    (dict(w=dict(scale=None)), "w: codes or scales"),
    (dict(a=dict(ld=288)), "a: ld"),
    (dict(w=dict(ld=310)), "multiple of 16"),
    (dict(a=dict(q=0x1008)), "16-byte"),
    (dict(w=dict(ld_scale=2)), "w: ld_scale"),
    (dict(w=dict(format=9)), "format"),
    (dict(a=dict(scale=0x2001)), "4-byte"),
])
def test_gemm_refuses(lib, kw, msg):
    d = dict(m=4, n=64, k=300, y=0x5000, ldy=64, y_type=B.SQZ_TYPE_F16)
    d.update({k: v for k, v in kw.items() if k not in "aw"})
    mats = []
    for name, q, s in (("a", 0x1000, 0x2000), ("w", 0x3000, 0x4000)):
        f = dict(q=q, ld=304, scale=s, ld_scale=3, format=0)
        f.update(kw.get(name, {}))
        mats.append(B.sqz_fp8_matrix(**f))
    st = lib.sqz_fp8_gemm(ctypes.byref(mats[0]), ctypes.byref(mats[1]), d["m"], d["n"], d["k"], d["y"], d["ldy"],
                          d["y_type"], None)
    assert st == B.SQZ_ERR_INVALID_ARG and msg in B.sqz_last_error()


def test_null_operands(lib):
    assert lib.sqz_fp8_gemm(None, None, 1, 1, 1, 0x1000, 1, 0, None) == B.SQZ_ERR_INVALID_ARG
    assert lib.sqz_fp8_status(None, None) == B.SQZ_ERR_INVALID_ARG


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros((4, 128), dtype=torch.float16)
    with pytest.raises(ValueError):
        B.sqz_fp8_quantize(x)
    with pytest.raises(ValueError):
        B.sqz_fp8_quantize(x[0])
    q = torch.zeros((4, 128), dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        B.sqz_fp8_gemm(q, torch.ones(4, 1), q, torch.ones(1, 1), torch.zeros(4, 4))


def test_pitch_of_views():
    t = torch.zeros((2, 3, 32), dtype=torch.uint8)
    assert B._pitch(t, "t") == 32 and B._pitch(t[0], "t") == 32 and B._pitch(t[:, :, :20], "t") == 32
    assert B._pitch(t[:1, :1, :20], "t") == 32  # one row: any pitch that holds it, a multiple of 16
    assert B._pitch(t[:, 1:2], "t") == 96
    for bad in (t[:, :2], t.transpose(1, 2), t[..., ::2]):
        with pytest.raises(ValueError):
            B._pitch(bad, "t")
