"""The mixture-of-experts entry points refuse bad arguments on the host, before any CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch

from lut_dequant_gemv_b200 import binding as B
from lut_dequant_gemv_b200 import build as build_mod


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


def desc(**kw):
    d = dict(experts=8, top_k=2, hidden=256, inter=128, x_type=B.SQZ_TYPE_F16, renormalize=1, router=0x1000,
             ld_router=256, w13=0x2000, w13_scale=0x3000, w2=0x4000, w2_scale=0x5000)
    d.update(kw)
    return B.sqz_moe_desc(**d)


@pytest.mark.parametrize("kw,msg", [
    (dict(experts=0), "experts"),
    (dict(experts=1025), "experts"),
    (dict(top_k=0), "top_k"),
    (dict(top_k=9), "top_k"),
    (dict(experts=64, top_k=17), "top_k"),
    (dict(hidden=250), "multiples of 16"),
    (dict(inter=0), "multiples of 16"),
    (dict(x_type=B.SQZ_TYPE_F32), "x_type"),
    (dict(renormalize=2), "renormalize"),
    (dict(router=None), "NULL"),
    (dict(w2_scale=None), "NULL"),
    (dict(ld_router=255), "ld_router"),
    (dict(w13=0x2008), "16-byte"),
    (dict(router=0x1001), "aligned"),
])
def test_create_refuses(lib, kw, msg):
    out = ctypes.c_void_p(0x1234)
    assert lib.sqz_create_moe(ctypes.byref(desc(**kw)), ctypes.byref(out)) == B.SQZ_ERR_INVALID_ARG
    assert out.value is None and msg in B.sqz_last_error()


def test_create_refuses_more_blocks_than_it_counts(lib):
    out = ctypes.c_void_p()
    big = 1 << 26
    st = lib.sqz_create_moe(ctypes.byref(desc(hidden=big, inter=big, ld_router=big)), ctypes.byref(out))
    assert st == B.SQZ_ERR_UNSUPPORTED and out.value is None


def test_null_handles(lib):
    n = ctypes.c_int64(5)
    assert lib.sqz_create_moe(None, ctypes.byref(ctypes.c_void_p())) == B.SQZ_ERR_INVALID_ARG
    assert lib.sqz_create_moe(ctypes.byref(desc()), None) == B.SQZ_ERR_INVALID_ARG
    assert lib.sqz_moe_workspace_bytes(None, 1, ctypes.byref(n)) == B.SQZ_ERR_INVALID_ARG and n.value == 0
    assert lib.sqz_moe_forward(None, 0x100, 1, 256, 0x200, 256, None, None, 0x300, 1 << 30, None) == \
        B.SQZ_ERR_INVALID_ARG
    assert lib.sqz_moe_status(None, None, None) == B.SQZ_ERR_INVALID_ARG
    assert lib.sqz_destroy_moe(None) == B.SQZ_OK


def test_binding_refuses_host_tensors():
    z = torch.zeros
    with pytest.raises(ValueError):
        B.sqz_create_moe(z(4, 256), z(4, 256, 256), z(4, 2, 1, 2), z(4, 256, 128), z(4, 2, 1), top_k=1)


@pytest.mark.parametrize("kw", [dict(hidden=(1 << 31) - 16, ld_router=1 << 31, inter=16), dict(inter=(1 << 31) - 16, hidden=16),
                                dict(hidden=(1 << 30) + 16, ld_router=1 << 31, inter=16)])
def test_create_refuses_sizes_beyond_its_32_bit_columns(lib, kw):
    """Columns are counted in 32 bits, in steps of the whole CTA and rounded up to blocks."""
    out = ctypes.c_void_p()
    assert lib.sqz_create_moe(ctypes.byref(desc(experts=1, top_k=1, **kw)), ctypes.byref(out)) == B.SQZ_ERR_UNSUPPORTED
    assert out.value is None and "too large" in B.sqz_last_error()
