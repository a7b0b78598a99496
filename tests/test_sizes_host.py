"""Sizes next to 2^31, which the kernels' 32-bit rounding up to whole tiles would not hold: refused on the host."""
import ctypes

import pytest

import sparse_mixture_experts_20_b200 as M
from test_few_host import call as few_call, config, size
from test_mxfp4_host import PTR, matmul, shape

TOP = 2 ** 31


@pytest.mark.parametrize("kw", [dict(rows=TOP - 1), dict(rows=TOP - 511), dict(n=TOP - 32, rows=1, n_seg=1),
                                dict(k=TOP - 128), dict(k=TOP - 384)])
def test_product(kw):
    s = shape(**{**dict(rows=1, n=32, k=128), **kw})
    n0, n = M.moe_kernel_launches(), ctypes.c_size_t(0)
    assert matmul(s) == M.MOE_ERR_UNSUPPORTED
    assert M.lib().moe_mxfp4_workspace_size(ctypes.byref(s), ctypes.byref(n)) == M.MOE_ERR_UNSUPPORTED
    assert M.moe_kernel_launches() == n0


@pytest.mark.parametrize("kw", [dict(rows=TOP - 512), dict(n=TOP - 512), dict(k=TOP - 512)])
def test_product_takes_what_fits(kw):
    s, n = shape(**{**dict(rows=1, n=32, k=128, n_seg=1), **kw}), ctypes.c_size_t(0)
    assert M.lib().moe_mxfp4_workspace_size(ctypes.byref(s), ctypes.byref(n)) == M.MOE_OK


def test_tiled_scales():
    for rows, cols in ((TOP - 1, 128), (TOP - 100, 128), (TOP - 511, 128)):
        n0 = M.moe_kernel_launches()
        assert M.lib().moe_mxfp4_tile_scales(PTR, 1, rows, cols, PTR, None) == M.MOE_ERR_UNSUPPORTED
        assert M.moe_kernel_launches() == n0


@pytest.mark.parametrize("dtype", [M.MOE_BF16, M.MOE_FP8_E4M3_BLOCK, M.MOE_MXFP4])
def test_few_tokens(dtype):
    for kw in (dict(d_ff=TOP - 128), dict(d_ff=TOP - 384), dict(d_ff=128, n_shared=1, d_ff_shared=TOP - 384)):
        cfg = config(dtype=dtype, T=1, d_model=128, n_routed=1, top_k=1, n_shared=kw.get("n_shared", 0),
                     **{k: v for k, v in kw.items() if k != "n_shared"})
        assert size(cfg)[0] == M.MOE_ERR_UNSUPPORTED
        assert few_call(cfg) == M.MOE_ERR_UNSUPPORTED
