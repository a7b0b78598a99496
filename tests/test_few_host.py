"""What the few-token layer refuses on the host, before anything is launched."""
import ctypes

import pytest
import torch

import sparse_mixture_experts_20_b200 as M

PTR = 0x10000          # aligned, never dereferenced: every call here is refused on the host
NAMES = ("x", "W_r", "logit_bias", "W1", "W1_scales", "b1", "W2", "W2_scales", "b2", "Ws1", "Ws1_scales", "bs1",
         "Ws2", "Ws2_scales", "bs2", "out", "f", "P", "loss", "topk_idx", "gates", "counts", "ws")


def config(**kw):
    d = dict(T=4, d_model=256, n_routed=8, top_k=2, d_ff=128, n_shared=1, d_ff_shared=128, dtype=M.MOE_MXFP4)
    d.update(kw)
    return M.make_config(**d)


def size(cfg):
    n = ctypes.c_size_t(0)
    return M.lib().moe_few_workspace_size(ctypes.byref(cfg), ctypes.byref(n)), n.value


def call(cfg, **kw):
    d = dict.fromkeys(NAMES, PTR)
    d.update(kw)
    return M.lib().moe_layer_forward_few(ctypes.byref(cfg), *[d[n] for n in NAMES], None)


@pytest.mark.parametrize("dtype", [M.MOE_BF16, M.MOE_FP8_E4M3_BLOCK, M.MOE_MXFP4])
def test_sizes_that_are_taken(dtype):
    for T in (1, 8, 9, 16):
        st, n = size(config(T=T, dtype=dtype))
        assert st == M.MOE_OK and n > 0 and n % 256 == 0
    assert size(config(T=17, dtype=dtype))[0] == M.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(dtype=M.MOE_F32), dict(T=17), dict(d_model=192), dict(d_ff=64),
                                dict(d_ff_shared=192), dict(dtype=M.MOE_FP8_E4M3_BLOCK, d_model=320),
                                dict(dtype=M.MOE_BF16, d_ff=96), dict(n_routed=300), dict(top_k=17, n_routed=64),
                                dict(n_shared=9)])
def test_unsupported(kw):
    n0 = M.moe_kernel_launches()
    assert size(config(**kw))[0] == M.MOE_ERR_UNSUPPORTED
    assert call(config(**kw)) == M.MOE_ERR_UNSUPPORTED
    assert M.moe_kernel_launches() == n0


@pytest.mark.parametrize("kw", [dict(T=0), dict(top_k=9), dict(dtype=4), dict(bias_mode=2), dict(capacity_factor=-1.0),
                                dict(overflow_mode=3), dict(d_ff=0)])
def test_invalid(kw):
    assert size(config(**kw))[0] == M.MOE_ERR_INVALID_ARG
    assert call(config(**kw)) == M.MOE_ERR_INVALID_ARG
    assert M.lib().moe_few_workspace_init(ctypes.byref(config(**kw)), PTR, None) == M.MOE_ERR_INVALID_ARG


def test_pointers():
    n0 = M.moe_kernel_launches()
    needed = [n for n in NAMES if n not in ("logit_bias", "topk_idx", "gates", "counts")]
    for n in needed:
        assert call(config(), **{n: None}) == M.MOE_ERR_INVALID_ARG, n
    for n in [n for n in needed if n not in ("f", "P", "loss")]:
        assert call(config(), **{n: PTR + 8}) == M.MOE_ERR_INVALID_ARG, n
    assert call(config(), ws=PTR + 128) == M.MOE_ERR_INVALID_ARG
    assert M.lib().moe_few_workspace_init(ctypes.byref(config()), PTR + 128, None) == M.MOE_ERR_INVALID_ARG
    assert M.lib().moe_few_workspace_init(ctypes.byref(config()), None, None) == M.MOE_ERR_INVALID_ARG
    assert M.lib().moe_layer_forward_few(None, *([PTR] * 23), None) == M.MOE_ERR_INVALID_ARG
    assert M.moe_kernel_launches() == n0


@pytest.mark.parametrize("dtype", [M.MOE_BF16, M.MOE_FP8_E4M3_BLOCK, M.MOE_MXFP4])
def test_widths_beyond_the_kernels_counting(dtype):
    """d_model up to which every slice of the router has a block; weights counted in 32 bits."""
    assert size(config(dtype=dtype, d_model=131072))[0] == M.MOE_OK
    wide = config(dtype=dtype, d_model=131072 + 128)
    long = config(dtype=dtype, T=16, d_model=131072, d_ff=131072, n_routed=256, top_k=8)
    n0 = M.moe_kernel_launches()
    for cfg in (wide, long):
        assert size(cfg)[0] == M.MOE_ERR_UNSUPPORTED
        assert call(cfg) == M.MOE_ERR_UNSUPPORTED
    assert M.moe_kernel_launches() == n0


@pytest.mark.parametrize("dtype,bits", [(M.MOE_BF16, 16), (M.MOE_FP8_E4M3_BLOCK, 8), (M.MOE_MXFP4, 4)])
def test_layer_refuses_small_weights(dtype, bits, monkeypatch):
    """The sizes that a layer checks before its first call, on a layer without a GPU."""
    monkeypatch.setattr(M, "moe_few_workspace_init", lambda cfg, ws: None)
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    sc = {M.MOE_FP8_E4M3_BLOCK: 4, M.MOE_MXFP4: 512}.get(dtype, 0)
    w = dict(W_r=u8(4 * 8 * 256), logit_bias=None, b1=u8(4 * 8 * 128), b2=u8(4 * 8 * 256), bs1=u8(4 * 128),
             bs2=u8(4 * 256), W1=u8(8 * 128 * 256 * bits // 8), W2=u8(8 * 128 * 256 * bits // 8),
             Ws1=u8(128 * 256 * bits // 8), Ws2=u8(128 * 256 * bits // 8))
    if sc:
        w.update(W1_scales=u8(8 * 2 * sc), W2_scales=u8(8 * 2 * sc), Ws1_scales=u8(2 * sc), Ws2_scales=u8(2 * sc))
    layer = M.MoELayer.__new__(M.MoELayer)
    layer.cfg, layer.w, layer.device = config(dtype=dtype), w, torch.device("cpu")
    layer._few_workspace()
    for name in w:
        if w[name] is not None:
            layer.w = {**w, name: w[name][:-1]}
            with pytest.raises(ValueError, match=name + " is smaller"):
                layer._few_workspace()
