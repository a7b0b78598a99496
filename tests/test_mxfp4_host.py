"""MXFP4 without a GPU: pins of the oracle, and what the entry points refuse
before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import oracle as O
import sparse_mixture_experts_20_b200 as M

PTR = 0x10000          # aligned, never dereferenced: every call here is refused on the host


# ---------------------------------------------------------------- oracle pins

def test_every_code_and_scale_decodes_to_its_value():
    codes = np.arange(16, dtype=np.uint8)
    row = (codes | (codes << 4))                                     # both nibbles
    want = [0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6]
    for s in (0, 1, 126, 127, 128, 254):
        v = O.mxfp4_decode(row[None], np.array([[s]], np.uint8))[0]
        assert np.array_equal(v[0::2], np.array(want) * 2.0 ** (s - 127)) and np.array_equal(v[0::2], v[1::2])
    assert np.all(np.isnan(O.mxfp4_decode(row[None], np.array([[255]], np.uint8))))


def test_nearest_code_by_exhaustion():
    """Against the nearest of all 15 values, ties to the even code."""
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-6, 6, 4000), [.25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -2.5, -5, 6, -6, 0]])
    v = np.concatenate([v, np.zeros(-len(v) % 31)]).reshape(-1, 31)
    v = np.concatenate([v, np.full((len(v), 1), 6.0)], 1)            # amax 6: scale 1
    codes, s = O.mxfp4_encode(v)
    assert np.all(s == 127)
    got = O.mxfp4_decode(codes, s)
    grid = O.GRID
    for x, y in zip(v.ravel(), got.ravel()):
        d = np.abs(grid - abs(x))
        best = np.flatnonzero(d == d.min())
        want = grid[best[best % 2 == 0][0] if len(best) > 1 else best[0]]
        assert abs(y) == want, (x, y)


@pytest.mark.parametrize("amax,k", [(6.0, 0), (np.nextafter(6.0, 7), 1), (3.0, -1), (12.0, 1), (4.0, 0), (0.0, 0),
                                    (2.0 ** -130, -126), (6 * 2.0 ** -126, -126), (np.finfo(np.float32).max, 126)])
def test_scale_is_the_smallest_that_holds_the_block(amax, k):
    assert O.mxfp4_scale(np.array(amax)) == k + 127


# ---------------------------------------------------------------- refusals

def q(x=PTR, dtype=M.MOE_BF16, rows=4, cols=64, codes=PTR, scales=PTR):
    return M.lib().moe_mxfp4_quantize(x, dtype, rows, cols, codes, scales, None)


def dq(codes=PTR, scales=PTR, rows=4, cols=64, out=PTR, dtype=M.MOE_BF16):
    return M.lib().moe_mxfp4_dequantize(codes, scales, rows, cols, out, dtype, None)


@pytest.mark.parametrize("call", [q, dq])
def test_quantiser_refusals(call):
    n0 = M.moe_kernel_launches()
    first = "x" if call is q else "out"
    for kw in (dict(dtype=M.MOE_FP8_E4M3_BLOCK), dict(dtype=M.MOE_MXFP4), dict(rows=-1), dict(cols=0),
               {first: None}, {first: PTR + 8}, dict(codes=None), dict(codes=PTR + 4), dict(scales=None)):
        assert call(**kw) == M.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(cols=48), dict(cols=33), dict(rows=1 << 42)):
        assert call(**kw) == M.MOE_ERR_UNSUPPORTED, kw
    assert call(rows=0) == M.MOE_OK
    assert M.moe_kernel_launches() == n0


def test_binding_checks_shapes():
    x = torch.zeros(4, 64)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    for bad in ((x.half(), u8(4, 32), u8(4, 2)), (x, u8(4, 31), u8(4, 2)), (x, u8(4, 32), u8(4, 3)),
                (x[:, :40], u8(4, 20), u8(4, 1)), (x, u8(4, 32).int(), u8(4, 2)),
                (x, u8(4, 32), u8(4, 2))):                           # the last: not on a GPU
        with pytest.raises(ValueError):
            M.moe_mxfp4_quantize(*bad)
        with pytest.raises(ValueError):
            M.moe_mxfp4_dequantize(bad[1], bad[2], bad[0])


def shape(**kw):
    d = dict(rows=10, n=64, k=256, n_mats=3, n_seg=2, activation=M.MOE_ACT_NONE, out_dtype=M.MOE_BF16)
    d.update(kw)
    return M.moe_mxfp4_shape(**d)


def matmul(s, **kw):
    names = ("a", "a_scales", "seg_offsets", "seg_mat", "w", "w_scales", "bias", "y", "y_scales", "ws")
    d = dict.fromkeys(names, PTR)
    d["y_scales"] = None
    d.update(kw)
    return M.lib().moe_mxfp4_matmul(ctypes.byref(s) if s else None, *[d[n] for n in names], None)


def test_matmul_refusals():
    n0 = M.moe_kernel_launches()
    for kw in (dict(rows=-1), dict(n=0), dict(k=0), dict(n_mats=0), dict(n_seg=0), dict(activation=2),
               dict(out_dtype=M.MOE_FP8_E4M3_BLOCK), dict(out_dtype=9)):
        assert matmul(shape(**kw)) == M.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(n=48), dict(k=64), dict(k=160), dict(n_mats=65536), dict(n_seg=257),
               dict(rows=2 ** 31 - 1, n=1 << 22)):
        assert matmul(shape(**kw)) == M.MOE_ERR_UNSUPPORTED, kw
    for kw in ({n: None} for n in ("a", "a_scales", "seg_offsets", "seg_mat", "w", "w_scales", "y", "ws")):
        assert matmul(shape(), **kw) == M.MOE_ERR_INVALID_ARG, kw
    for kw in ({n: PTR + 8} for n in ("a", "a_scales", "seg_offsets", "seg_mat", "w", "w_scales", "bias", "y", "ws")):
        assert matmul(shape(), **kw) == M.MOE_ERR_INVALID_ARG, kw
    assert matmul(shape(), ws=PTR + 16) == M.MOE_ERR_INVALID_ARG
    assert matmul(shape(), y_scales=PTR) == M.MOE_ERR_INVALID_ARG
    assert matmul(shape(out_dtype=M.MOE_MXFP4)) == M.MOE_ERR_INVALID_ARG
    assert matmul(None) == M.MOE_ERR_INVALID_ARG
    assert matmul(shape(rows=0)) == M.MOE_OK
    assert M.moe_kernel_launches() == n0


def test_layer_entry_points_reject_mxfp4():
    cfg = M.make_config(T=4, d_model=128, n_routed=8, top_k=2, d_ff=128, dtype=M.MOE_MXFP4)
    n = ctypes.c_size_t(0)
    assert M.lib().moe_workspace_size(ctypes.byref(cfg), ctypes.byref(n)) == M.MOE_ERR_INVALID_ARG


def test_tile_scales_refusals():
    n0 = M.moe_kernel_launches()

    def call(scales=PTR, n=2, rows=64, cols=256, tiled=PTR):
        return M.lib().moe_mxfp4_tile_scales(scales, n, rows, cols, tiled, None)

    for kw in (dict(n=-1), dict(rows=0), dict(cols=0), dict(scales=None), dict(tiled=None), dict(scales=PTR + 4),
               dict(tiled=PTR + 8)):
        assert call(**kw) == M.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(cols=192), dict(n=1 << 40)):
        assert call(**kw) == M.MOE_ERR_UNSUPPORTED, kw
    assert call(n=0) == M.MOE_OK
    assert M.moe_kernel_launches() == n0
    with pytest.raises(ValueError):
        M.moe_mxfp4_tile_scales(torch.zeros(4, 8, dtype=torch.uint8))
    with pytest.raises(ValueError):
        M.moe_mxfp4_tile_scales(torch.zeros(1, 4, 8))


def test_matmul_binding_checks_sizes():
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    s = M.make_mxfp4_shape(4, 64, 128, 2, 1, M.MOE_ACT_NONE, M.MOE_F32)
    good = dict(a=u8(256), a_scales=u8(16), seg_offsets=torch.zeros(2, dtype=torch.int32),
                seg_mat=torch.zeros(1, dtype=torch.int32), w=u8(2 * 64 * 64), w_scales=u8(2 * 64 * 4),
                bias=torch.zeros(128), y=torch.zeros(256), y_scales=None, ws=u8(256))
    for k in ("a", "a_scales", "seg_offsets", "seg_mat", "w", "w_scales", "bias", "y"):
        bad = dict(good)
        bad[k] = good[k][:-1]
        with pytest.raises(ValueError, match=k + " is smaller"):
            M.moe_mxfp4_matmul(s, *bad.values())
