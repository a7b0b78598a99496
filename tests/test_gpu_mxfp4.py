"""MXFP4 quantisation, its inverse and the grouped product against fp64."""
import numpy as np
import pytest
import torch

import oracle as O
import sparse_mixture_experts_20_b200 as M

pytestmark = pytest.mark.gpu


def quantize(x):
    codes = torch.empty((*x.shape[:-1], x.shape[-1] // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((*x.shape[:-1], x.shape[-1] // 32), dtype=torch.uint8, device="cuda")
    M.moe_mxfp4_quantize(x, codes, scales)
    return codes, scales


def hard_values(rows, cols, seed, dtype):
    """Blocks over the whole range of magnitudes, rounding ties, zeros, subnormals, the largest numbers, an
    infinity, a NaN."""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((rows, cols // 32, 32)) * 2.0 ** rng.integers(-140, 125, (rows, cols // 32, 1))
    flat = v.reshape(-1, 32)
    n = len(flat)
    pick = rng.permutation(n)
    ties = np.resize(np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5.0, 6.0]), 32)
    special = [np.zeros(32), ties, ties * 2.0 ** -100, np.full(32, 2.0 ** -149), np.full(32, -3.4e38),
               np.where(np.arange(32) == 7, np.inf, 1.0), np.where(np.arange(32) == 31, np.nan, 1.0),
               np.full(32, -0.0)]
    for i, s in enumerate(special[:n]):
        flat[pick[i]] = s
    return torch.tensor(v.reshape(rows, cols), dtype=torch.float64).to(torch.float32).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 96), (3, 4128), (257, 224), (129, 7168)])
def test_quantize_is_exact(rows, cols, dtype):
    x = hard_values(rows, cols, rows * cols, dtype)
    codes, scales = quantize(x.cuda())
    want_c, want_s = O.mxfp4_encode(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_dequantize_every_code_and_scale(dtype):
    codes = torch.randint(0, 256, (256, 16 * 5), dtype=torch.uint8, generator=torch.Generator().manual_seed(1))
    codes[:, :8] = torch.arange(8, dtype=torch.uint8) * 34 + 16      # every nibble
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 5)
    out = torch.empty((256, 160), dtype=dtype, device="cuda")
    M.moe_mxfp4_dequantize(codes.cuda(), scales.cuda(), out)
    want = torch.tensor(O.mxfp4_decode(codes.numpy(), scales.numpy())).float().to(dtype)
    assert torch.equal(torch.nan_to_num(out.cpu().float(), nan=-7.0), torch.nan_to_num(want.float(), nan=-7.0))


def test_quantize_leaves_its_neighbours_alone():
    """Rows of a larger buffer: nothing before or behind them is written."""
    x = torch.randn(5, 96, device="cuda")
    codes = torch.full((7, 48), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((7, 3), 0xCD, dtype=torch.uint8, device="cuda")
    M.moe_mxfp4_quantize(x, codes[1:6], scales[1:6])
    assert bool((codes[0] == 0xAB).all() and (codes[6] == 0xAB).all())
    assert bool((scales[0] == 0xCD).all() and (scales[6] == 0xCD).all())


# ---------------------------------------------------------------- the grouped product

def product(sizes, mats, n_mats, n, k, act, out, behind=0, bias=True, seed=0):
    """One call; returns (y as fp64 values, y_scales, z64, S): z64 the fp64 result of the same operands before the
    output's rounding, S the sum of the magnitudes each element adds up."""
    rng = np.random.default_rng(seed)
    rows = sum(sizes) + behind
    a64 = rng.standard_normal((rows, k)) * 2.0 ** rng.integers(-3, 4, (rows, 1))
    w64 = rng.standard_normal((n_mats, n, k)) / np.sqrt(k)
    b = rng.standard_normal((n_mats, n)).astype(np.float32) if bias else None
    ac, asc = O.mxfp4_encode(a64)
    wc, wsc = O.mxfp4_encode(w64.reshape(n_mats * n, k))
    dev = lambda t, dt=None: torch.as_tensor(t, dtype=dt).cuda().contiguous()  # noqa: E731
    offs = np.concatenate([[0], np.cumsum(sizes)])
    s = M.make_mxfp4_shape(rows, n, k, n_mats, len(sizes), act, out)
    ws = torch.empty(M.moe_mxfp4_workspace_size(s), dtype=torch.uint8, device="cuda")
    M.moe_mxfp4_workspace_init(s, ws)
    ysc = None
    if out == M.MOE_MXFP4:
        y = torch.full((rows, n // 2), 0x11, dtype=torch.uint8, device="cuda")
        ysc = torch.full((rows, n // 32), 0x22, dtype=torch.uint8, device="cuda")
    else:
        y = torch.full((rows, n), 77.0, dtype=torch.float32 if out == M.MOE_F32 else torch.bfloat16, device="cuda")
    M.moe_mxfp4_matmul(s, dev(ac), dev(asc), dev(offs, torch.int32), dev(mats, torch.int32), dev(wc), dev(wsc),
                       None if b is None else dev(b), y, ysc, ws)
    torch.cuda.synchronize()
    assert M.moe_mxfp4_get_device_status(s, ws) == 0
    av, wv = O.mxfp4_decode(ac, asc), O.mxfp4_decode(wc, wsc).reshape(n_mats, n, k)
    z, S = np.zeros((rows, n)), np.zeros((rows, n))
    for i, m in enumerate(mats):
        r = slice(offs[i], offs[i + 1])
        z[r] = av[r] @ wv[m].T
        S[r] = np.abs(av[r]) @ np.abs(wv[m]).T
        if b is not None:
            z[r] += b[m]
            S[r] += np.abs(b[m])
    return y.cpu(), None if ysc is None else ysc.cpu(), z, S, offs[-1]


def bounds(z, S, k, act):
    """The fp64 result and how far an fp32 kernel may be from it: k/64 accumulations of at most two fp32 steps of
    the running magnitude each, eight steps for the sums within them; SiLU's slope is at most 1.1, and its
    exponential and division add at most 2^-19 of the result and of the argument (relative error of the fast
    exponential: |z| 2^-22 and a few steps)."""
    tol = S * (k / 64 + 8) * 2.0 ** -22
    if act == M.MOE_ACT_SILU:
        tol = 1.1 * tol + 2.0 ** -19 * np.abs(z)
        z = z / (1 + np.exp(-z))
    return z, tol


SHAPES = [
    # sizes, mats, n_mats, n, k
    ([1], [0], 1, 32, 128),
    ([1, 1, 1], [2, 0, 2], 3, 96, 384),
    ([0, 5, 0, 130, 0], [1, 0, 0, 2, 1], 3, 224, 256),
    ([127, 128, 129], [1, 0, 1], 2, 256, 640),
    ([300], [0], 1, 544, 1408),
    ([17, 0, 64, 3, 201, 1, 33], [6, 5, 4, 3, 2, 1, 0], 7, 288, 2048),
    ([2] * 256, list(range(255, -1, -1)), 256, 64, 128),
    ([700, 20], [0, 0], 1, 1024, 7168),
]


@pytest.mark.parametrize("act", [M.MOE_ACT_NONE, M.MOE_ACT_SILU])
@pytest.mark.parametrize("out", [M.MOE_F32, M.MOE_BF16])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_matmul(case, out, act):
    sizes, mats, n_mats, n, k = SHAPES[case]
    y, _, z, S, end = product(sizes, mats, n_mats, n, k, act, out, behind=case % 3, seed=case)
    want, tol = bounds(z, S, k, act)
    got = y.double().numpy()
    if out == M.MOE_BF16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)          # half a bf16 step
    assert np.all(np.abs(got - want)[:end] <= tol[:end] + 1e-37)
    assert np.all(got[end:] == 77.0)                                     # rows behind the last segment


@pytest.mark.parametrize("act", [M.MOE_ACT_NONE, M.MOE_ACT_SILU])
@pytest.mark.parametrize("case", [0, 1, 2, 3, 5])
def test_matmul_to_mxfp4(case, act):
    """Scales equal unless the block's largest value is within the tolerance of a border; values within half a
    grid step of the fp64 result."""
    sizes, mats, n_mats, n, k = SHAPES[case]
    y, ysc, z, S, end = product(sizes, mats, n_mats, n, k, act, M.MOE_MXFP4, behind=2, seed=case, bias=case != 1)
    want, tol = bounds(z, S, k, act)
    want, tol = want[:end], tol[:end]
    top, slack = np.abs(want).reshape(end, -1, 32).max(-1), tol.reshape(end, -1, 32).max(-1)
    lo, hi = O.mxfp4_scale(np.maximum(top - slack, 0)), O.mxfp4_scale(top + slack)
    s = ysc.numpy()[:end]
    assert np.all((s == lo) | (s == hi))
    got = O.mxfp4_decode(y.numpy()[:end], s)
    unit = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=-1)
    a = np.abs(want) / unit
    half = np.where(a <= 2, 0.25, np.where(a <= 4, 0.5, 1.0)) * unit
    assert np.all(np.abs(got - want) <= half + tol * 2)
    assert np.all(y.numpy()[end:] == 0x11) and np.all(ysc.numpy()[end:] == 0x22)


def test_matmul_refused_segments_are_skipped_and_reported():
    """Bad bounds and bad matrices: their rows stay, the other segments are computed, the status says so."""
    k, n, rows = 128, 64, 40
    rng = np.random.default_rng(3)
    ac, asc = O.mxfp4_encode(rng.standard_normal((rows, k)))
    wc, wsc = O.mxfp4_encode(rng.standard_normal((2 * n, k)))
    dev = lambda t, dt=None: torch.as_tensor(t, dtype=dt).cuda()  # noqa: E731
    ref = O.mxfp4_decode(ac, asc) @ O.mxfp4_decode(wc, wsc).reshape(2, n, k)[1].T
    for offs, mats, good in (([0, 10, 20, 41], [1, 2, 1], (0, 10)), ([-3, 10, 20, 40], [1, 1, -1], (10, 20)),
                             ([0, 30, 20, 40], [70000, 1, 1], (20, 40))):
        s = M.make_mxfp4_shape(rows, n, k, 2, 3, M.MOE_ACT_NONE, M.MOE_F32)
        ws = torch.empty(M.moe_mxfp4_workspace_size(s), dtype=torch.uint8, device="cuda")
        M.moe_mxfp4_workspace_init(s, ws)
        y = torch.full((rows, n), 77.0, device="cuda")
        M.moe_mxfp4_matmul(s, dev(ac), dev(asc), dev(offs, torch.int32), dev(mats, torch.int32), dev(wc), dev(wsc),
                           None, y, None, ws)
        assert M.moe_mxfp4_get_device_status(s, ws, clear=True) == M.MOE_DEV_BAD_ROUTING
        assert M.moe_mxfp4_get_device_status(s, ws) == 0
        got = y.double().cpu().numpy()
        inside = np.zeros(rows, bool)
        inside[good[0]:good[1]] = True
        assert np.all(got[~inside] == 77.0)
        assert np.max(np.abs(got - ref)[inside]) < 1e-3


def test_nan_block_reaches_its_row_only():
    k, n, rows = 256, 64, 130
    x = torch.randn(rows, k, device="cuda")
    x[5, 40] = float("nan")
    x[129, 0] = float("inf")
    w = torch.randn(n, k, device="cuda")
    (ac, asc), (wc, wsc) = quantize(x), quantize(w)
    s = M.make_mxfp4_shape(rows, n, k, out_dtype=M.MOE_F32)
    ws = torch.zeros(M.moe_mxfp4_workspace_size(s), dtype=torch.uint8, device="cuda")
    y = torch.empty(rows, n, device="cuda")
    M.moe_mxfp4_matmul(s, ac, asc, torch.tensor([0, rows], dtype=torch.int32, device="cuda"),
                       torch.zeros(1, dtype=torch.int32, device="cuda"), wc, wsc, None, y, None, ws)
    bad = torch.isnan(y).any(1).nonzero().flatten().tolist()
    assert bad == [5, 129] and bool(torch.isnan(y[[5, 129]]).all())


@pytest.mark.parametrize("n,rows,cols", [(1, 1, 128), (3, 130, 256), (2, 256, 1408)])
def test_tile_scales(n, rows, cols):
    s = torch.randint(0, 256, (n, rows, cols // 32), dtype=torch.uint8, generator=torch.Generator().manual_seed(rows))
    got = M.moe_mxfp4_tile_scales(s.cuda()).cpu().numpy()
    tiles = (rows + 127) // 128
    assert got.shape == (n, tiles, cols // 128, 512)
    for m in range(n):
        for r in range(128 * tiles):
            at = 16 * (r % 32) + 4 * (r % 128 // 32)
            words = got[m, r // 128, :, at:at + 4].ravel()
            assert np.array_equal(words, s[m, r].numpy() if r < rows else np.full(cols // 32, 127))


def test_matmul_repeats_bit_for_bit_captured_and_on_a_side_stream():
    k, n, rows = 640, 352, 333
    gen = torch.Generator(device="cuda").manual_seed(0)
    (ac, asc), (wc, wsc) = (quantize(torch.randn(r, k, device="cuda", generator=gen)) for r in (rows, 2 * n))
    offs = torch.tensor([0, 200, rows], dtype=torch.int32, device="cuda")
    mats = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    s = M.make_mxfp4_shape(rows, n, k, 2, 2, M.MOE_ACT_SILU, M.MOE_BF16)
    ws = torch.zeros(M.moe_mxfp4_workspace_size(s), dtype=torch.uint8, device="cuda")
    y = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")

    def call():
        M.moe_mxfp4_matmul(s, ac, asc, offs, mats, wc, wsc, None, y, None, ws)

    call()
    first = y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(5):
            y.zero_()
            call()
        assert torch.equal(y, first)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        y.zero_()
        g.replay()
        assert torch.equal(y, first)


@pytest.mark.parametrize("seed,T,d,E,K,dff", [(0, 70, 256, 8, 2, 384), (1, 300, 640, 5, 3, 128)])
def test_experts_of_a_layer_in_four_bits(seed, T, d, E, K, dff):
    """Route, dispatch, quantise, two products (the hidden activation in MXFP4 between them) and combine, as a
    prompt goes through; then the first tokens through the few-token layer with the same weights."""
    from synthetic import MoEShape, make_inputs
    sh = MoEShape("four bits", T, d, E, K, dff, dtype=M.MOE_BF16)
    inp = make_inputs(sh, seed)
    w = {}
    for name in ("W1", "W2"):
        m = inp[name].double().numpy()
        codes, scales = O.mxfp4_encode(m.reshape(-1, m.shape[-1]))
        w[name] = O.mxfp4_decode(codes, scales).reshape(m.shape)
        inp[name] = torch.tensor(codes).reshape(*m.shape[:2], -1)
        inp[name + "_scales"] = torch.tensor(scales).reshape(*m.shape[:2], -1)
    g = {k: None if v is None else v.cuda() for k, v in inp.items()}
    cfg = M.make_config(sh)
    cap, r_cap, x_rows, _ = M.moe_buffer_rows(cfg)
    i32, f32, u8 = (dict(dtype=t, device="cuda") for t in (torch.int32, torch.float32, torch.uint8))
    ws = torch.empty(M.moe_workspace_size(cfg), **u8)
    M.moe_workspace_init(cfg, ws)
    idx, gates = torch.empty((T, K), **i32), torch.empty((T, K), **f32)
    counts, kept, offs = torch.empty(E, **i32), torch.empty(E, **i32), torch.empty(E + 1, **i32)
    slot_row, row_slot = torch.empty((T, K), **i32), torch.empty(r_cap, **i32)
    xd = torch.empty((x_rows, d), dtype=torch.bfloat16, device="cuda")
    M.moe_route(cfg, g["x"], g["W_r"], None, idx, gates, None, ws)
    M.moe_dispatch(cfg, g["x"], idx, counts, kept, offs, slot_row, row_slot, xd, None, ws)
    a, asc = quantize(xd)
    mats = torch.arange(E, **i32)
    s1 = M.make_mxfp4_shape(r_cap, dff, d, E, E, M.MOE_ACT_SILU, M.MOE_MXFP4)
    s2 = M.make_mxfp4_shape(r_cap, d, dff, E, E, M.MOE_ACT_NONE, M.MOE_BF16)
    mws = torch.empty(M.moe_mxfp4_workspace_size(s1), **u8)
    M.moe_mxfp4_workspace_init(s1, mws)
    h, hsc = torch.empty((r_cap, dff // 2), **u8), torch.empty((r_cap, dff // 32), **u8)
    y = torch.empty((r_cap, d), dtype=torch.bfloat16, device="cuda")
    M.moe_mxfp4_matmul(s1, a, asc, offs, mats, g["W1"], g["W1_scales"], g["b1"], h, hsc, mws)
    M.moe_mxfp4_matmul(s2, h, hsc, offs, mats, g["W2"], g["W2_scales"], g["b2"], y, None, mws)
    out = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    M.moe_combine(cfg, y, gates, slot_row, out)
    assert M.moe_get_device_status(cfg, ws) == 0 and M.moe_mxfp4_get_device_status(s1, mws) == 0

    x = inp["x"].double().numpy()
    idx_h, gates_h = idx.cpu().numpy(), gates.double().cpu().numpy()
    xq = O.mxfp4_decode(*O.mxfp4_encode(x))
    four, exact = np.zeros((T, d)), np.zeros((T, d))
    for t in range(T):
        for k in range(K):
            e = idx_h[t, k]
            b1, b2 = inp["b1"][e].double().numpy(), inp["b2"][e].double().numpy()
            silu = lambda z: z / (1 + np.exp(-z))  # noqa: E731
            hq = O.mxfp4_decode(*O.mxfp4_encode(silu(w["W1"][e] @ xq[t] + b1)[None]))[0]
            four[t] += gates_h[t, k] * (w["W2"][e] @ hq + b2)
            exact[t] += gates_h[t, k] * (w["W2"][e] @ silu(w["W1"][e] @ x[t] + b1) + b2)
    rel = lambda u, v: np.linalg.norm(u - v) / np.linalg.norm(v)  # noqa: E731
    # y and out rounded to bf16 (2^-8 at most, each on average less than half of it), and an h within fp32's error
    # of a border (one in some 10^4) rounded to its other side, a quarter of itself away: 0.25 / 100 of the norm
    assert rel(out.double().cpu().numpy(), four) < 2.0 ** -8 + 0.0025

    n = 5
    few = M.MoELayer(M.make_config(sh, T=n, dtype=M.MOE_MXFP4), g)
    got = few.forward_few(g["x"][:n])[0].double().cpu().numpy()
    assert np.array_equal(few.topk_idx.cpu().numpy(), idx_h[:n])
    assert rel(got, exact[:n]) < 2.0 ** -8


@pytest.mark.parametrize("k", [512, 1536, 2560, 4608])
def test_matmul_rows_of_scales_that_end_inside_a_read(k):
    y, _, z, S, end = product([130, 3, 90], [1, 0, 1], 2, 320, k, M.MOE_ACT_NONE, M.MOE_F32, behind=1, seed=k)
    want, tol = bounds(z, S, k, M.MOE_ACT_NONE)
    assert np.all(np.abs(y.double().numpy() - want)[:end] <= tol[:end] + 1e-37)


@pytest.mark.parametrize("out", [M.MOE_F32, M.MOE_BF16, M.MOE_MXFP4])
def test_matmul_operands_on_16_byte_boundaries(out):
    """The same bits whatever the multiple of 16 bytes at which scales and output start."""
    k, n, rows = 2048, 192, 200
    gen = torch.Generator(device="cuda").manual_seed(1)
    (ac, asc), (wc, wsc) = (quantize(torch.randn(r, k, device="cuda", generator=gen)) for r in (rows, n))
    offs, mats = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, rows], [0]))
    s = M.make_mxfp4_shape(rows, n, k, 1, 1, M.MOE_ACT_SILU, out)
    ws = torch.zeros(M.moe_mxfp4_workspace_size(s), dtype=torch.uint8, device="cuda")
    size = rows * n * {M.MOE_F32: 8, M.MOE_BF16: 4, M.MOE_MXFP4: 1}[out] // 2

    def at(off, t):
        buf = torch.zeros(t.numel() + 64, dtype=torch.uint8, device="cuda")
        buf[off:off + t.numel()] = t.reshape(-1)
        return buf[off:off + t.numel()]

    got = []
    for off in (0, 16):
        y = at(off, torch.zeros(size, dtype=torch.uint8, device="cuda"))
        ysc = torch.zeros((rows, n // 32), dtype=torch.uint8, device="cuda") if out == M.MOE_MXFP4 else None
        M.moe_mxfp4_matmul(s, ac, at(off, asc), offs, mats, wc, at(off, wsc), None, y, ysc, ws)
        got.append((y.clone(), ysc))
    assert torch.equal(got[0][0], got[1][0]) and bool(got[0][0].any())
    assert out != M.MOE_MXFP4 or torch.equal(got[0][1], got[1][1])
