"""The few-token layer against the definition in fp64, against the ordinary
layer, and as it is used: again and again, captured, on a side stream."""
import numpy as np
import pytest
import torch

import oracle as O
import sparse_mixture_experts_20_b200 as M
from moe_testlib import rel_frob, run_layer
from synthetic import MoEShape, make_inputs

pytestmark = pytest.mark.gpu

BF16, FP8, FP4 = M.MOE_BF16, M.MOE_FP8_E4M3_BLOCK, M.MOE_MXFP4
WEIGHTS = ("W1", "W2", "Ws1", "Ws2")


def inputs(sh, kind, seed):
    """(inputs on the GPU, the experts' weights as fp64 stacks on the CPU)."""
    host = make_inputs(sh.replace(dtype=FP8 if kind == FP8 else BF16), seed)
    plain = {}
    for n in WEIGHTS:
        if host[n] is None:
            continue
        if kind == FP8:
            plain[n] = np.stack([O.dequant_blocks_128x128(c.numpy(), s.double().numpy())
                                 for c, s in zip(host[n], host[n + "_scales"])])
        elif kind == FP4:
            e, r, c = host[n].shape
            codes, scales = O.mxfp4_encode(host[n].double().numpy().reshape(e * r, c))
            plain[n] = O.mxfp4_decode(codes, scales).reshape(e, r, c)
            host[n] = torch.tensor(codes).reshape(e, r, c // 2)
            host[n + "_scales"] = torch.tensor(scales).reshape(e, r, c // 32)
        else:
            plain[n] = host[n].double().numpy()
    return {k: None if v is None else v.cuda() for k, v in host.items()}, plain


def config(sh, kind):
    return M.make_config(sh, dtype=kind)


def run(sh, kind, inp):
    layer = M.MoELayer(config(sh, kind), inp)
    n0 = M.moe_kernel_launches()
    layer.forward_few(inp["x"])
    assert M.moe_kernel_launches() == n0 + 1                         # one kernel
    torch.cuda.synchronize()
    assert M.moe_get_device_status(layer.cfg, layer._few_ws) == 0
    return layer


def definition(sh, kind, inp, plain, idx, g):
    """out and its elementwise error bound, in fp64, with the experts idx (T, K) chosen and the gates g."""
    x = inp["x"].double().cpu().numpy()
    C = O.capacity_of(sh.T, sh.top_k, sh.n_routed, sh.capacity_factor)
    kept = O.dispatch_plan(idx, sh.n_routed, C, "slot" if sh.capacity_priority else "token")["slot_row"] >= 0
    xin = x
    if kind == FP8:
        xin = O.dequant_rows_1x128(*O.quantize_rows_1x128(x))
    half = {BF16: 2.0 ** -8, FP8: 2.0 ** -4, FP4: 2.0 ** -11}[kind]  # rounding of h
    fp32 = 2.0 ** -18                                                # sums, SiLU, gates: a few hundred fp32 steps
    out, tol = np.zeros_like(x), np.zeros_like(x)

    def add(t, w, W1, b1, W2, b2):
        z, S1 = W1 @ xin[t] + b1, np.abs(W1) @ np.abs(xin[t]) + np.abs(b1)
        h = z / (1 + np.exp(-z))
        hr = O.dequant_rows_1x128(*O.quantize_rows_1x128(h[None]))[0] if kind == FP8 else h
        y = W2 @ hr + b2
        dh = 1.1 * S1 * fp32 + (half + fp32) * np.abs(h) + np.abs(h).max() * 2.0 ** -38
        out[t] += w * y
        tol[t] += w * (np.abs(W2) @ dh + fp32 * (np.abs(W2) @ np.abs(h) + np.abs(b2)))

    f = lambda n: inp[n].double().cpu().numpy()  # noqa: E731
    b1, b2 = f("b1"), f("b2")
    for t in range(sh.T):
        for k, e in enumerate(idx[t]):
            if kept[t, k]:
                add(t, g[t, k], plain["W1"][e], b1[e], plain["W2"][e], b2[e])
            elif sh.overflow_mode:
                out[t] += g[t, k] * x[t]
                tol[t] += g[t, k] * np.abs(x[t]) * fp32
        for i in range(sh.n_shared):
            add(t, 1.0, plain["Ws1"][i], f("bs1")[i], plain["Ws2"][i], f("bs2")[i])
    return out, tol + 2.0 ** -8 * (np.abs(out) + tol)


def host_routing(inp):
    return {k: None if inp[k] is None else inp[k].cpu() for k in ("x", "W_r", "logit_bias")}


def check(sh, kind, seed=0, inp=None, plain=None):
    if inp is None:
        inp, plain = inputs(sh, kind, seed)
    o = run(sh, kind, inp)
    rt = O.route(sh.replace(dtype=FP8 if kind == FP8 else BF16), host_routing(inp))
    idx = o.topk_idx.cpu().numpy()
    # an fp32 logit: at most 16 steps of the sum of its terms' magnitudes (partial sums of d / 32 / slices terms a
    # lane, five additions across the warp, the slices)
    el = 16 * 2.0 ** -24 * (np.abs(inp["x"].double().cpu().numpy()) @ np.abs(inp["W_r"].double().cpu().numpy()).T).max(1)
    ok = rt["gap"] >= 2 * el
    # order within the chosen: equal up to logits that are as close as that
    key = rt["logits"] + (inp["logit_bias"].double().cpu().numpy() if sh.bias_mode and inp["logit_bias"] is not None
                          else 0.0)
    a, b = np.take_along_axis(key, idx, 1), np.take_along_axis(key, rt["idx"], 1)
    assert np.all((np.abs(a - b) <= 2 * el[:, None])[ok])
    assert all(len(set(r)) == sh.top_k for r in idx.tolist())
    s = O.softmax(rt["logits"])
    g = np.take_along_axis(s, idx, 1)
    # softmax moves by at most the largest change of a logit (relative 2 el)
    assert np.all(np.abs(o.gates.cpu().numpy() - g / g.sum(1, keepdims=True)) <= 2 * el[:, None] + 2.0 ** -20)
    counts = np.bincount(idx.ravel(), minlength=sh.n_routed)
    assert np.array_equal(o.counts.cpu().numpy(), counts)
    f, P = counts / (sh.T * sh.top_k), s.mean(0)
    assert np.max(np.abs(o.f.cpu().numpy() - f)) < 1e-6
    assert np.max(np.abs(o.P.cpu().numpy() - P)) <= np.mean(2 * el) + 2.0 ** -20
    loss = sh.alpha * sh.n_routed * (f * P).sum()
    assert abs(float(o.loss[0]) - loss) <= sh.alpha * sh.n_routed * (np.mean(2 * el) + 2.0 ** -20)
    want, tol = definition(sh, kind, inp, plain, idx, o.gates.double().cpu().numpy())
    got = o.out.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol)
    # in the 2-norm: the output's rounding (at most 2^-8, on average a good half of it) and that of h, which
    # averages out over the hidden columns; FP8: an h next to a border may round to the other side
    assert rel_frob(got, want) < (1e-2 if kind == FP8 else 5e-3)
    return o


def shape(T, d, E, K, dff, S=0, dffs=0, **kw):
    return MoEShape("few", T, d, E, K, dff, n_shared=S, d_ff_shared=dffs, **kw)


# T, d, E, K, dff, S, dffs: one token and sixteen, one expert and 256, widths from the smallest up, odd numbers of
# 128-byte pieces, more rows per block than one job holds
COMMON = [
    (1, 128, 1, 1, 128, 0, 0), (1, 128, 8, 2, 256, 0, 0), (2, 256, 3, 3, 128, 1, 128), (7, 640, 13, 4, 384, 2, 256),
    (8, 128, 256, 8, 128, 0, 0), (9, 384, 5, 2, 1408, 0, 0), (16, 1152, 64, 8, 256, 3, 128), (16, 128, 2, 1, 128, 8, 128),
    (3, 2048, 33, 16, 640, 1, 1280), (16, 256, 4, 4, 5120, 0, 0), (5, 4224, 6, 2, 896, 0, 0),
]


@pytest.mark.parametrize("kind", [BF16, FP8, FP4])
@pytest.mark.parametrize("case", range(len(COMMON)))
def test_against_definition(case, kind):
    check(shape(*COMMON[case]), kind, seed=case)


@pytest.mark.parametrize("dims", [(1, 64, 2, 1, 64, 0, 0), (4, 192, 7, 3, 64, 1, 64), (13, 320, 9, 2, 448, 2, 192)])
def test_bf16_multiples_of_64(dims):
    check(shape(*dims), BF16, seed=7)


@pytest.mark.parametrize("kind", [BF16, FP8, FP4])
@pytest.mark.parametrize("kw", [
    dict(capacity_factor=0.5), dict(capacity_factor=0.3, overflow_mode=1), dict(capacity_factor=0.6, capacity_priority=1),
    dict(capacity_factor=0.4, capacity_priority=1, overflow_mode=1, selection_bias=True, bias_mode=1),
    dict(selection_bias=True), dict(selection_bias=True, bias_mode=1), dict(zipf_logit_bias=True),
])
def test_routing_variants(kw, kind):
    check(shape(14, 256, 6, 3, 256, 1, 128, **kw), kind, seed=11)


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_same_layer_as_the_ordinary_one(kind):
    sh = shape(12, 512, 16, 4, 512, 1, 256, capacity_factor=1.0, overflow_mode=1, dtype=kind)
    inp, _ = inputs(sh, kind, 3)
    a, b = run(sh, kind, inp), run_layer(sh, inp)
    assert torch.equal(a.topk_idx, b["topk_idx"]) and torch.equal(a.counts, b["counts"])
    assert float((a.gates - b["gates"]).abs().max()) < 1e-5
    # the ordinary layer rounds every slot's output to bf16 as well
    assert rel_frob(a.out.double().cpu().numpy(), b["out"].double().cpu().numpy()) < 1e-2


def test_ties_go_to_the_lower_expert():
    sh = shape(3, 128, 40, 5, 128)
    inp, plain = inputs(sh, BF16, 5)
    inp["W_r"][7:31] = inp["W_r"][3]
    o = run(sh, BF16, inp)
    logits = inp["x"].double() @ inp["W_r"].double().T
    for t in range(3):
        row = o.topk_idx[t].tolist()
        want = sorted(range(40), key=lambda e: (-round(float(logits[t, e]), 4), e))[:5]
        assert row == want


@pytest.mark.parametrize("kind", [BF16, FP8, FP4])
def test_large_and_small_magnitudes(kind):
    """Tokens of very different size (and one of zeros) in one call."""
    sh = shape(6, 256, 4, 2, 256, 1, 128)
    inp, plain = inputs(sh, kind, 9)
    scale = torch.tensor([1e-30, 1e4, 0.0, 1.0, 1e-6, 3e2], device="cuda")
    inp["x"] = (inp["x"].float() * scale[:, None]).bfloat16()
    check(sh, kind, inp=inp, plain=plain)


@pytest.mark.parametrize("kind", [BF16, FP4])
def test_broken_weights_reach_only_their_tokens(kind):
    """An expert with NaN and infinite weights: the tokens that did not choose it do not see it."""
    sh = shape(10, 256, 4, 1, 256)
    inp, plain = inputs(sh, kind, 2)
    clean = run(sh, kind, inp).out.clone()
    idx = O.route(sh.replace(dtype=BF16), host_routing(inp))["idx"][:, 0]
    e = int(idx[0])
    if kind == BF16:
        inp["W2"][e, 17, 33] = float("nan")
        inp["W1"][e, 3, 5] = float("inf")
    else:
        inp["W2_scales"][e, 17, 1] = 255
        inp["W1_scales"][e, 3, 0] = 255
    out = run(sh, kind, inp).out
    hit = torch.tensor(idx == e)
    assert bool(hit.any()) and not bool(hit.all())
    assert torch.equal(out[~hit.cuda()], clean[~hit.cuda()])
    assert bool(torch.isnan(out[hit.cuda()]).any(1).all())


def test_nan_token_stays_alone():
    sh = shape(4, 256, 8, 2, 256, 1, 128)
    for kind in (BF16, FP4):
        inp, plain = inputs(sh, kind, 4)
        clean = run(sh, kind, inp).out.clone()
        inp["x"][2, 100] = float("nan")
        o = run(sh, kind, inp)
        rest = [0, 1, 3]
        assert torch.equal(o.out[rest], clean[rest])
        assert bool(torch.isnan(o.out[2]).all())
        row = o.topk_idx[2].tolist()
        assert len(set(row)) == 2 and all(0 <= e < 8 for e in row)


@pytest.mark.parametrize("kind", [BF16, FP8, FP4])
def test_calls_in_a_row_are_bit_identical(kind):
    sh = shape(11, 512, 16, 4, 384, 1, 128)
    inp, _ = inputs(sh, kind, 6)
    layer = run(sh, kind, inp)
    first = [t.clone() for t in (layer.out, layer.f, layer.P, layer.loss, layer.topk_idx, layer.gates)]
    for _ in range(20):
        layer.out.fill_(9.0)
        layer.forward_few(inp["x"])
        now = (layer.out, layer.f, layer.P, layer.loss, layer.topk_idx, layer.gates)
        assert all(torch.equal(a, b) for a, b in zip(first, now))


@pytest.mark.parametrize("kind", [BF16, FP8, FP4])
def test_captured_and_on_a_side_stream(kind):
    """A graph of two layers (one workspace each), replayed on new tokens, against calls on a side stream."""
    sh = shape(5, 256, 8, 2, 256, 1, 128)
    pair = [inputs(sh, kind, s)[0] for s in (1, 2)]
    layers = [M.MoELayer(config(sh, kind), i) for i in pair]
    x = pair[0]["x"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for la in layers:
            la.forward_few(x)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mid = layers[0].forward_few(x)[0]
        layers[1].forward_few(mid)
    for seed in (3, 4, 5):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))
        g.replay()
        got = layers[1].out.clone()
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layers[1].forward_few(layers[0].forward_few(x)[0])
        side.synchronize()
        assert torch.equal(got, layers[1].out)
        assert all(M.moe_get_device_status(la.cfg, la._few_ws) == 0 for la in layers)


def test_optional_outputs_may_be_left_out():
    sh = shape(3, 256, 8, 2, 256)
    inp, _ = inputs(sh, BF16, 8)
    ref = run(sh, BF16, inp)
    cfg = config(sh, BF16)
    ws = torch.empty(M.moe_few_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    M.moe_few_workspace_init(cfg, ws)
    out, f, P, loss = (torch.empty_like(t) for t in (ref.out, ref.f, ref.P, ref.loss))
    g = inp.get
    M.moe_layer_forward_few(cfg, inp["x"], g("W_r"), None, g("W1"), None, g("b1"), g("W2"), None, g("b2"), None, None,
                            None, None, None, None, out, f, P, loss, None, None, None, ws)
    assert torch.equal(out, ref.out) and torch.equal(P, ref.P) and torch.equal(loss, ref.loss)


def test_fp8_scales_that_differ_from_block_to_block():
    """Each weight block at its own size: a scale taken from a neighbouring block would show."""
    sh = shape(9, 512, 4, 2, 384, 1, 256)
    inp, plain = inputs(sh, FP8, 12)
    gen = torch.Generator().manual_seed(1)
    for n in WEIGHTS:
        s = inp[n + "_scales"]
        m = torch.randint(-3, 4, s.shape, generator=gen).cuda()
        s.mul_(2.0 ** m)
        plain[n] = plain[n] * np.repeat(np.repeat(2.0 ** m.double().cpu().numpy(), 128, 1), 128, 2)
    check(sh, FP8, inp=inp, plain=plain)


def test_rows_past_one_job_and_wide_layers():
    """d_model above 128 output rows per block on the whole device (two row ranges), MXFP4."""
    check(shape(2, 128 * 152, 2, 1, 128), FP4, seed=1)


@pytest.mark.parametrize("kind", [BF16, FP8, FP4])
def test_more_columns_than_one_job_holds(kind):
    """A row of weights longer than 64 pieces (of 64, 128 or 256 columns), with an odd number of them."""
    long = 128 * 129 if kind != FP4 else 128 * 259
    check(shape(3, long, 4, 2, 128, 1, 128), kind, seed=2)
    check(shape(3, 128, 4, 2, long, 1, 128), kind, seed=3)


@pytest.mark.parametrize("kind,wide", [(BF16, 0), (FP8, 0), (FP4, 0), (BF16, 19200), (FP8, 20480)])
def test_work_in_large_and_small_shares(kind, wide):
    """Enough weights that a block has 64 slots and more in both phases, where the last shares are small; and more
    tiles of output rows than there are blocks."""
    T, E, dff = 2, 4, 8448
    d = wide or {BF16: 4608, FP8: 9216, FP4: 18432}[kind]
    if wide:
        dff = 2560 if kind == BF16 else 5120
    gen = torch.Generator(device="cuda").manual_seed(5)

    def weights(rows, cols):
        """(stack as the layer takes it, its scales, expert e's matrix in fp64)."""
        if kind == FP4:
            codes = torch.randint(0, 256, (E, rows, cols // 2), dtype=torch.uint8, device="cuda", generator=gen)
            scales = torch.randint(118, 121, (E, rows, cols // 32), dtype=torch.uint8, device="cuda", generator=gen)

            def plain(e):
                out = torch.empty((rows, cols), device="cuda")
                M.moe_mxfp4_dequantize(codes[e], scales[e], out)
                return out.double()
            return codes, scales, plain
        w = torch.randn((E, rows, cols), device="cuda", generator=gen)
        if kind == BF16:
            w = (w / cols ** 0.5).bfloat16()
            return w, None, lambda e: w[e].double()
        w = w.to(torch.float8_e4m3fn)
        scales = 2.0 ** torch.randint(-8, -5, (E, (rows + 127) // 128, cols // 128), device="cuda", generator=gen)
        grid = lambda e: scales[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)[:rows]  # noqa: E731
        return w.view(torch.uint8), scales, lambda e: w[e].double() * grid(e)

    W1, s1, plain1 = weights(dff, d)
    W2, s2, plain2 = weights(d, dff)
    f32 = lambda *n: torch.randn(n, device="cuda", generator=gen) / 8  # noqa: E731
    inp = dict(x=torch.randn((T, d), device="cuda", generator=gen).bfloat16(), W_r=f32(E, d) / d ** 0.5, logit_bias=None,
               W1=W1, W1_scales=s1, b1=f32(E, dff), W2=W2, W2_scales=s2, b2=f32(E, d), Ws1=None, Ws1_scales=None,
               bs1=None, Ws2=None, Ws2_scales=None, bs2=None)
    o = run(shape(T, d, E, E, dff), kind, inp)
    x = inp["x"].double()
    q = lambda v: torch.tensor(O.dequant_rows_1x128(*O.quantize_rows_1x128(v.cpu().numpy()))).cuda()  # noqa: E731
    if kind == FP8:
        x = q(x)
    want = torch.zeros((T, d), dtype=torch.float64, device="cuda")
    for e in range(E):
        h = torch.nn.functional.silu(x @ plain1(e).T + inp["b1"][e].double())
        y = (q(h) if kind == FP8 else h) @ plain2(e).T + inp["b2"][e].double()
        want += torch.where(o.topk_idx == e, o.gates, 0.0).sum(1, dtype=torch.float64)[:, None] * y
    # as in check(): the output's rounding, and an FP8 h that rounds to the other side of a border
    assert float((o.out.double() - want).norm() / want.norm()) < (1e-2 if kind == FP8 else 5e-3)
    first = o.out.clone()
    for _ in range(5):
        o.forward_few(inp["x"])
        assert torch.equal(o.out, first)


def test_fp8_scales_far_apart_within_a_row():
    """Scales of neighbouring column blocks that differ by up to 2^16."""
    sh = shape(4, 1152, 3, 2, 640, 1, 256)
    inp, plain = inputs(sh, FP8, 13)
    gen = torch.Generator().manual_seed(2)
    for n in WEIGHTS:
        s = inp[n + "_scales"]
        m = torch.randint(-8, 9, s.shape, generator=gen).cuda()
        s.mul_(2.0 ** m)
        plain[n] = plain[n] * np.repeat(np.repeat(2.0 ** m.double().cpu().numpy(), 128, 1), 128, 2)
    check(sh, FP8, inp=inp, plain=plain)


@pytest.mark.parametrize("kind", [BF16, FP8, FP4])
def test_two_layers_at_once_on_two_streams(kind):
    """Each with its workspace, on streams that overlap, beside other kernels: the results of one after the other."""
    shapes = [shape(5, 1024, 16, 4, 512, 1, 256), shape(1, 128, 8, 2, 256)]
    made = [inputs(sh, kind, 20 + i)[0] for i, sh in enumerate(shapes)]
    layers = [M.MoELayer(config(sh, kind), inp) for sh, inp in zip(shapes, made)]
    want = []
    for la, inp in zip(layers, made):
        want.append(la.forward_few(inp["x"])[0].clone())
    streams = [torch.cuda.Stream() for _ in layers]
    got = [[], []]
    busy = torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    for _ in range(30):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(layers[i].forward_few(made[i]["x"])[0].clone())
        busy = busy * 1.0001
    torch.cuda.synchronize()
    for la, w, g in zip(layers, want, got):
        assert all(torch.equal(w, t) for t in g)
        assert M.moe_get_device_status(la.cfg, la._few_ws) == 0


@pytest.mark.parametrize("kind", [BF16, FP8, FP4])
def test_output_in_place_of_the_input(kind):
    sh = shape(7, 512, 12, 3, 256, 1, 128, capacity_factor=0.5, overflow_mode=1)
    inp, _ = inputs(sh, kind, 21)
    layer = run(sh, kind, inp)
    want = layer.out.clone()
    layer.out.copy_(inp["x"])
    layer.forward_few(layer.out)
    assert torch.equal(layer.out, want)
