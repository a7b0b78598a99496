"""The few-token layer with MXFP4 weights, where columns of very different size share a block of 32: x and the hidden
activation are held to the bound that the header states, not to their own roundings."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_20_b200 as M
from test_gpu_few import FP4, inputs, run, shape

pytestmark = pytest.mark.gpu

FP32 = 2.0 ** -18                                               # sums, SiLU, gates: a few hundred fp32 steps


def held(v):
    """How far a value may be from itself as an operand: max(amax / 12288, 2^-126) of its block of 32 columns."""
    b = np.abs(v).reshape(*v.shape[:-1], -1, 32).max(-1)
    return np.repeat(np.maximum(b / 12288, 2.0 ** -126), 32, axis=-1)


def check(sh, inp, plain):
    """The layer against fp64 on the experts and gates that it chose."""
    o = run(sh, FP4, inp)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    x, idx, g = f(inp["x"]), o.topk_idx.cpu().numpy(), f(o.gates)
    ex = held(x)
    out, tol = np.zeros_like(x), np.zeros_like(x)

    def add(t, w, W1, b1, W2, b2):
        z, S = W1 @ x[t] + b1, np.abs(W1) @ np.abs(x[t]) + np.abs(b1)
        with np.errstate(over="ignore"):
            h = z / (1 + np.exp(-z))
        dh = 1.1 * (np.abs(W1) @ ex[t] + S * FP32) + FP32 * np.abs(h)        # SiLU's slope is at most 1.1
        dh = dh + held(np.abs(h) + dh)
        out[t] += w * (W2 @ h + b2)
        tol[t] += w * (np.abs(W2) @ dh + FP32 * (np.abs(W2) @ np.abs(h) + np.abs(b2)))

    for t in range(sh.T):
        for k, e in enumerate(idx[t]):
            add(t, g[t, k], plain["W1"][e], f(inp["b1"][e]), plain["W2"][e], f(inp["b2"][e]))
        for i in range(sh.n_shared):
            add(t, 1.0, plain["Ws1"][i], f(inp["bs1"][i]), plain["Ws2"][i], f(inp["bs2"][i]))
    tol += 2.0 ** -8 * (np.abs(out) + tol)                                   # the output's rounding to bf16
    assert np.all(np.abs(f(o.out) - out) <= tol)
    return o


@pytest.mark.parametrize("loud", [8.0, 1e3, 1e5])
def test_one_large_column_in_every_block(loud):
    """In x, and through b1 in the hidden activation."""
    sh = shape(9, 256, 4, 2, 384, 1, 128)
    inp, plain = inputs(sh, FP4, 41)
    for name in ("x", "b1", "bs1"):
        for c in range(inp[name].shape[1] // 32):
            inp[name][:, 32 * c + (7 * c + 3) % 32] *= loud
    check(sh, inp, plain)


def test_blocks_at_the_lower_end_of_the_range():
    """Tokens down to where no plane but the first has a scale, through weights that bring them back up."""
    sh = shape(8, 256, 2, 2, 128, 1, 128)
    inp, plain = inputs(sh, FP4, 42)
    size = torch.tensor([2.0 ** -p for p in (106, 112, 114, 116, 118, 120, 122, 125)], device="cuda")
    inp["x"] = (inp["x"].float() * size[:, None]).bfloat16()
    for name in ("W1", "Ws1"):
        inp[name + "_scales"] += 110
        plain[name] = plain[name] * 2.0 ** 110
    check(sh, inp, plain)
