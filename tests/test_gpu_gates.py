"""Gates under a selection-only bias, where the experts chosen lie far below the largest logit: the softmax over the
chosen ones, as defined, whatever the other logits are."""
import numpy as np
import pytest
import torch

import moe_testlib as TL
import oracle as O
import sparse_mixture_experts_20_b200 as M
from synthetic import MoEShape
from test_gpu_backward import TOL, _grad_buffers
from test_gpu_few import BF16, FP4, FP8, host_routing, inputs, run

pytestmark = pytest.mark.gpu


def far(sh, kind, lead, seed):
    """Inputs where expert 0's logit is `lead` above zero for every token and a bias of -1e5 keeps it from being
    chosen; the gates by the definition, and how far an fp32 softmax over the chosen logits may be from them."""
    inp, _ = inputs(sh, kind, seed)
    inp["x"][:, 0] = 1.0
    inp["W_r"][0] = 0.0
    inp["W_r"][0, 0] = lead
    inp["logit_bias"] = torch.zeros(sh.n_routed, device="cuda")
    inp["logit_bias"][0] = -1e5
    h = host_routing(inp)
    x, W = h["x"].double().numpy(), h["W_r"].double().numpy()
    logits = x @ W.T
    order = np.argsort(-(logits + h["logit_bias"].double().numpy()), axis=1, kind="stable")[:, :sh.top_k]
    # a logit: at most 16 fp32 steps of the sum of its terms' magnitudes (an fp32 router; a three-plane bf16 one is
    # nearer); a gate moves by at most twice the largest change of a chosen logit, relative to itself
    el = 16 * 2.0 ** -24 * np.take_along_axis(np.abs(x) @ np.abs(W).T, order, 1).max(1)
    top = np.take_along_axis(logits, order, 1)
    e = np.exp(top - top.max(1, keepdims=True))
    return inp, logits, order, e / e.sum(1, keepdims=True), 2 * el[:, None] + 2.0 ** -20


def check(logits, idx, gates, order, want, tol):
    """Tokens whose chosen set is clear of ties: the same experts, the same gates."""
    idx, gates = idx.cpu().numpy(), gates.double().cpu().numpy()
    assert np.all(np.isfinite(gates))
    clear = np.all(idx == order, axis=1)
    assert clear.mean() > 0.9
    assert np.all(np.abs(gates - want)[clear] <= tol[clear] * want[clear] + 2.0 ** -24)
    assert np.all(idx != 0)


@pytest.mark.parametrize("lead", [20.0, 95.0, 150.0, 3e4])
@pytest.mark.parametrize("kind", [BF16, FP8, FP4])
def test_few_tokens(kind, lead):
    sh = MoEShape("few", 14, 256, 12, 4, 128, bias_mode=1)
    inp, logits, order, want, tol = far(sh, kind, lead, 31)
    o = run(sh, kind, inp)
    check(logits, o.topk_idx, o.gates, order, want, tol)
    assert bool(torch.isfinite(o.out.float()).all()) and bool((o.out != 0).any(1).all())
    # the probabilities stay those of all experts
    p = np.exp(logits - logits.max(1, keepdims=True))
    assert np.max(np.abs(o.P.double().cpu().numpy() - (p / p.sum(1, keepdims=True)).mean(0))) < 1e-4


# experts: the small router, the generic one (fp32) and the tensor-core one
@pytest.mark.parametrize("lead", [20.0, 95.0, 150.0, 3e4])
@pytest.mark.parametrize("dtype,E", [(M.MOE_F32, 8), (BF16, 8), (M.MOE_F32, 96), (BF16, 96), (FP8, 256)])
def test_ordinary_router(dtype, E, lead):
    sh = MoEShape("far", 70, 256, E, 4, 128, bias_mode=1, dtype=dtype)
    inp, logits, order, want, tol = far(sh, dtype, lead, 32)
    if dtype == M.MOE_F32:
        inp = {**TL.gpu_inputs(sh, 32), **{k: inp[k] for k in ("W_r", "logit_bias")}, "x": inp["x"].float()}
    o = TL.run_layer(sh, inp)
    check(logits, o["topk_idx"], o["gates"], order, want, tol)
    assert bool(torch.isfinite(o["out"].float()).all())


@pytest.mark.parametrize("lead", [20.0, 60.0, 75.0, 95.0, 150.0])
@pytest.mark.parametrize("dtype", [M.MOE_F32, BF16])
def test_backward(dtype, lead):
    """The gradients through those gates, against the oracle's in fp64."""
    sh = MoEShape("far", 60, 256, 8, 3, 128, bias_mode=1, dtype=dtype)
    inp = far(sh, BF16, lead, 33)[0]
    if dtype == M.MOE_F32:
        inp = {**TL.gpu_inputs(sh, 33), **{k: inp[k] for k in ("W_r", "logit_bias")}, "x": inp["x"].float()}
    o = TL.run_stages(sh, inp)
    dout = torch.randn(inp["x"].shape, generator=torch.Generator().manual_seed(1)).to(inp["x"].dtype)
    grads = _grad_buffers(sh, inp, "cuda")
    tensors = {k: inp[k] for k in ("x", "W_r", "W1", "b1", "W2", "b2")}
    tensors.update({k: o[k] for k in ("logits", "topk_idx", "gates", "counts", "offsets", "slot_row", "row_slot", "x_disp",
                                      "y")})
    bws = torch.empty(M.moe_backward_workspace_size(o["cfg"]), dtype=torch.uint8, device="cuda")
    M.moe_layer_backward(o["cfg"], 1.0, {**tensors, "dout": dout.cuda(), **grads}, bws)
    host = {k: TL.cpu(v) for k, v in inp.items()}
    rt = O.route(sh, host, logits=TL.cpu(o["logits"]).double().numpy())
    assert np.array_equal(rt["idx"], TL.cpu(o["topk_idx"]).numpy()) and not np.any(rt["idx"] == 0)
    ref = O.layer_backward(sh, host, O.to_f64(dout), lam=1.0, routing=rt)
    for k, v in grads.items():
        got, want = TL.cpu(v).double().numpy(), ref["logit_bias" if k == "d_logit_bias" else k[1:]]
        assert np.isfinite(got).all(), k
        if np.linalg.norm(want) == 0.0:
            assert np.all(got == 0.0), k
        else:
            assert TL.rel_frob(got, want) < TOL[dtype], k
