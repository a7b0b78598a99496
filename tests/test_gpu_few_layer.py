"""MoELayer.forward_few on streams of its own, and what the layer says of its calls."""
import pytest
import torch

import sparse_mixture_experts_20_b200 as M
from test_gpu_few import BF16, FP4, FP8, config, inputs, run, shape

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("kind", [BF16, FP8, FP4])
def test_first_call_on_a_given_stream(kind, raw):
    """While the current stream is busy with what was queued before the layer was built, and both streams' freed
    memory is full of ones."""
    sh = shape(6, 256, 8, 2, 256, 1, 128)
    inp, _ = inputs(sh, kind, 3)
    want = run(sh, kind, inp).out.clone()
    n = M.moe_few_workspace_size(config(sh, kind))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for st in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(st):
            dirty = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
            del dirty
    torch.cuda.synchronize()
    late = torch.zeros(n, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(20_000_000)                               # some 10 ms
    late.fill_(255)
    del late                                                    # the current stream still writes it
    layer = M.MoELayer(config(sh, kind), inp)
    for _ in range(3):
        layer.forward_few(inp["x"], stream=side.cuda_stream if raw else side)
    side.synchronize()
    assert torch.equal(layer.out, want)
    torch.cuda.synchronize()
    assert M.moe_get_device_status(layer.cfg, layer._few_ws) == 0


@pytest.mark.parametrize("kind", [BF16, FP8, FP4])
def test_first_call_within_a_capture(kind):
    """Refused where the graph alone would clear the workspace; then made before, captured and replayed."""
    sh = shape(3, 256, 8, 2, 128)
    inp, _ = inputs(sh, kind, 4)
    want = run(sh, kind, inp).out.clone()
    layer = M.MoELayer(config(sh, kind), inp)
    graph = torch.cuda.CUDAGraph()
    if kind != FP4:
        with pytest.raises(RuntimeError, match="before capturing"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                layer.forward_few(inp["x"])
        layer.forward_few(inp["x"])
        assert torch.equal(layer.out, want)
    with torch.cuda.graph(graph):
        layer.forward_few(inp["x"])
    for _ in range(2):
        layer.out.zero_()
        graph.replay()
        assert torch.equal(layer.out, want)


@pytest.mark.parametrize("kind", [BF16, FP8, FP4])
def test_device_status_reports_the_few_token_calls(kind):
    sh = shape(2, 256, 8, 2, 128)
    inp, _ = inputs(sh, kind, 5)
    layer = run(sh, kind, inp)
    assert layer.device_status() == 0
    layer._few_ws[:4].view(torch.int32).fill_(M.MOE_DEV_TIMEOUT)          # as a wait that gave up leaves it
    assert layer.device_status() == M.MOE_DEV_TIMEOUT
    side = torch.cuda.Stream()
    assert layer.device_status(clear=True, stream=side) == M.MOE_DEV_TIMEOUT
    side.synchronize()
    assert layer.device_status() == 0
    want = layer.out.clone()
    layer.forward_few(inp["x"])
    assert torch.equal(layer.out, want) and layer.device_status() == 0


def test_tiled_scales_on_a_given_stream():
    """While the current stream still writes what it has freed."""
    scales = torch.randint(0, 256, (5, 300, 64), dtype=torch.uint8, generator=torch.Generator().manual_seed(1)).cuda()
    want = M.moe_mxfp4_tile_scales(scales)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = torch.empty_like(want)
    torch.cuda._sleep(20_000_000)
    late.fill_(255)
    del late
    got = M.moe_mxfp4_tile_scales(scales, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("kind", [BF16, FP8, FP4])
def test_layers_of_several_lengths_share_their_weights(kind):
    sh = shape(6, 256, 8, 2, 256, 1, 128)
    inp, _ = inputs(sh, kind, 6)
    first = run(sh, kind, inp)
    for T in (1, 3, 6):
        other = M.MoELayer(M.make_config(sh, T=T, dtype=kind), first.w)
        assert all(other.w[k] is v for k, v in first.w.items())
        out = other.forward_few(inp["x"][:T])[0]
        assert torch.equal(out, first.out[:T]) and other.device_status() == 0
