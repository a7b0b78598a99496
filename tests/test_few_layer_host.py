"""MoELayer.forward_few around its launch, without a GPU: streams, and what it checks of its tensors."""
import contextlib
import types

import pytest
import torch

import sparse_mixture_experts_20_b200 as M


class Stream:
    def __init__(self, handle, capturing=False):
        self.cuda_stream, self.capturing, self.waited = handle, capturing, []

    def wait_stream(self, other):
        self.waited.append(other.cuda_stream)


@pytest.fixture
def world(monkeypatch):
    """Streams, the workspace's clearing and the launch, as a log of (what, stream handle)."""
    w = types.SimpleNamespace(now=Stream(0), log=[])

    @contextlib.contextmanager
    def stream(s):
        before = w.now
        w.now = before if s is None else s
        yield
        w.now = before

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: w.now)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: w.now.capturing)
    monkeypatch.setattr(M, "_p", lambda t: None if t is None else t.data_ptr())
    real = M.lib()

    def launch(*a):
        w.log.append(("launch", a[-1]))
        return M.MOE_OK

    fake = types.SimpleNamespace(moe_few_workspace_size=real.moe_few_workspace_size, moe_layer_forward_few=launch)
    monkeypatch.setattr(M, "lib", lambda: fake)
    monkeypatch.setattr(M, "moe_few_workspace_init",
                        lambda cfg, ws, stream=None: w.log.append(("clear", M._stream(stream))))
    return w


def layer(dtype=M.MOE_BF16, **weights):
    """A layer of T = 4, d = 256, 8 experts of 128 on the CPU, which only the launch above may run."""
    la = M.MoELayer.__new__(M.MoELayer)
    la.cfg = M.make_config(T=4, d_model=256, n_routed=8, top_k=2, d_ff=128, dtype=dtype)
    la._cfg_ref, la.device, la.w, la._few_ws = None, torch.device("cpu"), weights, None
    la.ws = torch.zeros(256, dtype=torch.uint8)
    la.out = torch.zeros(4, 256, dtype=torch.bfloat16)
    la.f = la.P = la.loss = la.topk_idx = la.gates = la.counts = None
    return la


def test_first_call_clears_the_workspace_on_its_own_stream(world):
    la, side = layer(), Stream(7)
    la.forward_few(la.out, stream=side)
    assert world.log == [("clear", 7), ("launch", 7)]
    assert side.waited == [0]                                   # the layer may just have been built there
    la.forward_few(la.out)
    assert world.log[2:] == [("launch", 0)]


def test_first_call_on_the_current_stream(world):
    la = layer()
    la.forward_few(la.out)
    assert world.log == [("clear", 0), ("launch", 0)]


def test_first_call_on_a_raw_handle(world, monkeypatch):
    made = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h: made.append(Stream(h)) or made[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: Stream(0))
    la = layer()
    la.forward_few(la.out, stream=9)
    assert world.log == [("clear", 9), ("launch", 9)] and made[0].waited == [0]
    la, world.now, world.log[:] = layer(), Stream(5), []
    la.forward_few(la.out, stream=0)
    assert world.log == [("clear", 0), ("launch", 0)]


def test_first_call_of_a_four_bit_layer_waits_for_its_building(world):
    la, side = layer(M.MOE_MXFP4), Stream(7)
    la.forward_few(la.out, stream=side)
    assert world.log == [("launch", 7)] and side.waited == [0]


@pytest.mark.parametrize("where", ["current", "given"])
def test_first_call_within_a_capture(world, where):
    """A bf16 layer's workspace would be cleared by the graph alone; a four-bit layer has its own already."""
    cap = Stream(7, capturing=True)
    stream = cap if where == "given" else None
    world.now = Stream(0) if where == "given" else cap
    la = layer()
    with pytest.raises(RuntimeError, match="before capturing"):
        la.forward_few(la.out, stream=stream)
    assert world.log == []
    four = layer(M.MOE_MXFP4)
    four.forward_few(four.out, stream=stream)
    assert world.log == [("launch", 7)] and cap.waited == [] and four._few_ws is None
    la._few_ws = torch.zeros(256, dtype=torch.uint8)
    la.forward_few(la.out, stream=stream)
    assert world.log[1:] == [("launch", 7)]


def test_device_status_holds_both_workspaces(monkeypatch):
    words = {}

    def read(cfg, ws, stream=None, clear=False):
        v = words[id(ws)]
        if clear:
            words[id(ws)] = 0
        return v

    monkeypatch.setattr(M, "moe_get_device_status", read)
    la = layer()
    words[id(la.ws)] = M.MOE_DEV_BAD_ROUTING
    assert la.device_status() == M.MOE_DEV_BAD_ROUTING          # no few-token call so far
    la._few_ws = torch.zeros(256, dtype=torch.uint8)
    words[id(la._few_ws)] = M.MOE_DEV_TIMEOUT
    assert la.device_status() == M.MOE_DEV_BAD_ROUTING | M.MOE_DEV_TIMEOUT
    assert la.device_status(clear=True) == M.MOE_DEV_BAD_ROUTING | M.MOE_DEV_TIMEOUT
    assert la.device_status() == 0


def weights(dtype):
    """The tensors of layer() as a user holds them (MXFP4 scales tiled)."""
    E, d, ff = 8, 256, 128
    w = dict(W_r=torch.zeros(E, d), logit_bias=torch.zeros(E), b1=torch.zeros(E, ff), b2=torch.zeros(E, d))
    for n, rows, cols in (("W1", ff, d), ("W2", d, ff)):
        if dtype == M.MOE_BF16:
            w[n] = torch.zeros(E, rows, cols, dtype=torch.bfloat16)
        elif dtype == M.MOE_FP8_E4M3_BLOCK:
            w[n] = torch.zeros(E, rows, cols, dtype=torch.float8_e4m3fn)
            w[n + "_scales"] = torch.zeros(E, rows // 128, cols // 128)
        else:
            w[n] = torch.zeros(E, rows, cols // 2, dtype=torch.uint8)
            w[n + "_scales"] = torch.zeros(E, rows // 128, cols // 128, 512, dtype=torch.uint8)
    return w


KINDS = [M.MOE_BF16, M.MOE_FP8_E4M3_BLOCK, M.MOE_MXFP4]


@pytest.mark.parametrize("dtype", KINDS)
def test_weights_of_the_layers_types_are_taken(dtype, monkeypatch):
    monkeypatch.setattr(M, "moe_few_workspace_init", lambda cfg, ws: None)
    w = weights(dtype)
    layer(dtype, **w)._few_workspace()
    layer(dtype, **{k: v.view(torch.uint8) for k, v in w.items()})._few_workspace()          # their bytes
    layer(dtype, **{k: v.flatten() for k, v in w.items()})._few_workspace()
    layer(dtype, **{k: torch.cat([v, v]) for k, v in w.items()})._few_workspace()            # more experts than routed


@pytest.mark.parametrize("dtype", KINDS)
def test_weights_of_other_types_are_refused(dtype, monkeypatch):
    """Larger ones too, which a comparison of sizes would let through."""
    monkeypatch.setattr(M, "moe_few_workspace_init", lambda cfg, ws: None)
    w = weights(dtype)
    for name, t in w.items():
        for other in (torch.float64, torch.float16, torch.int64, torch.bfloat16 if t.dtype != torch.bfloat16 else torch.float32):
            with pytest.raises(ValueError, match=f"{name} is torch"):
                layer(dtype, **{**w, name: torch.zeros(t.shape, dtype=other)})._few_workspace()
    # the matrices of another form: eight bits for four, twice the rows of half the length
    for name in ("W1", "W2"):
        for bad in (torch.cat([w[name], w[name]], -1), w[name].reshape(8, 2 * w[name].shape[1], -1)):
            with pytest.raises(ValueError, match=f"{name} has matrices of another shape"):
                layer(dtype, **{**w, name: bad})._few_workspace()


def test_weights_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(M, "moe_few_workspace_init", lambda cfg, ws: None)
    monkeypatch.setattr(M, "_on_current_device", lambda t, what: (_ for _ in ()).throw(ValueError("cuda:1")) if t is there else None)
    w = weights(M.MOE_BF16)
    for there in w.values():
        with pytest.raises(ValueError, match="cuda:1"):
            layer(**w)._few_workspace()


def test_layers_without_a_few_token_form_say_so():
    """Before anything is said of their weights: fp32, and more tokens than one kernel takes."""
    w = {k: v.float() for k, v in weights(M.MOE_BF16).items()}
    few = layer(M.MOE_F32, **w)
    many = layer(**weights(M.MOE_BF16))
    many.cfg.T = 17
    for la in (few, many):
        with pytest.raises(M.MoEError) as e:
            la._few_workspace()
        assert e.value.status == M.MOE_ERR_UNSUPPORTED


def test_tiled_scales_are_allocated_on_their_launch_stream(world, monkeypatch):
    """What the allocator gives on another stream may still be in use there."""
    real, fake = torch.empty, M.lib()
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: world.log.append(("empty", world.now.cuda_stream)) or real(*a, **kw))
    fake.moe_mxfp4_tile_scales = lambda *a: world.log.append(("launch", a[-1])) or M.MOE_OK
    scales = torch.zeros(2, 128, 8, dtype=torch.uint8)
    assert M.moe_mxfp4_tile_scales(scales, stream=Stream(7)).shape == (2, 1, 2, 512)
    M.moe_mxfp4_tile_scales(scales)
    assert world.log == [("empty", 7), ("launch", 7), ("empty", 0), ("launch", 0)]
