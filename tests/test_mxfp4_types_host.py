"""What the binding of the MXFP4 product says of its tensors' types, without a GPU."""
import pytest
import torch

import sparse_mixture_experts_20_b200 as M

OUT = {M.MOE_F32: torch.float32, M.MOE_BF16: torch.bfloat16, M.MOE_MXFP4: torch.uint8}
u8 = lambda *n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731


def operands(out):
    """Four rows of 128 columns, two segments, two matrices of 64 rows."""
    s = M.make_mxfp4_shape(4, 64, 128, 2, 2, M.MOE_ACT_NONE, out)
    y = u8(4, 32) if out == M.MOE_MXFP4 else torch.zeros(4, 64, dtype=OUT[out])
    return s, dict(a=u8(4, 64), a_scales=u8(4, 4), seg_offsets=torch.zeros(3, dtype=torch.int32),
                   seg_mat=torch.zeros(2, dtype=torch.int32), w=u8(2, 64, 64), w_scales=u8(2, 64, 4),
                   bias=torch.zeros(2, 64), y=y, y_scales=u8(4, 2) if out == M.MOE_MXFP4 else None, ws=u8(256))


@pytest.mark.parametrize("out", list(OUT))
def test_types_are_refused_whatever_their_size(out):
    s, good = operands(out)
    wrong = dict(a=torch.float32, a_scales=torch.bfloat16, seg_offsets=torch.int64, seg_mat=torch.int64, w=torch.bfloat16,
                 w_scales=torch.float32, bias=torch.float64, ws=torch.float32,
                 y=torch.bfloat16 if out == M.MOE_F32 else torch.float32, y_scales=torch.float32)
    for name, dtype in wrong.items():
        if good[name] is not None:
            bad = {**good, name: torch.zeros(good[name].shape, dtype=dtype)}
            with pytest.raises(ValueError, match=f"moe_mxfp4_matmul: {name} is torch"):
                M.moe_mxfp4_matmul(s, *bad.values())


@pytest.mark.parametrize("out", list(OUT))
def test_named_types_and_bytes_are_taken(out):
    """Up to the next check: none of these tensors is on a GPU."""
    s, good = operands(out)
    named = {**good, **{k: good[k].view(torch.float4_e2m1fn_x2) for k in ("a", "w")},
             **{k: good[k].view(torch.float8_e8m0fnu) for k in ("a_scales", "w_scales")}}
    raw = {k: None if t is None else t.view(torch.uint8) for k, t in good.items()}
    for case in (good, named, raw):
        with pytest.raises(ValueError, match="must live on a CUDA device"):
            M.moe_mxfp4_matmul(s, *case.values())


def test_small_workspace_is_refused():
    s, good = operands(M.MOE_F32)
    with pytest.raises(ValueError, match="ws is smaller"):
        M.moe_mxfp4_matmul(s, *{**good, "ws": u8(255)}.values())


class On(torch.Tensor):
    """A tensor that says it is on GPU `where`."""
    where = 0

    def get_device(self):
        return self.where


def test_every_operand_must_be_on_the_current_device(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    called = []
    fake = type("Lib", (), {"moe_mxfp4_matmul": staticmethod(lambda *a: called.append(a) or M.MOE_OK)})
    monkeypatch.setattr(M, "lib", lambda: fake)
    monkeypatch.setattr(M, "_stream", lambda s: 0)
    s, good = operands(M.MOE_MXFP4)
    good = {k: t.as_subclass(On) for k, t in good.items()}
    M.moe_mxfp4_matmul(s, *good.values())
    assert [p for p in called[0][1:-1]] == [t.data_ptr() for t in good.values()]
    for t in good.values():
        t.where = 1
        with pytest.raises(ValueError, match="every tensor must be on the current device"):
            M.moe_mxfp4_matmul(s, *good.values())
        t.where = 0
