"""Refusals of memory that is not what a call would take it for: workspaces,
status words, codes and scales whose elements do not lie where their count says."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def calls():
    import fp8_bf16_mxfp4_gb300 as mxg
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device=DEV)  # noqa: E731
    w13 = mxg.mx_quantize_rowwise_packed(z(2 * 256, 256), "e2m1", groups=2)
    w2 = mxg.mx_quantize_rowwise_packed(z(2 * 256, 128), "e2m1", groups=2)
    experts = dict(x=z(3, 256), ids=z(3, 2, d=torch.int32), weights=z(3, 2, d=torch.float32), W13=w13, W2=w2)
    lora = dict(y=z(3, 64), x=z(3, 128), A=z(2, 8, 128), B=z(2, 64, 8), ids=z(3, d=torch.int32))
    return {"moe_experts": (mxg.moe_experts, experts, mxg.moe_experts_workspace_size(3, 2, 2, 256, 128)),
            "lora_add": (mxg.lora_add, lora, mxg.lora_add_workspace_size(3, 128, 8))}


@pytest.mark.parametrize("name", ["moe_experts", "lora_add"])
def test_workspace_and_status(name):
    fn, args, need = calls()[name]
    u8 = torch.uint8
    whole = torch.zeros(2 * need, dtype=u8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    fn(**args, workspace=whole[:need], status=st, check=True)
    fn(**args, workspace=whole.view(2, need), check=True)
    for bad in (torch.zeros(1, dtype=u8, device=DEV).expand(need), whole[::2], whole.view(need, 2).t(),
                whole[: need // 4 * 4].view(torch.float32)):
        with pytest.raises(ValueError):
            fn(**args, workspace=bad)
    for bad in (torch.zeros(1, dtype=u8, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)):
        with pytest.raises(ValueError):
            fn(**args, status=bad)


@pytest.mark.parametrize("which", ["W13", "W2"])
def test_codes_and_scales_of_experts(which):
    import fp8_bf16_mxfp4_gb300 as mxg
    fn, args, _ = calls()["moe_experts"]
    op = args[which]
    op_of = lambda data, scale: mxg.MXOperand(data, scale, "e2m1", op.cols, "packed")  # noqa: E731
    rows, codes = op.data.shape
    wide = torch.zeros(rows, 2 * codes, dtype=torch.uint8, device=DEV)
    fn(**{**args, which: op_of(wide[:, :codes], op.scale)}, check=True)  # rows of a wider tensor
    one = torch.zeros(1, dtype=torch.uint8, device=DEV)
    for bad in (op_of(wide[:, -32:], op.scale), op_of(wide[:, ::2], op.scale), op_of(wide, op.scale),
                op_of(wide.view(-1)[: rows * codes], op.scale), op_of(op.data, one.expand(op.scale.numel())),
                op_of(op.data, torch.zeros(2 * op.scale.numel(), dtype=torch.uint8, device=DEV)[::2])):
        with pytest.raises(ValueError):
            fn(**{**args, which: bad})
