"""The serving operators and autograd: inputs that require grad are refused
(no gradient goes through these calls), and tensors that a call writes for the
caller count as modified, as with torch's in-place operations."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def calls():
    """name -> (function, arguments, those that can require grad, those that are written)"""
    import fp8_bf16_mxfp4_gb300 as mxg
    bf = lambda *s: torch.randn(*s, device=DEV).to(torch.bfloat16)  # noqa: E731
    w13 = mxg.mx_quantize_rowwise_packed(bf(2 * 256, 256), "e2m1", groups=2)
    w2 = mxg.mx_quantize_rowwise_packed(bf(2 * 256, 128), "e2m1", groups=2)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    f32 = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
    return {
        "moe_route": (mxg.moe_route, dict(logits=f32(3, 8), top_k=2, ids=i32(3, 2), weights=f32(3, 2)),
                      ("logits", "weights"), ("ids", "weights")),
        "moe_experts": (mxg.moe_experts, dict(x=bf(3, 256), ids=i32(3, 2), weights=f32(3, 2), W13=w13, W2=w2, out=bf(3, 256)),
                        ("x", "weights", "out"), ("out",)),
        "lora_add": (mxg.lora_add, dict(y=bf(3, 64), x=bf(3, 128), A=bf(2, 8, 128), B=bf(2, 64, 8), ids=i32(3),
                                        scale=f32(2), out=bf(3, 64)),
                     ("y", "x", "A", "B", "scale", "out"), ("out",)),
    }


@pytest.mark.parametrize("name", ["moe_route", "moe_experts", "lora_add"])
def test_inputs_that_require_grad_are_refused(name):
    fn, args, diff, written = calls()[name]
    fn(**args)
    for k in diff:
        asks = {**args, k: args[k].detach().clone().requires_grad_()}
        with pytest.raises(ValueError, match="forward only"):
            fn(**asks)
        with torch.no_grad():
            fn(**asks)
        with torch.inference_mode():
            fn(**asks)


@pytest.mark.parametrize("name", ["moe_route", "moe_experts", "lora_add"])
def test_written_tensors_count_as_modified(name):
    fn, args, diff, written = calls()[name]
    for k in written:
        v = args[k]._version
        fn(**args)
        assert args[k]._version == v + 1
    others = {k: t._version for k, t in args.items() if isinstance(t, torch.Tensor) and k not in written}
    fn(**args)
    assert all(args[k]._version == v for k, v in others.items())
    with torch.inference_mode():  # tensors without a version
        fn(**{k: t.clone() if k in written else t for k, t in args.items()})


def test_a_saved_projection_is_not_overwritten_unseen():
    fn, args, _, _ = calls()["lora_add"]
    y = args["y"]
    gate = torch.ones_like(y, requires_grad=True)
    loss = (gate * y).sum()  # saves y
    fn(**{**args, "out": y})
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
