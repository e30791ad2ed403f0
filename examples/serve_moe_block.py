"""One decode step of a mixture-of-experts block served from quantized weights.

    python examples/serve_moe_block.py [--tokens 16] [--steps 20]

The block as a server runs it, every part through the library:

  1. the shared projection over MXFP8 weights (mx_gemm_dense),
  2. each request's low-rank adapter added to it (lora_add),
  3. the router's logits (a plain product) and the top-k choice (moe_route),
  4. the chosen experts over MXFP4 weights (moe_experts), plus the residual.

The step is captured in a CUDA graph and replayed; the captured and the eager
results are compared, and the time per step is printed.
"""

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def build_block(hidden, inter, experts, adapters, rank, dev, seed=0):
    """Random weights of the block, quantized once."""
    import fp8_bf16_mxfp4_gb300 as mxg
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device=dev) * std).to(torch.bfloat16)  # noqa: E731
    return {
        "proj": mxg.mx_quantize_rowwise_packed(rnd(hidden, hidden, std=hidden ** -0.5), "e4m3", groups=1),
        "A": rnd(adapters, rank, hidden, std=hidden ** -0.5),
        "B": rnd(adapters, hidden, rank, std=rank ** -0.5),
        "scale": torch.full((adapters,), 0.5, device=dev),
        "router": rnd(experts, hidden, std=hidden ** -0.5),
        "w13": mxg.mx_quantize_rowwise_packed(rnd(experts * 2 * inter, hidden, std=hidden ** -0.5), "e2m1", groups=experts),
        "w2": mxg.mx_quantize_rowwise_packed(rnd(experts * hidden, inter, std=inter ** -0.5), "e2m1", groups=experts),
    }


def decode_step(x, adapter, block, top_k):
    """x BF16 [tokens, hidden], adapter int32 [tokens] (-1: none) -> (BF16
    [tokens, hidden], expert ids)."""
    import fp8_bf16_mxfp4_gb300 as mxg
    y = mxg.mx_gemm_dense(mxg.mx_quantize_rowwise(x, "e4m3"), block["proj"])
    y = mxg.lora_add(y, x, block["A"], block["B"], adapter, block["scale"], out=y)
    ids, weights = mxg.moe_route(y @ block["router"].t(), top_k)
    return y + mxg.moe_experts(y, ids, weights, block["w13"], block["w2"]), ids


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inter", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--adapters", type=int, default=8)
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    import fp8_bf16_mxfp4_gb300 as mxg
    dev = torch.device("cuda:0")
    block = build_block(a.hidden, a.inter, a.experts, a.adapters, a.rank, dev)
    x = torch.randn(a.tokens, a.hidden, device=dev).to(torch.bfloat16)
    adapter = (torch.arange(a.tokens, device=dev) % (a.adapters + 1) - 1).to(torch.int32)  # one in adapters + 1 has none
    want, ids = decode_step(x, adapter, block, a.top_k)
    mxg.check_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = decode_step(x, adapter, block, a.top_k)
    graph.replay()
    mxg.check_status()
    assert torch.equal(out, want), "the captured step differs from the eager one"
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        graph.replay()
    stop.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(stop) * 1e3 / a.steps
    print(f"{a.tokens} tokens, hidden {a.hidden}, {a.experts} experts top-{a.top_k}: "
          f"{len(torch.unique(ids))} experts used, {us:.1f} us a step")
    return us


if __name__ == "__main__":
    main()
