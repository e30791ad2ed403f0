"""Measured cases of the serving operators around the grouped MX GEMMs.

Three operators that a decode step of a mixture-of-experts model calls next to
the grouped GEMMs:

  route    top-k routing: router logits -> expert ids and combine weights;
  experts  the expert layer for a few tokens over MX-quantized weights:
             xq = mxfp8(x)                      (E4M3, one power-of-two scale per 32)
             g, u = W13[e] xq                   (gate rows first, then up rows)
             hq = mxfp8(g / (1 + exp(-g)) * u)
             y[t] = sum_j w[t, j] * W2[e_j] hq
  lora     low-rank adapters of many requests beside a shared projection:
             out[t] = y[t] + s[a] * B[a] (A[a] x[t]),  a = ids[t]  (a < 0: out = y)

``own`` selects the library's kernels (True) or the plain torch forms (False).
"""

import math

import numpy as np
import torch

own = False

F32, F64 = torch.float32, torch.float64
OUT = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------- cases


def listed():
    return [
        # one decoding request: the latency of a single row of logits
        dict(name="route_1tok", op="route", T=1, E=32, k=8, dtype="f32", renorm=True, masked=False),
        # a mixed batch over an odd expert count, BF16 logits (ties), some experts and whole rows masked
        dict(name="route_masked_odd", op="route", T=333, E=161, k=6, dtype="bf16", renorm=False, masked=True),
        # a training or prefill batch: 16384 tokens, top-8 of 32
        dict(name="route_16k", op="route", T=16384, E=32, k=8, dtype="f32", renorm=True, masked=False),
        # one decoding request over MXFP4 experts: 8 of 32 experts are read
        dict(name="experts_1tok_fp4", op="experts", T=1, E=32, k=8, H=7168, I=2048, fmt="e2m1", masked=False),
        # a small decode batch: most experts are read, one to nine tokens each
        dict(name="experts_13tok_fp4", op="experts", T=13, E=32, k=8, H=7168, I=2048, fmt="e2m1", masked=False),
        # a full decode batch: every expert is read, about 32 tokens each
        dict(name="experts_128tok_fp4", op="experts", T=128, E=32, k=8, H=7168, I=2048, fmt="e2m1", masked=False),
        # few wide experts, top-2 of 8, MXFP8 weights
        dict(name="experts_4tok_wide_fp8", op="experts", T=4, E=8, k=2, H=4096, I=14336, fmt="e4m3", masked=False),
        # a small model's layer, odd tile counts, a third of the slots empty (padding tokens, dropped slots)
        dict(name="experts_33tok_small", op="experts", T=33, E=12, k=3, H=1152, I=640, fmt="e4m3", masked=True),
        # one decoding request with its adapter
        dict(name="lora_1tok", op="lora", T=1, K=7168, N=4096, R=16, n=8, dtype="bf16", runs=1),
        # a decode batch in which nearly every request brings an adapter of its own
        dict(name="lora_64tok_mixed", op="lora", T=64, K=7168, N=7168, R=16, n=64, dtype="bf16", runs=1),
        # odd sizes, FP32 projection output, short prompts
        dict(name="lora_517tok_odd_f32", op="lora", T=517, K=1000, N=1544, R=8, n=5, dtype="f32", runs=37),
        # prompts of about a thousand tokens each beside a wide projection
        dict(name="lora_8k_prompts", op="lora", T=8192, K=8192, N=28672, R=32, n=16, dtype="bf16", runs=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "experts", "lora", "lora"])
    if op == "route":
        E = _log(rng, 2, 512)
        return dict(op=op, T=_log(rng, 1, 16384) if E <= 64 else _log(rng, 1, 1024), E=E, k=rng.randint(1, min(E, 8)),
                    dtype=rng.choice(["f32", "bf16"]), renorm=rng.random() < 0.5, masked=rng.random() < 0.5)
    if op == "experts":
        fmt = rng.choice(["e2m1", "e2m1", "e4m3"])
        room = (32 if fmt == "e2m1" else 16) * 2048 * 7168
        while True:
            H, I, E = 128 * _log(rng, 2, 56), 128 * _log(rng, 1, 112), _log(rng, 2, 64)
            if E * H * I <= room and 3072 not in (H, I, 2 * I):
                break
        return dict(op=op, T=_log(rng, 1, 128), E=E, k=rng.randint(1, min(E, 8)), H=H, I=I, fmt=fmt,
                    masked=rng.random() < 0.5)
    while True:
        T, K, N, R = _log(rng, 1, 8192), 8 * _log(rng, 16, 1024), 8 * _log(rng, 16, 3584), 8 * _log(rng, 1, 8)
        n = _log(rng, 1, 64)
        if T * (K + 2 * N) <= 8192 * (8192 + 2 * 28672) and 3072 not in (K, N, T):
            break
    return dict(op=op, T=T, K=K, N=N, R=R, n=n, dtype=rng.choice(["bf16", "bf16", "f32"]) if T < 2048 else "bf16",
                runs=rng.choice([1, 1, _log(rng, 1, 1024)]))


# --------------------------------------------------------------------------- inputs


def _pack_scales(s, cols):
    """[rows, cols/32] scale bytes (rows a multiple of 128) in the library's packed order: 512-byte chunks of 128
    rows x 4 blocks, k-chunk major; row i and block j of a chunk at (i % 32) * 16 + (i / 32) * 4 + j."""
    rt, kc = s.shape[0] // 128, cols // 128
    return s.view(rt, 4, 32, kc, 4).permute(3, 0, 2, 1, 4).contiguous().view(-1)


def _quantized_weights(gen, rows, cols, std, fmt, dev):
    """Normal weights in MXFP4 / MXFP8 (one shared power of two per 32): codes and packed scales."""
    codes, scales = [], []
    step = max(128, (1 << 26) // cols // 128 * 128)
    for r0 in range(0, rows, step):
        w = torch.randn(min(step, rows - r0), cols // 32, 32, generator=gen, device=dev) * std
        e = torch.frexp(w.abs().amax(-1, keepdim=True)).exponent - 1 - (2 if fmt == "e2m1" else 8)
        v = torch.ldexp(w, -e)
        scales.append((e.squeeze(-1) + 127).to(torch.uint8))
        if fmt == "e2m1":
            edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev)
            c = torch.bucketize(v.abs(), edges, out_int32=True).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
            c = c.view(-1, cols // 2, 2)
            codes.append(c[..., 0] | (c[..., 1] << 4))
        else:
            codes.append(v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, cols))
    return torch.cat(codes), _pack_scales(torch.cat(scales), cols)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=gen, device=dev)  # noqa: E731
    s, T = dict(case), case["T"]
    if case["op"] == "route":
        x = 1.5 * rnd(T, case["E"])
        if case["masked"]:  # experts that a token may not use, and padding rows
            x = x.masked_fill(uni(T, case["E"]) < 0.2, -math.inf).masked_fill(uni(T, 1) < 0.1, -math.inf)
        s["logits"] = x.to(OUT[case["dtype"]])
    elif case["op"] == "experts":
        E, H, I, k = case["E"], case["H"], case["I"], case["k"]
        top = torch.topk(rnd(T, E), k)
        s["x"] = rnd(T, H).to(torch.bfloat16)
        s["ids"] = top.indices.to(torch.int32)
        s["weights"] = torch.softmax(top.values, -1)
        if case["masked"]:
            s["ids"] = s["ids"].masked_fill(uni(T, k) < 0.33, -1)
        s["w13"] = _quantized_weights(gen, E * 2 * I, H, H ** -0.5, case["fmt"], dev)
        s["w2"] = _quantized_weights(gen, E * H, I, I ** -0.5, case["fmt"], dev)
    else:
        K, N, R, n = case["K"], case["N"], case["R"], case["n"]
        s["x"] = rnd(T, K).to(torch.bfloat16)
        s["y"] = rnd(T, N).to(OUT[case["dtype"]])
        s["A"] = (rnd(n, R, K) * K ** -0.5).to(torch.bfloat16)
        s["B"] = (rnd(n, N, R) * R ** -0.5).to(torch.bfloat16)
        s["scale"] = 0.5 + uni(n)
        # requests of `runs` consecutive tokens; one in about eleven uses no adapter
        req = torch.randint(-(n // 10 + 1), n, (-(-T // case["runs"]),), generator=gen, device=dev).clamp_(min=-1)
        s["ids"] = req.repeat_interleave(case["runs"])[:T].to(torch.int32).contiguous()
    return s


# --------------------------------------------------------------------------- plain forms


def _pow2(e):
    """2^e in FP32 for integer e in [-127, 127]."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(F32)


def _mxfp8(x):
    """FP32 rows rounded to MXFP8 values: e = max(floor(log2 amax) - 8, -127) per 32, elements to E4M3."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 9, -127).clamp(min=-127)
    q = (b * _pow2(-e)).clamp(-448, 448).to(torch.float8_e4m3fn).to(F32)
    return (q * _pow2(e)).flatten(-2)


def _dequantized(w, fmt, groups, cols, sel=None):
    """FP32 weights [groups (or sel), rows, cols] of one quantized matrix."""
    codes, packed = w
    dev = codes.device
    rows = codes.shape[0] // groups
    codes = codes.view(groups, rows, -1)
    sc = packed.view(cols // 128, groups, rows // 128, 32, 4, 4)
    if sel is not None:
        codes, sc = codes[sel], sc[:, sel]
    sc = sc.permute(1, 2, 4, 3, 0, 5).reshape(codes.shape[0], rows, cols // 32, 1).to(torch.int32)
    if fmt == "e2m1":
        half = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=dev, dtype=F32)
        nib = torch.cat([half, -half])
        table = torch.stack([nib.repeat(16), nib.repeat_interleave(16)], -1)
        v = table[codes.to(torch.int32)]
    else:
        v = codes.view(torch.float8_e4m3fn).to(F32)
    v = v.reshape(codes.shape[0], rows, cols // 32, 32)
    return (v * _pow2(sc - 127)).flatten(-2)


def _plain_route(s):
    x = s["logits"].to(F32)
    x = torch.where(x.isnan(), -math.inf, x)
    v, i = torch.sort(x, dim=-1, descending=True, stable=True)
    top = v[:, :1]
    z = lambda a: torch.where(top == -math.inf, 0.0, torch.where(a == top, 1.0, torch.exp(a - top)))  # noqa: E731
    v, i = v[:, : s["k"]], i[:, : s["k"]]
    p = z(v)
    tot = (p if s["renorm"] else z(x)).sum(-1, keepdim=True)
    return {"ids": torch.where(v == -math.inf, -1, i).to(torch.int32), "weights": p / tot.clamp(min=1.0)}


def _plain_experts(s):
    T, E, H, I, k = (s[n] for n in ("T", "E", "H", "I", "k"))
    xq = _mxfp8(s["x"].to(F32))
    ids = s["ids"].to(torch.int64)
    wts = torch.where(ids >= 0, s["weights"], 0.0)
    if T * k < E:  # fewer slots than experts: only the weights of the slots' experts
        sel = ids.clamp(min=0).flatten()
        xs = xq.repeat_interleave(k, 0).unsqueeze(1)
    else:
        sel, xs = None, xq
    gu = xs @ _dequantized(s["w13"], s["fmt"], E, H, sel).transpose(1, 2)
    g, u = gu[..., :I], gu[..., I:]
    h = _mxfp8(g / (1 + torch.exp(-g)) * u)
    y = h @ _dequantized(s["w2"], s["fmt"], E, I, sel).transpose(1, 2)
    if sel is not None:
        y = (y.view(T, k, H) * wts.unsqueeze(-1)).sum(1)
    else:
        full = torch.zeros(T, E, device=xq.device).scatter_add_(1, ids.clamp(min=0), wts)
        y = (y * full.t().unsqueeze(-1)).sum(0)
    return y.to(torch.bfloat16)


def _plain_lora(s):
    x, A, B = s["x"].to(F32), s["A"].to(F32), s["B"].to(F32)
    ids = s["ids"].to(torch.int64)
    on = ids >= 0
    a = ids.clamp(min=0)
    sc = torch.where(on, s["scale"][a], 0.0).unsqueeze(-1)
    if s["T"] < s["n"]:  # fewer tokens than adapters: each token's own
        u = (A[a] @ x.unsqueeze(-1)).squeeze(-1)
        d = (B[a] @ u.unsqueeze(-1)).squeeze(-1)
    else:
        u = (x @ A.flatten(0, 1).t()).view(s["T"], s["n"], s["R"])
        u = u * torch.nn.functional.one_hot(a, s["n"]).unsqueeze(-1)
        d = u.flatten(1) @ B.transpose(1, 2).flatten(0, 1)
    return (s["y"].to(F32) + sc * d).to(s["y"].dtype)


def run(state):
    s = state
    if not own:
        return {"route": _plain_route, "experts": _plain_experts, "lora": _plain_lora}[s["op"]](s)
    import fp8_bf16_mxfp4_gb300 as mxg
    if s["op"] == "route":
        ids, weights = mxg.moe_route(s["logits"], s["k"], renormalize=s["renorm"])
        return {"ids": ids, "weights": weights}
    if s["op"] == "experts":
        w13 = mxg.MXOperand(*s["w13"], s["fmt"], s["H"], "packed")
        w2 = mxg.MXOperand(*s["w2"], s["fmt"], s["I"], "packed")
        return mxg.moe_experts(s["x"], s["ids"], s["weights"], w13, w2)
    return mxg.lora_add(s["y"], s["x"], s["A"], s["B"], s["ids"], s["scale"])


# --------------------------------------------------------------------------- work


def work(case):
    T = case["T"]
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        return {"bytes": T * E * (4 if case["dtype"] == "f32" else 2) + T * k * 8, "flops": 4 * T * E}
    if case["op"] == "experts":
        E, H, I, k = case["E"], case["H"], case["I"], case["k"]
        slots = T * k * (0.67 if case["masked"] else 1.0)
        read = E * (1 - (1 - slots / T / E) ** T)  # experts that some token uses, routed uniformly
        per = (0.5 if case["fmt"] == "e2m1" else 1.0) + 1 / 32
        return {"bytes": read * 3 * H * I * per + T * H * 4 + T * k * 8, "flops": 6 * slots * H * I}
    K, N, R, n = case["K"], case["N"], case["R"], case["n"]
    reqs = -(-T // case["runs"])
    on = n / (n + n // 10 + 1)
    used = n * (1 - (1 - on / n) ** reqs)
    e = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": T * (2 * K + 2 * e * N + 4) + used * R * (K + N) * 2, "flops": 2 * T * on * R * (K + N)}


# --------------------------------------------------------------------------- 64-bit definition


def _round_e4m3(v):
    """Nearest E4M3 value, ties to even: 4 significant bits, subnormal step 2^-9, largest 448."""
    mag = v.abs()
    p = torch.floor(torch.log2(mag.clamp(min=2.0 ** -6)))
    p = torch.where(torch.exp2(p) > mag.clamp(min=2.0 ** -6), p - 1, p)
    step = torch.exp2(p - 3)
    return (torch.sign(v) * torch.round(mag / step) * step).clamp(-448, 448)


def _mxfp8_64(x):
    out = torch.empty_like(x)
    for c in range(0, x.shape[-1], 32):
        b = x[..., c:c + 32]
        amax = b.abs().max(-1, keepdim=True).values
        m, p = torch.frexp(amax)
        e = torch.where(amax > 0, (p - 9).to(F64), -127.0).clamp(-127, 127)
        out[..., c:c + 32] = _round_e4m3(b * torch.exp2(-e)) * torch.exp2(e)
    return out


def _expert_64(w, fmt, groups, cols, e):
    """Expert e's weights in 64 bits, decoded field by field."""
    codes, packed = w
    rows = codes.shape[0] // groups
    c = codes[e * rows:(e + 1) * rows].to(torch.int64)
    if fmt == "e2m1":
        c = torch.stack([c & 15, c >> 4], -1).flatten(1)
        ex, man, sign = (c >> 1) & 3, c & 1, c >> 3
        mag = torch.where(ex > 0, (2 + man) * torch.exp2((ex - 2).to(F64)), man * 0.5)
    else:
        ex, man, sign = (c >> 3) & 15, c & 7, c >> 7
        mag = torch.where(ex > 0, (8 + man) * torch.exp2((ex - 10).to(F64)), man * 2.0 ** -9)
    r = torch.arange(rows, device=c.device).view(-1, 1) + e * rows
    kb = torch.arange(cols // 32, device=c.device).view(1, -1)
    at = ((kb // 4) * (groups * rows // 128) + r // 128) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + kb % 4
    sc = torch.exp2(packed[at].to(F64) - 127)
    return torch.where(sign > 0, -mag, mag) * sc.repeat_interleave(32, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        x = s["logits"].cpu().numpy().astype(np.float64) if case["dtype"] == "f32" else s["logits"].float().cpu().numpy().astype(np.float64)
        w = np.zeros((case["T"], case["k"]))
        for t, row in enumerate(x):
            order = np.argsort(-row, kind="stable")[: case["k"]]
            if row[order[0]] == -np.inf:
                continue
            p = np.exp(row - row[order[0]])
            w[t] = p[order] / (p[order].sum() if case["renorm"] else p.sum())
        return {"ids": None, "weights": w}
    if case["op"] == "experts":
        E, H, I = case["E"], case["H"], case["I"]
        y = torch.zeros(case["T"], H, dtype=F64, device=s["x"].device)
        xq = _mxfp8_64(s["x"].to(F64))
        for e in torch.unique(s["ids"]).tolist():
            if e < 0:
                continue
            t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
            gu = xq[t] @ _expert_64(s["w13"], case["fmt"], E, H, e).t()
            g, u = gu[:, :I], gu[:, I:]
            h = _mxfp8_64(g * torch.sigmoid(g) * u)
            y.index_add_(0, t, (h @ _expert_64(s["w2"], case["fmt"], E, I, e).t()) * s["weights"][t, j].to(F64)[:, None])
        return y
    y = s["y"].to(F64)
    for a in torch.unique(s["ids"]).tolist():
        if a >= 0:
            t = torch.nonzero(s["ids"] == a).flatten()
            u = s["x"][t].to(F64) @ s["A"][a].to(F64).t()
            y[t] += float(s["scale"][a]) * (u @ s["B"][a].to(F64).t())
    return y
