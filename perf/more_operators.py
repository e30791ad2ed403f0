"""Measured cases of the operators that bring tokens to the experts and back, and
of the 8-bit integer products.

With slots (t, j) of T tokens and k choices each, P = T k:

  dispatch      ids [T, k] -> m_splits [E] and each slot's row in expert order
                (stable; an empty slot, id < 0, has a zero row behind all others,
                r, and the entry -1 - r; the last expert's split counts these),
                and xs[row] = x[t]
  combine       out[t] = sum_j w[t, j] y[row]   (w = 1 where there are no weights:
                the gradient of the copy above), empty slots adding nothing
  combine_grad  dy[row] = w[t, j] dout[t],  dw[t, j] = <dout[t], y[row]>;
                zeros for empty slots
  route_grad    s = sum_j w_j dw_j;  dl[id_j] = w_j (dw_j - s), zeros elsewhere
                (weights normalised over the chosen experts), or
                dl_e = [e = id_j] w_j dw_j - p_e s, p = softmax(logits)
  int8          a = max(max |x[t]|, 2^-100), sx = a / 127, qx = rint(x * (127 / a)),
                y[row, n] = sx sw[g, n] sum_k qx[k] qw[g, n, k], g the row's expert

``own`` selects the library's kernels (True) or the plain torch forms (False).
"""

import math

import numpy as np
import torch

own = False

F32, F64 = torch.float32, torch.float64
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------- cases


def listed():
    return [
        # a small decode step: eight tokens, latency
        dict(name="dispatch_8tok", op="dispatch", T=8, k=8, E=32, H=7168, dtype="bf16", masked=False),
        # a prefill or training batch, 65536 rows of 7168, some slots dropped
        dict(name="dispatch_8k", op="dispatch", T=8192, k=8, E=32, H=7168, dtype="bf16", masked=True),
        # a mixed batch of odd sizes in FP32 with dropped slots and padding tokens
        dict(name="combine_333tok_odd", op="combine", T=333, k=6, E=161, H=1160, dtype="f32", weighted=True, masked=True),
        # a prefill or training batch
        dict(name="combine_8k", op="combine", T=8192, k=8, E=32, H=7168, dtype="bf16", weighted=True, masked=False),
        # a short training sequence of a small FP32 model, slots dropped
        dict(name="combine_grad_517tok", op="combine_grad", T=517, k=3, E=12, H=1000, dtype="f32", masked=True),
        # a training batch
        dict(name="combine_grad_8k", op="combine_grad", T=8192, k=8, E=32, H=4096, dtype="bf16", masked=False),
        # a few tokens over an odd expert count, weights of all experts, some masked
        dict(name="route_grad_77tok", op="route_grad", T=77, k=6, E=161, dtype="bf16", renorm=False, masked=True),
        # a training batch over many experts
        dict(name="route_grad_16k", op="route_grad", T=16384, k=8, E=256, dtype="f32", renorm=False, masked=False),
        # one decoding request beside a dense projection
        dict(name="int8_1tok", op="int8", T=1, k=0, E=1, K=7168, N=4096, dtype="bf16"),
        # a decode batch over experts: 128 rows, every used expert's weights are read
        dict(name="int8_16tok_moe", op="int8", T=16, k=8, E=32, K=7168, N=4096, dtype="bf16"),
        # short prompts through a small layer of odd sizes, FP32 output
        dict(name="int8_173tok_odd", op="int8", T=173, k=3, E=5, K=1040, N=1096, dtype="f32"),
        # prompts through wide experts: bound by the products
        dict(name="int8_4k_wide", op="int8", T=4096, k=2, E=8, K=4096, N=14336, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_grad", "route_grad", "int8", "int8", "int8"])
    if op == "int8":
        while True:
            k = rng.choice([0, rng.randint(1, 8)])
            E = 1 if k == 0 else rng.randint(k, 32)
            T, K, N = _log(rng, 1, 8192), 16 * _log(rng, 4, 512), 8 * _log(rng, 4, 3584)
            if T * max(k, 1) * K * N <= 8192 * 4096 * 14336 and E * K * N <= 32 * 7168 * 4096 and T * max(k, 1) * N <= 8192 * 14336:
                return dict(op=op, T=T, k=k, E=E, K=K, N=N, dtype=rng.choice(["bf16", "bf16", "f32"]))
    E = _log(rng, 2, 512)
    k = rng.randint(1, min(E, 8))
    masked = rng.random() < 0.5
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "route_grad":
        T = _log(rng, 1, 16384)
        while T * E > 16384 * 256:
            T = _log(rng, 1, 16384)
        return dict(op=op, T=T, k=k, E=E, dtype=dtype, renorm=rng.random() < 0.5, masked=masked)
    most = 8192 * (4096 if op == "combine_grad" else 7168) * 8 * (1 if dtype == "bf16" else 0.5)
    while True:
        T, H = _log(rng, 1, 32768), 8 * _log(rng, 4, 2048)
        if T * k * H <= most:
            break
    c = dict(op=op, T=T, k=k, E=E, H=H, dtype=dtype, masked=masked)
    if op == "combine":
        c["weighted"] = rng.random() < 0.7
    return c


# --------------------------------------------------------------------------- inputs


def _sorted_rows(ids, E):
    """m_splits and rows of a routing (the plan that the later calls of a step take)."""
    flat = ids.flatten().to(torch.int64)
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True).indices
    rows = torch.empty_like(flat)
    rows[order] = torch.arange(flat.numel(), device=flat.device)
    rows = torch.where(flat < 0, -1 - rows, rows).view(ids.shape).to(torch.int32)
    splits = (key.unsqueeze(1) == torch.arange(E + 1, device=flat.device)).sum(0) if flat.numel() * E < 1 << 26 else \
        torch.stack([(key == e).sum() for e in range(E + 1)])
    splits[E - 1] += splits[E]
    return splits[:E].to(torch.int32), rows


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rnd = lambda *s, dt=F32: torch.randn(*s, generator=gen, device=dev, dtype=dt)  # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=gen, device=dev)  # noqa: E731
    s, op, T, k, E = dict(case), case["op"], case["T"], case["k"], case["E"]
    dt = DT[case["dtype"]]
    if k > 0:
        logits = 1.5 * rnd(T, E)
        if op == "route_grad":
            if case["masked"]:  # experts that a token may not use, and padding rows
                logits = logits.masked_fill(uni(T, E) < 0.2, -math.inf).masked_fill(uni(T, 1) < 0.1, -math.inf)
            logits = logits.to(dt)
        v, i = torch.sort(logits.to(F32), dim=-1, descending=True, stable=True)
        off = v[:, :k] == -math.inf
        if op != "route_grad" and case.get("masked"):  # slots over a capacity, and padding tokens
            off = off | (uni(T, k) < 0.15) | (uni(T, 1) < 0.1)
        top = torch.where(v[:, :1] == -math.inf, 0.0, v[:, :1])
        p = torch.exp(v - top)
        w = p[:, :k] / (p if not case.get("renorm", True) else p[:, :k]).sum(-1, keepdim=True).clamp(min=1.0)
        s["ids"] = torch.where(off, -1, i[:, :k]).to(torch.int32)
        s["weights"] = torch.where(off, 0.0, w)
    if op == "dispatch":
        s["x"] = rnd(T, case["H"]).to(dt)
    elif op == "route_grad":
        s["logits"] = logits
        s["dweights"] = rnd(T, k)
    elif op == "int8":
        K, N = case["K"], case["N"]
        s["x"] = rnd(T, K).to(torch.bfloat16)
        # weights quantized per channel: codes and scales of normal weights
        s["wq"] = torch.empty(E * N, K, dtype=torch.int8, device=dev)
        s["ws"] = torch.empty(E * N, device=dev)
        step = max(1, (1 << 27) // K)
        for r0 in range(0, E * N, step):
            w = rnd(min(step, E * N - r0), K) * K ** -0.5
            sc = w.abs().amax(-1, keepdim=True) / 127
            s["wq"][r0:r0 + step] = torch.round(w / sc).clamp(-127, 127).to(torch.int8)
            s["ws"][r0:r0 + step] = sc.squeeze(-1)
        if k > 0:
            s["m_splits"], s["rows"] = _sorted_rows(s["ids"], E)
    else:
        s["m_splits"], s["rows"] = _sorted_rows(s["ids"], E)
        H = case["H"]
        s["y"] = rnd(T * k, H, dt=dt)
        if op == "combine_grad":
            s["dout"] = rnd(T, H, dt=dt)
    return s


# --------------------------------------------------------------------------- plain forms


def _plain_dispatch(s):
    m_splits, rows = _sorted_rows(s["ids"], s["E"])
    xs = torch.zeros(s["T"] * s["k"], s["H"], dtype=s["x"].dtype, device=s["x"].device)
    for j in range(s["k"]):
        r = rows[:, j].to(torch.int64)
        xs[torch.where(r < 0, -1 - r, r)] = torch.where(r.unsqueeze(1) < 0, 0, s["x"])
    return {"m_splits": m_splits, "rows": rows, "xs": xs}


def _plain_combine(s):
    out = torch.zeros(s["T"], s["H"], device=s["y"].device)
    for j in range(s["k"]):
        r = s["rows"][:, j].to(torch.int64).unsqueeze(1)
        v = s["y"][r.squeeze(1).clamp(min=0)].to(F32)
        if s["weighted"]:
            v = v * s["weights"][:, j:j + 1]
        out += torch.where(r >= 0, v, 0.0)
    return out.to(s["y"].dtype)


def _plain_combine_grad(s):
    dt = s["y"].dtype
    dout = s["dout"].to(F32)
    dy, dw = torch.zeros_like(s["y"]), torch.zeros(s["T"], s["k"], device=dout.device)
    for j in range(s["k"]):
        r = s["rows"][:, j].to(torch.int64)
        on = r >= 0
        at = torch.where(on, r, -1 - r)
        dy[at] = torch.where(on.unsqueeze(1), dout * s["weights"][:, j:j + 1], 0.0).to(dt)
        dw[:, j] = torch.where(on, (dout * s["y"][at].to(F32)).sum(-1), 0.0)
    return {"dy": dy, "dweights": dw}


def _plain_route_grad(s):
    ids = s["ids"].to(torch.int64)
    w, dw = s["weights"], torch.where(ids >= 0, s["dweights"], 0.0)
    wd = w * dw
    tot = wd.sum(-1, keepdim=True)
    own_part = w * (dw - tot) if s["renorm"] else wd
    dl = torch.zeros(s["T"], s["E"] + 1, device=w.device)
    dl.scatter_(1, torch.where(ids < 0, s["E"], ids), own_part)  # empty slots into a column that is cut off
    dl = dl[:, :s["E"]]
    if not s["renorm"]:
        x = s["logits"].to(F32)
        top = x.amax(-1, keepdim=True)
        p = torch.where(x == -math.inf, 0.0, torch.exp(x - torch.where(top == -math.inf, 0.0, top)))
        dl = dl - p / p.sum(-1, keepdim=True).clamp(min=1.0) * tot
    return dl.to(s["logits"].dtype)


def _plain_int8(s):
    x = s["x"]
    a = x.to(F32).abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100)
    most = torch.full_like(a, 127)  # a tensor: torch divides by a number as a product with its inverse
    qx = torch.round(x.to(F64) * (most / a).to(F64)).to(F32)  # 64 bits: values next to a half
    sx = a / most
    if s["k"] == 0:
        y = qx @ s["wq"].to(F32).t() * sx * s["ws"]
        return y.to(DT[s["dtype"]])
    S, N, K = s["T"] * s["k"], s["N"], s["K"]
    q, sc = torch.empty(S, K, device=x.device), torch.empty(S, 1, device=x.device)
    for j in range(s["k"]):
        q[s["rows"][:, j].to(torch.int64)], sc[s["rows"][:, j].to(torch.int64)] = qx, sx
    y = torch.empty(S, N, dtype=DT[s["dtype"]], device=x.device)
    ends = torch.cumsum(s["m_splits"], 0).tolist()  # torch's products need the sizes on the host
    for g, end in enumerate(ends):
        r0 = ends[g - 1] if g else 0
        if end > r0:
            w, ws = s["wq"][g * N:(g + 1) * N].to(F32), s["ws"][g * N:(g + 1) * N]
            y[r0:end] = (q[r0:end] @ w.t() * sc[r0:end] * ws).to(y.dtype)
    return y


def run(state):
    s, op = state, state["op"]
    if not own:
        return {"dispatch": _plain_dispatch, "combine": _plain_combine, "combine_grad": _plain_combine_grad,
                "route_grad": _plain_route_grad, "int8": _plain_int8}[op](s)
    import fp8_bf16_mxfp4_gb300 as mxg
    if op == "dispatch":
        m_splits, rows = mxg.moe_sort(s["ids"], s["E"])
        return {"m_splits": m_splits, "rows": rows, "xs": mxg.moe_gather(s["x"], rows)}
    if op == "combine":
        return mxg.moe_combine(s["y"], s["rows"], s["weights"] if s["weighted"] else None)
    if op == "combine_grad":
        dy, dw = mxg.moe_combine_backward(s["dout"], s["y"], s["rows"], s["weights"])
        return {"dy": dy, "dweights": dw}
    if op == "route_grad":
        return mxg.moe_route_backward(s["dweights"], s["ids"], s["weights"], s["logits"], renormalize=s["renorm"])
    w = mxg.Int8Operand(s["wq"], s["ws"])
    if s["k"] == 0:
        return mxg.int8_gemm_dense(mxg.int8_quantize_rowwise(s["x"], codes="f16"), w, out_dtype=DT[s["dtype"]])
    a = mxg.int8_quantize_rowwise(s["x"], rows=s["rows"], codes="f16")
    return mxg.int8_grouped_gemm_fwd(a, w, s["m_splits"], s["N"], out_dtype=DT[s["dtype"]])


# --------------------------------------------------------------------------- work


def work(case):
    op, T, k, E = case["op"], case["T"], case["k"], case["E"]
    e = 2 if case["dtype"] == "bf16" else 4
    P = T * k
    if op == "dispatch":
        return {"bytes": (T + P) * case["H"] * e + 8 * P + 4 * E, "flops": P}
    on = 0.85 * 0.9 if case.get("masked") else 1.0
    if op == "combine":
        return {"bytes": (on * P + T) * case["H"] * e + (8 if case["weighted"] else 4) * P, "flops": 2 * on * P * case["H"]}
    if op == "combine_grad":
        return {"bytes": (T + P + on * P) * case["H"] * e + 12 * P, "flops": 3 * on * P * case["H"]}
    if op == "route_grad":
        return {"bytes": T * E * e * (1 if case["renorm"] else 2) + 12 * P, "flops": 4 * T * E + 4 * P}
    K, N, S = case["K"], case["N"], T * max(k, 1)
    used = E * (1 - (1 - max(k, 1) / E) ** T)  # experts that some token uses, routed uniformly
    return {"bytes": used * N * (K + 4) + T * K * 2 + S * N * e, "flops": 2 * S * N * K}


# --------------------------------------------------------------------------- 64-bit definition


def _slots(ids):
    """Rows of the slots, by walking the experts."""
    flat = ids.reshape(-1)
    rows = np.empty(flat.size, dtype=np.int64)
    at = 0
    for e in np.unique(flat[flat >= 0]):
        where = np.flatnonzero(flat == e)
        rows[where] = np.arange(at, at + where.size)
        at += where.size
    rows[flat < 0] = -1
    return rows


def exact(case, seed):
    s = prepare(case, seed)
    op, T, k, E = case["op"], case["T"], case["k"], case["E"]
    dev = s["x"].device if "x" in s else s["weights"].device
    if op == "dispatch":
        r = torch.from_numpy(_slots(s["ids"].cpu().numpy())).to(dev)
        xs = torch.zeros(T * k, case["H"], dtype=F64, device=dev)
        slot = torch.nonzero(r >= 0).flatten()
        xs[r[slot]] = s["x"].to(F64)[slot // k]
        return {"m_splits": None, "rows": None, "xs": xs}
    if op == "combine":
        r = torch.from_numpy(_slots(s["ids"].cpu().numpy())).to(dev).view(T, k)
        out = torch.zeros(T, case["H"], dtype=F64, device=dev)
        step = max(1, (1 << 25) // (k * case["H"]))
        for t0 in range(0, T, step):
            rr = r[t0:t0 + step]
            w = (rr >= 0).to(F64)
            if case["weighted"]:
                w = w * s["weights"][t0:t0 + step].to(F64)
            out[t0:t0 + step] = torch.einsum("tk,tkh->th", w, s["y"][rr.clamp(min=0)].to(F64))
        return out
    if op == "combine_grad":
        r = torch.from_numpy(_slots(s["ids"].cpu().numpy())).to(dev)
        slot = torch.nonzero(r >= 0).flatten()
        dy = torch.zeros(T * k, case["H"], dtype=F64, device=dev)
        dw = torch.zeros(T * k, dtype=F64, device=dev)
        step = max(1, (1 << 25) // case["H"])
        for i in range(0, slot.numel(), step):
            sl = slot[i:i + step]
            d = s["dout"][sl // k].to(F64)
            dw[sl] = torch.einsum("ph,ph->p", d, s["y"][r[sl]].to(F64))
            dy[r[sl]] = d * s["weights"].flatten()[sl].to(F64).unsqueeze(1)
        return {"dy": dy, "dweights": dw.view(T, k)}
    if op == "route_grad":
        x = s["logits"].to(F32).cpu().numpy().astype(np.float64)
        ids, w, dw = (s[n].cpu().numpy() for n in ("ids", "weights", "dweights"))
        dl = np.zeros((T, E))
        for t in range(T):
            on = ids[t] >= 0
            if not on.any():
                continue
            i, wt, g = ids[t][on], w[t][on].astype(np.float64), dw[t][on].astype(np.float64)
            tot = (wt * g).sum()
            if case["renorm"]:
                dl[t, i] = wt * (g - tot)
            else:
                p = np.exp(x[t] - x[t].max())
                dl[t] = -p / p.sum() * tot
                dl[t, i] += wt * g
        return torch.from_numpy(dl).to(dev)
    K, N = case["K"], case["N"]
    x = s["x"].to(F64)
    a = x.abs().max(dim=-1, keepdim=True).values.clamp(min=2.0 ** -100)
    inv = torch.from_numpy(np.float32(127) / a.cpu().numpy().astype(np.float32)).to(dev)  # rounded to 32 bits, by definition
    q = torch.round(x * inv.to(F64))
    sx = torch.from_numpy(a.cpu().numpy().astype(np.float32) / np.float32(127)).to(dev).to(F64)
    if k == 0:
        y = q @ s["wq"].to(F64).t()
        return y * sx * s["ws"].to(F64)
    flat = s["ids"].flatten()
    y = torch.empty(T * k, N, dtype=F64, device=dev)
    at = 0
    for g in range(E):
        slot = torch.nonzero(flat == g).flatten()
        if slot.numel():
            w = s["wq"][g * N:(g + 1) * N].to(F64)
            y[at:at + slot.numel()] = (q[slot // k] @ w.t()) * sx[slot // k] * s["ws"][g * N:(g + 1) * N].to(F64)
            at += slot.numel()
    return y
