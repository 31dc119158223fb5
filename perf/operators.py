"""The distillation path's operators as they are measured: RMS norms with the residual's addition (forward with 16-bit or
8-bit output, and backward), the 8-bit product with scales for tokens and channels, and the distillation loss on a
teacher's top logits (forward, backward, and both in one call).

``run`` computes them in plain torch operations in 32 bits where ``own`` is false, and through the framework's entry
points where it is true; ``exact`` computes them in 64 bits from their definitions.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
READ_BACK = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.bfloat16}    # 8-bit codes, as values
DEVICE = "cuda"
EPS = 1e-5
INF = float("inf")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token on its way through a layer: the norm before an 8-bit product, where latency counts
        {"name": "norm_int8_token", "op": "norm_int8", "rows": 1, "cols": 4096, "dtype": "bf16", "residual": True},
        # a long prompt or a packed batch of the 8-bit teacher
        {"name": "norm_int8_prompt", "op": "norm_int8", "rows": 8192, "cols": 4096, "dtype": "bf16", "residual": True},
        # a training step of a small student: forward and backward over a batch of packed sequences
        {"name": "norm_train", "op": "norm_train", "rows": 16384, "cols": 768, "dtype": "bf16", "residual": True},
        # fp32 training on an odd width that fills no vector, no residual
        {"name": "norm_train_odd", "op": "norm_train", "rows": 777, "cols": 1001, "dtype": "fp32", "residual": False},
        # one token through the widest projection: the weights' bytes
        {"name": "linear_token", "op": "linear", "m": 1, "n": 14336, "k": 4096, "dtype": "bf16", "bias": False},
        # a small batch of decoded tokens through the long reduction
        {"name": "linear_batch", "op": "linear", "m": 24, "n": 4096, "k": 14336, "dtype": "bf16", "bias": False},
        # odd sizes, activations quantised within the call, a bias
        {"name": "linear_odd", "op": "linear_dynamic", "m": 333, "n": 1001, "k": 777, "dtype": "fp16", "bias": True},
        # a prompt through the widest projection: matrix work
        {"name": "linear_prompt", "op": "linear", "m": 8192, "n": 14336, "k": 4096, "dtype": "bf16", "bias": False},
        # the loss of a few tokens, no gradient (evaluation)
        {"name": "distill_eval", "op": "distill_eval", "rows": 5, "vocab": 50257, "k": 32, "dtype": "fp32",
         "tdtype": "fp32", "pad": 0, "temperature": 1.0},
        # a training step of a small student: loss and gradient in one call, the vocabulary odd, rows padded to 64
        {"name": "distill_step", "op": "distill_step", "rows": 4096, "vocab": 50257, "k": 64, "dtype": "bf16",
         "tdtype": "bf16", "pad": 47, "temperature": 2.0},
        # fp32 logits, forward and backward apart as automatic differentiation calls them
        {"name": "distill_train", "op": "distill_train", "rows": 1021, "vocab": 32001, "k": 100, "dtype": "fp32",
         "tdtype": "fp32", "pad": 0, "temperature": 1.5},
        # the largest: a long batch over a large vocabulary
        {"name": "distill_step_large", "op": "distill_step", "rows": 8192, "vocab": 128256, "k": 128, "dtype": "bf16",
         "tdtype": "bf16", "pad": 0, "temperature": 1.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_int8", "norm_train", "linear", "linear_dynamic", "distill_eval", "distill_step",
                     "distill_train"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op.startswith("norm"):
        cols = _log_int(rng, 64, 16384)
        if rng.random() < 0.5:
            cols = max(64, cols // 64 * 64)
        rows = _log_int(rng, 1, min(16384, 8192 * 4096 // cols))
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "residual": rng.random() < 0.7}
    if op.startswith("linear"):
        k, n = _log_int(rng, 256, 14336), _log_int(rng, 256, 14336)
        if rng.random() < 0.6:
            k, n = max(256, k // 64 * 64), max(256, n // 64 * 64)
        m = _log_int(rng, 1, min(8192, 8192 * 14336 * 4096 // (n * k)))
        return {"op": op, "m": m, "n": n, "k": k, "dtype": dtype, "bias": rng.random() < 0.3}
    vocab = _log_int(rng, 1000, 131072)
    most = 8192 * 128256 // (2 if dtype == "fp32" else 1) // (2 if op == "distill_train" else 1)
    rows = _log_int(rng, 1, min(8192, most // (vocab + 64)))
    return {"op": op, "rows": rows, "vocab": vocab, "k": _log_int(rng, 1, 256), "dtype": dtype,
            "tdtype": rng.choice(["bf16", "fp32"]), "pad": rng.choice([0, 0, -vocab % 64]),
            "temperature": rng.choice([0.5, 1.0, 1.0, 2.0, 4.0])}


# ----------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    state = dict(case)
    if case["op"].startswith("norm"):
        dt, shape = DTYPES[case["dtype"]], (case["rows"], case["cols"])
        state["x"] = torch.randn(shape, generator=g, device=DEVICE, dtype=dt)
        # a residual stream: larger than what a layer adds, a few channels far larger than the others
        wide = torch.ones(case["cols"], device=DEVICE, dtype=dt)
        wide[torch.randint(case["cols"], (3,), generator=g, device=DEVICE)] = 12.0
        state["r"] = torch.randn(shape, generator=g, device=DEVICE, dtype=dt) * 2 * wide if case["residual"] else None
        state["w"] = 1 + 0.2 * torch.randn(case["cols"], generator=g, device=DEVICE, dtype=dt)
        if case["op"] == "norm_train":
            state["dy"] = torch.randn(shape, generator=g, device=DEVICE, dtype=dt) * 0.01
            state["dh"] = (torch.randn(shape, generator=g, device=DEVICE, dtype=dt) * 0.01 if case["residual"]
                           else None)
    elif case["op"].startswith("linear"):
        m, n, k = case["m"], case["n"], case["k"]
        if case["op"] == "linear":    # codes and scales that the norm before it wrote
            state["a"] = (torch.randn((m, k), generator=g, device=DEVICE) * 32).round().clamp(-127, 127).to(torch.int8)
            state["sa"] = 0.02 + 0.03 * torch.rand(m, generator=g, device=DEVICE)
        else:
            state["x"] = torch.randn((m, k), generator=g, device=DEVICE, dtype=torch.bfloat16)
        state["b"] = (torch.randn((n, k), generator=g, device=DEVICE) * 32).round().clamp(-127, 127).to(torch.int8)
        state["sb"] = (0.5 + torch.rand(n, generator=g, device=DEVICE)) / (32 * math.sqrt(k))
        state["bias"] = torch.randn(n, generator=g, device=DEVICE) if case["bias"] else None
    else:
        rows, vocab, k = case["rows"], case["vocab"], case["k"]
        dt = DTYPES[case["dtype"]]
        z = torch.randn((rows, vocab + case["pad"]), generator=g, device=DEVICE, dtype=dt)
        z = z.mul_(2.0)[:, :vocab]    # a padded vocabulary: rows further apart than they are long
        # distinct indices in each row: one from each of k strata of the vocabulary
        width = vocab // k
        idx = torch.randint(width, (rows, k), generator=g, device=DEVICE) + width * torch.arange(k, device=DEVICE)
        idx = idx[:, torch.randperm(k, generator=g, device=DEVICE)]
        # top logits, descending, on which the student mostly agrees
        t = 14 - torch.rand((rows, k), generator=g, device=DEVICE).mul(1.2 * 12 / k).cumsum(1)
        z.scatter_(1, idx, (t - 3 + torch.randn((rows, k), generator=g, device=DEVICE)).to(dt))
        # a teacher whose top set was cut at a share of the mass leaves its last places absent, and the tokens of the
        # instruction (one in 16) have no teacher at all
        cut = torch.randint(max(1, k // 2), k + 1, (rows, 1), generator=g, device=DEVICE)
        cut[15::16] = 0
        state["idx"] = torch.where(torch.arange(k, device=DEVICE) < cut, idx, -1)
        state["t"] = t.to(DTYPES[case["tdtype"]])
        state["z"] = z
        state["gl"] = torch.full((rows,), 1.0 / (rows - rows // 16), device=DEVICE)
    return state


# ------------------------------------------------------------ plain forms
def _norm(s):
    x = s["x"].float()
    if s["r"] is not None:
        x = x + s["r"].float()
    rstd = 1 / torch.sqrt((x * x).mean(1) + EPS)
    return x, rstd, x * rstd[:, None] * s["w"].float()


def _codes(y):
    amax = y.abs().amax(1)
    inv = torch.where(amax > 0, 127 / amax, 0)
    return torch.round(y * inv[:, None]), amax / 127


def _product(a, sa, b, sb, bias, dt):
    y = (a.float() @ b.float().t()) * sa[:, None] * sb
    if bias is not None:
        y = y + bias
    return y.to(dt)


def _teacher(s):
    temp, t, idx = s["temperature"], s["t"].float(), s["idx"]
    ok = (idx >= 0) & (idx < s["vocab"]) & (t != -INF)
    live = ok.any(1)
    top = torch.where(live, torch.where(ok, t, -INF).amax(1), 0)
    u = torch.where(ok, (t - top[:, None]) / temp, -INF)
    e = torch.exp(u)
    total = torch.where(live, e.sum(1), 1)[:, None]
    return torch.where(ok, idx, 0), live, e / total, u - torch.log(total)


def _loss(s, z, idx, live, p, logp):
    temp = s["temperature"]
    m = z.amax(1)
    logs = torch.log(torch.exp((z - m[:, None]) / temp).sum(1))
    logq = (z.gather(1, idx) - m[:, None]) / temp - logs[:, None]
    loss = temp * temp * torch.where(p > 0, p * (logp - logq), 0).sum(1)
    zero = torch.zeros_like(m)
    return torch.where(live, loss, zero), torch.where(live, m, zero), torch.where(live, logs, zero)


def _dlogits(s, z, idx, live, p, m, logs):
    temp = s["temperature"]
    d = torch.exp((z - m[:, None]) / temp - logs[:, None]).scatter_add_(1, idx, -p)
    d = d * (s["gl"] * temp)[:, None]
    return torch.where((live & (s["gl"] != 0))[:, None], d, 0).to(s["z"].dtype)


def _plain(s):
    op = s["op"]
    if op == "norm_int8":
        x, rstd, y = _norm(s)
        q, scale = _codes(y)
        out = {"y": (q * scale[:, None]).to(READ_BACK[s["dtype"]]), "scale": scale}
        if s["r"] is not None:
            out["h"] = x.to(s["x"].dtype)
        return out
    if op == "norm_train":
        x, rstd, y = _norm(s)
        dt = s["x"].dtype
        h, dy = x.to(dt).float(), s["dy"].float()
        gw = dy * s["w"].float()
        dx = rstd[:, None] * (gw - h * ((gw * h).mean(1) * rstd * rstd)[:, None])
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        out = {"y": y.to(dt), "dx": dx.to(dt), "dw": (dy * h * rstd[:, None]).sum(0).to(dt)}
        if s["r"] is not None:
            out["h"] = x.to(dt)
        return out
    if op == "linear":
        return _product(s["a"], s["sa"], s["b"], s["sb"], s["bias"], DTYPES[s["dtype"]])
    if op == "linear_dynamic":
        a, sa = _codes(s["x"].float())
        return _product(a, sa, s["b"], s["sb"], s["bias"], DTYPES[s["dtype"]])
    z = s["z"].float()
    teacher = _teacher(s)
    loss, m, logs = _loss(s, z, *teacher)
    if op == "distill_eval":
        return {"loss": loss}
    return {"loss": loss, "dlogits": _dlogits(s, z, *teacher[:3], m, logs)}


# ---------------------------------------------- the framework's operators
def _own(s):
    import orthogonalized_optimizer_step_amd as dion
    op = s["op"]
    if op == "norm_int8":
        q, scale, h = dion.rmsnorm_int8(s["x"], s["w"], residual=s["r"], eps=EPS)
        out = {"y": dion.int8_dequantize(q, scale, READ_BACK[s["dtype"]]), "scale": scale}
        if s["r"] is not None:
            out["h"] = h
        return out
    if op == "norm_train":
        y, h, rstd = dion.rmsnorm(s["x"], s["w"], residual=s["r"], eps=EPS)
        dx, dw = dion.rmsnorm_backward(s["dy"], h, s["w"], rstd, dh=s["dh"])
        out = {"y": y, "dx": dx, "dw": dw}
        if s["r"] is not None:
            out["h"] = h
        return out
    if op == "linear":
        return dion.int8_linear(s["a"], s["sa"], s["b"], s["sb"], bias=s["bias"], out_dtype=DTYPES[s["dtype"]])
    if op == "linear_dynamic":
        a, sa = dion.int8_quantize(s["x"])
        return dion.int8_linear(a, sa, s["b"], s["sb"], bias=s["bias"], out_dtype=DTYPES[s["dtype"]])
    temp = s["temperature"]
    if op == "distill_step":
        loss, dz = dion.distill_topk_step(s["z"], s["t"], s["idx"], s["gl"], temperature=temp)
        return {"loss": loss, "dlogits": dz}
    loss, stats = dion.distill_topk(s["z"], s["t"], s["idx"], temperature=temp)
    if op == "distill_eval":
        return {"loss": loss}
    return {"loss": loss, "dlogits": dion.distill_topk_backward(s["gl"], s["z"], stats, s["t"], s["idx"],
                                                                temperature=temp)}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op.startswith("norm"):
        e = case["rows"] * case["cols"]
        b = BYTES[case["dtype"]]
        passes = (2 if case["residual"] else 0) * b + b      # x, the residual and the stream carried on
        if op == "norm_int8":     # the values that the 8 bits stand for, in 16 bits
            return {"bytes": e * (passes + 2) + case["cols"] * b + 4 * case["rows"], "flops": 8 * e}
        back = (3 if case["residual"] else 2) * b            # dy, dx and the stream's gradient
        return {"bytes": e * (passes + b + back) + 2 * case["cols"] * b, "flops": 16 * e}
    if op.startswith("linear"):
        m, n, k = case["m"], case["n"], case["k"]
        a = m * k + 4 * m if op == "linear" else 2 * m * k
        return {"bytes": a + n * k + 4 * n + m * n * BYTES[case["dtype"]] + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    rows, vocab, k = case["rows"], case["vocab"], case["k"]
    b = BYTES[case["dtype"]]
    read = (rows - rows // 16) * vocab * b + rows * k * (8 + BYTES[case["tdtype"]]) + 4 * rows
    if op == "distill_eval":
        return {"bytes": read, "flops": 4 * rows * vocab}
    return {"bytes": read + rows * vocab * b + 4 * rows, "flops": 8 * rows * vocab}


# ------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = torch.float64
    if op.startswith("norm"):
        h = s["x"].to(d) if s["r"] is None else s["x"].to(d) + s["r"].to(d)
        n = h.shape[1]
        rms = (h.pow(2).sum(1, keepdim=True) / n + EPS).sqrt()
        y = h / rms * s["w"].to(d)
        stream = {} if s["r"] is None else {"h": h}
        if op == "norm_int8":
            step = y.abs().max(1, keepdim=True).values / 127
            return {"y": torch.round(y / step) * step, "scale": step[:, 0], **stream}
        # the gradient of sum(y * dy) + sum(h * dh)
        dy, unit = s["dy"].to(d), h / rms
        a = dy * s["w"].to(d)
        dx = (a - unit * (a * unit).sum(1, keepdim=True) / n) / rms
        if s["dh"] is not None:
            dx = dx + s["dh"].to(d)
        return {"y": y, "dx": dx, "dw": (dy * unit).sum(0), **stream}
    if op.startswith("linear"):
        if op == "linear":
            a = s["a"].to(d) * s["sa"].to(d)[:, None]
        else:
            x = s["x"].to(d)
            step = x.abs().max(1, keepdim=True).values / 127
            a = torch.round(x / step) * step
        y = a @ (s["b"].to(d) * s["sb"].to(d)[:, None]).t().contiguous()
        return y if s["bias"] is None else y + s["bias"].to(d)
    temp, vocab = case["temperature"], case["vocab"]
    losses, grads = [], []
    at_once = max(1, (1 << 28) // vocab)
    for lo in range(0, case["rows"], at_once):
        z = s["z"][lo:lo + at_once].to(d) / temp
        idx, t = s["idx"][lo:lo + at_once], s["t"][lo:lo + at_once].to(d) / temp
        has = idx >= 0
        some = has.any(1, keepdim=True)
        # the teacher as a distribution over the whole vocabulary
        share = torch.where(has, torch.exp(t - t.max(1, keepdim=True).values), 0)
        share = share / share.sum(1, keepdim=True).clamp_min(1e-300)
        p = torch.zeros_like(z).scatter_add_(1, idx.clamp_min(0), share)
        z = z - z.max(1, keepdim=True).values
        logq = z - z.exp().sum(1, keepdim=True).log()
        losses.append(temp ** 2 * (torch.special.xlogy(p, p) - p * logq).sum(1))
        if op != "distill_eval":
            grads.append((logq.exp() - p) * some * temp * s["gl"][lo:lo + at_once].to(d)[:, None])
    out = {"loss": torch.cat(losses)}
    if grads:
        out["dlogits"] = torch.cat(grads)
    return out
