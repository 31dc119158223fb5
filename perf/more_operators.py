"""More operators of a training step as they are measured: layer norms with the residual's addition (forward and
backward), microscaled 4-bit floating point (codes, values, product), and the log probabilities of given tokens with
entropy, top alternatives and gradient.

``run`` computes them in plain torch operations in 32 bits where ``own`` is false, and through the framework's entry
points where it is true; ``exact`` computes them in 64 bits from their definitions.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
DEVICE = "cuda"
EPS = 1e-5
INF = float("inf")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token on its way through a small model's layer, where latency counts
        {"name": "ln_token", "op": "ln", "rows": 1, "cols": 768, "dtype": "bf16", "residual": True, "bias": True},
        # a training step of a small student: forward and backward over a batch of packed sequences
        {"name": "ln_train", "op": "ln_train", "rows": 16384, "cols": 768, "dtype": "bf16", "residual": True,
         "bias": True},
        # fp32 training on an odd width that fills no vector, no residual
        {"name": "ln_train_odd", "op": "ln_train", "rows": 1021, "cols": 1601, "dtype": "fp32", "residual": False,
         "bias": True},
        # a long prompt's activations to 4-bit codes, and the values they stand for
        {"name": "mx_codes", "op": "mx_codes", "rows": 8192, "cols": 4096, "dtype": "bf16"},
        # one token through the widest projection: the weights' bytes
        {"name": "mx_token", "op": "mx", "m": 1, "n": 14336, "k": 4096, "dtype": "bf16", "bias": False},
        # a small batch of decoded tokens through the long reduction
        {"name": "mx_batch", "op": "mx", "m": 24, "n": 4096, "k": 14336, "dtype": "bf16", "bias": False},
        # odd sizes, k inside a block of 32, activations quantised within the call, a bias
        {"name": "mx_odd", "op": "mx_dynamic", "m": 333, "n": 1001, "k": 777, "dtype": "fp16", "bias": True},
        # a prompt through the widest projection, activations quantised within the call: matrix work
        {"name": "mx_prompt", "op": "mx_dynamic", "m": 8192, "n": 14336, "k": 4096, "dtype": "bf16", "bias": False},
        # a served token: its log probability and the 20 best alternatives
        {"name": "lp_token", "op": "lp_top", "rows": 1, "vocab": 128256, "dtype": "bf16", "pad": 0, "top": 20,
         "temperature": 1.0, "masked": False},
        # evaluation of constrained answers in fp32: some rows' masks leave a few tokens only
        {"name": "lp_eval", "op": "lp_top", "rows": 333, "vocab": 32001, "dtype": "fp32", "pad": 0, "top": 5,
         "temperature": 0.7, "masked": True},
        # a training step on log probabilities and entropy, the vocabulary odd, rows padded to 64
        {"name": "lp_train", "op": "lp_train", "rows": 4096, "vocab": 50257, "dtype": "bf16", "pad": 47, "top": 0,
         "temperature": 1.0, "masked": False},
        # the largest: a teacher's top entries over a long batch
        {"name": "lp_teacher", "op": "lp_top", "rows": 8192, "vocab": 128256, "dtype": "bf16", "pad": 0, "top": 64,
         "temperature": 1.0, "masked": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln", "ln_train", "mx_codes", "mx", "mx_dynamic", "lp_top", "lp_top", "lp_train"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("ln", "ln_train", "mx_codes"):
        cols = _log_int(rng, 64, 16384)
        if rng.random() < 0.5:
            cols = max(64, cols // 64 * 64)
        rows = _log_int(rng, 1, min(16384, 8192 * 4096 // cols))
        if op == "mx_codes":
            return {"op": op, "rows": rows, "cols": cols, "dtype": dtype}
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "residual": rng.random() < 0.7,
                "bias": rng.random() < 0.8}
    if op.startswith("mx"):
        k, n = _log_int(rng, 256, 14336), _log_int(rng, 256, 14336)
        if rng.random() < 0.6:
            k, n = max(256, k // 64 * 64), max(256, n // 64 * 64)
        m = _log_int(rng, 1, min(8192, 8192 * 14336 * 4096 // (n * k)))
        return {"op": op, "m": m, "n": n, "k": k, "dtype": dtype, "bias": rng.random() < 0.3}
    vocab = _log_int(rng, 1000, 131072)
    most = 8192 * 128256 // (2 if dtype == "fp32" else 1) // (4 if op == "lp_train" else 1)
    rows = _log_int(rng, 1, min(8192, most // (vocab + 64)))
    return {"op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "pad": rng.choice([0, 0, -vocab % 64]),
            "top": _log_int(rng, 1, 128) if op == "lp_top" else 0, "temperature": rng.choice([0.5, 1.0, 1.0, 2.0]),
            "masked": rng.random() < 0.3}


# ----------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    state = dict(case)
    if case["op"].startswith("ln"):
        dt, shape, cols = DTYPES[case["dtype"]], (case["rows"], case["cols"]), case["cols"]
        state["x"] = torch.randn(shape, generator=g, device=DEVICE, dtype=dt) + 0.25
        # a residual stream: larger than what a layer adds, its tokens off centre, a few channels far larger
        wide = torch.ones(cols, device=DEVICE, dtype=dt)
        wide[torch.randint(cols, (3,), generator=g, device=DEVICE)] = 12.0
        off = torch.randn((case["rows"], 1), generator=g, device=DEVICE, dtype=dt)
        state["r"] = torch.randn(shape, generator=g, device=DEVICE, dtype=dt) * 2 * wide + off if case["residual"] else None
        state["w"] = 1 + 0.2 * torch.randn(cols, generator=g, device=DEVICE, dtype=dt)
        state["b"] = 0.2 * torch.randn(cols, generator=g, device=DEVICE, dtype=dt) if case["bias"] else None
        if case["op"] == "ln_train":
            state["dy"] = torch.randn(shape, generator=g, device=DEVICE, dtype=dt) * 0.01
            state["dh"] = (torch.randn(shape, generator=g, device=DEVICE, dtype=dt) * 0.01 if case["residual"]
                           else None)
    elif case["op"] == "mx_codes":
        # activations behind a norm: a few channels far larger than the others
        wide = torch.ones(case["cols"], device=DEVICE)
        wide[torch.randint(case["cols"], (3,), generator=g, device=DEVICE)] = 12.0
        state["x"] = (torch.randn((case["rows"], case["cols"]), generator=g, device=DEVICE) * wide).to(
            DTYPES[case["dtype"]])
    elif case["op"].startswith("mx"):
        m, n, k = case["m"], case["n"], case["k"]
        x = torch.randn((m, k), generator=g, device=DEVICE)
        if case["op"] == "mx":    # codes that the quantisation before it wrote
            state["a"], state["sa"] = _pack(*_mx_codes(x))
        else:
            state["x"] = x.to(torch.bfloat16)
        # the weights' codes: laid out once
        w = torch.randn((n, k), generator=g, device=DEVICE) * (0.5 + torch.rand((n, 1), generator=g, device=DEVICE))
        state["w"], state["sw"] = _pack(*_mx_codes(w / math.sqrt(k)))
        state["bias"] = torch.randn(n, generator=g, device=DEVICE) if case["bias"] else None
    else:
        rows, vocab = case["rows"], case["vocab"]
        dt = DTYPES[case["dtype"]]
        z = torch.randn((rows, vocab + case["pad"]), generator=g, device=DEVICE, dtype=dt)
        z = z.mul_(2.0)[:, :vocab]    # a padded vocabulary: rows further apart than they are long
        # the tokens, on which the model mostly agrees, and a few tokens that it holds for likely
        tokens = torch.randint(vocab, (rows,), generator=g, device=DEVICE)
        some = torch.randint(vocab, (rows, 8), generator=g, device=DEVICE)
        some[:, 0] = tokens
        z.scatter_add_(1, some, (8 * torch.rand((rows, 8), generator=g, device=DEVICE)).to(dt))
        if case["masked"]:    # one row in four may answer with a few tokens only
            keep = torch.zeros((rows, vocab), dtype=torch.bool, device=DEVICE).scatter_(1, some, True)
            keep[torch.arange(rows, device=DEVICE) % 4 != 3] = True
            z.masked_fill_(~keep, -INF)
        tokens[15::16] = -100    # tokens of a prompt or padding: left out
        state["z"], state["tokens"] = z, tokens
        if case["op"] == "lp_train":
            state["gl"] = torch.randn(rows, generator=g, device=DEVICE) / rows
            state["ge"] = torch.full((rows,), -0.01 / rows, device=DEVICE)
    return state


# ------------------------------------------------------------ plain forms
def _norm(s):
    x = s["x"].float()
    if s["r"] is not None:
        x = x + s["r"].float()
    mean = x.sum(1) / x.shape[1]
    d = x - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).sum(1) / x.shape[1] + EPS)
    y = d * rstd[:, None] * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    return x, mean, rstd, y


def _mx_codes(x):
    """4-bit floating point: codes (sign, two bits of exponent, one of mantissa) and the exponent of each block of 32"""
    rows, cols = x.shape
    x = x.float()
    if cols % 32:
        x = torch.cat([x, x.new_zeros((rows, -cols % 32))], 1)
    x = x.view(rows, -1, 32)
    amax = x.abs().amax(2)
    part, e = torch.frexp(amax)    # amax = part 2^e, part in [0.5, 1)
    e = torch.where(amax > 0, e - 3 + (part >= 0.875), -127).clamp_min(-127)    # the least with amax < 7 2^e
    v = torch.ldexp(torch.ldexp(x, -(e // 2)[:, :, None]), -(e - e // 2)[:, :, None])
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp_max(6)
    code = torch.where(a <= 2, 2 * a, torch.where(a <= 4, a + 2, 7.0)).to(torch.uint8) | (v < 0).to(torch.uint8) * 8
    return code.view(rows, -1)[:, :cols], (e + 127).to(torch.uint8)


def _pack(code, scale):
    """two codes a byte, the even one low"""
    if code.shape[1] % 2:
        code = torch.cat([code, code.new_zeros((code.shape[0], 1))], 1)
    return code[:, ::2] | code[:, 1::2] << 4, scale


def _mx_values(codes, scale, cols):
    code = torch.stack([codes & 15, codes >> 4], 2).view(codes.shape[0], -1)[:, :cols].int()
    mag = code & 7
    v = torch.where(mag < 4, 0.5 * mag, torch.where(mag < 6, mag - 2.0, 2.0 * mag - 8))
    v = torch.where(code >= 8, -v, v)
    e = scale.int().repeat_interleave(32, 1)[:, :cols] - 127
    return torch.ldexp(torch.ldexp(v, e // 2), e - e // 2)


def _logprobs(s, z):
    """maximum, log of the sum, log probabilities and entropy of each row"""
    u = z / s["temperature"]
    m = u.amax(1, keepdim=True)
    u = u - m
    e = torch.exp(u)
    total = e.sum(1, keepdim=True)
    logq = u - torch.log(total)
    q = e / total
    return logq, q, -torch.where(q > 0, q * logq, 0).sum(1)


def _token(s, logq):
    t = s["tokens"]
    has = (t >= 0) & (t < s["vocab"])
    at = torch.where(has, t, 0)[:, None]
    return has, at, torch.where(has, logq.gather(1, at)[:, 0], 0)


def _top(s, z, logq):
    """the largest, equal ones by their index: both in one whole number"""
    bits = (z + 0.0).view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32
    order |= 0xFFFFFFFF - torch.arange(z.shape[1], device=z.device)
    index = 0xFFFFFFFF - (torch.topk(order, s["top"], dim=1).values & 0xFFFFFFFF)
    top = logq.gather(1, index)
    return top, torch.where(z.gather(1, index) == -INF, -1, index)


def _plain(s):
    op = s["op"]
    if op.startswith("ln"):
        x, mean, rstd, y = _norm(s)
        dt = s["x"].dtype
        out = {"y": y.to(dt)}
        if s["r"] is not None:
            out["h"] = x.to(dt)
        if op == "ln":
            return out
        n = x.shape[1]
        dy = s["dy"].float()
        u = (x.to(dt).float() - mean[:, None]) * rstd[:, None]
        g = dy * s["w"].float()
        dx = rstd[:, None] * (g - g.sum(1, keepdim=True) / n - u * ((g * u).sum(1, keepdim=True) / n))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        out.update(dx=dx.to(dt), dw=(dy * u).sum(0).to(dt))
        if s["b"] is not None:
            out["db"] = dy.sum(0).to(dt)
        return out
    if op == "mx_codes":
        return _mx_values(*_pack(*_mx_codes(s["x"])), s["cols"]).to(s["x"].dtype)
    if op.startswith("mx"):
        a, sa = (s["a"], s["sa"]) if op == "mx" else _pack(*_mx_codes(s["x"]))
        y = _mx_values(a, sa, s["k"]) @ _mx_values(s["w"], s["sw"], s["k"]).t()
        if s["bias"] is not None:
            y = y + s["bias"]
        return y.to(DTYPES[s["dtype"]])
    z = s["z"].float()
    logq, q, entropy = _logprobs(s, z)
    has, at, logprob = _token(s, logq)
    out = {"logprob": logprob, "entropy": entropy}
    if op == "lp_top":
        out["top"], out["index"] = _top(s, z, logq)
        return out
    gl = torch.where(has, s["gl"], 0)[:, None]
    slope = gl + s["ge"][:, None] * (logq + entropy[:, None])
    d = torch.where(q > 0, -q * slope, 0).scatter_add_(1, at, gl) / s["temperature"]
    out["dlogits"] = d.to(s["z"].dtype)
    return out


# ---------------------------------------------- the framework's operators
def _own(s):
    import orthogonalized_optimizer_step_amd as dion
    op = s["op"]
    if op.startswith("ln"):
        y, h, mean, rstd = dion.layernorm(s["x"], s["w"], s["b"], residual=s["r"], eps=EPS)
        out = {"y": y}
        if s["r"] is not None:
            out["h"] = h
        if op == "ln":
            return out
        out["dx"], out["dw"], db = dion.layernorm_backward(s["dy"], h, s["w"], mean, rstd, dh=s["dh"],
                                                           bias=s["b"] is not None)
        if s["b"] is not None:
            out["db"] = db
        return out
    if op == "mx_codes":
        return dion.mxfp4_dequantize(*dion.mxfp4_quantize(s["x"]), dtype=s["x"].dtype, cols=s["cols"])
    if op.startswith("mx"):
        a, sa = (s["a"], s["sa"]) if op == "mx" else dion.mxfp4_quantize(s["x"])
        return dion.mxfp4_linear(a, sa, s["w"], s["sw"], bias=s["bias"], out_dtype=DTYPES[s["dtype"]])
    temp = s["temperature"]
    if op == "lp_top":
        top, index, logprob, entropy = dion.top_logprobs(s["z"], s["top"], s["tokens"], temperature=temp)
        return {"logprob": logprob, "entropy": entropy, "top": top, "index": index}
    logprob, entropy, stats = dion.token_logprobs(s["z"], s["tokens"], temperature=temp)
    return {"logprob": logprob, "entropy": entropy,
            "dlogits": dion.token_logprobs_backward(s["gl"], s["ge"], s["z"], stats, s["tokens"], temperature=temp)}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    b = BYTES[case["dtype"]]
    if op.startswith("ln"):
        e, vectors = case["rows"] * case["cols"], (2 if case["bias"] else 1) * case["cols"] * b
        forward = (4 if case["residual"] else 2) * b         # x, the residual and the stream carried on, y
        if op == "ln":
            return {"bytes": e * forward + vectors, "flops": 9 * e}
        back = (3 if case["residual"] else 2) * b            # dy, dx and the stream's gradient
        return {"bytes": e * (forward + back) + 2 * vectors, "flops": 23 * e}
    if op == "mx_codes":
        e = case["rows"] * case["cols"]
        return {"bytes": 2 * e * b, "flops": 4 * e}
    if op.startswith("mx"):
        m, n, k = case["m"], case["n"], case["k"]
        scales = (k + 31) // 32
        a = m * ((k + 1) // 2 + scales) if op == "mx" else 2 * m * k
        return {"bytes": a + n * ((k + 1) // 2 + scales) + m * n * b + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    rows, vocab = case["rows"], case["vocab"]
    read = rows * vocab * b + 8 * rows
    if op == "lp_top":
        return {"bytes": read + rows * (8 + 12 * case["top"]), "flops": 6 * rows * vocab}
    return {"bytes": read + rows * vocab * b + 16 * rows, "flops": 12 * rows * vocab}


# ------------------------------------------------- definitions in 64 bits
def _mx_exact(x):
    """the values that 4 bits leave of x: the nearest of 15, equally near ones to the even code"""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x.double(), (0, -cols % 32)).view(rows, -1, 32)
    top = x.abs().max(2, keepdim=True).values
    # candidates 2^e for the scale, the least of them with top < 7 2^e
    e = torch.log2(torch.where(top > 0, top, 1) / 7).floor()
    e = torch.where(torch.exp2(e) * 7 > top, e, e + 1)
    scale = torch.where(top > 0, torch.exp2(e.clamp_min(-127)), 1)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    a = x.abs() / scale
    best, gap = torch.zeros_like(a), a.clone()
    for i in range(1, 8):
        far = (a - grid[i]).abs()
        nearer = far < gap if i % 2 else far <= gap    # from a tie with the odd code below, up to the even one
        best, gap = torch.where(nearer, grid[i], best), torch.where(nearer, far, gap)
    return (torch.sign(x) * best * scale).view(rows, -1)[:, :cols]


def _mx_read(codes, scale, cols):
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=codes.device)
    grid = torch.cat([grid, -grid])
    out = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device=codes.device)
    out[:, 0::2], out[:, 1::2] = grid[(codes % 16).long()], grid[(codes // 16).long()]
    out = out[:, :cols]
    block = torch.arange(cols, device=codes.device) // 32
    return out * torch.exp2(scale.double() - 127)[:, block]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = torch.float64
    if op.startswith("ln"):
        h = s["x"].to(d) if s["r"] is None else s["x"].to(d) + s["r"].to(d)
        unit = h - h.mean(1, keepdim=True)
        std = (unit.pow(2).mean(1, keepdim=True) + EPS).sqrt()
        unit = unit / std
        w = s["w"].to(d)
        out = {"y": unit * w if s["b"] is None else unit * w + s["b"].to(d)}
        if s["r"] is not None:
            out["h"] = h
        if op == "ln":
            return out
        # the gradient of sum(y * dy) + sum(h * dh)
        dy = s["dy"].to(d)
        a = dy * w
        dx = (a - a.mean(1, keepdim=True) - unit * (a * unit).mean(1, keepdim=True)) / std
        out["dx"] = dx if s["dh"] is None else dx + s["dh"].to(d)
        out["dw"] = (dy * unit).sum(0)
        if s["b"] is not None:
            out["db"] = dy.sum(0)
        return out
    if op == "mx_codes":
        return torch.cat([_mx_exact(x) for x in s["x"].split(max(1, (1 << 25) // case["cols"]))])
    if op.startswith("mx"):
        k = case["k"]
        a = _mx_read(s["a"], s["sa"], k) if op == "mx" else _mx_exact(s["x"])
        y = a @ _mx_read(s["w"], s["sw"], k).t().contiguous()
        return y if s["bias"] is None else y + s["bias"].to(d)
    temp, vocab = case["temperature"], case["vocab"]
    parts = []
    at_once = max(1, (1 << 27) // vocab)
    for lo in range(0, case["rows"], at_once):
        z = s["z"][lo:lo + at_once].to(d)
        t = s["tokens"][lo:lo + at_once]
        q = torch.softmax(z / temp, 1)
        logq = torch.log_softmax(z / temp, 1)
        hit = torch.arange(vocab, device=z.device) == t[:, None]
        entropy = -torch.special.xlogy(q, q).sum(1)
        part = [torch.where(hit, logq, 0).sum(1), entropy]
        if op == "lp_top":
            value, index = torch.sort(z, dim=1, descending=True, stable=True)
            value, index = value[:, :case["top"]], index[:, :case["top"]]
            part += [logq.gather(1, index), torch.where(value > -INF, index, -1)]
        else:
            gl, ge = s["gl"][lo:lo + at_once, None].to(d), s["ge"][lo:lo + at_once, None].to(d)
            some = hit.any(1, keepdim=True)
            centred = torch.special.xlogy(q, q) + q * entropy[:, None]
            part.append(((hit.to(d) - q) * some * gl - centred * ge) / temp)
        parts.append(part)
    joined = [torch.cat(p) for p in zip(*parts)]
    return dict(zip(["logprob", "entropy"] + (["top", "index"] if op == "lp_top" else ["dlogits"]), joined))
