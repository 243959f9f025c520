"""The dense feed-forward operators around the experts, as cases to be timed and compared.

Three operators, each in its plain form (elementary torch operations in 32 bits, rounded once at
the end) and as the calls a user makes of this package:

* ``fp8_linear``: y = deq(q(x)) deq(W)^T with 8-bit floating-point (e4m3) operands, one fp32 scale
  for each 128 consecutive K elements of a row of x and one for each 128 x 128 block of W;
* ``gated_linear``: h = act(x Wg^T) * (x Wu^T), and its backward pass (dx, dWg, dWu);
* ``residual_norm``: the norm after a block, its gate and residual scale, the residual sum and the
  norm before the next block, and its backward pass.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one decoded token through an 8-bit projection of the model width (latency; weight bytes)
        {"name": "fp8 one token", "op": "fp8", "m": 1, "k": 7168, "n": 2048, "type": "bf16"},
        # a decode batch of an odd number of sequences through the wide, short projection
        {"name": "fp8 odd batch", "op": "fp8", "m": 37, "k": 1536, "n": 16384, "type": "fp16"},
        # a small prefill chunk, sizes that end inside the scale blocks and the tiles
        {"name": "fp8 ragged chunk", "op": "fp8", "m": 333, "k": 2000, "n": 1137, "type": "bf16"},
        # a whole prefill of 4096 tokens through a square projection (tensor-bound)
        {"name": "fp8 prefill", "op": "fp8", "m": 4096, "k": 7168, "n": 7168, "type": "bf16"},
        # one decoded token through gate and up of a shared-expert-sized block
        {"name": "gated one token", "op": "gated", "t": 1, "h": 7168, "i": 2048, "type": "bf16", "act": "silu", "train": False},
        # a ragged chunk forward, widths that end inside the tiles
        {"name": "gated ragged chunk", "op": "gated", "t": 333, "h": 1544, "i": 1000, "type": "fp16", "act": "gelu", "train": False},
        # a small training step with an odd number of tokens
        {"name": "gated odd step", "op": "gated", "t": 517, "h": 1536, "i": 2048, "type": "fp16", "act": "gelu_tanh", "train": True},
        # a full training step: forward, input gradient and both weight gradients
        {"name": "gated training step", "op": "gated", "t": 4096, "h": 7168, "i": 2048, "type": "bf16", "act": "silu", "train": True},
        # one decoded token between two blocks (latency)
        {"name": "norm one token", "op": "norm", "m": 1, "k": 7168, "type": "bf16", "rtype": "bf16", "gate": "none", "scale": 1.0,
         "after": True, "before": True, "train": False},
        # a prefill's tokens between two blocks: one pass over memory
        {"name": "norm prefill", "op": "norm", "m": 4096, "k": 7168, "type": "bf16", "rtype": "bf16", "gate": "channel", "scale": 0.22,
         "after": True, "before": True, "train": False},
        # a training step with an fp32 residual stream, odd sizes and a gate for each token
        {"name": "norm odd step", "op": "norm", "m": 1001, "k": 1544, "type": "fp16", "rtype": "fp32", "gate": "token", "scale": 0.5,
         "after": True, "before": True, "train": True},
        # a training step at full width, a gate for each of eight sequences and channel
        {"name": "norm training step", "op": "norm", "m": 8192, "k": 7168, "type": "bf16", "rtype": "bf16", "gate": "sequence", "scale": 1.0,
         "after": True, "before": True, "train": True},
    ]


def _spread(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread evenly over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return min(high, max(low, int(round(v / step)) * step)) // step * step


def draw(rng):
    op = rng.choice(["fp8", "gated", "norm"])
    if op == "fp8":
        k, n = _spread(rng, 256, 7168, 16), _spread(rng, 128, 16384, rng.choice([1, 8, 8, 128]))
        m = _spread(rng, 1, min(4096, 4096 * 7168 * 7168 // (k * n)))
        return {"op": op, "m": m, "k": k, "n": n, "type": rng.choice(["bf16", "fp16"])}
    if op == "gated":
        h, i = _spread(rng, 256, 7168, 8), _spread(rng, 256, 4096, 8)
        t = _spread(rng, 1, min(4096, 4096 * 7168 * 2048 // (h * i)))
        return {"op": op, "t": t, "h": h, "i": i, "type": rng.choice(["bf16", "fp16"]), "act": rng.choice(["silu", "gelu", "gelu_tanh"]),
                "train": rng.random() < 0.5}
    k = _spread(rng, 256, 8192, 8)
    m = _spread(rng, 1, 8192 * 7168 // k if k > 7168 else 8192)
    gate = rng.choice(["none", "channel", "token", "sequence"])
    if gate == "sequence":
        m = max(8, m // 8 * 8)
    kind = rng.choice(["bf16", "fp16"])
    after = rng.random() < 0.7
    return {"op": op, "m": m, "k": k, "type": kind, "rtype": rng.choice([kind, "fp32"]), "gate": gate, "scale": rng.choice([1.0, 0.5, 0.22]),
            "after": after, "before": not after or rng.random() < 0.7, "train": rng.random() < 0.5}


# --------------------------------------------------------------------------- inputs


def _blocks(v, rows):
    """(R, K) -> (R / rows, rows, K / 128, 128), zero-padded to whole blocks."""
    r, k = v.shape
    v = torch.nn.functional.pad(v, (0, -k % 128, 0, -r % rows))
    return v.view(v.shape[0] // rows, rows, v.shape[1] // 128, 128)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    if case["op"] == "fp8":
        m, k, n = case["m"], case["k"], case["n"]
        # activations with channels of different size, as after a norm; weights as trained ones
        x = (normal(m, k) * torch.exp(0.7 * normal(k))).to(dt)
        w = _blocks(normal(n, k) * (k ** -0.5), 128)
        ws = w.abs().amax(dim=(1, 3)) / 448.0
        wq = (w / ws[:, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        wq = wq.view(w.shape[0] * 128, -1)[:n, :k].contiguous()
        return {"case": case, "x": x, "w": wq, "ws": ws.contiguous()}
    if case["op"] == "gated":
        t, h, i = case["t"], case["h"], case["i"]
        s = {"case": case, "x": normal(t, h).to(dt), "wg": (normal(i, h) * (h ** -0.5)).to(dt), "wu": (normal(i, h) * (h ** -0.5)).to(dt)}
        if case["train"]:
            s["dh"] = (normal(t, i) * (0.05 if dt == torch.float16 else 1e-3)).to(dt)
        return s
    m, k = case["m"], case["k"]
    s = {"case": case, "f": (normal(m, k) * 3.0).to(dt), "r": (normal(m, k) * torch.exp(0.5 * normal(k))).to(TYPES[case["rtype"]]),
         "ga": (1.0 + 0.1 * normal(k)).to(dt) if case["after"] else None, "gb": (1.0 + 0.1 * normal(k)).to(dt) if case["before"] else None}
    shape = {"none": None, "channel": (k,), "token": (m, 1), "sequence": (8, k)}[case["gate"]]
    s["gate"] = None if shape is None else (0.5 * normal(*shape)).to(dt)
    if case["train"]:
        s["dr_out"] = normal(m, k).to(TYPES[case["rtype"]])
        s["dy"] = normal(m, k).to(dt) if case["before"] else None
    return s


# --------------------------------------------------------------------------- plain forms


def _plain_fp8(x, w, ws):
    m, k = x.shape
    n = w.shape[0]
    xb = _blocks(x.float(), 1)
    s = xb.abs().amax(dim=3, keepdim=True)
    s = s / torch.full_like(s, 448.0)  # a tensor: division by a Python number multiplies by its rounded reciprocal
    q = (xb / torch.where(s > 0, s, torch.ones_like(s))).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    a = (q * s).view(m, -1)[:, :k]
    b = (_blocks(w.float(), 128) * ws[:, None, :, None]).view(ws.shape[0] * 128, -1)[:n, :k]
    return (a @ b.T).to(x.dtype)


def _act(g, kind):
    """act(g) and its derivative."""
    if kind == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    if kind == "gelu":
        c = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * c, c + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    b = math.sqrt(2.0 / math.pi)
    t = torch.tanh(b * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * b * (1.0 + 3.0 * 0.044715 * g * g)


def _plain_gated(s):
    dt, kind = s["x"].dtype, s["case"]["act"]
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    g, u = x @ wg.T, x @ wu.T
    a, da = _act(g, kind)
    out = {"h": (a * u).to(dt)}
    if s["case"]["train"]:
        dh = s["dh"].float()
        dg, du = dh * u * da, dh * a
        out |= {"dx": (dg @ wg + du @ wu).to(dt), "dwg": (dg.T @ x).to(dt), "dwu": (du.T @ x).to(dt)}
    return out


def _gate_rows(gate, m):
    """The gate as a factor that broadcasts against (m, K)."""
    if gate is None:
        return 1.0
    if gate.dim() == 1 or gate.shape[0] == m:
        return gate
    return gate.repeat_interleave(m // gate.shape[0], dim=0)


def _plain_norm(s):
    c, dt, rt = s["case"], s["f"].dtype, s["r"].dtype
    m = c["m"]
    f, r = s["f"].float(), s["r"].float()
    ga = None if s["ga"] is None else s["ga"].float()
    gb = None if s["gb"] is None else s["gb"].float()
    gate = _gate_rows(None if s["gate"] is None else s["gate"].float(), m)
    if ga is not None:
        ia = 1.0 / torch.sqrt((f * f).mean(dim=1, keepdim=True) + EPS)
        fh = f * ia
        n = fh * ga
    else:
        n = f
    ro = r + c["scale"] * gate * n
    out = {"r_out": ro.to(rt)}
    if gb is not None:
        ib = 1.0 / torch.sqrt((ro * ro).mean(dim=1, keepdim=True) + EPS)
        rh = ro * ib
        out["y"] = (rh * gb).to(dt)
    if not c["train"]:
        return out
    dro = s["dr_out"].float()
    if gb is not None:
        dy = s["dy"].float()
        v = dy * gb
        dro = dro + ib * (v - rh * (v * rh).mean(dim=1, keepdim=True))
        out["dgb"] = (dy * rh).sum(dim=0)
    out["dr"] = dro.to(rt)
    dn = c["scale"] * gate * dro
    if s["gate"] is not None:
        p = c["scale"] * dro * n
        if c["gate"] == "channel":
            out["dgate"] = p.sum(dim=0)
        elif c["gate"] == "token":
            out["dgate"] = p.sum(dim=1, keepdim=True)
        else:
            out["dgate"] = p.view(8, m // 8, -1).sum(dim=1)
    if ga is not None:
        out["dga"] = (dn * fh).sum(dim=0)
        v = dn * ga
        out["df"] = (ia * (v - fh * (v * fh).mean(dim=1, keepdim=True))).to(dt)
    else:
        out["df"] = dn.to(dt)
    return out


# --------------------------------------------------------------------------- one pass


def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "fp8":
            return {"y": _plain_fp8(s["x"], s["w"], s["ws"])}
        return _plain_gated(s) if c["op"] == "gated" else _plain_norm(s)
    from nvfp4_block_scaled_quant_gb300 import ops

    if c["op"] == "fp8":
        return {"y": ops.fp8_linear(s["x"], s["w"], s["ws"])}
    if c["op"] == "gated":
        if not c["train"]:
            return {"h": ops.gated_linear(s["x"], s["wg"], s["wu"], activation=c["act"])}
        h, gu = ops.gated_linear(s["x"], s["wg"], s["wu"], activation=c["act"], save=True)
        dx, dwg, dwu = ops.gated_linear_backward(s["dh"], s["x"], s["wg"], s["wu"], gu, activation=c["act"])
        return {"h": h, "dx": dx, "dwg": dwg, "dwu": dwu}
    kw = {"gamma_after": s["ga"], "gate": s["gate"], "scale": c["scale"], "gamma_before": s["gb"], "eps": EPS}
    if not c["train"]:
        r_out, y = ops.residual_norm(s["f"], s["r"], **kw)
        return {"r_out": r_out} if y is None else {"r_out": r_out, "y": y}
    r_out, y, stats = ops.residual_norm(s["f"], s["r"], save=True, **kw)
    df, dr, dga, dgate, dgb = ops.residual_norm_backward(s["dr_out"], s["dy"], s["f"], s["r"], stats, **kw)
    out = {"r_out": r_out, "y": y, "df": df, "dr": dr, "dga": dga, "dgate": dgate, "dgb": dgb}
    return {k: v for k, v in out.items() if v is not None}


def work(case):
    if case["op"] == "fp8":
        m, k, n = case["m"], case["k"], case["n"]
        scales = -(-n // 128) * -(-k // 128) * 4
        return {"bytes": 2 * m * k + n * k + scales + 2 * m * n, "flops": 2 * m * n * k}
    if case["op"] == "gated":
        t, h, i = case["t"], case["h"], case["i"]
        if not case["train"]:
            return {"bytes": 2 * (t * h + 2 * i * h + t * i), "flops": 4 * t * h * i}
        # x, both weights and dh in; h, dx and both weight gradients out
        return {"bytes": 2 * (2 * t * h + 4 * i * h + 2 * t * i), "flops": 12 * t * h * i}
    m, k = case["m"], case["k"]
    a, b = 2, 4 if case["rtype"] == "fp32" else 2
    y = a if case["before"] else 0
    params = {"none": 0, "channel": k, "token": m, "sequence": 8 * k}[case["gate"]] + k * (case["after"] + case["before"])
    bytes_ = m * k * (a + 2 * b + y) + a * params
    if case["train"]:  # dr_out and dy in; df, dr and the parameters' gradients out (f and r are the same inputs)
        bytes_ += m * k * (b + y + a + b) + 4 * params
    return {"bytes": bytes_, "flops": m * k * (40 if case["train"] else 12)}


# --------------------------------------------------------------------------- the definition in 64 bits


def _e4m3(v):
    """Round float64 values to e4m3, ties to even, saturating at 448."""
    a = v.abs().clamp(max=448.0)
    e = torch.frexp(a).exponent.to(torch.float64) - 1.0
    q = torch.exp2(e.clamp(min=-6.0) - 3.0)
    return torch.sign(v) * (torch.round(a / q) * q)


def _exact_fp8(s):
    x, w, ws = s["x"].double(), s["w"].to(torch.float32).double(), s["ws"].double()
    m, k = x.shape
    n = w.shape[0]
    y = torch.zeros(m, n, dtype=torch.float64, device=x.device)
    for b in range(0, k, 128):
        xb = x[:, b:b + 128]
        # the scale and the quotient are 32-bit values by the operator's definition
        sc = (xb.abs().amax(dim=1, keepdim=True) / 448.0).float().double()
        q = _e4m3((xb / torch.where(sc > 0, sc, 1.0)).float().double())
        rows = ws[:, b // 128].repeat_interleave(128)[:n]
        y += (q @ w[:, b:b + 128].T) * sc * rows
    return {"y": y}


def _exact_gated(s):
    x, wg, wu = s["x"].double(), s["wg"].double(), s["wu"].double()
    g, u = x @ wg.T, x @ wu.T
    kind = s["case"]["act"]
    if kind == "silu":
        sig = torch.sigmoid(g)
        a, da = g * sig, sig + g * sig * torch.sigmoid(-g)
    elif kind == "gelu":
        phi = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        a, da = g * phi, phi + g * torch.exp(-g * g / 2.0) / math.sqrt(2.0 * math.pi)
    else:
        z = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
        dz = math.sqrt(2.0 / math.pi) * (1.0 + 0.134145 * g ** 2)
        p = torch.sigmoid(2.0 * z)  # (1 + tanh z) / 2
        a, da = g * p, p + 2.0 * g * p * torch.sigmoid(-2.0 * z) * dz
    out = {"h": a * u}
    if s["case"]["train"]:
        dh = s["dh"].double()
        dg, du = dh * u * da, dh * a
        out["dx"] = dg @ wg + du @ wu
        out["dwg"], out["dwu"] = dg.T @ x, du.T @ x
    return out


def _exact_norm(s):
    c = s["case"]
    m, k = c["m"], c["k"]
    f, r = s["f"].double(), s["r"].double()
    gate = torch.ones(m, k, dtype=torch.float64, device=f.device)
    if s["gate"] is not None:
        gd = s["gate"].double()
        groups = 1 if c["gate"] == "channel" else gd.shape[0]
        gate = gd.reshape(groups, 1, -1).expand(groups, m // groups, k).reshape(m, k)
    ia = (f.square().mean(1, keepdim=True) + EPS).rsqrt()
    n = f * ia * s["ga"].double() if s["ga"] is not None else f
    ro = torch.addcmul(r, gate, n, value=c["scale"])
    out = {"r_out": ro}
    ib = (ro.square().mean(1, keepdim=True) + EPS).rsqrt()
    if s["gb"] is not None:
        out["y"] = ro * ib * s["gb"].double()
    if not c["train"]:
        return out
    total = s["dr_out"].double()
    if s["gb"] is not None:
        dy = s["dy"].double()
        out["dgb"] = torch.einsum("mk,mk,m->k", dy, ro, ib[:, 0])
        t = dy * s["gb"].double()
        total = total + ib * t - ro * ib ** 3 * ((t * ro).sum(1, keepdim=True) / k)
    out["dr"] = total
    dn = c["scale"] * total * gate
    if s["gate"] is not None:
        p = c["scale"] * total * n
        out["dgate"] = {"channel": lambda: p.sum(0), "token": lambda: p.sum(1, keepdim=True),
                        "sequence": lambda: p.reshape(8, -1, k).sum(1)}[c["gate"]]()
    if s["ga"] is not None:
        out["dga"] = torch.einsum("mk,mk,m->k", dn, f, ia[:, 0])
        t = dn * s["ga"].double()
        out["df"] = ia * t - f * ia ** 3 * ((t * f).sum(1, keepdim=True) / k)
    else:
        out["df"] = dn
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"fp8": _exact_fp8, "gated": _exact_gated, "norm": _exact_norm}[case["op"]](s)
