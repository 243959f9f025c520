"""Checkpoint weights of 4 bits with group scales, made from a seed, and what the operators on them compute, in 64
bits with bounds of the kernels' errors, both from the definitions alone."""

import math

import torch

F64 = torch.float64
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(dt):
    """A rounding to dt is off by at most this, relative to the value."""
    return torch.finfo(dt).eps / 2


def checkpoint(gen, shape, group, zeros, dt, device):
    """Random codes (..., N, K / 2), scales and zero points (or None) of matrices of the given shape (..., N, K)."""
    *lead, K = shape
    codes = torch.randint(0, 256, (*lead, K // 2), generator=gen, device=device, dtype=torch.uint8)
    groups = (*lead, -(-K // group))
    scales = (torch.rand(groups, generator=gen, device=device) * 0.9 + 0.1) * K ** -0.5 / 4
    z = torch.randint(0, 16, groups, generator=gen, device=device, dtype=torch.uint8) if zeros else None
    return codes, scales.to(dt), z


def weight(ck, group):
    """(W, B) of one checkpoint matrix: the real numbers it stands for, and s (c + z), the size of the terms that
    the kernels add up for an element."""
    codes, scales, zeros = ck
    N, half = codes.shape
    c = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(N, 2 * half).to(F64)
    s = scales.to(F64).repeat_interleave(group, dim=1)[:, :2 * half]
    z = torch.full_like(c, 8.0) if zeros is None else zeros.to(F64).repeat_interleave(group, dim=1)[:, :2 * half]
    return (c - z) * s, (c + z) * s


def product(x, ck, group):
    """(y, e) of x W^T: the product and a bound of the fp32 sums' error.  An element passes at most 8 MMAs of
    its group's sum, the difference and the product with the scale, one addition per group, and 16 over warps and
    CTAs; each is off by at most 2^-23 (the MMA may cut instead of rounding) of the sum of the terms' sizes.
    Activations lose what is below 2^-36 of their row's largest."""
    w, b = weight(ck, group)
    steps = 8 + 2 + -(-x.shape[1] // group) + 16
    size = x.abs() + 2.0 ** -13 * x.abs().amax(dim=1, keepdim=True) / steps if x.shape[0] else x
    return x @ w.T, steps * 2.0 ** -23 * (size @ b.T)


def act(kind, g):
    if kind == "silu":
        return g * torch.sigmoid(g)
    if kind == "gelu":
        return g * 0.5 * torch.erfc(-g / math.sqrt(2.0))
    return g * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))


def expert(x, w13, w2, group, kind, dt):
    """(y, e) of one expert.  |act'| < 1.13 for the three activations; the fast logistic function's error stays below 2^-19 of
    h; h is rounded to dt once."""
    gu, e = product(x, w13, group)
    I = gu.shape[1] // 2
    g, u, eg, eu = gu[:, :I], gu[:, I:], e[:, :I], e[:, I:]
    h = act(kind, g) * u
    eh = 1.13 * eg * (u.abs() + eu) + act(kind, g).abs() * eu + 2.0 ** -19 * h.abs()
    # a value under the type's normal range rounds by half of its smallest step
    eh = eh + half_step(dt) * (h.abs() + eh) + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
    y, e2 = product(h, w2, group)
    w, _ = weight(w2, group)
    return y, eh @ w.abs().T + e2


def moe(x, router, w13, w2, topk, group, kind, dt, shared=None):
    """(y, e, ids, sure): the layer, a bound of its error, the chosen experts, and whether the choice is beyond the worst error
    of fp32 logits: every token's last chosen and first left-out expert are further apart than twice the bound of H / 16
    MMAs and 16 additions, each off by at most 2^-23 of the sum of the terms' sizes."""
    logits = x @ router.to(F64).T
    error = (x.shape[1] / 16 + 16) * 2.0 ** -23 * (x.abs() @ router.to(F64).abs().T)
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids = order.indices[:, :topk]
    p = torch.softmax(order.values[:, :topk], dim=1)
    sure = router.shape[0] == topk or bool((order.values[:, topk - 1] - order.values[:, topk] > 2 * error.amax(dim=1)).all())
    y, e = torch.zeros_like(x), torch.zeros_like(x)
    if shared is not None:
        y, e = expert(x, *shared, group, kind, dt)
    for j in torch.unique(ids).tolist():
        t, at = torch.nonzero(ids == j, as_tuple=True)
        yj, ej = expert(x[t], tuple(None if v is None else v[j] for v in w13), tuple(None if v is None else v[j] for v in w2), group, kind, dt)
        pj = p[t, at, None]
        # the weights: logits off by 2^-23 of their terms each of up to 2^14, exp and division by a few steps
        ep = 2.0 ** -12 * pj * 2.0 ** -4
        y[t] += pj * yj
        e[t] += pj * ej + ep * (yj.abs() + ej)
    return y, e + (topk + 1) * 2.0 ** -24 * (y.abs() + e), ids, sure


def check(got, want, err, dt, what=""):
    """got (dt) is within err and one rounding of want."""
    bound = err + half_step(dt) * (want.abs() + err) + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
    off = (got.to(F64) - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = tuple(int(v) for v in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; at {i} got {float(got[i])!r}, want "
                             f"{float(want[i])!r} within {float(bound[i])!r}")
