"""Residual norm and its gradients on the GPU against their formulas in 64 bits.

Bounds: half a step of the output type, plus 64 fp32 half steps (2^-24) of the sum of the absolute
values of the terms that make an element: a row's statistics and sums are chains of at most 16 terms
per thread and 10 shuffle steps, each element passes through fewer than 20 products and sums.
Column sums over M rows add M / 8 steps of the sum of absolute terms.
"""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5


def case(M, K, dtype, rtype, gate, seed, after=True, before=True, groups=1):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g, device=DEV)

    shape = {"none": None, "channel": (K,), "groups": (groups, K), "row": (M, 1)}[gate]
    return dict(f=(3 * normal(M, K)).to(dtype), r=normal(M, K).to(rtype),
                gamma_after=(1 + 0.2 * normal(K)).to(dtype) if after else None,
                gate=None if shape is None else normal(*shape).to(dtype), scale=0.37,
                gamma_before=(1 + 0.2 * normal(K)).to(dtype) if before else None), normal(M, K).to(rtype), (
                    normal(M, K).to(dtype) if before else None)


def reference(c, dr_out, dy):
    """{name: (value, sum of absolute terms, additions beyond a row)} in float64."""
    f, r, sc = c["f"].double(), c["r"].double(), c["scale"]
    M, K = f.shape
    gate = c["gate"]
    if gate is None:
        gk = torch.ones(M, K, dtype=torch.float64, device=DEV)
    elif gate.dim() == 2 and gate.shape == (M, 1):
        gk = gate.double().expand(M, K)
    else:
        gg = gate.double().reshape(-1, K)
        gk = gg.repeat_interleave(M // gg.shape[0], 0)
    fh, ia = f, torch.ones(M, 1, dtype=torch.float64, device=DEV)
    if c["gamma_after"] is not None:
        ia = 1 / (f.square().mean(1, keepdim=True) + EPS).sqrt()
        fh = f * ia
        n = fh * c["gamma_after"].double()
    else:
        n = f
    ro, mag = r + sc * gk * n, r.abs() + (sc * gk * n).abs()
    out = {"r_out": (ro, mag, 0)}
    d = torch.zeros_like(f) if dr_out is None else dr_out.double()
    dmag = d.abs()
    if c["gamma_before"] is not None:
        gb = c["gamma_before"].double()
        ib = 1 / (ro.square().mean(1, keepdim=True) + EPS).sqrt()
        rh, rm = ro * ib, mag * ib
        # rstd(r') carries the relative error of the row's squares, mean(|r'| mag) / mean(r'^2)
        rm = rm + rh.abs() * ((ro.abs() * mag).mean(1, keepdim=True) * ib * ib)
        out["y"] = (rh * gb, (rm * gb).abs(), 0)
        if dy is not None:
            v = dy.double() * gb
            d = d + ib * (v - rh * (v * rh).mean(1, keepdim=True))
            ibm = ib * (1 + (ro.abs() * mag).mean(1, keepdim=True) * ib * ib)
            dmag = dmag + ibm * (v.abs() + rm * (v.abs() * rm).mean(1, keepdim=True))
            out["dgamma_before"] = ((dy.double() * rh).sum(0), (dy.double().abs() * rm).sum(0), M)
        else:
            out["dgamma_before"] = (torch.zeros(K, dtype=torch.float64, device=DEV), torch.zeros(K, dtype=torch.float64, device=DEV), 0)
    out["dr"] = (d, dmag, 0)
    dn, dnm = sc * gk * d, (sc * gk).abs() * dmag
    if c["gamma_after"] is not None:
        ga = c["gamma_after"].double()
        out["dgamma_after"] = ((dn * fh).sum(0), (dnm * fh.abs()).sum(0), M)
        v, vm = dn * ga, dnm * ga.abs()
        out["df"] = (ia * (v - fh * (v * fh).mean(1, keepdim=True)), ia * (vm + fh.abs() * (vm * fh.abs()).mean(1, keepdim=True)), 0)
    else:
        out["df"] = (dn, dnm, 0)
    if gate is not None:
        p, pm = sc * d * n, abs(sc) * dmag * n.abs()
        if gate.dim() == 2 and gate.shape == (M, 1):
            out["dgate"] = (p.sum(1, keepdim=True), pm.sum(1, keepdim=True), 0)
        else:
            shape = (gate.reshape(-1, K).shape[0], -1, K)
            out["dgate"] = (p.reshape(shape).sum(1).reshape(gate.shape), pm.reshape(shape).sum(1).reshape(gate.shape), M)
    return out


def held(name, got, ref):
    want, mag, rows = ref
    u = torch.finfo(got.dtype).eps / 2
    bound = u * want.abs() + u * torch.finfo(got.dtype).smallest_normal + (64 + rows / 8) * 2.0 ** -24 * mag * (1 + u)
    off = (got.double() - want).abs()
    assert got.shape == want.shape and torch.isfinite(got).all(), name
    assert (off <= bound).all(), f"{name}: worst excess {(off - bound).max().item()}, {(off > bound).sum().item()} elements"


def check(c, dr_out, dy):
    r_out, y, stats = ops.residual_norm(eps=EPS, save=True, **c)
    plain = ops.residual_norm(eps=EPS, **c)
    assert torch.equal(plain[0], r_out) and (y is None or torch.equal(plain[1], y))
    df, dr, dga, dgate, dgb = ops.residual_norm_backward(dr_out, dy, c["f"], c["r"], stats, eps=EPS,
                                                         **{k: v for k, v in c.items() if k not in "fr"})
    ref = reference(c, dr_out, dy)
    got = {"r_out": r_out, "y": y, "df": df, "dr": dr, "dgamma_after": dga, "dgate": dgate, "dgamma_before": dgb}
    for name, t in got.items():
        assert (t is None) == (name not in ref), name
        if t is not None:
            held(name, t, ref[name])
    assert ops.device_error() == (0, 0)


@pytest.mark.parametrize("M,K", [(1, 8), (1, 7168), (3, 264), (5, 1544), (40, 512), (160, 7168), (700, 1024), (33, 8192), (9, 8200), (6, 16384)])
@pytest.mark.parametrize("gate", ["none", "channel", "row"])
@pytest.mark.parametrize("dtype,rtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                         (torch.float16, torch.float16), (torch.float16, torch.float32)])
def test_forward_and_gradients(M, K, gate, dtype, rtype):
    check(*case(M, K, dtype, rtype, gate, seed=M + K))


@pytest.mark.parametrize("M,groups", [(8, 2), (8, 8), (600, 3), (600, 600), (600, 150), (1200, 300), (456, 152)])
@pytest.mark.parametrize("K", [64, 2048])
def test_gates_of_groups_of_rows(M, groups, K):
    check(*case(M, K, torch.bfloat16, torch.float32, "groups", seed=M + groups, groups=groups))


@pytest.mark.parametrize("after,before", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("gate", ["none", "channel", "row"])
@pytest.mark.parametrize("M", [3, 400])
def test_either_norm_may_be_absent(after, before, gate, M):
    check(*case(M, 1024, torch.bfloat16, torch.bfloat16, gate, seed=M, after=after, before=before))


@pytest.mark.parametrize("which", ["dr_out", "dy"])
def test_either_gradient_may_be_absent(which):
    c, dr_out, dy = case(50, 512, torch.bfloat16, torch.float32, "channel", seed=9)
    check(c, None if which == "dr_out" else dr_out, None if which == "dy" else dy)


def test_gradient_against_differences():
    """The formulas of reference() are the derivative: central differences in 64 bits of
    sum(r_out a) + sum(y b) along random directions, with an error of O(d^2) of the third derivative."""
    c, dr_out, dy = case(6, 64, torch.float16, torch.float32, "groups", seed=4, groups=2)
    ref = reference(c, dr_out, dy)
    names = {"f": "df", "r": "dr", "gamma_after": "dgamma_after", "gate": "dgate", "gamma_before": "dgamma_before"}
    g = torch.Generator(device=DEV).manual_seed(2)
    for k, grad in names.items():
        v = torch.randn(c[k].shape, generator=g, device=DEV, dtype=torch.float64)

        def loss(s):
            o = reference({**c, k: c[k].double() + s * v}, dr_out, dy)
            return (o["r_out"][0] * dr_out.double()).sum() + (o["y"][0] * dy.double()).sum()

        diff = (loss(1e-4) - loss(-1e-4)) / 2e-4
        assert (diff - (ref[grad][0] * v).sum()).abs() <= 1e-6 * ((ref[grad][0] * v).abs().sum() + 1), k


def test_strides_in_place_and_rows_behind():
    c, dr_out, dy = case(37, 512, torch.bfloat16, torch.float32, "channel", seed=5)
    r_out, y, stats = ops.residual_norm(eps=EPS, save=True, **c)
    wide = {k: torch.zeros(37, 1024 + 8, dtype=t.dtype, device=DEV) for k, t in (("f", c["f"]), ("r", c["r"]), ("d", dr_out), ("y", dy))}
    views = {}
    for k, t in (("f", c["f"]), ("r", c["r"]), ("d", dr_out), ("y", dy)):
        views[k] = wide[k][:, 16:16 + 512]
        views[k].copy_(t)
    s = {**c, "f": views["f"], "r": views["r"]}
    r2, y2, st2 = ops.residual_norm(eps=EPS, save=True, **s)
    assert torch.equal(r_out, r2) and torch.equal(y, y2) and torch.equal(stats, st2)
    rest = {k: v for k, v in c.items() if k not in "fr"}
    a = ops.residual_norm_backward(dr_out, dy, c["f"], c["r"], stats, eps=EPS, **rest)
    b = ops.residual_norm_backward(views["d"], views["y"], views["f"], views["r"], stats, eps=EPS, **rest)
    for x, z in zip(a, b):
        assert torch.equal(x, z)
    buf = torch.full((38, 512), 3.0, device=DEV)
    buf[:37] = c["r"]
    r3, y3 = ops.residual_norm(eps=EPS, out=buf[:37], **{**c, "r": buf[:37]})
    assert torch.equal(r3, r_out) and torch.equal(y3, y) and (buf[37] == 3.0).all()


def test_zero_rows_of_f_and_r():
    """A row of zeros has rstd = 1 / sqrt(eps): finite outputs and gradients; eps = 0 gives the
    formula's own 0 * inf = NaN in that row only."""
    c, dr_out, dy = case(4, 256, torch.bfloat16, torch.float32, "channel", seed=6)
    c["f"][1] = 0
    c["r"][1] = 0
    check(c, dr_out, dy)
    r_out, y = ops.residual_norm(eps=0.0, **c)
    assert torch.isnan(r_out[1]).all() and torch.isfinite(r_out[[0, 2, 3]]).all() and torch.isfinite(y[[0, 2, 3]]).all()


def test_nan_stays_in_its_row():
    c, dr_out, dy = case(30, 256, torch.bfloat16, torch.bfloat16, "channel", seed=7)
    clean = ops.residual_norm(eps=EPS, **c)
    c["f"][4, 3] = float("nan")
    r_out, y = ops.residual_norm(eps=EPS, **c)
    keep = [i for i in range(30) if i != 4]
    assert torch.isnan(r_out[4]).all() and torch.isnan(y[4]).all()
    assert torch.equal(r_out[keep], clean[0][keep]) and torch.equal(y[keep], clean[1][keep])


def test_no_rows():
    c, dr_out, dy = case(0, 64, torch.bfloat16, torch.bfloat16, "channel", seed=1)
    r_out, y, stats = ops.residual_norm(eps=EPS, save=True, **c)
    assert r_out.shape == (0, 64) and y.shape == (0, 64)
    grads = ops.residual_norm_backward(dr_out, dy, c["f"], c["r"], stats, gamma_after=c["gamma_after"], gate=c["gate"],
                                       gamma_before=c["gamma_before"])
    assert all((g == 0).all() for g in grads[2:])


def test_capture_and_determinism():
    c, dr_out, dy = case(500, 1024, torch.bfloat16, torch.float32, "row", seed=8)
    rest = {k: v for k, v in c.items() if k not in "fr"}

    def step():
        r_out, y, stats = ops.residual_norm(eps=EPS, save=True, **c)
        return [r_out, y, *ops.residual_norm_backward(dr_out, dy, c["f"], c["r"], stats, eps=EPS, **rest)]

    first = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        for a, b in zip(got, first):
            assert torch.equal(a, b)


def test_refusals():
    c, dr_out, dy = case(6, 64, torch.bfloat16, torch.bfloat16, "channel", seed=1)
    _, _, stats = ops.residual_norm(save=True, **c)
    f, r = c["f"], c["r"]
    for call in [lambda: ops.residual_norm(f, r.half()), lambda: ops.residual_norm(f.float(), r.float()),
                 lambda: ops.residual_norm(f, r[:3]), lambda: ops.residual_norm(f, r, gamma_after=c["gamma_after"].float()),
                 lambda: ops.residual_norm(f, r, gate=torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)),
                 lambda: ops.residual_norm(f, r, gate=torch.zeros(6, dtype=torch.bfloat16, device=DEV)),
                 lambda: ops.residual_norm(f.cpu(), r), lambda: ops.residual_norm(f, r, out=torch.empty(6, 64, device=DEV)),
                 lambda: ops.residual_norm_backward(dr_out, dy, f, r, stats),  # dy without gamma_before
                 lambda: ops.residual_norm_backward(dr_out.float(), None, f, r, stats)]:
        with pytest.raises(ValueError):
            call()
    big = torch.zeros(2, 16392, dtype=torch.bfloat16, device=DEV)
    for call in [lambda: ops.residual_norm(big, big), lambda: ops.residual_norm(f[:, :60], r[:, :60]),
                 lambda: ops.residual_norm(f, r, scale=float("inf")), lambda: ops.residual_norm(f, r, eps=-1.0)]:
        with pytest.raises(RuntimeError, match="nvfp4 status"):
            call()
