"""The mixture-of-experts layer for a few tokens on 4-bit weights, against its definition in 64 bits."""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import ops
from w4_reference import F64, TYPES, check, checkpoint, moe

pytestmark = pytest.mark.gpu


class Layer:
    def __init__(self, T, H, I, E, topk, shared, group=128, zeros=False, kind="bf16", act="silu", seed=0):
        g = torch.Generator(device="cuda").manual_seed(77 * seed + T + H + I + E)
        dt = TYPES[kind]
        self.topk, self.group, self.act, self.dt = topk, group, act, dt
        self.x = torch.randn(T, H, generator=g, device="cuda").to(dt)
        self.router = (torch.randn(E, H, generator=g, device="cuda") * H ** -0.5).to(dt)
        self.w13 = checkpoint(g, (E, 2 * I, H), group, zeros, dt, "cuda")
        self.w2 = checkpoint(g, (E, H, I), group, zeros, dt, "cuda")
        self.s13 = checkpoint(g, (2 * I, H), group, zeros, dt, "cuda") if shared else None
        self.s2 = checkpoint(g, (H, I), group, zeros, dt, "cuda") if shared else None
        self.p13, self.p2 = ops.w4_prepare(*self.w13, group=group, gated=True), ops.w4_prepare(*self.w2, group=group)
        self.q13 = ops.w4_prepare(*self.s13, group=group, gated=True) if shared else None
        self.q2 = ops.w4_prepare(*self.s2, group=group) if shared else None

    def run(self, x=None, **kw):
        return ops.w4_moe(self.x if x is None else x, self.router, self.p13, self.p2, self.topk, shared13=self.q13, shared2=self.q2,
                          activation=self.act, **kw)

    def want(self, x=None):
        return moe((self.x if x is None else x).to(F64), self.router, self.w13, self.w2, self.topk, self.group, self.act, self.dt,
                   None if self.s13 is None else (self.s13, self.s2))

    def verify(self, y, x=None):
        want, err, ids, sure = self.want(x)
        check(y, want, err, self.dt, "" if sure else "the choice of experts may hang on the sums' order")
        return ids


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, False), (128, True)])
@pytest.mark.parametrize("T,H,I,E,topk,shared,act", [(1, 256, 128, 8, 2, True, "silu"), (3, 264, 40, 24, 4, False, "gelu"),
                                                     (13, 520, 200, 10, 3, True, "gelu_tanh"), (33, 136, 264, 6, 2, True, "silu")])
def test_sizes(T, H, I, E, topk, shared, act, group, zeros, kind):
    layer = Layer(T, H, I, E, topk, shared, group, zeros, kind, act)
    layer.verify(layer.run())


@pytest.mark.parametrize("T,H,I,E,topk,shared", [(1, 8, 8, 1, 1, False), (2, 16, 8, 2, 2, True), (64, 64, 32, 8, 8, True), (5, 72, 1000, 3, 1, False),
                                                 (32, 128, 64, 300, 16, False), (64, 256, 64, 1024, 8, True), (7, 2056, 24, 129, 5, True),
                                                 (1, 7168, 512, 64, 8, True), (16, 1024, 2048, 40, 6, False), (50, 64, 32, 385, 10, True)])
def test_small_large_and_odd(T, H, I, E, topk, shared):
    layer = Layer(T, H, I, E, topk, shared, seed=1)
    layer.verify(layer.run())


@pytest.mark.parametrize("T", [9, 24, 64])
def test_all_tokens_on_the_same_experts(T):
    layer = Layer(T, 128, 96, 16, 3, True, 32, True, seed=2)
    layer.x[:] = layer.x[:1] * torch.linspace(0.5, 1.5, T, device="cuda")[:, None].to(layer.dt)
    layer.router[:] = layer.router * 0.1
    for e, v in [(3, 1.0), (7, 2.0), (12, 3.0)]:
        layer.router[e] = (layer.x[0].float() * v * 0.05).to(layer.dt)
    ids = layer.verify(layer.run())
    assert sorted(set(ids.flatten().tolist())) == [3, 7, 12]


def test_ties_go_to_the_lowest_expert():
    layer = Layer(4, 64, 32, 40, 2, False, seed=3)
    layer.router[5] = layer.router[33]
    layer.router[9] = layer.router[33]
    layer.x[:] = (layer.router[33].float() * 20).to(layer.dt)
    want, err, ids, _ = layer.want()
    assert (ids == torch.tensor([5, 9], device="cuda")).all()
    check(layer.run(), want, err, layer.dt)


def test_repeats_strides_out_and_workspace():
    layer = Layer(11, 392, 136, 20, 4, True, 64, seed=4)
    y = layer.run()
    layer.verify(y)
    ws = ops.w4_moe_workspace(11, 392, 136, 20, 4, True, "cuda")
    out = torch.empty_like(y)
    wide = torch.full((11, 512), float("nan"), device="cuda", dtype=layer.dt)
    wide[:, 24:416] = layer.x
    for k in range(5):
        ws.fill_(0xFF if k % 2 else 0x11)  # the workspace needs no initialisation
        out.zero_()
        assert layer.run(wide[:, 24:416], out=out, workspace=ws) is out
        assert torch.equal(out, y)


def test_tokens_do_not_mix():
    layer = Layer(12, 128, 64, 8, 2, True, seed=5)
    y = layer.run()
    bad = layer.x.clone()
    bad[7, 3] = float("nan")
    z = layer.run(bad)
    keep = torch.arange(12, device="cuda") != 7
    assert torch.equal(z[keep], y[keep])
    assert torch.isnan(z[7]).all()


def test_no_tokens():
    layer = Layer(1, 64, 32, 4, 2, False, seed=6)
    assert layer.run(layer.x[:0]).shape == (0, 64)


def test_stream_and_graph():
    layer = Layer(6, 256, 96, 16, 4, True, seed=7)
    want = layer.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = layer.run(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    static = layer.x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.run(static)
        z = layer.run(static)
    for k in range(4):
        static.copy_(torch.roll(layer.x, k, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, torch.roll(want, k, 0)) and torch.equal(z, y)


def test_two_streams_at_once():
    """Layers that run beside one another, each larger than half of the GPU."""
    layers = [Layer(8, 1024, 512, 32, 4, True, seed=8 + k) for k in range(2)]
    wants = [layer.run() for layer in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k in range(2):
            got[k].append(layers[k].run(stream=streams[k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(v, wants[k]) for v in got[k])
    assert ops.device_error() == (0, 0)
