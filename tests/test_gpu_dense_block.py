"""The dense feed-forward operators run together, as a layer uses them: residual norm -> gated linear ->
FP8 down projection -> residual norm, forward and backward, queued back to back, captured, on two
streams, and between NVFP4 calls.

Each call's result depends on its inputs alone, so a chain queued without waiting has to give the bits
of the same calls with a synchronisation after each: a kernel that starts before its input is
complete, or two that share scratch, would not.
"""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import model, ops, workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Block:
    def __init__(self, H, I, seed, dtype=torch.bfloat16):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def normal(*s):
            return torch.randn(*s, generator=g, device=DEV)

        self.wg, self.wu = ((normal(I, H) * H ** -0.5).to(dtype) for _ in range(2))
        self.down = ops.fp8_quantize_weight((normal(H, I) * I ** -0.5).to(dtype))
        self.ga, self.gb = ((1 + 0.1 * normal(H)).to(dtype) for _ in range(2))
        self.gate = normal(H).to(dtype)

    def __call__(self, f, r, wait=lambda: None):
        out = []
        r, y = ops.residual_norm(f, r, gamma_after=self.ga, gate=self.gate, scale=0.5, gamma_before=self.gb)
        wait()
        h = ops.gated_linear(y, self.wg, self.wu)
        wait()
        f = ops.fp8_linear(h, *self.down)
        wait()
        out += [r, y, h, f]
        r, y = ops.residual_norm(f, r, gamma_after=self.ga, gamma_before=self.gb)
        wait()
        return out + [r, y]

    def train(self, f, r, dr, dy, wait=lambda: None):
        r1, y, st = ops.residual_norm(f, r, gamma_after=self.ga, gate=self.gate, gamma_before=self.gb, save=True)
        wait()
        h, gu = ops.gated_linear(y, self.wg, self.wu, save=True)
        wait()
        dyi, dwg, dwu = ops.gated_linear_backward(dy, y, self.wg, self.wu, gu)
        wait()
        grads = ops.residual_norm_backward(dr, dyi, f, r, st, gamma_after=self.ga, gate=self.gate, gamma_before=self.gb)
        wait()
        return [r1, y, h, dyi, dwg, dwu, *grads]


def inputs(M, H, I, seed, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(M, n, generator=g, device=DEV).to(t) for n, t in ((H, dtype), (H, torch.float32), (H, torch.float32), (I, dtype))]


def same(a, b):
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("M", [1, 24, 70, 300, 1500])
@pytest.mark.parametrize("train", [False, True])
def test_queued_chain_gives_the_bits_of_single_calls(M, train):
    H, I = 1024, 768
    b = Block(H, I, seed=M)
    sets = [inputs(M, H, I, seed=10 * M + i) for i in range(4)]

    def run(s, **kw):
        return b.train(*s, **kw) if train else b(s[0], s[1], **kw)

    want = [run(s, wait=torch.cuda.synchronize) for s in sets]
    got = [run(sets[i % 4]) for i in range(40)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        same(g, want[i % 4])
    assert ops.device_error() == (0, 0)


@pytest.mark.parametrize("M", [1, 300])
def test_two_captured_chains_replayed_in_turn(M):
    H, I = 512, 384
    b = Block(H, I, seed=1)
    s1, s2 = inputs(M, H, I, 1), inputs(M, H, I, 2)
    w1, w2 = b(s1[0], s1[1]) + b.train(*s1), b(s2[0], s2[1]) + b.train(*s2)
    graphs = []
    for s in (s1, s2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = b(s[0], s[1]) + b.train(*s)
        graphs.append((g, out))
    for _ in range(5):
        for g, _ in graphs:
            g.replay()
        eager = b(s1[0], s1[1]) + b.train(*s1)  # an eager chain between replays
        torch.cuda.synchronize()
        same(graphs[0][1], w1)
        same(graphs[1][1], w2)
        same(eager, w1)


@pytest.mark.parametrize("M", [2, 40, 300])
def test_two_streams_at_once(M):
    H, I = 1024, 512
    b = Block(H, I, seed=3)
    s1, s2 = inputs(M, H, I, 5), inputs(M, H, I, 6)
    w1, w2 = b(s1[0], s1[1]) + b.train(*s1), b(s2[0], s2[1]) + b.train(*s2)
    a, c = torch.cuda.Stream(), torch.cuda.Stream()
    a.wait_stream(torch.cuda.current_stream())
    c.wait_stream(torch.cuda.current_stream())
    got = {a: [], c: []}
    for _ in range(10):
        for st, s in ((a, s1), (c, s2)):
            with torch.cuda.stream(st):
                got[st].append(b(s[0], s[1]) + b.train(*s))
    torch.cuda.synchronize()
    for st, want in ((a, w1), (c, w2)):
        for g in got[st]:
            same(g, want)


def test_between_nvfp4_calls():
    """The NVFP4 linear before and after the new operators on one stream keeps its bits, and theirs."""
    M, H, I = 40, 1536, 512
    b = Block(H, I, seed=4)
    s = inputs(M, H, I, 7)
    dw = model.make_dense_weight(H, H, seed=9, device=DEV)
    x = workloads.activations(M, H, seed=8, device=DEV)
    want_l = ops.linear(x, dw.w, dw.sf, dw.ws2, H)[0]
    want_b = b(s[0], s[1])
    for _ in range(5):
        l1 = ops.linear(x, dw.w, dw.sf, dw.ws2, H)[0]
        got = b(l1, s[1])
        l2 = ops.linear(x, dw.w, dw.sf, dw.ws2, H)[0]
        got2 = b(s[0], s[1])
        torch.cuda.synchronize()
        assert torch.equal(l1, want_l) and torch.equal(l2, want_l)
        same(got2, want_b)
        same(got, b(want_l, s[1]))


def test_gradients_of_the_chain_against_autograd():
    """norm -> gated, end to end, against torch's own differentiation in 64 bits.  At most five 16-bit
    roundings (y, h or its gradient's operands, dx, df) lie on a path, each within u = 2^-8 of its
    value, so the 2-norm of each error is within 5 u of the gradient's."""
    M, H, I = 96, 512, 384
    b = Block(H, I, seed=11)
    f, r, dr, dy = inputs(M, H, I, 12)
    got = dict(zip(("r", "y", "h", "dyi", "dwg", "dwu", "df", "dr", "dga", "dgate", "dgb"), b.train(f, r, dr, dy)))
    p = {k: v.double().requires_grad_() for k, v in dict(f=f, r=r, wg=b.wg, wu=b.wu, ga=b.ga, gate=b.gate, gb=b.gb).items()}

    def norm(v, g):
        return v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt() * g

    r1 = p["r"] + p["gate"] * norm(p["f"], p["ga"])
    y = norm(r1, p["gb"])
    h = torch.nn.functional.silu(y @ p["wg"].T) * (y @ p["wu"].T)
    ((r1 * dr.double()).sum() + (h * dy.double()).sum()).backward()
    for mine, theirs in (("df", "f"), ("dr", "r"), ("dwg", "wg"), ("dwu", "wu"), ("dga", "ga"), ("dgate", "gate"), ("dgb", "gb")):
        want = p[theirs].grad
        assert (got[mine].double() - want).norm() <= 5 * 2.0 ** -8 * want.norm(), mine
