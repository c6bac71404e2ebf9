"""The microscaled experts and the balance loss together, as a layer in training and in serving uses them: route, balance
loss, grouping, gate/up products, SwiGLU, down products, combine, and back to the tokens; captured and replayed in a
graph, on a stream of its own, and from two graphs that take turns."""
import numpy as np
import pytest

import mx4_ref
from gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu


class Layer:
    """A small routed layer with one shared expert, its weights quantised by the framework."""

    def __init__(self, seed, E=12, H=256, I=96, k=3):
        torch = torch_cuda()
        import bit_quantized_moe_topk_amd as moe
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.E, self.H, self.I, self.k = E, H, I, k
        self.router = (torch.randn((E, H), generator=g, device="cuda") / H ** 0.5).bfloat16()
        self.up = moe.mx4_quantize(torch.randn((E + 1, 2 * I, H), generator=g, device="cuda") / H ** 0.5)
        self.down = moe.mx4_quantize(torch.randn((E + 1, H, I), generator=g, device="cuda") / I ** 0.5)
        self.d = torch.tensor([0.01, 0.001], device="cuda")

    def step(self, x, dy):
        """Forward and backward of the layer for x [T, H] float32: everything a training step returns."""
        torch = torch_cuda()
        import bit_quantized_moe_topk_amd as moe
        T, k, I = x.shape[0], self.k, self.I
        logits = moe.router_logits(x, self.router)
        idx, gates = moe.route_topk(logits, k)
        bl = moe.balance_loss(logits, idx)
        dlogits = moe.balance_loss_backward(logits, bl, self.d)
        grp = moe.group(idx, self.E, True)
        gu = moe.mx4_experts_matmul(x, self.up, grp, tokens=T)
        sig = torch.sigmoid(gu[:, :I])
        h = gu[:, :I] * sig * gu[:, I:]
        o = moe.mx4_experts_matmul(h, self.down, grp)
        of = grp.slot_of.long()
        routed = o[of[:T * k]].view(T, k, self.H)
        y = (routed * gates.unsqueeze(2)).sum(1) + o[of[T * k:]]
        # back: each assignment's share of dy, through down, SwiGLU and gate/up to the tokens
        weight = torch.cat([gates.flatten(), torch.ones(T, device=x.device)])
        ids = grp.perm.long()
        do = dy[torch.where(ids < T * k, ids // k, ids - T * k)] * weight[ids].unsqueeze(1)
        dh = moe.mx4_experts_matmul_backward(do, self.down, grp)
        dg = dh * gu[:, I:] * sig * (1 + gu[:, :I] * (1 - sig))
        du = dh * gu[:, :I] * sig
        dx = moe.mx4_experts_matmul_backward(torch.cat([dg, du], 1), self.up, grp, tokens=T)
        return y, dx, dlogits, bl.losses, bl.counts, idx, gates

    def reference(self, x, dy, idx, gates):
        """The same in float64, by expert and token."""
        q = lambda m: mx4_ref.values(m.codes.cpu().numpy(), m.scales.cpu().numpy(), m.K)  # noqa: E731
        up, down, I = q(self.up), q(self.down), self.I
        y, dx = np.zeros_like(x), np.zeros_like(x)
        for t in range(x.shape[0]):
            for e, w in list(zip(idx[t], gates[t])) + [(self.E, 1.0)]:
                g, u = up[e][:I] @ x[t], up[e][I:] @ x[t]
                s = 1 / (1 + np.exp(-g))
                y[t] += w * (down[e] @ (g * s * u))
                dh = down[e].T @ (w * dy[t])
                dx[t] += up[e][:I].T @ (dh * u * s * (1 + g * (1 - s))) + up[e][I:].T @ (dh * g * s)
        return y, dx


def inputs(seed, T, H):
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((T, H), generator=g, device="cuda"), torch.randn((T, H), generator=g, device="cuda")


@pytest.mark.parametrize("T", [1, 5, 64, 200])
def test_layer_step(T):
    """Two products in a row in float32: each is within (3 n + 2) 2^-24 of a sum of magnitudes that here is at most 30
    times the result's norm, so rows agree to a relative 1e-4 with room for SwiGLU's own float32."""
    lay = Layer(T)
    x, dy = inputs(T, T, lay.H)
    y, dx, dlogits, losses, counts, idx, gates = lay.step(x, dy)
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    ry, rdx = lay.reference(n(x), n(dy), idx.cpu().numpy(), n(gates))
    for name, got, ref in (("y", y, ry), ("dx", dx, rdx)):
        err = np.linalg.norm(n(got) - ref, axis=1) / np.linalg.norm(ref, axis=1)
        log(f"[mx4 layer] T={T} {name}: {err.max():.2e}")
        assert err.max() <= 1e-4
    assert np.array_equal(counts.cpu().numpy(), np.bincount(idx.cpu().numpy().ravel(), minlength=lay.E))


def test_layer_in_a_graph_replayed():
    """One graph over the step, replayed with new inputs between eager work on the same tensors' values."""
    torch = torch_cuda()
    lay = Layer(7)
    x, dy = inputs(1, 70, lay.H)
    lay.step(x, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        out = lay.step(x, dy)
    torch.cuda.current_stream().wait_stream(side)
    for rep in range(4):
        a, b = inputs(50 + rep, 70, lay.H)
        x.copy_(a)
        dy.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for i, (got, want) in enumerate(zip(out, lay.step(a, b))):
            assert torch.equal(got, want), (rep, i)
        torch.cuda.synchronize()


def test_two_graphs_and_a_stream_of_its_own():
    """Two layers' graphs replayed on two streams at once, beside an eager step on a third, give what each gives alone."""
    torch = torch_cuda()
    lays = [Layer(20 + i) for i in range(3)]
    data = [inputs(30 + i, 64, l.H) for i, l in enumerate(lays)]
    alone = [[t.clone() for t in l.step(*d)] for l, d in zip(lays, data)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in lays]
    graphs, outs = [], []
    for l, d, s in list(zip(lays, data, streams))[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            outs.append(l.step(*d))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = lays[2].step(*data[2])
        torch.cuda.synchronize()
        for got, want in zip([*outs, eager], alone):
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graphs_of_many_rows_take_turns_with_one_workspace():
    """More tiles than CUs: two graphs and an eager call use one workspace, one after the other, whatever it holds."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    gen = torch.Generator(device="cuda").manual_seed(8)
    T, k, E, N, K = 1200, 3, 200, 640, 512
    w = moe.mx4_quantize(torch.randn((E + 1, N, K), generator=gen, device="cuda"))
    idx, _ = moe.route_topk(torch.randn((T, E), generator=gen, device="cuda"), k)
    grp = moe.group(idx, E, True)
    A = T * (k + 1)
    room = torch.empty(moe.lib().moe_mx4_experts_matmul_backward_workspace_size(T, k, 1, K, 1), dtype=torch.uint8, device="cuda")

    def step(x, dy):
        y = moe.mx4_experts_matmul(x, w, grp, tokens=T, workspace=room)
        y4 = moe.mx4_experts_matmul(moe.mx4_quantize(x), w, grp, tokens=T, workspace=room)
        return y, y4, moe.mx4_experts_matmul_backward(dy, w, grp, tokens=T, workspace=room)

    data = [(torch.randn((T, K), generator=gen, device="cuda").bfloat16(),
             torch.randn((A, N), generator=gen, device="cuda").bfloat16()) for _ in range(3)]
    alone = [[t.clone() for t in step(*d)] for d in data]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for d in data[:2]:
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            outs.append(step(*d))
        graphs.append(g)
    for rep in range(3):
        for g, out, want in zip(graphs, outs, alone):
            room.random_(0, 256)
            for t in out:
                t.zero_()
            g.replay()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), rep
        assert all(torch.equal(a, b) for a, b in zip(step(*data[2]), alone[2]))
        torch.cuda.synchronize()


def test_four_bit_rows_of_a_decode_window():
    """Quantised activations through the grouped product: the same rows as values through it give the same sums."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    lay = Layer(9)
    x, _ = inputs(3, 4, lay.H)
    idx, _ = moe.route_topk(moe.router_logits(x, lay.router), lay.k)
    grp = moe.group(idx, lay.E, True)
    q = moe.mx4_quantize(x)
    y4 = moe.mx4_experts_matmul(q, lay.up, grp, tokens=4, dtype=torch.float32)
    yb = moe.mx4_experts_matmul(moe.mx4_dequantize(q, torch.bfloat16), lay.up, grp, tokens=4, dtype=torch.float32)
    size = moe.mx4_experts_matmul(moe.mx4_dequantize(q).abs(), moe.Mx4(lay.up.codes & 0x77, lay.up.scales, lay.H), grp, tokens=4)
    # two float32 sums of the same exact terms
    assert ((y4 - yb).abs() <= 2 * (lay.H + 2) * 2.0 ** -24 * size * 1.01).all()
