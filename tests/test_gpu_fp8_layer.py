"""The norm, routing by scores and the 8-bit experts together, as a layer in training and in serving uses them: residual and norm,
router product, scores, grouping, gate/up products, SwiGLU, down products, combine, and the gradients back to x; captured and
replayed in a graph, on a stream of its own, and from two graphs that take turns."""
import numpy as np
import pytest

import blocks_ref as ref
from gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu


class Layer:
    """A small routed layer with one shared expert, its weights quantised by the framework."""

    def __init__(self, seed, E=16, H=256, I=128, k=3):
        torch = torch_cuda()
        import bit_quantized_moe_topk_amd as moe
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.E, self.H, self.I, self.k = E, H, I, k
        self.router = (torch.randn((E, H), generator=g, device="cuda") / H ** 0.5).bfloat16()
        self.bias = 0.05 * torch.randn(E, generator=g, device="cuda")
        self.norm = 1 + 0.1 * torch.randn(H, generator=g, device="cuda")
        self.up = moe.fp8_quantize(torch.randn((E + 1, 2 * I, H), generator=g, device="cuda") / H ** 0.5, 128)
        self.down = moe.fp8_quantize(torch.randn((E + 1, H, I), generator=g, device="cuda") / I ** 0.5, 128)
        self.how = dict(score="sigmoid", renormalize=True, scale=1.5)

    def step(self, x, residual, dy):
        """Forward and backward for x and residual [T, H]: everything that a training step returns."""
        torch = torch_cuda()
        import bit_quantized_moe_topk_amd as moe
        T, k, I, H = x.shape[0], self.k, self.I, self.H
        f32 = torch.float32
        n = moe.rms_norm(x, self.norm, residual, fp8=True)
        logits = moe.router_logits(n.y, self.router)
        idx, gates = moe.route_scores(logits, k, self.bias, groups=4, keep_groups=2, **self.how)
        grp = moe.group(idx, self.E, True)
        gu = moe.fp8_experts_matmul(n.fp8, self.up, grp, tokens=T, dtype=f32)
        sig = torch.sigmoid(gu[:, :I])
        h = moe.fp8_quantize(gu[:, :I] * sig * gu[:, I:])
        o = moe.fp8_experts_matmul(h, self.down, grp, dtype=f32)
        of = grp.slot_of.long()
        routed = o[of[:T * k]].view(T, k, H)
        y = n.total + (routed * gates.unsqueeze(2)).sum(1) + o[of[T * k:]]
        # back
        d_gates = (routed * dy.unsqueeze(1)).sum(2)
        dlogits = moe.route_scores_backward(logits, idx, d_gates, **self.how)
        weight = torch.cat([gates.flatten(), torch.ones(T, device=x.device)])
        ids = grp.perm.long()
        do = moe.fp8_quantize(dy[torch.where(ids < T * k, ids // k, ids - T * k)] * weight[ids].unsqueeze(1))
        dh = moe.fp8_experts_matmul_backward(do, self.down, grp, dtype=f32)
        dgu = torch.cat([dh * gu[:, I:] * sig * (1 + gu[:, :I] * (1 - sig)), dh * gu[:, :I] * sig], 1)
        dgu = moe.fp8_quantize(dgu)
        dn = moe.fp8_experts_matmul_backward(dgu, self.up, grp, tokens=T, dtype=f32) + dlogits @ self.router.float()
        dx, dw = moe.rms_norm_backward(dn, n.total, self.norm, dy)
        return dict(y=y, dx=dx, dw=dw, dlogits=dlogits, idx=idx, gates=gates, total=n.total, normed=n.y, codes=n.fp8.codes.view(torch.uint8),
                    scales=n.fp8.scales, logits=logits, gu=gu, h=h.codes.view(torch.uint8), hs=h.scales, do=do.codes.view(torch.uint8),
                    ds=do.scales, dgu=dgu.codes.view(torch.uint8), dgs=dgu.scales, dn=dn, d_gates=d_gates, perm=grp.perm, offsets=grp.offsets)


def inputs(seed, T, H):
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((T, H), generator=g, device="cuda") for _ in range(3)]


@pytest.mark.parametrize("T", [1, 5, 64, 300])
def test_layer_step(T):
    """Each 8-bit operand that the step made is taken as it is, so that every product and sum is held to float32: sums of up to
    a few hundred terms, at most 300 2^-24 of magnitudes that here are at most 30 times the result's norm: 1e-3 with all of them in
    one direction, of which rows stay far short."""
    lay = Layer(T)
    x, residual, dy = inputs(T, T, lay.H)
    s = {k: v.double().cpu().numpy() if v.is_floating_point() else v.cpu().numpy() for k, v in lay.step(x, residual, dy).items()}
    k, I, H, E = lay.k, lay.I, lay.H, lay.E
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    mats = lambda q: ref.values(q.codes.view(torch_cuda().uint8).cpu().numpy(), n(q.scales), q.K, 128)  # noqa: E731
    up, down = mats(lay.up), mats(lay.down)

    def near(name, want, bound=1e-3):
        err = np.linalg.norm(s[name] - want) / np.linalg.norm(want)
        log(f"[fp8 layer] T={T} {name}: {err:.2e}")
        assert err <= bound, name
    total = n(x) + n(residual)
    near("total", total, 1e-6)
    near("normed", ref.norm(total, n(lay.norm), 1e-6), 1e-5)
    near("logits", s["normed"] @ n(lay.router).T, 1e-5)
    idx, gates = ref.route(s["logits"], k, n(lay.bias), groups=4, keep_groups=2, **lay.how)
    assert np.array_equal(idx, s["idx"])
    near("gates", gates, 1e-6)
    assert np.array_equal(s["codes"], ref.quantize(s["normed"])[0])
    token = np.where(s["perm"] < T * k, s["perm"] // k, s["perm"] - T * k)
    expert = np.searchsorted(s["offsets"][1:], np.arange(len(token)), side="right")
    xv = ref.values(s["codes"], s["scales"], H)
    near("gu", np.stack([up[e] @ xv[t] for e, t in zip(expert, token)]), 1e-5)
    hv = ref.values(s["h"], s["hs"], I)
    o = np.stack([down[e] @ v for e, v in zip(expert, hv)])
    weight = np.concatenate([s["gates"].ravel(), np.ones(T)])[s["perm"]]
    y = total.copy()
    np.add.at(y, token, o * weight[:, None])
    near("y", y, 1e-5)
    near("dlogits", ref.route_gradient(s["logits"], s["idx"], s["d_gates"], **lay.how)[0], 1e-5)
    dgu = ref.values(s["dgu"], s["dgs"], 2 * I)
    dn = s["dlogits"] @ n(lay.router)
    np.add.at(dn, token, np.stack([v @ up[e] for e, v in zip(expert, dgu)]))
    near("dn", dn, 1e-5)
    dx, dw, _, _ = ref.norm_gradients(s["dn"], s["total"], n(lay.norm), n(dy), 1e-6)
    near("dx", dx, 1e-5)
    near("dw", dw, 1e-5)


def test_layer_in_a_graph_replayed():
    """One graph over the step, replayed with new inputs between eager work on the same tensors' values."""
    torch = torch_cuda()
    lay = Layer(7)
    data = inputs(1, 300, lay.H)
    lay.step(*data)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        out = lay.step(*data)
    torch.cuda.current_stream().wait_stream(side)
    for rep in range(4):
        new = inputs(50 + rep, 300, lay.H)
        for a, b in zip(data, new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        want = lay.step(*new)
        for name in want:
            assert torch.equal(out[name], want[name]), (rep, name)
        torch.cuda.synchronize()


def test_two_graphs_and_a_stream_of_its_own():
    """Two layers' graphs replayed on two streams at once, beside an eager step on a third, give what each gives alone."""
    torch = torch_cuda()
    lays = [Layer(20 + i) for i in range(3)]
    data = [inputs(30 + i, 256, l.H) for i, l in enumerate(lays)]
    alone = [{k: v.clone() for k, v in l.step(*d).items()} for l, d in zip(lays, data)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in lays]
    graphs, outs = [], []
    for l, d, s in list(zip(lays, data, streams))[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            outs.append(l.step(*d))
        graphs.append(g)
    torch.cuda.synchronize()
    for rep in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            third = lays[2].step(*data[2])
        torch.cuda.synchronize()
        for got, want in zip([*outs, third], alone):
            for name in want:
                assert torch.equal(got[name], want[name]), (rep, name)


@pytest.mark.parametrize("shape", [(9, 256, 384, 700, 4), (64, 800, 2048, 700, 3)], ids=["dealt", "taken"])
def test_two_graphs_share_a_workspace_in_turn(shape):
    """Two captured products with one workspace, replayed one after the other (the larger takes its tiles from counters there)."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    g = torch.Generator(device="cuda").manual_seed(3)
    E, N, K, T, k = shape
    w = moe.fp8_quantize(torch.randn((E, N, K), generator=g, device="cuda"), 128)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    grp = moe.group(idx, E, False)
    dy = moe.fp8_quantize(torch.randn((T * k, N), generator=g, device="cuda"))
    n = moe.lib().moe_fp8_experts_matmul_backward_workspace_size(T, k, 0, K, 1)
    room = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    calls = [lambda: moe.fp8_experts_matmul_backward(dy, w, grp, workspace=room),
             lambda: moe.fp8_experts_matmul_backward(dy, w, grp, tokens=T, workspace=room)]
    want = [c().clone() for c in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(c())
        graphs.append(graph)
    for rep in range(4):
        for graph in graphs:
            graph.replay()
        for c in calls if rep == 2 else []:
            c()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), rep
