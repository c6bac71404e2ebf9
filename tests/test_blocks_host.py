"""Host checks of the 8-bit calls, the RMS norm and routing by scores: refusals before any launch, workspace sizes, and the
tests' own float64 forms against torch and against differences. No GPU work."""
import ctypes as C
import os

import numpy as np
import pytest
import torch

import blocks_ref as ref

moe = pytest.importorskip("bit_quantized_moe_topk_amd")
if not os.path.exists(moe.LIB_PATH):
    pytest.skip("libmoe.so not built (run __graft_entry__.build())", allow_module_level=True)

INV, UNS, WSP, OK = moe.ERR_INVALID_ARG, moe.ERR_UNSUPPORTED, moe.ERR_WORKSPACE, moe.OK
MB = 1 << 20
P = lambda a: C.c_void_p(a)  # noqa: E731
AT = {n: i * 1024 * MB for i, n in enumerate(("x", "xs", "w", "ws", "y", "room", "offsets", "perm", "more", "last"), 1)}  # far apart
BIG = 1 << 40


# ---- refusals -------------------------------------------------------------------------


def quantize(x=AT["x"], t=moe.BF16, ld=256, mats=1, rows=4, K=256, block=1, codes=AT["y"], scales=AT["ws"]):
    return moe.lib().moe_fp8_quantize(P(x), t, ld, mats, rows, K, block, P(codes), P(scales), None)


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_refuses(block):
    for bad in (dict(K=0), dict(rows=-1), dict(mats=-1), dict(ld=255), dict(t=7), dict(block=2), dict(x=0), dict(codes=0),
                dict(scales=0), dict(codes=AT["y"] + 8), dict(scales=AT["ws"] + 2), dict(x=AT["x"] + 1)):
        assert quantize(**{"block": block, **bad}) == INV, bad
    for bad in (dict(K=(1 << 19) + 1, ld=1 << 20), dict(ld=BIG + 1), dict(mats=1 << 16, rows=1 << 16)):
        assert quantize(**{"block": block, **bad}) == UNS, bad
    # results over the rows, or over each other
    for bad in (dict(codes=AT["x"]), dict(scales=AT["x"] + 16), dict(codes=AT["x"] + 3 * 512), dict(scales=AT["y"] + 16)):
        assert quantize(**{"block": block, **bad}) == INV, bad
    if block == 128:  # one workgroup a block: no more than a launch holds
        assert quantize(block=128, mats=1 << 24, rows=1, K=1) == UNS and quantize(block=128, mats=1 << 23, rows=1, K=129) == UNS
    assert quantize(rows=0, x=0, codes=0, scales=0) == OK and quantize(mats=0, x=0, codes=0, scales=0) == OK


def test_dequantize_refuses():
    def call(c=AT["x"], s=AT["xs"], mats=1, rows=4, K=256, block=1, t=moe.F32, y=AT["y"]):
        return moe.lib().moe_fp8_dequantize(P(c), P(s), mats, rows, K, block, t, P(y), None)
    for bad in (dict(K=0), dict(rows=-1), dict(t=5), dict(block=64), dict(c=0), dict(s=0), dict(y=0), dict(c=AT["x"] + 8),
                dict(y=AT["x"]), dict(y=AT["xs"]), dict(y=AT["y"] + 2)):
        assert call(**bad) == INV, bad
    assert call(K=(1 << 19) + 1) == UNS and call(rows=0, c=0, s=0, y=0) == OK


def matmul(back, x=AT["x"], xs=AT["xs"], T=4, w=AT["w"], ws=AT["ws"], N=256, K=512, y=AT["y"], t=moe.BF16):
    fn = moe.lib().moe_fp8_matmul_backward if back else moe.lib().moe_fp8_matmul
    return fn(P(x), P(xs), T, P(w), P(ws), N, K, P(y), t, None)


@pytest.mark.parametrize("back", [False, True])
def test_matmul_refuses(back):
    for bad in (dict(T=-1), dict(N=0), dict(K=0), dict(t=4), dict(x=0), dict(xs=0), dict(w=0), dict(ws=0), dict(y=0),
                dict(x=AT["x"] + 8), dict(w=AT["w"] + 4), dict(xs=AT["xs"] + 1), dict(ws=AT["ws"] + 2), dict(y=AT["y"] + 1)):
        assert matmul(back, **bad) == INV, bad
    for bad in (dict(N=(1 << 19) + 1), dict(K=(1 << 19) + 1), dict(T=(1 << 22) + 1)):
        assert matmul(back, **bad) == UNS, bad
    n_in = 256 if back else 512
    for base, size in (("x", 4 * n_in), ("xs", 4 * n_in // 128 * 4), ("w", 256 * 512), ("ws", 2 * 4 * 4)):
        for at in (AT[base], AT[base] + size - 16):
            assert matmul(back, y=at) == INV, base
    assert matmul(back, T=0, x=0, xs=0, w=0, ws=0, y=0) == OK


def experts(back, x=AT["x"], xs=AT["xs"], T=300, k=8, E=16, shared=1, gather=1, offsets=AT["offsets"], perm=AT["perm"],
            w=AT["w"], ws=AT["ws"], N=256, K=512, y=AT["y"], t=moe.BF16, room=AT["room"], n=1 << 30):
    fn = moe.lib().moe_fp8_experts_matmul_backward if back else moe.lib().moe_fp8_experts_matmul
    return fn(P(x), P(xs), T, k, E, shared, gather, P(offsets), P(perm), P(w), P(ws), N, K, P(y), t, *((P(room), n) if back else ()), None)


@pytest.mark.parametrize("back", [False, True])
def test_experts_refuse(back):
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(shared=2), dict(gather=3), dict(offsets=0), dict(perm=0), dict(N=0), dict(K=0),
                dict(x=0), dict(xs=0), dict(w=0), dict(ws=0), dict(y=0), dict(t=4), dict(w=AT["w"] + 8),
                dict(y=AT["offsets"]), dict(y=AT["perm"] + 16), dict(y=AT["w"]), dict(y=AT["ws"] + 16)):
        assert experts(back, **bad) == INV, bad
    for bad in (dict(y=AT["room"] + 512), dict(room=AT["x"]), dict(room=AT["w"] + 1024), dict(room=AT["offsets"]), dict(room=AT["perm"])):
        assert not back or experts(back, **bad) == INV, bad
    for bad in (dict(E=2049), dict(T=1 << 22), dict(k=1 << 23), dict(N=(1 << 19) + 1)):
        assert experts(back, **bad) == UNS, bad
    for bad in (dict(room=0), dict(n=64), dict(room=AT["room"] + 8)):
        assert not back or experts(back, **bad) == WSP, bad
    assert experts(back, T=0, x=0, xs=0, w=0, ws=0, y=0, offsets=0, perm=0, room=0, n=0) == OK


def test_workspace_sizes():
    L = moe.lib()
    assert L.moe_fp8_experts_matmul_backward_workspace_size(8192, 10, 1, 100, 0) > 0
    assert L.moe_fp8_experts_matmul_backward_workspace_size(-1, 10, 1, 100, 0) == 0
    assert L.moe_fp8_experts_matmul_backward_workspace_size(10, 2, 1, 100, 1) >= 30 * 100 * 4
    assert L.moe_fp8_experts_matmul_backward_workspace_size(10, 2, 1, 100, 0) == 0
    assert L.moe_rms_norm_backward_workspace_size(5, 64) >= 64 * 4 and L.moe_rms_norm_backward_workspace_size(0, 64) == 0


def norm(x=AT["x"], t=moe.BF16, ldx=256, r=AT["xs"], ldr=256, w=AT["w"], wt=moe.F32, eps=1e-6, T=4, H=256, total=AT["y"],
         y=AT["room"], codes=AT["more"], scales=AT["last"]):
    return moe.lib().moe_rms_norm(P(x), t, ldx, P(r), ldr, P(w), wt, eps, T, H, P(total), P(y), P(codes), P(scales), None)


def test_norm_refuses():
    for bad in (dict(T=-1), dict(H=0), dict(ldx=255), dict(ldr=255), dict(t=4), dict(wt=9), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(x=0), dict(w=0), dict(scales=0), dict(codes=0), dict(total=0, y=0, codes=0, scales=0),
                dict(x=AT["x"] + 1), dict(codes=AT["more"] + 8), dict(y=AT["x"]), dict(y=AT["xs"] + 16), dict(codes=AT["w"]),
                dict(total=AT["x"] + 16), dict(total=AT["x"], ldx=512), dict(y=AT["y"]), dict(scales=AT["room"]), dict(total=AT["w"])):
        assert norm(**bad) == INV, bad
    for bad in (dict(H=32769, ldx=40000, ldr=40000), dict(T=(1 << 22) + 1), dict(ldx=BIG + 1), dict(ldr=BIG + 1)):
        assert norm(**bad) == UNS, bad
    assert norm(T=0, x=0, w=0) == OK


def norm_back(dy=AT["x"], ldd=256, h=AT["xs"], ldh=256, t=moe.BF16, w=AT["w"], wt=moe.F32, d=AT["ws"], ldt=256, eps=1e-6, T=4, H=256,
              dh=AT["y"], dw=AT["more"], room=AT["room"], n=1 << 24):
    return moe.lib().moe_rms_norm_backward(P(dy), ldd, P(h), ldh, t, P(w), wt, P(d), ldt, eps, T, H, P(dh), P(dw), P(room), n, None)


def test_norm_backward_refuses():
    for bad in (dict(T=-1), dict(H=0), dict(ldd=255), dict(ldh=255), dict(ldt=255), dict(t=4), dict(wt=4), dict(eps=-1.0), dict(dy=0),
                dict(h=0), dict(w=0), dict(dh=0), dict(dw=AT["more"] + 2), dict(dh=AT["x"]), dict(dh=AT["xs"]), dict(dh=AT["ws"]),
                dict(dw=AT["w"]), dict(dw=AT["y"]), dict(room=AT["x"]), dict(room=AT["y"])):
        assert norm_back(**bad) == INV, bad
    for bad in (dict(H=32769, ldd=40000, ldh=40000, ldt=40000), dict(T=(1 << 22) + 1), dict(ldd=BIG + 1)):
        assert norm_back(**bad) == UNS, bad
    for bad in (dict(room=0), dict(n=16), dict(room=AT["room"] + 4)):
        assert norm_back(**bad) == WSP, bad
    assert norm_back(T=0, dw=0, dy=0, h=0, w=0, dh=0) == OK


def route(x=AT["x"], t=moe.F32, ld=64, T=4, E=64, bias=AT["xs"], score=0, groups=8, keep=4, top=2, k=6, renorm=1, scale=1.0,
          idx=AT["y"], gates=AT["ws"]):
    return moe.lib().moe_route_scores(P(x), t, ld, T, E, P(bias), score, groups, keep, top, k, renorm, scale, P(idx), P(gates), None)


def test_route_refuses():
    for bad in (dict(T=-1), dict(E=0), dict(ld=63), dict(t=4), dict(score=2), dict(groups=0), dict(groups=7), dict(keep=0), dict(keep=9),
                dict(top=0), dict(top=3), dict(k=0), dict(k=33), dict(scale=float("inf")), dict(scale=float("nan")), dict(x=0), dict(idx=0),
                dict(gates=0), dict(x=AT["x"] + 2), dict(idx=AT["x"]), dict(gates=AT["xs"]), dict(gates=AT["y"])):
        assert route(**bad) == INV, bad
    for bad in (dict(E=4096, ld=4096), dict(E=130, ld=130, groups=65, keep=65), dict(T=(1 << 22) + 1), dict(ld=BIG + 1)):
        assert route(**bad) == UNS, bad
    assert route(T=0, x=0, idx=0, gates=0) == OK


def test_route_backward_refuses():
    def call(x=AT["x"], t=moe.F32, ld=64, T=4, E=64, k=6, score=0, renorm=1, scale=1.0, idx=AT["xs"], d=AT["w"], out=AT["y"]):
        return moe.lib().moe_route_scores_backward(P(x), t, ld, T, E, k, score, renorm, scale, P(idx), P(d), P(out), None)
    for bad in (dict(T=-1), dict(E=0), dict(ld=63), dict(t=4), dict(score=-1), dict(k=0), dict(scale=float("nan")), dict(x=0), dict(idx=0),
                dict(d=0), dict(out=0), dict(out=AT["x"]), dict(out=AT["xs"]), dict(out=AT["w"])):
        assert call(**bad) == INV, bad
    assert call(E=4096, ld=4096) == UNS and call(k=2049) == UNS and call(T=0, x=0, idx=0, d=0, out=0) == OK


def test_python_refuses_what_is_not_on_the_gpu():
    x = torch.zeros(4, 256)
    for call in (lambda: moe.fp8_quantize(x), lambda: moe.route_scores(x, 2), lambda: moe.rms_norm(x, torch.ones(256)),
                 lambda: moe.fp8_quantize(x, 3), lambda: moe.Fp8(torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2), 256),
                 lambda: moe.fp8_matmul(x, x), lambda: moe.rms_norm_backward(x, x, x[0])):
        with pytest.raises((ValueError, TypeError)):
            call()


# ---- the float64 forms ------------------------------------------------------------------


def test_codes_are_torchs():
    c = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(c, ref.CODES, equal_nan=True)
    v = np.concatenate([ref.GRID, (ref.GRID[1:] + ref.GRID[:-1]) / 2, np.linspace(0, 448, 4001)])
    got = torch.from_numpy(v).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    keep = v == v.astype(np.float32)
    assert np.array_equal(got[keep], ref.nearest(v)[keep])


def test_quantize_form():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((200, 300)) * np.exp(rng.standard_normal((200, 1)))).astype(np.float32)
    for block in (1, 128):
        c, s = ref.quantize(x, block)
        v = ref.values(c, s, 300, block)
        top = np.repeat(np.repeat(s, 128, 1), block, 0)[:200, :300].astype(np.float64)
        assert (np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, top * 2.0 ** -10) * (1 + 1e-7)).all()
        assert (c[:, 300:] == 0).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_form(score, renorm):
    """The formula against central differences of the gates, with the selection held."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 7))
    idx, _ = ref.route(x, 3, None, score, 1, 1, 2, renorm, 1.5)
    d = rng.standard_normal((3, 3))

    def gates(x):
        q = np.take_along_axis(ref.scores(x, score), idx.astype(np.int64), 1)
        return 1.5 * (q / q.sum(1, keepdims=True) if renorm else q)
    got, _ = ref.route_gradient(x, idx, d, score, renorm, 1.5)
    for e in range(7):
        h = np.zeros_like(x)
        h[:, e] = 1e-5
        diff = ((gates(x + h) - gates(x - h)) * d).sum(1) / 2e-5
        assert np.allclose(got[:, e], diff, atol=1e-8)


def test_norm_gradient_form():
    rng = np.random.default_rng(2)
    h, dy, dt, w = rng.standard_normal((4, 9)), rng.standard_normal((4, 9)), rng.standard_normal((4, 9)), rng.standard_normal(9)
    f = lambda h, w: (ref.norm(h, w, 1e-3) * dy).sum() + (h * dt).sum()  # noqa: E731
    dh, dw, _, _ = ref.norm_gradients(dy, h, w, dt, 1e-3)
    for i in range(9):
        e = np.zeros(9)
        e[i] = 1e-6
        assert abs((f(h, w + e) - f(h, w - e)) / 2e-6 - dw[i]) < 1e-7
        for t in range(4):
            m = np.zeros((4, 9))
            m[t, i] = 1e-6
            assert abs((f(h + m, w) - f(h - m, w)) / 2e-6 - dh[t, i]) < 1e-7


def test_route_form_by_hand():
    """Two groups of three: the second has the larger sum of two, the first the largest score alone."""
    x = np.array([[4.0, -3.0, -3.0, 2.0, 2.5, -1.0]])
    idx, gates = ref.route(x, 2, None, "sigmoid", 2, 1, 2, True, 1.0)
    assert idx.tolist() == [[4, 3]] and abs(gates.sum() - 1) < 1e-12
    idx, _ = ref.route(x, 2, None, "sigmoid", 2, 1, 1, True, 1.0)
    assert idx.tolist() == [[0, 1]]
    idx, _ = ref.route(x, 2, np.array([0, 0, 0, 0, 0, 9.0]), "softmax", 2, 2, 2, True, 1.0)
    assert idx.tolist() == [[5, 0]]
    idx, gates = ref.route(np.full((1, 4), -np.inf), 2, None, "softmax", 1, 1, 2, True, 1.0)
    assert idx.tolist() == [[0, 1]] and gates.tolist() == [[0, 0]]
