"""RMS norm, its 8-bit rows and its gradients on the GPU against float64.

With u = 2^-24: a float32 sum of H squares is off by at most (H + 1) u relative, 1 / sqrt of it by half of that and 3 u, the value
by three more products; a residual's sum by u. So v is off by at most (H / 2 + 8) u |v|, plus, where a residual is added, u times
what its own rounding moves (|x| + |residual|) q w. Results are rounded by half a step of their type. An 8-bit value lies within half a
step of a code (2^-4 of it, or 2^-10 of the scale for the smallest), one that lies that near a border within a whole step.
Gradients: float32 sums of n terms, (n + 16) u of the sum of their magnitudes.
"""
import numpy as np
import pytest

import blocks_ref as ref
from gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6


def lib():
    torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    return moe


def dtype_of(kind):
    torch = torch_cuda()
    return {"f32": torch.float32, "bf16": torch.bfloat16}[kind]


def as64(t):
    return t.double().cpu().numpy()


def half(t):
    return torch_cuda().finfo(t.dtype).eps / 2


def rows(seed, T, H, kind, gap=0):
    torch = torch_cuda()
    g = torch.Generator().manual_seed(seed)
    v = torch.randn((T, H + gap), generator=g) * torch.exp(torch.randn((T, 1), generator=g))
    return v.to(dtype_of(kind)).cuda()[:, gap // 2:gap // 2 + H] if gap else v.to(dtype_of(kind)).cuda()


def weight(seed, H, kind):
    torch = torch_cuda()
    return (1 + 0.3 * torch.randn(H, generator=torch.Generator().manual_seed(seed))).to(dtype_of(kind)).cuda()


def check_rows(n, x, residual, w, H):
    x64, w64 = as64(x), as64(w)
    r = x64 if residual is None else x64 + as64(residual)
    size = np.abs(x64) if residual is None else np.abs(x64) + np.abs(as64(residual))
    v = ref.norm(r, w64, EPS)
    q = 1 / np.sqrt((r * r).mean(1, keepdims=True) + EPS)
    err = (H / 2 + 8) * U * np.abs(v) + U * size * q * np.abs(w64)
    worst = {}
    if residual is not None:
        worst["total"] = np.max(np.abs(as64(n.total) - r) / (half(x) * np.abs(r) + U * size + 1e-37))
    else:
        assert n.total is None
    if n.y is not None:
        assert n.y.dtype == x.dtype
        worst["y"] = np.max(np.abs(as64(n.y) - v) / (err + half(x) * (np.abs(v) + err) + 1e-37))
    if n.fp8 is not None:
        torch, moe = torch_cuda(), lib()
        B = -(-H // 128)
        pad = np.zeros((x.shape[0], B * 128))
        pad[:, :H] = np.abs(v)
        top = pad.reshape(-1, B, 128).max(2)
        pad[:, :H] = err
        slack = pad.reshape(-1, B, 128).max(2)
        s = as64(n.fp8.scales)
        want = np.maximum(top, ref.LEAST) / 448
        worst["scales"] = np.max(np.abs(s - want) / (slack / 448 + 2 * U * want))
        assert (n.fp8.codes.view(torch.uint8)[:, H:] == 0).all()
        # the codes are those of a value within err: between the codes of v - err and v + err
        full = np.repeat(s, 128, 1)[:, :H]
        c = ref.CODES[n.fp8.codes.view(torch.uint8).cpu().numpy()[:, :H]]
        lo, hi = ((v + d) / full for d in (-err, err))
        code = lambda m: np.sign(m) * ref.GRID[ref.nearest(np.abs(m))]  # noqa: E731
        assert ((c >= code(lo)) & (c <= code(hi))).all()
        assert np.array_equal(as64(moe.fp8_dequantize(n.fp8)), (c * full).astype(np.float32).astype(np.float64))
    log(f"[norm] {tuple(x.shape)} {x.dtype}: " + ", ".join(f"{k} {v:.3f}" for k, v in worst.items()))
    assert all(v <= 1 for v in worst.values()), worst


SHAPES = [(1, 1), (1, 2048), (3, 127), (5, 128), (4, 130), (2, 512), (9, 513), (33, 1000), (7, 1024), (300, 2048), (6, 4096), (5, 5000),
          (3, 8192), (2, 16384), (2, 30001), (1, 32768)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm(T, H, kind, residual):
    moe = lib()
    x, r = rows(1, T, H, kind), rows(2, T, H, kind) if residual else None
    for wk, y, q in (("f32", True, True), ("bf16", True, False), ("bf16", False, True)):
        w = weight(H, H, wk)
        n = moe.rms_norm(x, w, r, eps=EPS, rows=y, fp8=q)
        assert (n.y is not None) == y and (n.fp8 is not None) == q
        check_rows(n, x, r, w, H)


@pytest.mark.parametrize("T", [2000, 5000])
def test_norm_many_rows(T):
    """More rows than workgroups: each takes several."""
    moe = lib()
    for H in (300, 2048):
        x, r, w = rows(1, T, H, "bf16"), rows(2, T, H, "bf16"), weight(3, H, "f32")
        check_rows(moe.rms_norm(x, w, r, eps=EPS, fp8=True), x, r, w, H)


def test_norm_strides_and_places():
    torch, moe = torch_cuda(), lib()
    for kind in ("f32", "bf16"):
        for gap in (2, 16, 64):
            x, r, w = rows(1, 37, 1000, kind, gap), rows(2, 37, 1000, kind), weight(1, 1000, "f32")
            n = moe.rms_norm(x, w, r, eps=EPS, fp8=True)
            check_rows(n, x, r, w, 1000)
            m = moe.rms_norm(x.contiguous(), w, r, eps=EPS, fp8=True)
            assert torch.equal(n.y, m.y) and torch.equal(n.total, m.total) and torch.equal(n.fp8.codes.view(torch.uint8), m.fp8.codes.view(torch.uint8))
            # the sum in the residual's place, and in x's
            for own in ("r", "x"):
                a, b = x.contiguous().clone(), r.clone()
                out = moe.Norm(b if own == "r" else a, torch.empty_like(r), None)
                moe.rms_norm(a, w, b, eps=EPS, out=out)
                assert torch.equal(out.total, n.total) and torch.equal(out.y, n.y)
    # a weight that lies on no 16 bytes
    w = weight(1, 1001, "bf16")[1:]
    x = rows(1, 5, 1000, "bf16")
    check_rows(moe.rms_norm(x, w, eps=EPS), x, None, w, 1000)


def test_norm_special_rows():
    torch, moe = torch_cuda(), lib()
    x = rows(1, 8, 300, "f32")
    x[1] = 0
    x[2, 7] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 1e30   # its squares are infinite
    x[5] = 1e-30  # its squares are 0
    w = torch.ones(300, device="cuda")
    n = moe.rms_norm(x, w, eps=EPS, fp8=True)
    v = moe.fp8_dequantize(n.fp8)
    assert (n.y[1] == 0).all() and (v[1] == 0).all()
    assert torch.isnan(n.y[2]).all() and torch.isnan(v[2]).all()
    assert torch.isnan(n.y[3, 7]) and (n.y[3, :7] == 0).all()
    assert (n.y[4] == 0).all()
    assert torch.allclose(n.y[5], torch.full_like(n.y[5], 1e-27), rtol=1e-5)
    assert torch.isfinite(n.y[[0, 6, 7]]).all()
    assert moe.rms_norm(torch.empty((0, 300), device="cuda"), w, fp8=True).y.shape == (0, 300)


@pytest.mark.parametrize("through", [False, True])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", SHAPES + [(1100, 256), (2500, 1000), (777, 1000)])
def test_norm_backward(T, H, kind, through):
    torch, moe = torch_cuda(), lib()
    h, dy = rows(1, T, H, kind), rows(2, T, H, kind, 8)
    d = rows(3, T, H, kind) if through else None
    for wk in ("f32", "bf16"):
        w = weight(H, H, wk)
        dh, dw = moe.rms_norm_backward(dy, h, w, d, eps=EPS)
        want, wdw, size, wsize = ref.norm_gradients(as64(dy), as64(h), as64(w), None if d is None else as64(d), EPS)
        err = (H + 16) * U * size
        a = np.max(np.abs(as64(dh) - want) / (err + half(h) * (np.abs(want) + err) + 1e-37))
        b = np.max(np.abs(as64(dw) - wdw) / ((T + H / 2 + 16) * U * wsize + 1e-37))
        log(f"[norm] backward {T}x{H} {kind}: dh {a:.3f}, dweight {b:.3f}")
        assert a <= 1 and b <= 1 and dw.dtype == torch.float32
        again = moe.rms_norm_backward(dy, h, w, d, eps=EPS)
        assert torch.equal(again[0], dh) and torch.equal(again[1], dw)
        alone, none = moe.rms_norm_backward(dy, h, w, d, eps=EPS, out=(torch.empty_like(h), None))
        assert none is None and torch.equal(alone, dh)


def test_norm_backward_of_nothing():
    torch, moe = torch_cuda(), lib()
    e = torch.empty((0, 300), device="cuda")
    dh, dw = moe.rms_norm_backward(e, e, torch.ones(300, device="cuda"))
    assert dh.shape == (0, 300) and (dw == 0).all()


def test_norm_refusals_with_tensors():
    torch, moe = torch_cuda(), lib()
    x, w = rows(1, 4, 256, "f32"), weight(1, 256, "f32")
    for call in (lambda: moe.rms_norm(x, w[:100]), lambda: moe.rms_norm(x, w, x[:2]), lambda: moe.rms_norm(x, w, x.bfloat16()),
                 lambda: moe.rms_norm(x.t(), weight(1, 4, "f32")), lambda: moe.rms_norm(x, w, rows=False), lambda: moe.rms_norm(x.half(), w),
                 lambda: moe.rms_norm_backward(x[:2], x, w), lambda: moe.rms_norm_backward(None, x, w),
                 lambda: moe.rms_norm_backward(x, x, w, out=(torch.empty((4, 255), device="cuda"), None))):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(moe.MoeError):
        moe.rms_norm(x, w, eps=-1.0)
