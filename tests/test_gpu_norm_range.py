"""The RMS norm and its gradients at the ends of float32's range, against float64, with the bounds of test_gpu_norm: (H / 2 + 8) u of a
value and half a step of its type; (H + 16) u of the magnitudes that a gradient's entry adds up."""
import numpy as np
import pytest

import blocks_ref as ref
from gpu_util import log, torch_cuda
from test_gpu_norm import U, as64, half, lib, rows, weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(3, 64), (5, 1000), (4, 2048), (6, 4096), (3, 8192), (2, 16384), (2, 20000), (1, 32768)])
def test_rows_near_the_range(T, H, kind):
    """Magnitudes up to 2^61, whose squares add up past 2^128, and rows below eps: norm and gradients are those of any row."""
    torch, moe = torch_cuda(), lib()
    for size, eps in ((2.0 ** 61, 1e-6), (1.5e18, 0.0), (1e17, 1e-6), (1e-15, 0.0)):
        h = (rows(1, T, H, "f32").clamp(-1, 1) * size).to(torch.float32 if kind == "f32" else torch.bfloat16)
        dy, d, w = rows(2, T, H, kind), rows(3, T, H, kind), weight(H, H, "f32")
        h64, w64 = as64(h), as64(w)
        y = as64(moe.rms_norm(h, w, eps=eps).y)
        v = ref.norm(h64, w64, float(np.float32(eps)))
        err = (H / 2 + 8) * U * np.abs(v)
        assert np.all(np.abs(y - v) <= err + half(h) * (np.abs(v) + err) + 1e-37)
        for through in (None, d):
            dh, dw = moe.rms_norm_backward(dy, h, w, through, eps=eps)
            want, wdw, mags, wmags = ref.norm_gradients(as64(dy), h64, w64, None if through is None else as64(through), float(np.float32(eps)))
            err = (H + 16) * U * mags
            a = np.max(np.abs(as64(dh) - want) / (err + half(h) * (np.abs(want) + err) + 1e-37))
            b = np.max(np.abs(as64(dw) - wdw) / ((T + H / 2 + 16) * U * wmags + 1e-37))
            log(f"[norm] range {T}x{H} {kind} {size:g}: dh {a:.3f}, dweight {b:.3f}")
            assert a <= 1 and b <= 1, (size, a, b)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("H", [5, 300, 2048, 20000])
def test_weights_that_are_not_finite(H, kind):
    """An infinite weight gives infinities of the value's sign, NaN where the value is 0; a NaN weight NaN; others what they gave."""
    torch, moe = torch_cuda(), lib()
    for wk in ("f32", "bf16"):
        x, w = rows(1, 7, H, kind), weight(2, H, wk)
        x[1, 0] = 0
        clean = moe.rms_norm(x, w).y
        bad = w.clone()
        bad[0], bad[3] = float("inf"), -float("inf")
        bad[4] = float("nan")
        n = moe.rms_norm(x, bad, fp8=True)
        want = clean.clone()
        for c in (0, 3):
            want[:, c] = (x[:, c].float() * bad[c].float()).to(x.dtype)
        want[:, 4] = float("nan")
        assert torch.equal(n.y.nan_to_num(1234.0, posinf=1e30, neginf=-1e30), want.nan_to_num(1234.0, posinf=1e30, neginf=-1e30))
        assert torch.isnan(n.y[1, 0]) and torch.isinf(n.y[0, 0])
        v = moe.fp8_dequantize(n.fp8)
        assert torch.isnan(v[:, :128]).all() and torch.isfinite(v[:, 128:]).all()
        # the largest finite weight: a product past the range is infinite, others are values
        bad = w.clone()
        bad[0] = torch.finfo(w.dtype).max
        y = moe.rms_norm(x, bad).y
        v = ref.norm(as64(x), as64(bad), 1e-6)[:, 0]
        with np.errstate(over="ignore"):
            past = np.abs(v) > float(torch.finfo(x.dtype).max) * (1 + 2.0 ** -8)
        inside = np.abs(v) < float(torch.finfo(x.dtype).max) * (1 - 2.0 ** -8)
        y0 = as64(y[:, 0])
        assert (np.isinf(y0[past]) & (np.sign(y0[past]) == np.sign(v[past]))).all()
        assert np.all(np.abs(y0[inside] - v[inside]) <= ((H / 2 + 8) * U + half(x)) * 1.01 * np.abs(v[inside]))
        assert torch.equal(y[:, 1:], clean[:, 1:])
