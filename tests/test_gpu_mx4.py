"""Microscaled 4-bit quantisation and products on the GPU against float64.

Quantisation is exact: codes and scales equal the reference's. A product's terms are exact (a weight has two
significant bits, a bfloat16 row eight, a float32 row enters in three exact parts), so its error is that of a float32
sum of n terms in some order, at most (n + 2) 2^-24 sum |x w| (n = 3 K or 3 N terms for float32 rows, plus the rows
that a token's gradient adds up), and of one rounding to the result's type, half a step (finfo.eps / 2).
"""
import numpy as np
import pytest

import mx4_ref
from gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu


def types():
    torch = torch_cuda()
    return {"f32": torch.float32, "bf16": torch.bfloat16}


def as64(t) -> np.ndarray:
    return t.double().cpu().numpy()


def check(name, got, ref, size, terms):
    torch = torch_cuda()
    half = torch.finfo(got.dtype).eps / 2
    g = as64(got)
    sums = (terms + 2) * 2.0 ** -24 * size
    bound = sums + half * (np.abs(ref) + sums) + 1e-37
    assert g.shape == ref.shape and np.isfinite(g).all(), name
    worst = np.max(np.abs(g - ref) / bound, initial=0.0)
    log(f"[mx4] {name}: error / bound {worst:.3f}")
    assert worst <= 1, name


def random_matrix(rng, shape, K, lo=110, hi=131):
    """Random codes (zeros past K) and scales: an Mx4 and its values."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    B = -(-K // 32)
    codes = rng.integers(0, 256, (*shape, 16 * B), dtype=np.uint8)
    if K % 32:
        n = np.arange(32 * B).reshape(-1, 2)
        codes &= ((n[:, 0] < K) * 15 + (n[:, 1] < K) * 240).astype(np.uint8)
    scales = rng.integers(lo, hi, (*shape, B), dtype=np.uint8)
    return moe.Mx4(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), K), mx4_ref.values(codes, scales, K)


def random_rows(rng, R, n, kind, strided=False):
    """An operand of R rows and its values."""
    torch = torch_cuda()
    if kind == "mx4":
        return random_matrix(rng, (R,), n)
    v = torch.from_numpy(rng.standard_normal((R, n + 24 if strided else n)) * np.exp(rng.standard_normal((R, 1))))
    t = v.to(types()[kind]).cuda()
    t = t[:, 8:8 + n] if strided else t
    return t, as64(t)


def grouping_of(rng, T, k, E, shared, skew=0.0, quiet=0):
    """A grouping by the framework; `quiet` experts get nothing."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    logits = rng.standard_normal((T, E)) - skew * np.log(1 + np.arange(E))
    if quiet:
        logits[:, rng.permutation(E)[:quiet]] -= 100
    idx, _ = moe.route_topk(torch.from_numpy(logits.astype(np.float32)).cuda(), k)
    return moe.group(idx, E, shared)


# ---- quantisation ---------------------------------------------------------------------


def nasty(rng, rows, K):
    v = rng.standard_normal((rows, K)) * np.exp(4 * rng.standard_normal((rows, 1)))
    v = v.astype(np.float32)
    flat = v.reshape(-1)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 7.999, 4, -0.25, -0.75, -5, 0.0, -0.0], np.float32)
    flat[: min(flat.size, 16)] = ties[: min(flat.size, 16)]
    for i, s in enumerate((2.0 ** -126, 2.0 ** -149, 3e38, 1e-38, 0.0, 2.0 ** -124)):
        if i < rows - 1:
            v[i + 1] = (rng.standard_normal(K) * s).clip(-3.4e38, 3.4e38).astype(np.float32)
    if rows > 8:
        v[8, 0], v[7, K - 1], v[8, K // 2] = np.nan, np.inf, -np.inf
    return v


@pytest.mark.parametrize("rows,K", [(1, 1), (1, 32), (3, 31), (9, 33), (17, 100), (33, 256), (70, 1000), (2, 4096)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_quantize_is_exact(rows, K, kind):
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    x = torch.from_numpy(nasty(np.random.default_rng(rows * K), rows, K)).to(types()[kind])
    codes, scales = mx4_ref.quantize(x.float().numpy())
    wide = torch.zeros((rows, K + 9), dtype=x.dtype).cuda()
    wide[:, 5:5 + K] = x.cuda()
    for name, t in (("adjacent", x.cuda()), ("strided", wide[:, 5:5 + K])):
        q = moe.mx4_quantize(t)
        assert np.array_equal(q.scales.cpu().numpy(), scales), name
        assert np.array_equal(q.codes.cpu().numpy(), codes), name
    want = mx4_ref.values(codes, scales, K)
    for dt in types().values():
        got = moe.mx4_dequantize(q, dt)
        assert got.dtype == dt and np.array_equal(as64(got), want, equal_nan=True)


def test_dequantize_every_code_and_scale():
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    codes = np.tile(np.arange(16, dtype=np.uint8) * 17, (256, 1))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    q = moe.Mx4(torch.from_numpy(codes).cuda(), torch.from_numpy(scales.copy()).cuda(), 32)
    with np.errstate(over="ignore"):
        want = mx4_ref.values(codes, scales, 32).astype(np.float32).astype(np.float64)
    for dt in types().values():
        assert np.array_equal(as64(moe.mx4_dequantize(q, dt)), want, equal_nan=True)


def test_quantize_three_dimensions_and_out():
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    x = torch.randn(3, 5, 70, device="cuda")
    q = moe.mx4_quantize(x)
    assert q.shape == (3, 5, 70) and q.codes.shape == (3, 5, 48) and q.scales.shape == (3, 5, 3)
    again = moe.mx4_quantize(2 * x, out=moe.Mx4(torch.empty_like(q.codes), torch.empty_like(q.scales), 70))
    assert torch.equal(again.codes, q.codes) and torch.equal(again.scales, q.scales + 1)
    assert moe.mx4_quantize(x[:, :0].contiguous()).shape == (3, 0, 70)


# ---- one matrix -----------------------------------------------------------------------

SIZES = [(1, 1, 1), (1, 1024, 2048), (3, 17, 33), (4, 256, 96), (16, 130, 64), (17, 500, 1000), (33, 64, 2048),
         (65, 48, 160), (100, 1000, 31), (130, 257, 544), (300, 384, 512)]


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "f32", "mx4"])
def test_matmul(T, N, K, kind):
    torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(T * N + K)
    w, wv = random_matrix(rng, (N,), K)
    for strided in (False, True)[: 1 if kind == "mx4" else 2]:
        x, xv = random_rows(rng, T, K, kind, strided)
        ref, size = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
        for dt in types().values():
            y = moe.mx4_matmul(x, w, dtype=dt)
            assert y.dtype == dt
            check(f"{kind} {T}x{N}x{K} strided={strided} -> {dt}", y, ref, size, K * (3 if kind == "f32" else 1))


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_matmul_backward(T, N, K, kind):
    torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(T + N * K)
    w, wv = random_matrix(rng, (N,), K)
    for strided in (False, True):
        d, dv = random_rows(rng, T, N, kind, strided)
        ref, size = dv @ wv, np.abs(dv) @ np.abs(wv)
        for dt in types().values():
            check(f"gradient {kind} {T}x{N}x{K} strided={strided} -> {dt}", moe.mx4_matmul_backward(d, w, dtype=dt), ref,
                  size, N * (3 if kind == "f32" else 1))


# Rows enough for the tile kernels, each form of them: strips of 512, 256 and 128 matrix rows, scales
# four and sixteen at a time, one at a time; columns in no whole step or block; rows that end a run,
# a tile, or one past it.
MANY = [(33000, 260, 512), (33025, 260, 384), (33000, 130, 256), (1100, 1040, 512), (1153, 1040, 384), (1100, 1040, 100),
        (2000, 800, 72), (4100, 513, 640)]


@pytest.mark.parametrize("T,N,K", MANY)
@pytest.mark.parametrize("kind", ["bf16", "f32", "mx4"])
def test_matmul_many_rows(T, N, K, kind):
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(T + N + K)
    w, wv = random_matrix(rng, (N,), K)
    x, xv = random_rows(rng, T, K, kind, strided=kind == "bf16" and T % 2 == 1)
    ref, size = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    y = moe.mx4_matmul(x, w)
    check(f"{kind} {T}x{N}x{K}", y, ref, size, K * (3 if kind == "f32" else 1))
    assert torch.equal(moe.mx4_matmul(x, w), y)
    if kind != "f32":
        check(f"{kind} {T}x{N}x{K} -> f32", moe.mx4_matmul(x, w, dtype=torch.float32), ref, size, K)


MANY_BACK = [(1300, 192, 2176), (1301, 64, 2176), (1300, 200, 2176), (1300, 192, 2100), (2600, 70, 2100), (33000, 128, 512),
             (40000, 64, 2176), (40100, 64, 1100), (40000, 60, 1000)]


@pytest.mark.parametrize("T,N,K", MANY_BACK)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_matmul_backward_many_rows(T, N, K, kind):
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(T + N + K)
    w, wv = random_matrix(rng, (N,), K)
    d, dv = random_rows(rng, T, N, kind)
    ref, size = dv @ wv, np.abs(dv) @ np.abs(wv)
    g = moe.mx4_matmul_backward(d, w)
    check(f"gradient {kind} {T}x{N}x{K}", g, ref, size, N * (3 if kind == "f32" else 1))
    assert torch.equal(moe.mx4_matmul_backward(d, w), g)
    if kind == "bf16":
        check(f"gradient {kind} {T}x{N}x{K} -> f32", moe.mx4_matmul_backward(d, w, dtype=torch.float32), ref, size, N)


def test_gradient_against_differences():
    """The product is linear in x, so a difference quotient is exact up to its own roundings: with x, h and the
    weights small integers over powers of two every sum here is exact in float32, and so both sides are equal."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(5)
    T, N, K = 5, 40, 70
    w, _ = random_matrix(rng, (N,), K, lo=127, hi=128)
    x = torch.from_numpy(rng.integers(-8, 9, (T, K))).float().cuda()
    d = torch.from_numpy(rng.integers(-8, 9, (T, N))).float().cuda()
    g = moe.mx4_matmul_backward(d, w)
    for k in range(0, K, 7):
        h = torch.zeros_like(x)
        h[:, k] = 2
        quotient = ((moe.mx4_matmul(x + h, w) - moe.mx4_matmul(x - h, w)) * d).sum(1) / 4
        assert torch.equal(quotient, g[:, k])


@pytest.mark.parametrize("kind", ["bf16", "f32", "mx4"])
def test_special_values(kind):
    """NaN blocks reach their own outputs alone; infinities and huge, tiny and subnormal rows keep their class."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(11)
    T, N, K = 20, 40, 128
    w, wv = random_matrix(rng, (N,), K, 120, 126)
    w.scales[7, 2] = 255
    x, xv = random_rows(rng, T, K, kind)
    if kind == "mx4":
        x.scales[3, 1] = 255
        x.scales[5], xv[5] = 0, xv[5] * 2.0 ** (-x.scales[5].cpu().numpy().astype(float)).repeat(32)
    else:
        x[3, 40] = float("nan")
        x[4, 9] = float("inf")
        x[5] *= 2.0 ** -120
        x[6] *= 2.0 ** 100
        xv = as64(x)
    y = as64(moe.mx4_matmul(x, w, dtype=torch.float32))
    assert np.isnan(y[3]).all() and np.isnan(y[:, 7]).all()
    rest = np.delete(np.arange(N), 7)
    if kind != "mx4":
        bad = y[4][rest]
        assert not np.isfinite(bad[wv[rest, 9] != 0]).any() and np.isnan(bad[wv[rest, 9] == 0]).all()
    rows = np.delete(np.arange(T), [3, 4] if kind != "mx4" else [3])
    ref, size = xv[rows] @ wv[rest].T, np.abs(xv[rows]) @ np.abs(wv[rest]).T
    err = np.abs(y[np.ix_(rows, rest)] - ref) / ((3 * K + 3) * 2.0 ** -24 * size + 2.0 ** -148)
    assert err.max() <= 1, err.max()
    if kind != "mx4":
        d, dv = random_rows(rng, T, N, kind)
        d[:, 7] = 0
        d[2, 3] = float("nan")
        g = as64(moe.mx4_matmul_backward(d, w, dtype=torch.float32))
        assert np.isnan(g[2]).all() and np.isnan(g[:, 64:96]).all()   # 0 times NaN is NaN
        assert np.isfinite(np.delete(g, 2, 0)[:, :64]).all() and np.isfinite(np.delete(g, 2, 0)[:, 96:]).all()


@pytest.mark.parametrize("T,N,K", [(1, 40, 70), (9, 33, 130), (40, 300, 100), (300, 300, 100), (1100, 1040, 33), (1100, 200, 2100)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_what_lies_around_the_rows_is_not_read_into_them(T, N, K, kind):
    """Rows cut out of a wider array of NaN, products and gradients of them: every result is a number."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(T + N + K)
    w, wv = random_matrix(rng, (N,), K)
    terms = 3 if kind == "f32" else 1
    for n, ref_of, call in ((K, wv.T, moe.mx4_matmul), (N, wv, moe.mx4_matmul_backward)):
        for lead in (8, 3):
            room = torch.full((T + 2, n + 48), float("nan"), device="cuda", dtype=types()[kind])
            x = room[1:-1, lead:lead + n]
            x.copy_(torch.from_numpy(rng.standard_normal((T, n))))
            xv = as64(x)
            check(f"{call.__name__} {kind} {T}x{N}x{K} among NaN", call(x, w), xv @ ref_of, np.abs(xv) @ np.abs(ref_of), n * terms)


@pytest.mark.parametrize("T,N,K", [(300, 520, 512), (300, 520, 384), (1100, 1040, 512), (1100, 1040, 100), (2100, 1100, 1024)])
@pytest.mark.parametrize("kind", ["bf16", "f32", "mx4"])
def test_special_values_of_many_rows(T, N, K, kind):
    """NaN blocks, infinities and overflow reach their own outputs alone in the tile kernels too."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(T + N + K)
    w, wv = random_matrix(rng, (N,), K, 120, 126)
    w.scales[7, 2], w.scales[N - 1, -1] = 255, 255
    rest = np.setdiff1d(np.arange(N), [7, N - 1])
    x, xv = random_rows(rng, T, K, kind)
    if kind == "mx4":
        x.scales[T - 1, 1] = 255
        lost = [T - 1]
    else:
        x[T - 1, K - 1], x[4, 9] = float("nan"), float("inf")
        x[6] *= 2.0 ** 100
        xv, lost = as64(x), [4, T - 1]
    y = as64(moe.mx4_matmul(x, w, dtype=torch.float32))
    assert np.isnan(y[T - 1]).all() and np.isnan(y[:, [7, N - 1]]).all()
    if kind != "mx4":
        bad = y[4][rest]
        assert not np.isfinite(bad[wv[rest, 9] != 0]).any() and np.isnan(bad[wv[rest, 9] == 0]).all()
    rows = np.setdiff1d(np.arange(T), lost)
    ref, size = xv[rows] @ wv[rest].T, np.abs(xv[rows]) @ np.abs(wv[rest]).T
    assert (np.abs(y[np.ix_(rows, rest)] - ref) <= (3 * K + 3) * 2.0 ** -24 * size + 2.0 ** -148).all()


@pytest.mark.parametrize("at", [1, 2, 4])
@pytest.mark.parametrize("T", [3, 1100, 33000])
def test_scales_that_start_anywhere(T, at):
    """Scales need no alignment: those of a matrix and of rows that start 1, 2 or 4 bytes into a buffer."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(T + at)
    N, K = 300, 512

    def moved(q):
        room = torch.empty(q.scales.numel() + 16, dtype=torch.uint8, device="cuda")
        s = room[at:at + q.scales.numel()].view(q.scales.shape)
        s.copy_(q.scales)
        return moe.Mx4(q.codes, s, q.K)

    w, wv = random_matrix(rng, (N,), K)
    x, xv = random_rows(rng, T, K, "bf16")
    q, qv = random_matrix(rng, (T,), K)
    d, dv = random_rows(rng, T, 320, "bf16")
    v, vv = random_matrix(rng, (320,), K)
    assert torch.equal(moe.mx4_dequantize(moved(w)), moe.mx4_dequantize(w))
    for name, y, left, right in (("rows", moe.mx4_matmul(x, moved(w)), xv, wv.T),
                                 ("four bits", moe.mx4_matmul(moved(q), moved(w)), qv, wv.T),
                                 ("gradient", moe.mx4_matmul_backward(d, moved(v)), dv, vv)):
        check(f"{name} T={T} at {at}", y, left @ right, np.abs(left) @ np.abs(right), left.shape[1])


def test_results_repeat_and_leave_the_rest_alone():
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(3)
    for T, N, K in ((5, 70, 300), (200, 300, 256)):
        w, _ = random_matrix(rng, (N,), K)
        x, _ = random_rows(rng, T, K, "bf16")
        room = torch.full((T + 2, N), 7.0, device="cuda", dtype=torch.bfloat16)
        y = moe.mx4_matmul(x, w, out=room[1:-1])
        assert (room[0] == 7).all() and (room[-1] == 7).all()
        for _ in range(3):
            assert torch.equal(moe.mx4_matmul(x, w), y)
        d, _ = random_rows(rng, T, N, "f32")
        g = moe.mx4_matmul_backward(d, w)
        for _ in range(3):
            assert torch.equal(moe.mx4_matmul_backward(d, w), g)
    assert moe.mx4_matmul(x[:0], w).shape == (0, N) and moe.mx4_matmul_backward(d[:0], w).shape == (0, K)


@pytest.mark.parametrize("T,N,K", [(260, 2048, 96), (250, 2047, 260), (1030, 520, 1000), (600, 1030, 33), (2100, 300, 256)])
def test_matmul_float32_of_some_hundred_rows(T, N, K):
    """Sixteen rows a tile: columns in no whole block or stage, rows that end inside a tile, odd strides, ends of strips."""
    torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(T + N + K)
    w, wv = random_matrix(rng, (N,), K)
    for strided in (False, True):
        x, xv = random_rows(rng, T, K, "f32", strided)
        x = x if not strided else x[:, :K]
        ref, size = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
        for dt in types().values():
            check(f"f32 {T}x{N}x{K} strided={strided} -> {dt}", moe.mx4_matmul(x, w, dtype=dt), ref, size, 3 * K)


# ---- experts --------------------------------------------------------------------------

GROUPS = [  # T, k, E, shared, N, K, skew, experts that get nothing
    (1, 1, 1, False, 16, 32, 0, 0), (1, 2, 8, True, 40, 70, 0, 3), (4, 10, 64, True, 128, 256, 1, 20),
    (37, 3, 5, False, 100, 96, 1, 1), (64, 8, 300, True, 64, 64, 1, 100), (130, 2, 4, True, 272, 160, 1, 1),
    (300, 4, 16, False, 130, 288, 0.5, 4), (1500, 2, 6, True, 64, 128, 2, 2),
    # more tiles than CUs, taken from the queues; long and short rows; a crowded group among empty ones
    (1200, 3, 400, True, 600, 512, 0.3, 50), (1100, 2, 300, True, 640, 384, 0, 0), (900, 6, 2047, True, 128, 256, 0.5, 900),
    (700, 3, 300, True, 576, 1024, 3, 0),
    # groups of a few rows, in more tiles than run at once; columns and matrix rows in no whole stage or strip
    (90, 4, 500, True, 1030, 200, 0.5, 100), (64, 8, 120, False, 520, 1100, 0, 0), (40, 10, 512, True, 2048, 72, 1, 0),
    (300, 2, 64, True, 2050, 129, 2, 10)]


@pytest.mark.parametrize("T,k,E,shared,N,K,skew,quiet", GROUPS)
@pytest.mark.parametrize("kind", ["bf16", "f32", "mx4"])
def test_experts_matmul(T, k, E, shared, N, K, skew, quiet, kind):
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(T * k + N)
    g = grouping_of(rng, T, k, E, shared, skew, quiet)
    off, perm, A = g.offsets.cpu().numpy(), g.perm.cpu().numpy(), T * (k + shared)
    w, wv = random_matrix(rng, (E + shared, N), K)
    terms = K * (3 if kind == "f32" else 1)
    x, xv = random_rows(rng, T, K, kind)
    ref, size = mx4_ref.grouped(xv[mx4_ref.token_rows(perm, T, k)], wv, off)
    y = moe.mx4_experts_matmul(x, w, g, tokens=T)
    check(f"experts {kind} T={T} by token", y, ref, size, terms)
    assert torch.equal(moe.mx4_experts_matmul(x, w, g, tokens=T), y)
    x, xv = random_rows(rng, A, K, kind)
    ref, size = mx4_ref.grouped(xv, wv, off)
    for dt in types().values():
        check(f"experts {kind} T={T} in order -> {dt}", moe.mx4_experts_matmul(x, w, g, dtype=dt), ref, size, terms)


@pytest.mark.parametrize("T,k,E,shared,N,K,skew,quiet", GROUPS)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_experts_matmul_backward(T, k, E, shared, N, K, skew, quiet, kind):
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(T * k + K)
    g = grouping_of(rng, T, k, E, shared, skew, quiet)
    off, perm, A = g.offsets.cpu().numpy(), g.perm.cpu().numpy(), T * (k + shared)
    w, wv = random_matrix(rng, (E + shared, N), K)
    d, dv = random_rows(rng, A, N, kind, strided=True)
    ref, size = mx4_ref.grouped(dv, wv.transpose(0, 2, 1), off)
    terms = N * (3 if kind == "f32" else 1)
    for dt in types().values():
        check(f"experts gradient {kind} T={T} in order -> {dt}", moe.mx4_experts_matmul_backward(d, w, g, dtype=dt), ref,
              size, terms)
    dx, total = np.zeros((T, K)), np.zeros((T, K))
    np.add.at(dx, mx4_ref.token_rows(perm, T, k), ref)
    np.add.at(total, mx4_ref.token_rows(perm, T, k), size)
    got = moe.mx4_experts_matmul_backward(d, w, g, tokens=T)
    assert got.shape == (T, K)
    check(f"experts gradient {kind} T={T} by token", got, dx, total, terms + k + 1)
    assert torch.equal(moe.mx4_experts_matmul_backward(d, w, g, tokens=T), got)


def test_rows_of_no_group_stay_and_bad_ids_stay_in_bounds():
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(9)
    E, N, K, A = 4, 32, 64, 40
    w, wv = random_matrix(rng, (E, N), K)
    off = torch.tensor([0, 0, 7, 7, 29, 29], dtype=torch.int32, device="cuda")
    g = moe.Grouping(torch.zeros(E + 1, dtype=torch.int32, device="cuda"), off,
                     torch.arange(A, dtype=torch.int32, device="cuda"), torch.arange(A, dtype=torch.int32, device="cuda"))
    x, xv = random_rows(rng, A, K, "bf16")
    room = torch.full((A, N), 7.0, device="cuda", dtype=torch.bfloat16)
    y = moe.mx4_experts_matmul(x, w, g, out=room)
    ref, size = mx4_ref.grouped(xv, wv, off.cpu().numpy())
    check("seven and 22 rows", y[:29], ref[:29], size[:29], K)
    assert (room[29:] == 7).all()
    d, _ = random_rows(rng, A, N, "bf16")
    room = torch.full((A, K), 7.0, device="cuda", dtype=torch.bfloat16)
    moe.mx4_experts_matmul_backward(d, w, g, out=room)
    assert (room[29:] == 7).all() and not (room[:29] == 7).all()
    # ids past the assignments read as rows of zeros
    g.perm[3], g.perm[20] = 1 << 30, -5
    y = moe.mx4_experts_matmul(x, w, g, tokens=A)
    assert not y[3].any() and not y[20].any()
    check("rows beside bad ids", y[4:20], ref[4:20], size[4:20], K)
    # offsets past the rows are cut
    g.offsets = torch.tensor([0, 0, 7, 7, 1 << 30, 29], dtype=torch.int32, device="cuda")
    ref, size = mx4_ref.grouped(xv, wv, np.array([0, 0, 7, 7, A]))
    check("a cut offset", moe.mx4_experts_matmul(x, w, g), ref, size, K)


@pytest.mark.parametrize("kind", ["f32", "bf16", "mx4"])
@pytest.mark.parametrize("E,N", [(4, 32), (300, 1000)])
def test_bad_ids_of_few_rows(E, N, kind):
    """Ids out of range and rows in no group, for each type and in more tiles than CUs: neighbours are right, the rest stays."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(E + N)
    K, A = 96, 700
    w, wv = random_matrix(rng, (E, N), K)
    off = np.minimum(np.sort(rng.integers(0, A - 60, E + 2)), A - 61).astype(np.int32)
    ids = rng.permutation(A).astype(np.int32)
    wild = rng.permutation(A)[:40]
    perm = ids.copy()
    perm[wild] = rng.choice(np.array([-1, A, 2 ** 31 - 1, -2 ** 31], np.int64), 40).astype(np.int32)
    g = moe.Grouping(torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.from_numpy(off).cuda(),
                     torch.from_numpy(perm).cuda(), torch.from_numpy(perm).cuda())
    x, xv = random_rows(rng, A, K, kind)
    room = torch.full((A, N), 7.0, device="cuda")
    y = moe.mx4_experts_matmul(x, w, g, tokens=A, dtype=torch.float32, out=room)
    ref, size = mx4_ref.grouped(xv[ids], wv, off[:E + 1])
    inside = np.zeros(A, bool)
    inside[off[0]:off[E]] = True
    tame = inside.copy()
    tame[wild] = False
    at = torch.from_numpy(np.flatnonzero(tame)).cuda()
    check(f"{kind} among bad ids", y[at], ref[tame], size[tame], K * (3 if kind == "f32" else 1))
    assert (y[torch.from_numpy(np.flatnonzero(~inside)).cuda()] == 7).all()


@pytest.mark.parametrize("K", [64, 66])
def test_gradient_of_tokens_whose_rows_are_in_no_group(K):
    """A grouping that leaves rows out at both ends: they add nothing to their tokens, whatever the workspace holds."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(K)
    E, N, T, k = 4, 32, 12, 2  # the last of the four is the shared expert
    A = T * (k + 1)
    w, wv = random_matrix(rng, (E, N), K)
    off = np.array([3, 3, 10, 22, 29, 29], np.int32)
    perm = rng.permutation(A).astype(np.int32)
    slot = np.empty(A, np.int32)
    slot[perm] = np.arange(A)
    g = moe.Grouping(torch.zeros(E, dtype=torch.int32, device="cuda"), *(torch.from_numpy(v).cuda() for v in (off, perm, slot)))
    d, dv = random_rows(rng, A, N, "bf16")
    rows, sizes = np.zeros((A, K)), np.zeros((A, K))
    for e in range(E):
        rows[off[e]:off[e + 1]] = dv[off[e]:off[e + 1]] @ wv[e]
        sizes[off[e]:off[e + 1]] = np.abs(dv[off[e]:off[e + 1]]) @ np.abs(wv[e])
    ref, size = np.zeros((T, K)), np.zeros((T, K))
    np.add.at(ref, mx4_ref.token_rows(perm, T, k), rows)
    np.add.at(size, mx4_ref.token_rows(perm, T, k), sizes)
    n = moe.lib().moe_mx4_experts_matmul_backward_workspace_size(T, k, 1, K, 1)
    room = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN
    check("rows in no group", moe.mx4_experts_matmul_backward(d, w, g, tokens=T, workspace=room), ref, size, N + k + 1)


def test_experts_refusals():
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(2)
    g = grouping_of(rng, 6, 2, 4, True)
    w, _ = random_matrix(rng, (5, 16), 64)
    x, _ = random_rows(rng, 6, 64, "bf16")
    flat, _ = random_matrix(rng, (16,), 64)
    four, _ = random_matrix(rng, (4, 16), 64)
    bad = [lambda: moe.mx4_experts_matmul(x, flat, g, tokens=6), lambda: moe.mx4_experts_matmul(x, four, g, tokens=6),
           lambda: moe.mx4_experts_matmul(x, w, g), lambda: moe.mx4_experts_matmul(x, w, g, tokens=5),
           lambda: moe.mx4_experts_matmul(x[:, :32], w, g, tokens=6), lambda: moe.mx4_experts_matmul(x[:5], w, g, tokens=6),
           lambda: moe.mx4_experts_matmul(x.t(), w, g, tokens=6), lambda: moe.mx4_matmul(x, w),
           lambda: moe.mx4_matmul(x[:, ::2], flat), lambda: moe.mx4_matmul(x[:1].expand(4, 64), flat),
           lambda: moe.mx4_matmul(x, flat, out=torch.empty(6, 17, device="cuda", dtype=torch.bfloat16)),
           lambda: moe.mx4_matmul_backward(x, flat), lambda: moe.mx4_experts_matmul_backward(x, w, g, tokens=6),
           lambda: moe.Mx4(w.codes[..., :16], w.scales, 64), lambda: moe.Mx4(w.codes, w.scales, 65),
           lambda: moe.Mx4(w.codes.transpose(0, 1), w.scales.transpose(0, 1), 64)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: moe.mx4_quantize(x.half()), lambda: moe.mx4_matmul(x.half(), flat),
              lambda: moe.mx4_matmul(x, flat, dtype=torch.float16)):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(moe.MoeError) as e:
        moe.mx4_experts_matmul_backward(torch.zeros(18, 16, device="cuda"), w, g, tokens=6,
                                        workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == moe.ERR_WORKSPACE


def test_sizes_past_the_calls_are_refused():
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    tall = torch.empty((2 ** 31 + 3, 1), dtype=torch.bfloat16, device="cuda")
    w = moe.Mx4(torch.zeros((4, 16), dtype=torch.uint8, device="cuda"), torch.zeros((4, 1), dtype=torch.uint8, device="cuda"), 1)
    for f in (lambda: moe.mx4_quantize(tall), lambda: moe.mx4_quantize(tall.view(1, -1)), lambda: moe.mx4_matmul(tall, w),
              lambda: moe.mx4_quantize(tall.view(2 ** 31 + 3, 1, 1)),
              lambda: moe.balance_loss(tall, torch.zeros((2 ** 31 + 3, 0), dtype=torch.int32, device="cuda")),
              lambda: moe.Mx4(tall.view(torch.uint8)[:, :1].contiguous().expand(-1, 16), tall.view(torch.uint8)[:, :1].contiguous(), 32)):
        with pytest.raises(ValueError):
            f()


def test_offsets_past_32_bits():
    """More than 4 GiB of codes, and more than 2^31 results: the last expert's rows and the last rows are right."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(4)
    E, N, K = 2049, 2048, 2048
    last, lv = random_matrix(rng, (N,), K)
    codes = torch.zeros((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((E, N, K // 32), dtype=torch.uint8, device="cuda")
    codes[-1], scales[-1] = last.codes, last.scales
    x, xv = random_rows(rng, 5, K, "bf16")
    off = torch.zeros(E + 2, dtype=torch.int32, device="cuda")
    off[E:] = 5
    g = moe.Grouping(torch.zeros(E + 1, dtype=torch.int32, device="cuda"), off,
                     torch.arange(5, dtype=torch.int32, device="cuda"), torch.arange(5, dtype=torch.int32, device="cuda"))
    w = moe.Mx4(codes, scales, K)
    check("last of 2049 experts", moe.mx4_experts_matmul(x, w, g), xv @ lv.T, np.abs(xv) @ np.abs(lv).T, K)
    check("its gradient", moe.mx4_experts_matmul_backward(x, w, g), xv @ lv, np.abs(xv) @ np.abs(lv), N)
    del codes, scales, w
    T, N, K = (1 << 20) + 3, 2100, 32
    w, wv = random_matrix(rng, (N,), K)
    x = torch.randn((T, K), device="cuda").bfloat16()
    y = moe.mx4_matmul(x, w)
    at = [0, T // 2, T - 1]
    xv = as64(x[at])
    check("2^31 results", y[at], xv @ wv.T, np.abs(xv) @ np.abs(wv).T, K)
