"""8-bit quantisation and products on the GPU against float64.

Quantisation is exact: codes and scales equal the reference's. A product's terms are exact in float32 (two codes have eight
significant bits together) and added up in float32, block sums times two scales: for float32 results the error is at most
(n + 3 B + 4) 2^-24 sum |x w| for n terms in B blocks (a sum of n terms in some order, and per block the product of the
scales, the product by it and one more addition), plus the rows that a token's gradient adds up. For bfloat16 results the
8-bit matrix cores may drop less than 2^-12 of a block's largest product from each (blocks_ref.cut), and the result is
rounded by half a step (finfo.eps / 2); that bound is wide for one value, so the rows' norm is held to half a step too.
"""
import numpy as np
import pytest

import blocks_ref as ref
from gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu


def lib():
    torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    return moe


def dtype_of(kind):
    torch = torch_cuda()
    return {"f32": torch.float32, "bf16": torch.bfloat16}[kind]


def as64(t) -> np.ndarray:
    return t.double().cpu().numpy()


def check(name, got, y, size, lost, n, rows_added=0):
    torch = torch_cuda()
    half = torch.finfo(got.dtype).eps / 2
    g = as64(got)
    err = (n + 3 * (-(-n // 128)) + 4 + rows_added) * 2.0 ** -24 * size
    if got.dtype == torch.bfloat16:
        err = err + lost
    bound = err + half * (np.abs(y) + err) + 1e-37
    assert g.shape == y.shape and np.isfinite(g).all(), name
    worst = np.max(np.abs(g - y) / bound, initial=0.0)
    rel = np.linalg.norm(g - y) / max(np.linalg.norm(y), 1e-300)
    log(f"[fp8] {name}: error / bound {worst:.3f}, norm {rel:.2e}")
    assert worst <= 1, name
    assert rel <= max(half, 2.0 ** -19), name


def random_fp8(rng, shape, K, block_rows=1, wide=False):
    """Rows of normal values (wide: of every magnitude) quantised by the reference: an Fp8 and its values."""
    torch, moe = torch_cuda(), lib()
    v = rng.standard_normal((*shape, K)) * np.exp(rng.standard_normal((*shape[:-1], shape[-1], 1)))
    if wide:
        v *= np.exp(1.5 * rng.standard_normal(v.shape))
    c, s = ref.quantize(v.astype(np.float32), block_rows)
    q = moe.Fp8(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), K, block_rows)
    return q, ref.values(c, s, K, block_rows)


def grouping_of(rng, T, k, E, shared, skew=0.0, quiet=0):
    torch, moe = torch_cuda(), lib()
    logits = rng.standard_normal((T, E)) - skew * np.log(1 + np.arange(E))
    if quiet:
        logits[:, rng.permutation(E)[:quiet]] -= 100
    idx, _ = moe.route_topk(torch.from_numpy(logits.astype(np.float32)).cuda(), k)
    return moe.group(idx, E, shared)


# ---- quantisation ---------------------------------------------------------------------


def nasty(rng, R, K):
    v = (rng.standard_normal((R, K)) * np.exp(4 * rng.standard_normal((R, 1)))).astype(np.float32)
    flat = v.reshape(-1)
    # a block whose scale is 1, with every border between codes, both signs, and their neighbours
    mid = np.concatenate([(ref.GRID[1:] + ref.GRID[:-1]) / 2, ref.GRID]).astype(np.float32)
    ties = np.concatenate([mid, -mid, np.nextafter(mid, np.float32(np.inf)), np.nextafter(mid, np.float32(0)), [0.0, -0.0]]).astype(np.float32)
    ties = ties[np.abs(ties) <= 448]
    flat[:min(len(ties), flat.size)] = ties[:flat.size]
    if K >= 128:
        v[0, ::128] = 448
    if R > 3:
        v[1] = 0
        v[1, ::2] = -0.0
        v[2] = v[2] / np.abs(v[2]).max() * np.float32(1e-38)
        v[3] = v[3] / np.abs(v[3]).max() * np.float32(3e38)
    if R > 6:
        v[4] = v[4] / np.abs(v[4]).max() * np.float32(2.0 ** -50)
        v[5] = np.float32(1e-44)
        v[6] = np.float32(2.0 ** -40)
    return v


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("R,K", [(1, 1), (1, 128), (3, 129), (9, 1000), (128, 256), (130, 384), (257, 130), (1000, 2048)])
def test_quantize(R, K, block, kind):
    torch, moe = torch_cuda(), lib()
    x = torch.from_numpy(nasty(np.random.default_rng(R * K), R, K)).to(dtype_of(kind)).cuda()
    c, s = ref.quantize(as64(x.float()), block)
    q = moe.fp8_quantize(x, block)
    assert np.array_equal(q.scales.cpu().numpy(), s)
    got = q.codes.view(torch.uint8).cpu().numpy()
    assert np.array_equal(got, c), np.argwhere(got != c)[:4]
    v = ref.values(c, s, K, block)
    assert np.array_equal(as64(moe.fp8_dequantize(q)), v.astype(np.float32).astype(np.float64))
    back = moe.fp8_dequantize(q, torch.bfloat16)
    assert torch.equal(back, torch.from_numpy(v.astype(np.float32)).cuda().bfloat16())


def test_quantize_short_quotients():
    """bfloat16 rows of few magnitudes: many quotients lie on a border between codes, or one rounding away from it."""
    torch, moe = torch_cuda(), lib()
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.integers(-64, 65, (4000, 128)) * 2.0 ** rng.integers(-20, 20, (4000, 1))).bfloat16().cuda()
    q = moe.fp8_quantize(x)
    c, s = ref.quantize(as64(x.float()))
    assert np.array_equal(q.scales.cpu().numpy(), s) and np.array_equal(q.codes.view(torch.uint8).cpu().numpy(), c)


def test_quantize_strided_matrices_and_nothing():
    torch, moe = torch_cuda(), lib()
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((50, 400)).astype(np.float32)).cuda()[:, 3:260]
    for block in (1, 128):
        q = moe.fp8_quantize(x, block)
        c, s = ref.quantize(as64(x), block)
        assert np.array_equal(q.codes.view(torch.uint8).cpu().numpy(), c) and np.array_equal(q.scales.cpu().numpy(), s)
    x = torch.from_numpy(rng.standard_normal((3, 2, 140, 200)).astype(np.float32)).cuda()
    for block in (1, 128):
        q = moe.fp8_quantize(x, block)
        c, s = ref.quantize(as64(x), block)
        assert q.shape == (3, 2, 140, 200)
        assert np.array_equal(q.codes.view(torch.uint8).cpu().numpy(), c) and np.array_equal(q.scales.cpu().numpy(), s)
        out = moe.fp8_quantize(torch.zeros_like(x), block, out=q)
        assert out is q and (q.codes.view(torch.uint8) == 0).all()
    for shape in ((0, 256), (4, 0, 256), (0, 7, 256)):
        assert moe.fp8_dequantize(moe.fp8_quantize(torch.empty(shape, device="cuda"), 128)).shape == shape


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_not_finite(bad):
    torch, moe = torch_cuda(), lib()
    x = torch.ones((140, 300), device="cuda")
    x[2, 130] = bad
    q = moe.fp8_quantize(x)
    v = moe.fp8_dequantize(q)
    assert torch.isnan(v[2, 128:256]).all() and not torch.isnan(v).sum() > 128
    assert (q.codes.view(torch.uint8)[2, 128:256] == 0).all() and torch.isnan(q.scales[2, 1])
    v = moe.fp8_dequantize(moe.fp8_quantize(x, 128))
    assert torch.isnan(v[:128, 128:256]).all() and torch.isnan(v).sum() == 128 * 128


# ---- products with one matrix -----------------------------------------------------------

SHAPES = [(1, 16, 128), (1, 1, 1), (1, 1024, 2048), (2, 17, 127), (5, 130, 300), (15, 64, 129), (16, 500, 1000), (17, 256, 512),
          (33, 300, 256), (64, 512, 384), (77, 500, 1000), (129, 260, 640), (300, 1024, 512), (257, 100, 2048)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_matmul(T, N, K, back, kind):
    moe = lib()
    rng = np.random.default_rng(T * N + K)
    w, wv = random_fp8(rng, (N,), K, 128)
    x, xv = random_fp8(rng, (T,), N if back else K, wide=T % 2 == 0)
    m = wv if not back else wv.T
    y, size = ref.products(xv, m)
    some = np.s_[:8] if T * N * K > 1 << 24 else np.s_[:]
    got = (moe.fp8_matmul_backward if back else moe.fp8_matmul)(x, w, dtype=dtype_of(kind))
    lost = ref.cut(xv[some], m) if kind == "bf16" else 0
    check(f"{'back' if back else 'matmul'} {T}x{N}x{K} {kind}", got[some], y[some], size[some], lost, xv.shape[1])
    again = (moe.fp8_matmul_backward if back else moe.fp8_matmul)(x, w, dtype=dtype_of(kind))
    assert bool((got == again).all())
    if kind == "f32":
        check("all rows", got, y, size, 0, xv.shape[1])


@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("back", [False, True])
def test_matmul_not_finite(T, back):
    """A NaN block of a row, or of the matrix, reaches the results that it enters and no others."""
    torch, moe = torch_cuda(), lib()
    rng = np.random.default_rng(T)
    w, _ = random_fp8(rng, (300,), 400, 128)
    x, _ = random_fp8(rng, (T,), 300 if back else 400)
    run = moe.fp8_matmul_backward if back else moe.fp8_matmul
    clean = run(x, w)
    x.scales[1, 2] = float("nan")
    y = run(x, w)
    assert torch.isnan(y[1]).all() and torch.equal(y[2:], clean[2:]) and torch.equal(y[0], clean[0])
    x.scales[1, 2] = 1.0
    clean = run(x, w)
    w.scales[1, 0] = float("inf")
    w.codes.view(torch.uint8)[128, 0] = 0
    y = run(x, w)
    hit = np.s_[:, 0:128] if back else np.s_[:, 128:256]
    assert not torch.isfinite(y[hit]).any()
    rest = torch.ones(y.shape[1], dtype=torch.bool, device="cuda")
    rest[hit[1]] = False
    assert torch.equal(y[:, rest], clean[:, rest])
    w.scales[1, 0] = 1.0
    w.codes.view(torch.uint8)[200, 5] = 0x7F
    y = run(x, w)
    col = 5 if back else 200
    assert torch.isnan(y[:, col]).all() and torch.isfinite(y[:, :col]).all() and torch.isfinite(y[:, col + 1:]).all()


def test_matmul_far_results_and_nothing():
    """No rows; results past 2^31 bytes."""
    torch, moe = torch_cuda(), lib()
    w = moe.fp8_quantize(torch.randn((256, 256), device="cuda"), 128)
    for back in (False, True):
        run = moe.fp8_matmul_backward if back else moe.fp8_matmul
        assert run(moe.fp8_quantize(torch.empty((0, 256), device="cuda")), w).shape == (0, 256)
    T = (1 << 22) - 5
    row = torch.randn((1, 256), device="cuda")
    x = moe.fp8_quantize(row.expand(T, 256).contiguous())
    y = moe.fp8_matmul(x, w, dtype=torch.float32)
    one = moe.fp8_matmul(moe.fp8_quantize(row.expand(300, 256).contiguous()), w, dtype=torch.float32)[:1]
    for part in y.split(1 << 20):
        assert torch.equal(part, one.expand_as(part))


# ---- products by expert -----------------------------------------------------------------

GROUPED = [  # T, k, E, shared, N, K, skew, quiet
    (1, 1, 1, False, 16, 128, 0, 0), (1, 10, 64, True, 64, 256, 0, 0), (4, 10, 512, True, 128, 128, 1, 0),
    (7, 3, 5, False, 33, 200, 0, 0), (40, 4, 12, True, 300, 256, 1, 3), (64, 2, 100, False, 100, 130, 0, 50),
    (200, 8, 16, True, 256, 384, 1, 2), (333, 3, 7, False, 260, 512, 0.5, 0), (700, 4, 9, True, 128, 256, 0, 0)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "x".join(map(str, c)))
def test_experts(case, back, gather, kind):
    torch, moe = torch_cuda(), lib()
    T, k, E, shared, N, K, skew, quiet = case
    rng = np.random.default_rng(T * k + E)
    grp = grouping_of(rng, T, k, E, shared, skew, quiet)
    A = T * (k + shared)
    w, wv = random_fp8(rng, (E + shared, N), K, 128)
    off, perm, slot = (t.cpu().numpy() for t in (grp.offsets, grp.perm, grp.slot_of))
    token = np.where(perm < T * k, perm // k, perm - T * k)
    rows = T if gather and not back else A
    x, xv = random_fp8(rng, (rows,), N if back else K)
    full = xv[token] if gather and not back else xv
    outs = K if back else N
    y, size, lost = np.zeros((A, outs)), np.zeros((A, outs)), np.zeros((A, outs))
    for e in range(E + shared):
        a, b = off[e], off[e + 1]
        m = wv[e].T if back else wv[e]
        y[a:b], size[a:b] = ref.products(full[a:b], m)
        if kind == "bf16":
            lost[a:b] = ref.cut(full[a:b], m)
    if gather and back:
        y, size, lost = (np.add.reduce([v[slot[:T * k].reshape(T, k)[:, j]] for j in range(k)]
                                       + ([v[slot[T * k:]]] if shared else [])) for v in (y, size, lost))
    run = moe.fp8_experts_matmul_backward if back else moe.fp8_experts_matmul
    got = run(x, w, grp, tokens=T if gather else None, dtype=dtype_of(kind))
    check(f"experts {case} back={back} gather={gather} {kind}", got, y, size, lost, xv.shape[1], k + 1)
    assert torch.equal(got, run(x, w, grp, tokens=T if gather else None, dtype=dtype_of(kind)))


@pytest.mark.parametrize("T", [5, 600])
@pytest.mark.parametrize("back", [False, True])
def test_experts_rows_behind_the_groups(T, back):
    """Groups that end early, start late and lie beyond the rows; ids out of range: other rows keep what they had."""
    torch, moe = torch_cuda(), lib()
    rng = np.random.default_rng(T)
    k, E, N, K = 4, 6, 256, 256
    grp = grouping_of(rng, T, k, E, False)
    A = T * k
    w, wv = random_fp8(rng, (E, N), K, 128)
    x, xv = random_fp8(rng, (A,), 256)
    off = grp.offsets.cpu().numpy().copy()
    off[:E + 1] = np.clip(off[:E + 1], 3, A - 7)
    off[E] = A - 7
    grp.offsets = torch.from_numpy(off).cuda()
    run = moe.fp8_experts_matmul_backward if back else moe.fp8_experts_matmul
    out = torch.full((A, 256), 7.0, device="cuda")
    got = run(x, w, grp, dtype=torch.float32, out=out)
    assert (got[:3] == 7).all() and (got[A - 7:] == 7).all()
    y, size = np.zeros((A, 256)), np.zeros((A, 256))
    for e in range(E):
        a, b = off[e], off[e + 1]
        y[a:b], size[a:b] = ref.products(xv[a:b], wv[e].T if back else wv[e])
    check("inner rows", got[3:A - 7], y[3:A - 7], size[3:A - 7], 0, 256)
    # offsets past the rows and below zero count as cut to them
    off[0], off[E] = -5, A + 1000
    grp.offsets = torch.from_numpy(off).cuda()
    got = run(x, w, grp, dtype=torch.float32)
    for e, (a, b) in ((0, (0, off[1])), (E - 1, (off[E - 1], A))):
        y, size = ref.products(xv[a:b], wv[e].T if back else wv[e])
        check("cut groups", got[a:b], y, size, 0, 256)
    if back:  # slots out of range, and of rows in no group, add nothing
        grp = grouping_of(rng, T, k, E, False)
        slot = grp.slot_of.clone()
        slot[:k] = torch.tensor([A, -1, -A, 2 ** 31 - 1], device="cuda", dtype=torch.int32)
        grp.slot_of = slot
        got = run(x, w, grp, tokens=T, dtype=torch.float32)
        assert (got[0] == 0).all() and (got[1:] != 0).any(1).all()
    else:
        grp = grouping_of(rng, T, k, E, False)
        clean = run(moe.Fp8(x.codes[:T], x.scales[:T], K), w, grp, tokens=T)
        perm = grp.perm.clone()
        perm[2], perm[A - 1] = -1, A
        grp.perm = perm
        got = run(moe.Fp8(x.codes[:T], x.scales[:T], K), w, grp, tokens=T)
        same = torch.ones(A, dtype=torch.bool, device="cuda")
        same[2] = same[A - 1] = False
        assert torch.equal(got[same], clean[same])


def test_refusals_with_tensors():
    torch, moe = torch_cuda(), lib()
    w = moe.fp8_quantize(torch.randn((64, 256), device="cuda"), 128)
    x = moe.fp8_quantize(torch.randn((4, 256), device="cuda"))
    for call in (lambda: moe.fp8_matmul(x, x), lambda: moe.fp8_matmul(w, w), lambda: moe.fp8_matmul_backward(x, w),
                 lambda: moe.fp8_matmul(x, w, out=torch.empty((4, 65), device="cuda", dtype=torch.bfloat16)),
                 lambda: moe.fp8_matmul(x, w, out=torch.empty((4, 64), device="cuda")),
                 lambda: moe.fp8_quantize(torch.randn((4, 256), device="cuda").half()),
                 lambda: moe.fp8_quantize(torch.randn((256, 4), device="cuda").t()),
                 lambda: moe.Fp8(x.codes, x.scales, 300), lambda: moe.Fp8(x.codes, x.scales, 256, 128),
                 lambda: moe.fp8_experts_matmul(x, w, None)):
        with pytest.raises((ValueError, TypeError)):
            call()
    grp = grouping_of(np.random.default_rng(0), 4, 2, 3, False)
    we = moe.fp8_quantize(torch.randn((5, 64, 256), device="cuda"), 128)
    with pytest.raises(ValueError):
        moe.fp8_experts_matmul(x, we, grp, tokens=4)
    with pytest.raises(ValueError):
        moe.fp8_experts_matmul(x, moe.fp8_quantize(torch.randn((3, 64, 256), device="cuda"), 128), grp)
