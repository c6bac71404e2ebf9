"""Every result of every kernel of the 8-bit products in bfloat16, element by element. Codes are whole numbers from -4 to 4, so that a
block's products are at most 16, and their sums at most 2^11: the 8-bit cores, which keep 13 bits below the largest product, drop
nothing, and block sums are exact. What is left is (3 B + 4 + rows added) 2^-24 sum |x w| of the scaled sums of B blocks and half a step
of bfloat16. (Any other codes are cut within a block, by a bound that is wide for one element: test_gpu_blocks.)"""
import numpy as np
import pytest

import blocks_ref as ref
from gpu_util import log, torch_cuda
from test_gpu_blocks import as64, grouping_of, lib
from test_gpu_fp8_forms import DENSE, GROUPED, run_named

pytestmark = pytest.mark.gpu
WHOLE = np.array([int(np.argwhere(ref.GRID == m)[0, 0]) for m in range(5)], np.uint8)  # the codes of 0 .. 4


def whole_fp8(rng, shape, K, block_rows=1):
    """Rows of codes of whole numbers with scales of their own: an Fp8 and its values."""
    torch, moe = torch_cuda(), lib()
    B = -(-K // 128)
    v = rng.integers(-4, 5, (*shape, K))
    c = np.zeros((*shape, 128 * B), np.uint8)
    c[..., :K] = WHOLE[np.abs(v)] + np.where(v < 0, 128, 0).astype(np.uint8)
    s = np.exp(rng.standard_normal((*shape[:-1], -(-shape[-1] // block_rows), B))).astype(np.float32)
    q = moe.Fp8(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), K, block_rows)
    return q, ref.values(c, s, K, block_rows)


def check(name, got, y, size, n, rows_added=0):
    g = as64(got)
    err = (3 * -(-n // 128) + 4 + rows_added) * 2.0 ** -24 * size
    worst = np.max(np.abs(g - y) / (err + 2.0 ** -8 * (np.abs(y) + err) + 1e-37))
    log(f"[fp8] elements {name}: {worst:.3f}")
    assert g.shape == y.shape and worst <= 1, name


@pytest.mark.parametrize("case", DENSE, ids=lambda c: "-".join(map(str, c)))
def test_dense_elements(case):
    moe = lib()
    name, T, N, K, back = case
    rng = np.random.default_rng(T + K)
    w, wv = whole_fp8(rng, (N,), K, 128)
    x, xv = whole_fp8(rng, (T,), N if back else K)
    got = run_named(name, lambda: (moe.fp8_matmul_backward if back else moe.fp8_matmul)(x, w))
    y, size = ref.products(xv, wv.T if back else wv)
    check(name, got, y, size, xv.shape[1])


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "-".join(map(str, c)))
def test_grouped_elements(case, gather):
    moe = lib()
    name, T, k, E, shared, N, K, back = case
    rng = np.random.default_rng(T + K)
    grp = grouping_of(rng, T, k, E, shared, 0.3)
    A = T * (k + shared)
    w, wv = whole_fp8(rng, (E + shared, N), K, 128)
    off, perm, slot = (t.cpu().numpy() for t in (grp.offsets, grp.perm, grp.slot_of))
    token = np.where(perm < T * k, perm // k, perm - T * k)
    x, xv = whole_fp8(rng, (T if gather and not back else A,), N if back else K)
    full = xv[token] if gather and not back else xv
    outs = K if back else N
    y, size = np.zeros((A, outs)), np.zeros((A, outs))
    for e in range(E + shared):
        y[off[e]:off[e + 1]], size[off[e]:off[e + 1]] = ref.products(full[off[e]:off[e + 1]], wv[e].T if back else wv[e])
    if gather and back:
        parts = lambda v: np.add.reduce([v[slot[:T * k].reshape(T, k)[:, j]] for j in range(k)] + ([v[slot[T * k:]]] if shared else []))  # noqa: E731
        y, size = parts(y), parts(size)
    run = moe.fp8_experts_matmul_backward if back else moe.fp8_experts_matmul
    got = run_named(name, lambda: run(x, w, grp, tokens=T if gather else None))
    check(f"{name} {gather}", got, y, size, xv.shape[1], k + 1)
