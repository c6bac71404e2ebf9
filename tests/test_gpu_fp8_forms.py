"""Every kernel of the 8-bit products, named: each case has to run the one that it is for, in both result types, and agrees with
float64 as in test_gpu_blocks (whose bounds these are); rows and matrices past 4 GiB."""
import numpy as np
import pytest

import blocks_ref as ref
from gpu_util import log, torch_cuda
from test_gpu_blocks import as64, check, dtype_of, grouping_of, lib, random_fp8

pytestmark = pytest.mark.gpu

DENSE = [  # kernel, T, N, K of the stored matrix, back
    ("f8_rows", 16, 40, 700, False), ("f8_tiles_strip128", 31, 9000, 300, False), ("f8_rows", 1, 300, 2000, False),
    ("f8_rows", 32, 130, 129, False), ("f8_rows", 200, 500, 1300, False), ("f8_rows", 47, 5000, 1300, False),
    ("f8_tiles_strip128", 20, 8300, 129, False), ("f8_tiles_strip128", 700, 700, 1300, False),
    ("f8_tiles", 2000, 4100, 260, False), ("f8_tiles", 4097, 2048, 130, False), ("f8_tiles", 8300, 1030, 100, False),
    ("f8_tiles_back_strip128", 1, 300, 130, True), ("f8_tiles_back_strip128", 150, 1300, 500, True),
    ("f8_tiles_back", 2000, 260, 4100, True), ("f8_tiles_back", 4097, 130, 2048, True), ("f8_tiles_back", 8300, 100, 1030, True)]


def run_named(name, call):
    """The call's result, and that its product ran on kernel `name`."""
    moe = lib()
    moe.profile_begin(64)
    y = call()
    torch_cuda().cuda.synchronize()
    ran = [k for k in moe.profile_end() if k not in ("mx4_zero", "mx4_sum_tokens")]
    assert ran == [name], (ran, name)
    return y


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("case", DENSE, ids=lambda c: "-".join(map(str, c)))
def test_dense(case, kind):
    moe = lib()
    name, T, N, K, back = case
    rng = np.random.default_rng(T + N)
    w, wv = random_fp8(rng, (N,), K, 128)
    x, xv = random_fp8(rng, (T,), N if back else K)
    got = run_named(name, lambda: (moe.fp8_matmul_backward if back else moe.fp8_matmul)(x, w, dtype=dtype_of(kind)))
    m = wv.T if back else wv
    y, size = ref.products(xv, m)
    if kind == "f32":
        check(name, got, y, size, 0, xv.shape[1])
        return
    # the bound of what the 8-bit cores drop, at some rows and results; the norm of all
    n = m.shape[0]
    rows, cols = np.unique(np.r_[:4, T - 4:T, rng.integers(0, T, 12)].clip(0, T - 1)), np.unique(np.r_[:64, n - 70:n].clip(0, n - 1))
    check(name, got[rows.tolist()][:, cols.tolist()], y[np.ix_(rows, cols)], size[np.ix_(rows, cols)], ref.cut(xv[rows], m[cols]), xv.shape[1])
    off = np.linalg.norm(as64(got) - y, axis=1) / np.linalg.norm(y, axis=1)
    assert off.max() <= 2.0 ** -8, off.max()


GROUPED = [  # kernel, T, k, E, shared, N, K, back
    ("f8_rows", 3, 2, 9, True, 130, 260, False), ("f8_rows", 30, 1, 2, False, 530, 700, False),
    ("f8_tiles_strip128", 3, 2, 9, True, 2000, 260, False), ("f8_tiles_strip128", 300, 4, 6, False, 384, 640, False),
    ("f8_tiles", 900, 2, 40, True, 2300, 200, False), ("f8_tiles_192", 900, 3, 16, True, 3100, 200, False),
    ("f8_tiles_192", 1500, 2, 20, False, 3000, 400, False),
    ("f8_tiles_back_strip128", 3, 2, 9, True, 130, 260, True), ("f8_tiles_back_strip128", 300, 4, 6, False, 384, 640, True),
    ("f8_tiles_back", 900, 2, 40, True, 200, 2300, True), ("f8_tiles_back", 700, 3, 64, False, 800, 2100, True),
    ("f8_tiles_back_192", 900, 3, 16, True, 200, 3100, True),
    ("f8_tiles_back_192", 1500, 2, 20, False, 400, 3000, True)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "-".join(map(str, c)))
def test_grouped(case, gather, kind):
    torch, moe = torch_cuda(), lib()
    name, T, k, E, shared, N, K, back = case
    rng = np.random.default_rng(T + N)
    grp = grouping_of(rng, T, k, E, shared, 0.3)
    A = T * (k + shared)
    w, wv = random_fp8(rng, (E + shared, N), K, 128)
    off, perm, slot = (t.cpu().numpy() for t in (grp.offsets, grp.perm, grp.slot_of))
    token = np.where(perm < T * k, perm // k, perm - T * k)
    x, xv = random_fp8(rng, (T if gather and not back else A,), N if back else K)
    full = xv[token] if gather and not back else xv
    outs = K if back else N
    y, size = np.zeros((A, outs)), np.zeros((A, outs))
    for e in range(E + shared):
        y[off[e]:off[e + 1]], size[off[e]:off[e + 1]] = ref.products(full[off[e]:off[e + 1]], wv[e].T if back else wv[e])
    if gather and back:
        parts = lambda v: np.add.reduce([v[slot[:T * k].reshape(T, k)[:, j]] for j in range(k)] + ([v[slot[T * k:]]] if shared else []))  # noqa: E731
        y, size = parts(y), parts(size)
    run = moe.fp8_experts_matmul_backward if back else moe.fp8_experts_matmul
    got = run_named(name, lambda: run(x, w, grp, tokens=T if gather else None, dtype=dtype_of(kind)))
    if kind == "f32":
        check(f"{name} {gather}", got, y, size, 0, xv.shape[1], k + 1)
    else:
        off = np.linalg.norm(as64(got) - y, axis=1) / np.linalg.norm(y, axis=1)
        log(f"[fp8] {name} {gather}: rows' norm {off.max():.2e}")
        assert off.max() <= 2.0 ** -8
    again = run(x, w, grp, tokens=T if gather else None, dtype=dtype_of(kind))
    assert torch.equal(got, again)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("back", [False, True])
def test_past_4_gib(back, kind):
    """Rows of codes past 2^32 bytes, and a matrix of that size, run on the rows' kernels, with 64-bit offsets."""
    torch, moe = torch_cuda(), lib()
    rng = np.random.default_rng(1)
    wide, T = 4096, (1 << 20) + 100
    few = 16
    w, wv = random_fp8(rng, (wide, ) if back else (few, ), few if back else wide, 128)
    x, xv = random_fp8(rng, (64,), wide)
    index = torch.arange(T, device="cuda") * 7 % 64
    rows = moe.Fp8(x.codes.view(torch.uint8)[index].view(torch.float8_e4m3fn), x.scales[index], wide)
    name = "f8_rows_back" if back else "f8_rows"
    got = run_named(name, lambda: (moe.fp8_matmul_backward if back else moe.fp8_matmul)(rows, w, dtype=dtype_of(kind)))
    m = wv.T if back else wv
    y, size = ref.products(xv, m)
    lost = ref.cut(xv, m) if kind == "bf16" else 0
    first = got[:64][torch.argsort(index[:64])]
    check(name, first, y, size, lost, wide)
    for part, at in zip(got.split(1 << 18), index.split(1 << 18)):
        assert torch.equal(part, first[at])
    if kind == "bf16" and not back:  # a matrix of 2^19 x 8300 codes
        N, K = 1 << 19, 8300
        m, mv = random_fp8(rng, (128,), K, 128)
        B = -(-K // 128)
        big = moe.Fp8(m.codes.view(torch.uint8).repeat(N // 128, 1).view(torch.float8_e4m3fn), m.scales.repeat(N // 128, 1), K, 128)
        x, xv = random_fp8(rng, (40,), K)
        got = run_named("f8_rows", lambda: moe.fp8_matmul(x, big))
        y, size = ref.products(xv, mv)
        check("matrix", got[:, :128], y, size, ref.cut(xv, mv), K)
        assert torch.equal(got.view(40, N // 128, 128), got[:, None, :128].expand(40, N // 128, 128))
