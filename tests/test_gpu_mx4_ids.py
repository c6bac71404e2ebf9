"""Offsets and ids outside their range, as the header describes them: offsets count as cut to the rows, the row of an id
that is none is a row of zeros or not specified, and its neighbours are right."""
import numpy as np
import pytest

from gpu_util import torch_cuda
from test_gpu_mx4_forms import check, grouped, launched, random_mx4, random_rows

pytestmark = pytest.mark.gpu


def grouping(off, perm):
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    dev = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32).cuda()  # noqa: E731
    return moe.Grouping(torch.zeros(len(off) - 1, dtype=torch.int32, device="cuda"), dev(off), dev(perm), dev(perm))


# offsets (one more than groups, and one that is not looked at), rows: few rows for the units, more for the tiles
OFFSETS = [([-5, -3, 10, 10, 30, 30], 30), ([-2 ** 31, -1, -1, 5, 24, 30], 30), ([-40, -17, 3, 28, 2 ** 31 - 1, 0], 30),
           ([-7, -2, 250, 250, 2000, 0], 900), ([-2 ** 31, -2 ** 31, -9, 600, 700, 0], 900)]


@pytest.mark.parametrize("off,A", OFFSETS)
@pytest.mark.parametrize("kind", ["bf16", "f32", "mx4"])
def test_offsets_are_cut(off, A, kind):
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    gen = torch.Generator(device="cuda").manual_seed(A)
    E, N, K = 4, 48, 96
    w = random_mx4(gen, (E, N), K)
    g = grouping(off, np.arange(A))
    cut = np.clip(np.array(off, np.int64), 0, A)
    inside = torch.zeros(A, dtype=torch.bool, device="cuda")
    inside[cut[0]:cut[E]] = True
    for back in (False, True)[: 1 if kind == "mx4" else 2]:
        x, xv = random_rows(gen, A, N if back else K, kind)
        ref, size = grouped(xv, w, cut, back)
        out = torch.full(ref.shape, 7.0, device="cuda")
        call = moe.mx4_experts_matmul_backward if back else moe.mx4_experts_matmul
        y = call(x, w, g, dtype=torch.float32, out=out)
        check(f"{kind} back={back} {off}", y, ref, size, (N if back else K) * 3, inside)
        assert bool((y[~inside] == 7).all())


@pytest.mark.parametrize("T,k,E,N,kind,kernel", [(8, 3, 4, 40, "bf16", "mx4_rows"), (8, 3, 4, 40, "f32", "mx4_rows"), (8, 3, 4, 40, "mx4", "mx4_rows"),
                                                 (200, 3, 60, 1000, "bf16", "mx4_few"), (200, 3, 60, 600, "f32", "mx4_few"),
                                                 (400, 3, 20, 600, "bf16", "mx4_tiles"), (400, 3, 6, 600, "f32", "mx4_tiles")])
def test_negative_ids_are_rows_of_zeros(T, k, E, N, kind, kernel):
    """-1 to -(k - 1) divided by k round to 0: they are no ids of token 0."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    gen = torch.Generator(device="cuda").manual_seed(T)
    K, A = 100, T * k
    w = random_mx4(gen, (E, N), K)
    off = np.concatenate([np.linspace(0, A, E + 1).astype(np.int64), [A]])
    perm = np.random.default_rng(T).permutation(A)
    bad = np.arange(0, A, 5)
    perm[bad] = np.resize([-1, -2, -k, A, A + 1], len(bad))
    g = grouping(off, perm)
    x, xv = random_rows(gen, T, K, kind)
    at = torch.from_numpy(np.where((perm >= 0) & (perm < A), perm // k, 0)).cuda()
    ref, size = grouped(xv[at], w, off)
    y, names = launched(lambda: moe.mx4_experts_matmul(x, w, g, tokens=T, dtype=torch.float32))
    assert names == {kernel}
    wrong = torch.zeros(A, dtype=torch.bool, device="cuda")
    wrong[torch.from_numpy(bad).cuda()] = True
    check(f"{kernel} {kind}", y, ref, size, 3 * K, ~wrong)
    assert not bool(y[wrong].any())
