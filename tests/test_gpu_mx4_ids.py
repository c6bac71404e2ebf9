"""Offsets outside the rows, as the header describes them: they count as cut to the rows."""
import numpy as np
import pytest

from gpu_util import torch_cuda
from test_gpu_mx4_forms import check, grouped, random_mx4, random_rows

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
