"""The ends of the number range in the microscaled products: weights of 2^128 and more (scale bytes 253 and 254), and
float32 values whose low bits lie below what a bfloat16 part can hold."""
import numpy as np
import pytest

from gpu_util import torch_cuda
from test_gpu_mx4_forms import EXACT, check, groups, launched, lone_values, random_mx4, random_rows, values

pytestmark = pytest.mark.gpu

# T, N, K, experts (0: one matrix), type, kernel forward, kernel backward: each kernel that takes float32 or bf16 rows
FORMS = [(T, N, K, E, "f32", f, b) for T, N, K, E, f, b in EXACT] + [
    (5, 70, 100, 0, "bf16", "mx4_rows", "mx4_rows_grad"), (8200, 600, 100, 0, "bf16", "mx4_tiles", "mx4_rows_grad"),
    (8200, 1030, 1024, 0, "bf16", "mx4_stream_256", "mx4_grad_tiles"), (400, 1030, 96, 40, "bf16", "mx4_few", "mx4_grad_tiles"),
    (3000, 320, 512, 30, "bf16", "mx4_stream_128", "mx4_grad_stream")]


def calls(gen, w, T, E, seed):
    """The two products with the experts w (E of them, or one matrix), and the expert of each row."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    if not E:
        one = moe.Mx4(w.codes[0], w.scales[0], w.K)
        return lambda x: moe.mx4_matmul(x, one, dtype=torch.float32), \
            lambda d: moe.mx4_matmul_backward(d, one, dtype=torch.float32), torch.zeros(T, dtype=torch.long, device="cuda")
    g, off, _ = groups(seed, T, 1, E, 0, quiet=2)
    of = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.from_numpy(np.diff(off[:E + 1])).cuda())
    return lambda x: moe.mx4_experts_matmul(x, w, g, dtype=torch.float32), \
        lambda d: moe.mx4_experts_matmul_backward(d, w, g, dtype=torch.float32), of


def classes(x, m, of):
    """Of every result of rows x with matrices m [E, in, out]: the finite sum, its magnitudes, and how many terms are
    +infinity, -infinity and NaN (0 times infinity), where weights from 2^128 on are infinite."""
    torch = torch_cuda()
    big = m.abs() >= 2.0 ** 128
    parts = [torch.where(big, 0.0, m), torch.where(big, 0.0, m).abs(), (big & (m > 0)).double(), (big & (m < 0)).double(), big.double()]
    out = [torch.empty((x.shape[0], m.shape[2]), dtype=torch.float64, device="cuda") for _ in range(5)]
    pos, neg, nil = (x > 0).double(), (x < 0).double(), (x == 0).double()
    for e in of.unique().tolist():
        r = of == e
        p = [t[e].contiguous() for t in parts]
        out[0][r], out[1][r] = x[r] @ p[0], x[r].abs() @ p[1]
        out[2][r], out[3][r], out[4][r] = pos[r] @ p[2] + neg[r] @ p[3], pos[r] @ p[3] + neg[r] @ p[2], nil[r] @ p[4]
    return out


@pytest.mark.parametrize("T,N,K,E,kind,forward,backward", FORMS)
def test_infinite_weights(T, N, K, E, kind, forward, backward):
    """Infinite weights make the results that they reach infinite, NaN where they meet a zero or one another (with float32
    rows: one of the two), and leave the others as they are."""
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(T + N + K)
    w = random_mx4(gen, (max(E, 1), N), K, 110, 118)
    some = torch.rand(w.scales.shape, generator=gen, device="cuda") < 1.0 / N
    some[:, 1] = False
    w.scales[some] = torch.randint(253, 255, (int(some.sum()),), generator=gen, device="cuda", dtype=torch.uint8)
    w.scales[:, 1, 0] = 254
    w.codes[:, 1, :16] = 0  # 0, 6, 1, 0, 0, -6, and zeros: one positive and one negative infinity
    w.codes[:, 1, :3] = torch.tensor([0x70, 0x02, 0xF0], dtype=torch.uint8, device="cuda")
    m = values(w)
    f, b, of = calls(gen, w, T, E, T)
    for n, call, mats, kernel in ((K, f, m.transpose(1, 2), forward), (N, b, m, backward)):
        x, xv = random_rows(gen, T, n, kind)
        x[:, : n // 2] = x[:, : n // 2].bfloat16().to(x.dtype)  # values without lower parts
        x[0, 1] = x[T - 1, 0] = 0
        xv = x.double()
        y, names = launched(lambda: call(x))
        assert names - {"mx4_zero"} == {kernel}
        ref, size, pos, neg, nan = classes(xv, mats, of)
        # finite weights of the two top bytes reach 2^127 x: results past float32 are infinite too
        bad = (nan > 0) | ((pos > 0) & (neg > 0))
        reached = (pos > 0) | (neg > 0) | (nan > 0)
        assert not bool(y[reached].isfinite().any())
        if kind == "bf16":
            assert bool(y[bad].isnan().all())
            assert bool((y[(pos > 0) & ~bad & (size < 2.0 ** 127)] == float("inf")).all())
            assert bool((y[(neg > 0) & ~bad & (size < 2.0 ** 127)] == -float("inf")).all())
        rest = ~reached & (size < 2.0 ** 127)
        assert bool(rest.any()) and bool(bad.any()) and bool(((pos > 0) & ~bad).any())
        bound = ((3 * n + 2) * 2.0 ** -24 * size + 2.0 ** -24 * ref.abs() + 1e-37)[rest]
        assert bool(((y[rest].double() - ref[rest]).abs() <= bound).all())


@pytest.mark.parametrize("T,N,K,E,kernel", [(20, 70, 100, 0, "mx4_rows"), (1100, 1040, 512, 0, "mx4_tiles4_wide"), (700, 300, 384, 4, "mx4_tiles4_quads")])
def test_large_weights_with_four_bit_rows(T, N, K, E, kernel):
    """Against microscaled rows the same weights are what they are: scales meet as exponents."""
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(T)
    w = random_mx4(gen, (max(E, 1), N), K, 245, 255)
    x = random_mx4(gen, (T,), K, 20, 40)
    f, _, of = calls(gen, w, T, E, T)
    y, names = launched(lambda: f(x))
    assert names == {kernel}
    xv, m = values(x), values(w)
    for e in of.unique().tolist():
        r = of == e
        check(f"{kernel} expert {e}", y[r], xv[r] @ m[e].t().contiguous(), xv[r].abs() @ m[e].abs().t().contiguous(), K)


@pytest.mark.parametrize("T,N,K,E,forward,backward", EXACT)
def test_small_float32_values(T, N, K, E, forward, backward):
    """One value a row, weights powers of two: values from 2^-110 on enter whole, smaller ones to within 2^-133, and the
    product is one float32 (its exponent far from either end here)."""
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(T + N + K)
    w = random_mx4(gen, (max(E, 1), N), K, 200, 220)
    powers = torch.tensor([2, 4, 10, 12], dtype=torch.uint8, device="cuda")  # of 1, 2
    nibble = powers[torch.randint(0, 4, (*w.codes.shape, 2), generator=gen, device="cuda")]
    there = torch.arange(32 * w.scales.shape[-1], device="cuda").view(-1, 2) < K
    w.codes.copy_(nibble[..., 0] * there[:, 0] | (nibble[..., 1] * there[:, 1]) << 4)
    m = values(w)
    f, b, of = calls(gen, w, T, E, T)
    for n, call, kernel, back in ((K, f, forward, False), (N, b, backward, True)):
        x, at = lone_values(gen, T, n)
        x = (x.double() * 2.0 ** -110 * torch.exp2(-torch.randint(0, 24, (T, 1), generator=gen, device="cuda").double())).float()
        x[:T // 2] *= 2.0 ** 44  # one half from 2^-110 on, and one row below for sure
        x[T - 1] = torch.where(x[T - 1] != 0, (1 + 2.0 ** -20) * 2.0 ** -120, 0.0)
        y, names = launched(lambda: call(x))
        assert names - {"mx4_zero"} == {kernel}
        v = x.double().sum(1, keepdim=True)
        weight = m[of, at] if back else m[of, :, at]
        off = (y.double() - v * weight).abs()
        large = (v.abs() >= 2.0 ** -110).squeeze(1)
        assert bool(large.any()) and bool((~large).any()) and not bool(off[large].any())
        assert bool((off <= (2.0 ** -133 + 2.0 ** -24 * v.abs()) * weight.abs()).all())
