"""Every form of the microscaled products' kernels against float64 on the GPU, each case with the kernels that it has to
reach: the names of its launches are read back, so a rule that sends it elsewhere fails the test.

Tolerances as for the other products: terms are exact, a float32 sum of n of them is off by at most (n + 2) 2^-24 sum
|x w| (n three times the terms for float32 rows, which enter in three parts), then one rounding to the result's type.
"""
import numpy as np
import pytest

from gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu

CODES = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def launched(call):
    """What `call` returns, and the names of the kernels it launched."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    moe.profile_begin(64)
    out = call()
    torch.cuda.synchronize()
    return out, set(moe.profile_end())


def values(q):
    """The float64 values of an Mx4, from the format's definition."""
    torch = torch_cuda()
    table = torch.tensor(CODES + [-v for v in CODES], dtype=torch.float64, device="cuda")
    v = table[torch.stack([q.codes & 15, q.codes >> 4], -1).flatten(-2).long()]
    s = torch.exp2(q.scales.double() - 127)
    s[q.scales == 255] = float("nan")
    return (v * s.repeat_interleave(32, -1))[..., :q.K]


def random_mx4(gen, shape, K, lo=118, hi=131):
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    B = -(-K // 32)
    codes = torch.randint(0, 256, (*shape, 16 * B), generator=gen, device="cuda", dtype=torch.uint8)
    if K % 32:
        at = torch.arange(16 * B, device="cuda") * 2
        codes &= ((at < K) * 15 + (at + 1 < K) * 240).to(torch.uint8)
    return moe.Mx4(codes, torch.randint(lo, hi, (*shape, B), generator=gen, device="cuda", dtype=torch.uint8), K)


def random_rows(gen, R, n, kind, room=0):
    """Rows and their values; `room`: cut out of a wider array of NaN, that many values from one row to the next."""
    torch = torch_cuda()
    if kind == "mx4":
        q = random_mx4(gen, (R,), n)
        return q, values(q)
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    x = torch.randn((R, n), generator=gen, device="cuda").to(dt)
    if room:
        wide = torch.full((R + 2, n + room), float("nan"), device="cuda", dtype=dt)
        wide[1:-1, room // 2:room // 2 + n] = x
        x = wide[1:-1, room // 2:room // 2 + n]
    return x, x.double()


def groups(seed, T, k, E_tot, shared, quiet=0, lead=0, tail=0):
    """A grouping of T tokens' assignments, in groups of random sizes: `quiet` of them empty, rows in none at both ends."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    rng = np.random.default_rng(seed)
    A = T * (k + shared)
    weight = rng.random(E_tot) + 0.2
    weight[rng.permutation(E_tot)[:quiet]] = 0
    sizes = rng.multinomial(A - lead - tail, weight / weight.sum())
    off = np.concatenate([[lead], lead + np.cumsum(sizes), [A]]).astype(np.int32)
    perm = rng.permutation(A).astype(np.int32)
    slot = np.empty(A, np.int32)
    slot[perm] = np.arange(A)
    dev = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    g = moe.Grouping(torch.zeros(E_tot - shared + 1, dtype=torch.int32, device="cuda"), dev(off), dev(perm), dev(slot))
    return g, off, dev(np.where(perm < T * k, perm // k, perm - T * k)).long()


def grouped(x, w, off, back=False):
    """Rows x of the groups through the matrices (or, back, their transposes), and the sums of magnitudes."""
    torch = torch_cuda()
    n = w.K if back else w.codes.shape[-2]
    y = torch.zeros((x.shape[0], n), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(y)
    import bit_quantized_moe_topk_amd as moe
    for e in range(w.codes.shape[0]):
        a, b = int(off[e]), int(off[e + 1])
        if a < b:
            m = values(moe.Mx4(w.codes[e], w.scales[e], w.K))
            m = m if back else m.t().contiguous()
            y[a:b] = x[a:b] @ m
            size[a:b] = x[a:b].abs() @ m.abs()
    return y, size


def check(name, got, ref, size, terms, rows=slice(None)):
    torch = torch_cuda()
    half = torch.finfo(got.dtype).eps / 2
    sums = (terms + 2) * 2.0 ** -24 * size[rows]
    bound = sums + half * (ref[rows].abs() + sums) + 1e-37
    g = got[rows].double()
    assert g.shape == ref[rows].shape and bool(torch.isfinite(g).all()), name
    worst = float(((g - ref[rows]).abs() / bound).max()) if g.numel() else 0.0
    log(f"[mx4 forms] {name}: error / bound {worst:.3f}")
    assert worst <= 1, name


# T, k, E_tot, shared, N, K, type, kernel: more tiles than CUs, so tiles come from the queues
FORWARD = [
    (1200, 3, 201, 1, 1040, 1024, "bf16", "mx4_stream_512_wide"), (1200, 3, 201, 1, 1040, 1536, "bf16", "mx4_stream_512_wide"),
    (1200, 3, 201, 1, 1030, 2048, "bf16", "mx4_stream_512_wide"), (1500, 4, 150, 0, 2060, 512, "bf16", "mx4_stream_512_wide"),
    (1200, 3, 201, 1, 1040, 1152, "bf16", "mx4_stream_512"), (1200, 3, 301, 1, 700, 384, "bf16", "mx4_stream_512"),
    (800, 3, 80, 0, 1040, 768, "bf16", "mx4_stream_256"), (1200, 3, 301, 1, 200, 512, "bf16", "mx4_stream_256"),
    (1300, 3, 301, 1, 100, 640, "bf16", "mx4_stream_128"), (800, 3, 40, 0, 900, 256, "bf16", "mx4_stream_128"),
    (1200, 3, 201, 1, 1040, 1000, "bf16", "mx4_tiles"), (1200, 3, 201, 1, 515, 72, "bf16", "mx4_tiles"),
    (1200, 3, 201, 1, 700, 33, "bf16", "mx4_tiles"),
    (1500, 2, 30, 0, 1300, 1000, "f32", "mx4_tiles"), (1500, 2, 30, 0, 2570, 33, "f32", "mx4_tiles"),
    (1100, 3, 40, 1, 1290, 72, "f32", "mx4_tiles"), (1500, 2, 30, 0, 1300, 100, "f32", "mx4_tiles"),
    (2200, 1, 26, 1, 1300, 544, "f32", "mx4_tiles"),
    (1200, 3, 201, 1, 1040, 1024, "mx4", "mx4_tiles4_wide"), (1200, 3, 201, 1, 515, 1536, "mx4", "mx4_tiles4_wide"),
    (1200, 3, 201, 1, 1040, 640, "mx4", "mx4_tiles4_quads"), (1200, 3, 201, 1, 515, 128, "mx4", "mx4_tiles4_quads"),
    (1200, 3, 201, 1, 700, 1000, "mx4", "mx4_tiles4_wide"),
    (1200, 3, 201, 1, 1040, 1100, "mx4", "mx4_tiles4_bytes"), (1200, 3, 201, 1, 515, 33, "mx4", "mx4_tiles4_bytes"),
]


@pytest.mark.parametrize("T,k,E_tot,shared,N,K,kind,kernel", FORWARD)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_forward(T, k, E_tot, shared, N, K, kind, kernel, gather):
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    g, off, token = groups(N * K, T, k, E_tot, shared, quiet=E_tot // 8, lead=3, tail=37)
    A = T * (k + shared)
    w = random_mx4(gen, (E_tot, N), K)
    # rows that lie apart where they may (a multiple of 16 bytes apart for the streamed forms)
    x, xv = random_rows(gen, T if gather else A, K, kind, room=0 if kind == "mx4" else 16 if "stream" in kernel else 7)
    ref, size = grouped(xv[token] if gather else xv, w, off)
    if gather and kind != "mx4":  # ids that are none: their own rows alone are not specified
        wild = torch.randperm(A, generator=torch.Generator().manual_seed(K))[:20].cuda()
        g.perm[wild] = torch.tensor([-1, -2, A, 2 ** 31 - 1, -2 ** 31] * 4, dtype=torch.int32, device="cuda")
    tame = torch.zeros(A, dtype=torch.bool, device="cuda")
    tame[int(off[0]):int(off[E_tot])] = True
    outside = ~tame
    if gather and kind != "mx4":
        tame[wild] = False
    room = torch.full((A, N), 7.0, device="cuda", dtype=torch.bfloat16)
    call = lambda: moe.mx4_experts_matmul(x, w, g, tokens=T if gather else None, dtype=torch.bfloat16, out=room)  # noqa: E731
    y, names = launched(call)
    assert names == {kernel, "mx4_zero"}
    check(f"{kernel} {kind} T={T} N={N} K={K} gather={gather}", y, ref, size, K * (3 if kind == "f32" else 1), tame)
    assert bool((y[outside] == 7).all())
    first = y.clone()
    assert torch.equal(call()[tame], first[tame])
    f = moe.mx4_experts_matmul(x, w, g, tokens=T if gather else None, dtype=torch.float32)
    check(f"{kernel} {kind} -> f32", f, ref, size, K * (3 if kind == "f32" else 1), tame)


BACKWARD = [
    (1200, 3, 201, 1, 1024, 1130, "bf16", "mx4_grad_stream"), (1200, 3, 201, 1, 192, 2048, "bf16", "mx4_grad_stream"),
    (1200, 3, 301, 1, 64, 512, "bf16", "mx4_grad_stream"), (2500, 2, 30, 0, 320, 4096, "bf16", "mx4_grad_stream"),
    (1200, 3, 201, 1, 200, 1030, "bf16", "mx4_grad_tiles"), (1200, 3, 201, 1, 33, 1030, "bf16", "mx4_grad_tiles"),
    (1200, 3, 201, 1, 1000, 700, "f32", "mx4_grad_tiles"), (1200, 3, 201, 1, 33, 515, "f32", "mx4_grad_tiles"),
    (1500, 2, 30, 0, 130, 1300, "f32", "mx4_grad_tiles"), (1200, 3, 201, 1, 64, 512, "f32", "mx4_grad_tiles"),
]


@pytest.mark.parametrize("T,k,E_tot,shared,N,K,kind,kernel", BACKWARD)
def test_grouped_backward(T, k, E_tot, shared, N, K, kind, kernel):
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    g, off, token = groups(N * K, T, k, E_tot, shared, quiet=E_tot // 8, lead=3, tail=37)
    A = T * (k + shared)
    w = random_mx4(gen, (E_tot, N), K)
    d, dv = random_rows(gen, A, N, kind, room=16 if "stream" in kernel else 7)
    ref, size = grouped(dv, w, off, back=True)
    inside = torch.zeros(A, dtype=torch.bool, device="cuda")
    inside[int(off[0]):int(off[E_tot])] = True
    room = torch.full((A, K), 7.0, device="cuda", dtype=torch.bfloat16)
    terms = N * (3 if kind == "f32" else 1)
    y, names = launched(lambda: moe.mx4_experts_matmul_backward(d, w, g, dtype=torch.bfloat16, out=room))
    assert names == {kernel, "mx4_zero"}
    check(f"{kernel} {kind} T={T} N={N} K={K}", y, ref, size, terms, inside)
    assert bool((y[~inside] == 7).all())
    dx, names = launched(lambda: moe.mx4_experts_matmul_backward(d, w, g, tokens=T))
    assert names == {kernel, "mx4_zero", "mx4_sum_tokens"}
    total = torch.zeros((T, K), dtype=torch.float64, device="cuda").index_add_(0, token, ref)
    sizes = torch.zeros_like(total).index_add_(0, token, size)
    check(f"{kernel} {kind} by token", dx, total, sizes, terms + k + 1)
    assert torch.equal(moe.mx4_experts_matmul_backward(d, w, g, tokens=T), dx)


# One matrix: T, N, K, type, kernel, columns from row to row beyond K
ONE = [
    (8200, 600, 33, "f32", "mx4_tiles", 0), (8200, 600, 72, "f32", "mx4_tiles", 5), (8200, 600, 100, "f32", "mx4_tiles", 4),
    (8200, 600, 1000, "f32", "mx4_tiles", 0), (8200, 600, 1000, "f32", "mx4_tiles", 24),
    (8200, 600, 33, "bf16", "mx4_tiles", 0), (8200, 600, 1000, "bf16", "mx4_tiles", 7),
    (33000, 1030, 1536, "bf16", "mx4_stream_512_wide", 16), (20000, 1030, 1152, "bf16", "mx4_stream_512", 16),
    (1000, 600, 1000, "f32", "mx4_few", 3), (1200, 600, 72, "f32", "mx4_few", 0), (50, 600, 100, "f32", "mx4_rows", 9),
]


@pytest.mark.parametrize("T,N,K,kind,kernel,room", ONE)
def test_one_matrix(T, N, K, kind, kernel, room):
    """Ragged columns, strides and rows among NaN; NaN, infinite, huge and small values reach their own results alone."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    gen = torch.Generator(device="cuda").manual_seed(T + N + K)
    w = random_mx4(gen, (N,), K)
    x, _ = random_rows(gen, T, K, kind, room=room)
    w.scales[7, 0], w.scales[N - 1, -1] = 255, 255
    w.codes[:, 4] = torch.randint(0, 2, (N,), generator=gen, device="cuda", dtype=torch.uint8) * 0x22  # columns 8 and 9: 0 or 1
    x[T - 1, K - 1], x[4, 9] = float("nan"), float("inf")
    x[6] *= 2.0 ** 100
    x[8] *= 2.0 ** -90
    y, names = launched(lambda: moe.mx4_matmul(x, w, dtype=torch.float32))
    assert names == {kernel}
    wv = values(w)
    assert bool(y[T - 1].isnan().all()) and bool(y[:, [7, N - 1]].isnan().all())
    fine = torch.ones(N, dtype=torch.bool, device="cuda")
    fine[[7, N - 1]] = False
    zero = wv[:, 9] == 0
    assert bool(y[4][fine & zero].isnan().all()) and bool(y[4][fine & ~zero].isinf().all())
    rows = torch.ones(T, dtype=torch.bool, device="cuda")
    rows[[4, T - 1]] = False
    xv, m = x[rows].double(), wv[fine].t().contiguous()
    check(f"{kernel} {kind} T={T} N={N} K={K} among NaN", y[rows][:, fine], xv @ m, xv.abs() @ m.abs(),
          K * (3 if kind == "f32" else 1))


# Float32 rows of one 24-bit value each, weights powers of two: a result is one product, which float32 holds, so the
# three parts that a value enters in have to add up to it bit by bit.
EXACT = [  # T, N, K, experts (0: one matrix), kernel forward, kernel backward
    (5, 70, 100, 0, "mx4_rows", "mx4_rows_grad"), (1000, 600, 130, 0, "mx4_few", "mx4_rows_grad"),
    (8200, 600, 100, 0, "mx4_tiles", "mx4_rows_grad"), (8200, 100, 1200, 0, "mx4_few", "mx4_grad_tiles"),
    (8200, 64, 1024, 0, "mx4_few", "mx4_grad_tiles"), (20, 64, 96, 6, "mx4_rows", "mx4_rows_grad"),
    (600, 515, 96, 40, "mx4_few", "mx4_grad_tiles"), (3000, 1300, 160, 30, "mx4_tiles", "mx4_grad_tiles"),
]


def lone_values(gen, T, n):
    """[T, n] float32, one value a row that is not 0, of 24 significant bits, within 2^-20 .. 2^20; its column."""
    torch = torch_cuda()
    at = torch.randint(0, n, (T,), generator=gen, device="cuda")
    odd = torch.randint(2 ** 22, 2 ** 23, (T,), generator=gen, device="cuda") * 2 + 1
    sign = torch.randint(0, 2, (T,), generator=gen, device="cuda") * 2 - 1
    v = (sign * odd).double() * torch.exp2(torch.randint(-43, -3, (T,), generator=gen, device="cuda").double())
    return torch.zeros((T, n), device="cuda").index_put_((torch.arange(T, device="cuda"), at), v.float()), at


@pytest.mark.parametrize("T,N,K,E,forward,backward", EXACT)
def test_float32_values_enter_whole(T, N, K, E, forward, backward):
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    gen = torch.Generator(device="cuda").manual_seed(T + N + K)
    w = random_mx4(gen, (max(E, 1), N), K)
    powers = torch.tensor([1, 2, 4, 6, 9, 10, 12, 14], dtype=torch.uint8, device="cuda")  # of 1/2, 1, 2, 4
    pick = lambda: powers[torch.randint(0, 8, w.codes.shape, generator=gen, device="cuda")]  # noqa: E731
    there = torch.arange(32 * w.scales.shape[-1], device="cuda").view(-1, 2) < K
    w = moe.Mx4(pick() * there[:, 0] | (pick() * there[:, 1]) << 4, w.scales, K)
    wv = values(w)
    if E:
        g, off, _ = groups(T, T, 1, E, 0, quiet=2)
        of = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.from_numpy(np.diff(off[:E + 1])).cuda())
        f, b = lambda x: moe.mx4_experts_matmul(x, w, g), lambda d: moe.mx4_experts_matmul_backward(d, w, g)
    else:
        one = moe.Mx4(w.codes[0], w.scales[0], K)
        of = torch.zeros(T, dtype=torch.long, device="cuda")
        f, b = lambda x: moe.mx4_matmul(x, one), lambda d: moe.mx4_matmul_backward(d, one)
    x, at = lone_values(gen, T, K)
    y, names = launched(lambda: f(x))
    assert names - {"mx4_zero"} == {forward}
    assert torch.equal(y.double(), x.double().sum(1, keepdim=True) * wv[of, :, at])
    d, at = lone_values(gen, T, N)
    dx, names = launched(lambda: b(d))
    assert names - {"mx4_zero"} == {backward}
    assert torch.equal(dx.double(), d.double().sum(1, keepdim=True) * wv[of, at])
