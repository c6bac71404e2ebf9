"""Results that lie over operands are refused on the host by the microscaled products, the quantiser and the balance
loss's gradient; results beside them, or in the gaps between rows, are not. (Nothing is launched: where a call would be
taken, a last argument that is checked later is wrong, or there is no GPU to launch on.)"""
import ctypes as C
import os

import pytest
import torch

moe = pytest.importorskip("bit_quantized_moe_topk_amd")
if not os.path.exists(moe.LIB_PATH):
    pytest.skip("libmoe.so not built (run __graft_entry__.build())", allow_module_level=True)
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: not where a call that is taken would launch")

INV = moe.ERR_INVALID_ARG
MB = 1 << 20
X, XS, W, WS, Y, G, ROOM = (i * 64 * MB for i in range(1, 8))  # far apart


def P(a):
    return C.c_void_p(a)


def product(back, T=64, N=256, K=512, ld=None, **at):
    a = dict(x=X, wc=W, ws=WS, y=Y, xs=None, t=moe.BF16)
    a.update(at)
    L = moe.lib()
    if back:
        return L.moe_mx4_matmul_backward(P(a["x"]), a["t"], ld or N, T, P(a["wc"]), P(a["ws"]), N, K, P(a["y"]), moe.BF16, None)
    return L.moe_mx4_matmul(P(a["x"]), P(a["xs"]), a["t"], ld or K, T, P(a["wc"]), P(a["ws"]), N, K, P(a["y"]), moe.BF16, None)


@pytest.mark.parametrize("back", [False, True])
def test_products(back):
    n_in, n_out = (256, 512) if back else (512, 256)
    x, y, codes, scales = 64 * n_in * 2, 64 * n_out * 2, 256 * 512 // 2, 256 * 512 // 32
    assert product(back) != INV
    for base, size in ((X, x), (W, codes), (WS, scales)):
        for at in (base, base + 16, base + size - 16, base - 16, base - y + 16):
            assert product(back, y=at) == INV, (base, at)
        assert product(back, y=base + size) != INV and product(back, y=base - y) != INV
    # between two rows that lie far apart there is room for results, over one of them there is none
    step = 2 * y
    assert product(back, ld=step // 2, y=X + step + 2 * n_in) != INV
    assert product(back, ld=step // 2, y=X + 5 * step - 16) == INV
    assert product(back, ld=step // 2, y=X + 64 * step) != INV
    assert product(back, ld=step // 2, y=X + 63 * step + 2 * n_in) != INV
    assert product(back, ld=step // 2, y=X + 63 * step + 2 * n_in - 16) == INV


def test_four_bit_rows():
    at = dict(t=moe.MX4, xs=XS)
    assert product(False, **at) != INV
    for y in (X, X + 64 * 256 - 16, XS, XS + 64 * 16 - 2):
        assert product(False, y=y, **at) == INV
    assert product(False, y=X + 64 * 256, **at) != INV and product(False, y=XS + 64 * 16, **at) != INV


@pytest.mark.parametrize("gather", [0, 1])
def test_experts(gather):
    T, k, E, N, K = 1024, 2, 4, 64, 128
    A, L = T * (k + 1), moe.lib()

    def forward(y=Y, ws=ROOM):
        n = L.moe_mx4_experts_matmul_workspace_size(T, k, 1)
        return L.moe_mx4_experts_matmul(P(X), None, moe.BF16, K, T, k, E, 1, gather, P(G), P(G), P(W), P(WS), N, K, P(y),
                                        moe.BF16, P(ws), n, None)

    def backward(dx=Y, ws=ROOM):
        n = L.moe_mx4_experts_matmul_backward_workspace_size(T, k, 1, K, gather)
        return L.moe_mx4_experts_matmul_backward(P(X), moe.BF16, N, T, k, E, 1, gather, P(G), P(G), P(W), P(WS), N, K, P(dx),
                                                 moe.BF16, P(ws), n, None)

    assert forward() != INV and backward() != INV
    assert forward(y=X) == INV and forward(ws=X) == INV and forward(y=W + 16) == INV and forward(y=ROOM + 16) == INV
    assert forward(y=W + 5 * N * K // 2 - 16) == INV and forward(y=W + 5 * N * K // 2) != INV   # the shared matrix's end
    assert forward(y=X + (T if gather else A) * K * 2) != INV
    assert backward(dx=X) == INV and backward(ws=X) == INV and backward(dx=W) == INV and backward(dx=ROOM + 16) == INV
    assert backward(ws=WS) == INV and backward(dx=X + A * N * 2) != INV


def test_quantiser_and_balance():
    L = moe.lib()
    q = lambda codes=W, scales=WS: L.moe_mx4_quantize(P(X), moe.F32, 64, 8, 64, P(codes), P(scales), None)  # noqa: E731
    assert q() != INV and q(codes=X) == INV and q(scales=X + 8 * 256 - 1) == INV and q(scales=W + 1) == INV
    d = lambda y: L.moe_mx4_dequantize(P(W), P(WS), 8, 64, moe.F32, P(y), None)  # noqa: E731
    assert d(Y) != INV and d(W) == INV and d(WS) == INV
    b = lambda out, ld=64: L.moe_balance_loss_backward(P(X), moe.F32, ld, 8, 64, 2, None, P(W), P(WS), P(G), P(out), None)  # noqa: E731
    assert b(Y) != INV and b(X) != INV and b(X + 256) == INV and b(X, ld=72) == INV and b(X + 8 * 256) != INV
