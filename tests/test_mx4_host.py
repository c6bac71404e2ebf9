"""Host side of the microscaled 4-bit calls and the balance loss, without a GPU: the float64 reference against
hand-made values, and what the C ABI and the binding refuse before anything is launched."""
import ctypes as C
import os

import numpy as np
import pytest
import torch

import mx4_ref

moe = pytest.importorskip("bit_quantized_moe_topk_amd")
if not os.path.exists(moe.LIB_PATH):
    pytest.skip("libmoe.so not built (run __graft_entry__.build())", allow_module_level=True)

FAKE = C.c_void_p(0x10000)  # 16-byte aligned, never dereferenced by the host checks
ODD = C.c_void_p(0x10008)
INV, UNS, WSP, OK = moe.ERR_INVALID_ARG, moe.ERR_UNSUPPORTED, moe.ERR_WORKSPACE, moe.OK


def test_reference_quantisation():
    x = np.zeros((1, 40), np.float32)
    x[0, :10] = [6, -5, 2.5, 3.5, 1.25, -0.75, 0.25, 0.26, 7.9, -1.75]
    x[0, 32:36] = [2.0 ** -126, 2.0 ** -128, 0, -0.0]
    codes, scales = mx4_ref.quantize(x)
    assert scales.tolist() == [[127, 0]]
    assert mx4_ref.values(codes, scales, 40)[0, :10].tolist() == [6, -4, 2, 4, 1, -1, 0, 0.5, 6, -2]
    assert mx4_ref.values(codes, scales, 40)[0, 32:34].tolist() == [2.0 ** -126, 2.0 ** -128]
    x[0, 3], x[0, 39] = np.nan, np.inf
    codes, scales = mx4_ref.quantize(x)
    assert scales.tolist() == [[255, 255]] and not codes.any()


def test_quantize_refusals():
    q = moe.lib().moe_mx4_quantize
    assert q(FAKE, moe.F32, 63, 4, 64, FAKE, FAKE, None) == INV     # rows overlap
    assert q(FAKE, 3, 64, 4, 64, FAKE, FAKE, None) == INV
    assert q(FAKE, moe.F32, 64, -1, 64, FAKE, FAKE, None) == INV
    assert q(FAKE, moe.F32, 64, 4, 0, FAKE, FAKE, None) == INV
    assert q(None, moe.F32, 64, 4, 64, FAKE, FAKE, None) == INV
    assert q(FAKE, moe.F32, 64, 4, 64, ODD, FAKE, None) == INV
    assert q(C.c_void_p(0x10002), moe.F32, 64, 4, 64, FAKE, FAKE, None) == INV
    assert q(FAKE, moe.F32, 1 << 20, 4, 1 << 20, FAKE, FAKE, None) == UNS
    assert q(None, moe.F32, 64, 0, 64, None, None, None) == OK
    d = moe.lib().moe_mx4_dequantize
    assert d(FAKE, FAKE, 4, 64, moe.MX4, FAKE, None) == INV
    assert d(FAKE, None, 4, 64, moe.F32, FAKE, None) == INV
    assert d(None, None, 0, 64, moe.F32, None, None) == OK


def test_matmul_refusals():
    f = moe.lib().moe_mx4_matmul

    def call(**kw):
        a = dict(x=FAKE, xs=None, t=moe.BF16, ld=64, T=4, wc=FAKE, ws=FAKE, N=16, K=64, y=FAKE, yt=moe.BF16)
        a.update(kw)
        return f(*a.values(), None)

    assert call(T=0, x=None, wc=None, ws=None, y=None) == OK
    for bad in (dict(T=-1), dict(N=0), dict(K=0), dict(t=2), dict(yt=moe.MX4), dict(ld=63), dict(x=None),
                dict(wc=None), dict(ws=None), dict(y=None), dict(wc=ODD), dict(t=moe.MX4), dict(xs=FAKE),
                dict(t=moe.MX4, xs=FAKE, x=ODD), dict(x=C.c_void_p(0x10001)), dict(y=C.c_void_p(0x10001))):
        assert call(**bad) == INV, bad
    for bad in (dict(N=(1 << 19) + 1), dict(K=(1 << 19) + 1, ld=1 << 20), dict(T=(1 << 23) + 1), dict(ld=1 << 41)):
        assert call(**bad) == UNS, bad
    b = moe.lib().moe_mx4_matmul_backward
    assert b(FAKE, moe.MX4, 16, 4, FAKE, FAKE, 16, 64, FAKE, moe.F32, None) == INV
    assert b(FAKE, moe.F32, 15, 4, FAKE, FAKE, 16, 64, FAKE, moe.F32, None) == INV
    assert b(None, moe.F32, 16, 0, None, None, 16, 64, None, moe.F32, None) == OK


def test_experts_refusals():
    f = moe.lib().moe_mx4_experts_matmul

    def call(**kw):
        a = dict(x=FAKE, xs=None, t=moe.BF16, ld=64, T=4, k=2, E=8, sh=1, ga=1, off=FAKE, perm=FAKE, wc=FAKE, ws=FAKE,
                 N=16, K=64, y=FAKE, yt=moe.BF16, wk=None, nb=0)
        a.update(kw)
        return f(*a.values(), None)

    assert call(T=0, x=None, off=None, perm=None, wc=None, ws=None, y=None) == OK
    assert moe.lib().moe_mx4_experts_matmul_workspace_size(4, 2, 1) == 0
    need = moe.lib().moe_mx4_experts_matmul_workspace_size(4096, 2, 1)
    assert need > 0
    assert call(T=4096) == WSP and call(T=4096, wk=FAKE, nb=need - 1) == WSP and call(T=4096, wk=ODD, nb=need) == WSP
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(sh=2), dict(ga=2), dict(off=None), dict(perm=None), dict(N=0),
                dict(ld=63), dict(t=moe.MX4), dict(xs=FAKE), dict(y=None)):
        assert call(**bad) == INV, bad
    assert call(E=moe.MAX_E + 1, sh=1) == UNS
    assert call(T=1 << 22, k=2) == UNS
    b, size = moe.lib().moe_mx4_experts_matmul_backward, moe.lib().moe_mx4_experts_matmul_backward_workspace_size
    need = size(4, 2, 1, 64, 1)
    assert need == 12 * 64 * 4 and size(4, 2, 1, 64, 0) == 0 and size(4, 0, 1, 64, 1) == 0

    def back(**kw):
        a = dict(dy=FAKE, t=moe.BF16, ld=16, T=4, k=2, E=8, sh=1, ga=1, off=FAKE, so=FAKE, wc=FAKE, ws=FAKE, N=16,
                 K=64, dx=FAKE, dt=moe.BF16, wk=FAKE, nb=need)
        a.update(kw)
        return b(*a.values(), None)

    assert back(nb=need - 1) == WSP and back(wk=None) == WSP and back(wk=ODD) == WSP
    for bad in (dict(t=moe.MX4), dict(so=None), dict(off=None), dict(ld=15), dict(dx=None)):
        assert back(**bad) == INV, bad
    assert back(T=0, dy=None, dx=None, wk=None, nb=0) == OK


def test_experts_sizes_past_every_integer():
    """Sums and products of the sizes that pass 32 bits are refused, not wrapped."""
    f, b = moe.lib().moe_mx4_experts_matmul, moe.lib().moe_mx4_experts_matmul_backward
    top = 2 ** 31 - 1
    for T, k, E, shared in ((4, top, 8, 1), (top, top, 8, 1), (4, 2, top, 1), (4, 2, top, 0), (0, top, 8, 1), (2, 2 ** 30, 8, 0)):
        for gather in (0, 1):
            assert f(FAKE, None, moe.BF16, 64, T, k, E, shared, gather, FAKE, FAKE, FAKE, FAKE, 16, 64, FAKE, moe.BF16,
                     FAKE, 1 << 40, None) == UNS, (T, k, E, shared)
            assert b(FAKE, moe.BF16, 64, T, k, E, shared, gather, FAKE, FAKE, FAKE, FAKE, 16, 64, FAKE, moe.BF16, FAKE,
                     1 << 40, None) == UNS, (T, k, E, shared)
        assert moe.lib().moe_mx4_experts_matmul_workspace_size(T, k, shared) == 0 or E == top
        assert moe.lib().moe_mx4_experts_matmul_backward_workspace_size(T, k, shared, 64, 1) == 0 or E == top


def test_balance_refusals():
    f, size = moe.lib().moe_balance_loss, moe.lib().moe_balance_loss_workspace_size
    need = size(64, 10, 512)
    assert need > 0 and size(64, 0, 512) == 0 and size(64, 10, moe.MAX_E + 1) == 0 and size(-1, 10, 512) == 0

    def call(**kw):
        a = dict(x=FAKE, t=moe.F32, ld=512, T=64, E=512, k=10, idx=FAKE, m=None, lo=FAKE, c=FAKE, n=FAKE, ws=FAKE, nb=need)
        a.update(kw)
        return f(*a.values(), None)

    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(ld=511), dict(t=moe.MX4), dict(x=None), dict(idx=None),
                dict(lo=None), dict(c=None), dict(n=None)):
        assert call(**bad) == INV, bad
    assert call(E=moe.MAX_E + 1, ld=4096) == UNS
    assert call(nb=need - 1) == WSP and call(ws=None) == WSP
    b = moe.lib().moe_balance_loss_backward
    assert b(FAKE, moe.F32, 512, 64, 512, 10, None, FAKE, FAKE, None, FAKE, None) == INV
    assert b(FAKE, moe.F32, 511, 64, 512, 10, None, FAKE, FAKE, FAKE, FAKE, None) == INV
    assert b(None, moe.F32, 512, 0, 512, 10, None, None, None, None, None, None) == OK


def test_balance_sizes_past_the_launches():
    f, b, n = moe.lib().moe_balance_loss, moe.lib().moe_balance_loss_backward, moe.lib().moe_balance_loss_workspace_size
    for T, k in ((2 ** 31 - 1, 1), (2 ** 30 + 1, 1), (2 ** 29, 3), (2, 2 ** 30), (2 ** 31 - 1, 2 ** 31 - 1)):
        assert n(T, k, 1) == 0
        assert f(FAKE, moe.BF16, 1, T, 1, k, FAKE, None, FAKE, FAKE, FAKE, FAKE, 1 << 40, None) == UNS
        assert b(FAKE, moe.BF16, 1, T, 1, k, None, FAKE, FAKE, FAKE, FAKE, None) == UNS
    assert n(2 ** 30, 1, 1) > 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64)
    codes, scales = torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(16, 2, dtype=torch.uint8)
    for call in (lambda: moe.mx4_quantize(x), lambda: moe.mx4_quantize(x[0]), lambda: moe.Mx4(codes, scales, 64),
                 lambda: moe.mx4_matmul(x, None), lambda: moe.mx4_matmul_backward(x, None),
                 lambda: moe.balance_loss(x, torch.zeros(4, 2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()


def test_grouping_keeps_its_four_fields():
    g = moe.Grouping(1, 2, 3, 4)
    assert (g.counts, g.offsets, g.perm, g.slot_of, g.has_shared) == (1, 2, 3, 4, None)
