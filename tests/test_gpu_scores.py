"""Routing by scores and the gates' gradient on the GPU against float64: indices equal, gates off by at most a float32 sum
of E exponentials ((E + 8) 2^-24 relative), gradients by (E + k + 24) 2^-24 of the magnitudes that they add up, and half a step of
their type."""
import numpy as np
import pytest

import blocks_ref as ref
from gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def lib():
    torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    return moe


def as64(t):
    return t.double().cpu().numpy()


def make(seed, T, E, kind, bias, off=0, gap=0):
    torch = torch_cuda()
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, E + gap)) * 2
    if off:
        x[:, rng.permutation(E)[:off]] = -np.inf
    x = torch.from_numpy(x.astype(np.float32)).to(torch.float32 if kind == "f32" else torch.bfloat16).cuda()[:, :E]
    b = torch.from_numpy((0.2 * rng.standard_normal(E)).astype(np.float32)).cuda() if bias else None
    return x, b, rng


def check(x, b, k, **how):
    moe = lib()
    idx, gates = moe.route_scores(x, k, b, **how)
    want, wg = ref.route(as64(x), k, None if b is None else as64(b), **{"score": "sigmoid", **how})
    got = idx.cpu().numpy()
    assert np.array_equal(got, want), [(t, got[t].tolist(), want[t].tolist()) for t in np.argwhere((got != want).any(1)).ravel()[:3]]
    assert np.all(np.abs(as64(gates) - wg) <= (x.shape[1] + 8) * U * np.abs(wg) + 1e-37)
    return idx, gates


CASES = [  # T, E, k, groups, keep, top
    (1, 1, 1, 1, 1, 1), (5, 7, 3, 1, 1, 2), (4, 512, 10, 8, 4, 2), (3, 64, 64, 1, 1, 1), (9, 100, 8, 5, 3, 1), (17, 100, 40, 5, 2, 2),
    (6, 130, 12, 2, 1, 2), (33, 256, 8, 8, 4, 2), (2, 2048, 16, 64, 7, 2), (3, 2048, 100, 1, 1, 2), (2, 300, 300, 3, 3, 1), (5, 64, 2, 64, 2, 2),
    (8, 1000, 12, 8, 3, 1), (4, 192, 6, 16, 5, 2), (3, 600, 90, 4, 1, 2)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_route(case, score, bias, kind):
    T, E, k, groups, keep, top = case
    for off in (0, E // 10):
        x, b, _ = make(E * k + off, T, E, kind, bias, off, gap=3 if T % 2 else 0)
        for renorm in (False, True):
            check(x, b, k, score=score, groups=groups, keep_groups=keep, group_top=top, renormalize=renorm, scale=2.5)


def test_route_matches_topk():
    """Softmax scores without a bias or groups, renormalised: route_topk's own selection and gates."""
    torch, moe = torch_cuda(), lib()
    x, _, _ = make(1, 700, 512, "f32", False)
    idx, gates = moe.route_scores(x, 10, score="softmax")
    i2, g2 = moe.route_topk(x, 10)
    assert torch.equal(idx, i2) and torch.allclose(gates, g2, rtol=1e-5, atol=0)


def test_route_many_near_ties():
    """Scores that differ in the last places of 32 bits: the order is that of 64."""
    torch = torch_cuda()
    rng = np.random.default_rng(7)
    base = np.float32(1.25)
    for bias in (False, True):
        x = np.full((300, 256), base, np.float32)
        steps = rng.integers(0, 4, x.shape).astype(np.int32)
        x = (x.view(np.int32) + steps).view(np.float32)
        b = torch.from_numpy((np.float32(0.5).view(np.int32) + rng.integers(0, 3, 256).astype(np.int32)).view(np.float32)).cuda() if bias else None
        t = torch.from_numpy(x).cuda()
        for score in ("sigmoid", "softmax"):
            for groups, keep, top in ((1, 1, 1), (8, 3, 2), (8, 3, 1)):
                check(t, b, 9, score=score, groups=groups, keep_groups=keep, group_top=top)
        t = torch.from_numpy((rng.standard_normal((300, 256)) + 0 * x).astype(np.float32)).cuda()
        t[:, 100:140] = torch.from_numpy(x[:, :40] + np.float32(3)).cuda()
        for groups, keep, top in ((1, 1, 1), (8, 3, 2)):
            check(t, b, 9, groups=groups, keep_groups=keep, group_top=top)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_ties_and_switched_off(score):
    torch = torch_cuda()
    for E, groups, keep in ((64, 1, 1), (512, 8, 3), (100, 5, 2), (2048, 16, 16)):
        x = torch.zeros((4, E), device="cuda")
        b = torch.zeros(E, device="cuda")
        x[1, ::3] = -float("inf")
        x[2] = -float("inf")                      # nothing is left: the lowest indices, gates 0
        x[3, 5:] = -float("inf")                  # fewer are left than are asked for
        for bias in (None, b, b - 2):
            for top in (1, 2):
                check(x, bias, 12, score=score, groups=groups, keep_groups=keep, group_top=top)
                check(x, bias, 12, score=score, groups=groups, keep_groups=keep, group_top=top, renormalize=False)
        b = b.clone()
        b[1::2] = -float("inf")                   # switched off by the bias
        check(x, b, 12, score=score, groups=groups, keep_groups=keep)
        # the type's lowest value is a value, not a switch
        x[0, 1::2] = torch.finfo(torch.float32).min
        check(x, None, 12, score=score, groups=groups, keep_groups=keep)
    # bfloat16: many logits alike
    x, b, _ = make(3, 200, 512, "bf16", True)
    check((x * 2).round() / 2, b.bfloat16().float().round(), 10, score=score, groups=8, keep_groups=4)
    check((x * 2).round() / 2, None, 10, score=score, groups=8, keep_groups=4)


def test_route_not_finite():
    """NaN and +inf logits: indices stay distinct and in range, other tokens are not touched."""
    torch, moe = torch_cuda(), lib()
    x, b, _ = make(5, 40, 512, "f32", True)
    for score in ("sigmoid", "softmax"):
        for bias in (None, b):
            clean = moe.route_scores(x, 10, bias, score=score, groups=8, keep_groups=4)
            y = x.clone()
            y[3] = float("nan")
            y[7, 100] = float("nan")
            y[9, 200] = float("inf")
            y[11, 3:400] = float("nan")
            idx, gates = moe.route_scores(y, 10, bias, score=score, groups=8, keep_groups=4)
            for t in range(40):
                row = idx[t].tolist()
                assert len(set(row)) == 10 and 0 <= min(row) and max(row) < 512
                if t not in (3, 7, 9, 11):
                    assert torch.equal(idx[t], clean[0][t]) and torch.equal(gates[t], clean[1][t])
            assert torch.isnan(gates[3]).all()
            if score == "softmax":
                assert torch.isnan(gates[7]).all() and torch.isnan(gates[9]).all()
            else:
                assert 100 not in idx[7].tolist() and torch.isfinite(gates[7]).all()
                # a score of 1: with a bias others may still come before it
                assert score == "softmax" or bias is not None or 200 in idx[9].tolist()
    big = torch.tensor([[200.0, -200.0, 90.0, -90.0]], device="cuda")
    check(big, None, 4, renormalize=False)


def test_route_out_and_nothing():
    torch, moe = torch_cuda(), lib()
    x, b, _ = make(5, 40, 100, "f32", True)
    want = moe.route_scores(x, 7, b)
    out = (torch.empty((40, 7), dtype=torch.int32, device="cuda"), torch.empty((40, 7), device="cuda"))
    got = moe.route_scores(x, 7, b, out=out)
    assert got[0] is out[0] and torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert moe.route_scores(x[:0], 7, b)[0].shape == (0, 7)
    assert moe.route_scores_backward(x[:0], want[0][:0], want[1][:0]).shape == (0, 100)
    for call in (lambda: moe.route_scores(x, 7, b[:5]), lambda: moe.route_scores(x, 7, score="relu"), lambda: moe.route_scores(x, 0),
                 lambda: moe.route_scores(x, 7, out=(out[0][:3], out[1])), lambda: moe.route_scores(x.t(), 7),
                 lambda: moe.route_scores_backward(x, want[0], want[1][:, :3]), lambda: moe.route_scores_backward(x, want[0].long(), want[1])):
        with pytest.raises((ValueError, TypeError)):
            call()
    for how in (dict(groups=3), dict(groups=5, keep_groups=6), dict(group_top=3), dict(groups=50, keep_groups=3)):
        with pytest.raises(moe.MoeError):
            moe.route_scores(x, 7, **how)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (4, 512, 10), (9, 100, 8), (3, 2048, 100), (30, 63, 5), (2, 65, 65), (700, 256, 6), (5, 1000, 64)])
def test_route_backward(T, E, k, score, renorm, kind):
    torch, moe = torch_cuda(), lib()
    x, b, rng = make(E + k, T, E, kind, True, E // 10, gap=5 if T % 2 else 0)
    idx, _ = moe.route_scores(x, k, b, score=score, renormalize=renorm, scale=2.5)
    d = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    got = moe.route_scores_backward(x, idx, d, score=score, renormalize=renorm, scale=2.5)
    want, size = ref.route_gradient(as64(x), idx.cpu().numpy(), as64(d), score, renorm, 2.5)
    err = (E + k + 24) * U * size
    half = torch.finfo(x.dtype).eps / 2
    worst = np.max(np.abs(as64(got) - want) / (err + half * (np.abs(want) + err) + 1e-37))
    log(f"[scores] backward {T}x{E}x{k} {score} {renorm} {kind}: {worst:.3f}")
    assert got.dtype == x.dtype and worst <= 1
    assert torch.equal(got, moe.route_scores_backward(x, idx, d, score=score, renormalize=renorm, scale=2.5))


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_backward_bad_and_repeated_ids(score, renorm):
    """An index twice counts twice; ids out of range are not there; a token whose experts are all off has no gradient."""
    torch, moe = torch_cuda(), lib()
    x, _, rng = make(4, 6, 90, "f32", False)
    x[2] = -float("inf")
    idx = torch.from_numpy(rng.integers(0, 90, (6, 8)).astype(np.int32)).cuda()
    idx[0, 1] = idx[0, 0]
    idx[1, :] = 5
    idx[3, 2], idx[3, 3], idx[3, 4] = -1, 90, 2 ** 31 - 1
    idx[4] = -1
    d = torch.from_numpy(rng.standard_normal((6, 8)).astype(np.float32)).cuda()
    got = as64(moe.route_scores_backward(x, idx, d, score=score, renormalize=renorm))
    want, size = ref.route_gradient(as64(x), idx.cpu().numpy(), as64(d), score, renorm)
    assert np.all(np.abs(got - want) <= (90 + 8 + 24) * U * (size + np.abs(want)) + 1e-37)
    assert (got[2] == 0).all() and (got[4] == 0).all()
