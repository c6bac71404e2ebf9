"""Routing by scores at the ends of its range, against float64: gradients of very low and very high logits, groups whose best two
values nearly cancel or pass float32's range, and group counts that leave lanes without an expert.

Bounds, as in test_gpu_scores: (E + k + 24) 2^-24 of the magnitudes that a gradient's entry adds up, and half a step of its type. A
sigmoid's entry is d s (1 - s), so its magnitudes carry both factors here: 1 - s is the score of the other sign."""
import numpy as np
import pytest

import blocks_ref as ref
from gpu_util import log, torch_cuda
from test_gpu_scores import U, as64, check, lib

pytestmark = pytest.mark.gpu


def gradient(x, idx, d_gates, renorm, scale):
    """The gradient of sigmoid gates in float64 without cancellation: (dlogits, the magnitudes that each adds up)."""
    T, E = x.shape
    s, rest = ref.scores(x, "sigmoid"), ref.scores(-x, "sigmoid")
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        e = idx[t]
        d = np.float64(np.float32(scale)) * d_gates[t]
        q, m = s[t][e], np.abs(d)
        total = 1.0
        if renorm:
            total = q.sum()
            if total == 0:
                continue
            d, m = d - (d * q).sum() / total, m + (m * q).sum() / total
        np.add.at(out[t], e, d * (q / total) * rest[t][e])
        np.add.at(size[t], e, m * (q / total) * rest[t][e])
    return out, size


def check_gradient(x, idx, d, renorm, name):
    torch, moe = torch_cuda(), lib()
    got = moe.route_scores_backward(x, idx, d, score="sigmoid", renormalize=renorm, scale=2.5)
    want, size = gradient(as64(x), idx.cpu().numpy(), as64(d), renorm, 2.5)
    err = (x.shape[1] + idx.shape[1] + 24) * U * size
    half = torch.finfo(x.dtype).eps / 2
    g = as64(got)
    worst = np.max(np.abs(g - want) / (err + half * (np.abs(want) + err) + 1e-37))
    log(f"[scores] gradient {name}: {worst:.3f}")
    assert np.isfinite(g).all() and worst <= 1, name
    return got


def typed(v, kind):
    torch = torch_cuda()
    return torch.from_numpy(v.astype(np.float32)).to(torch.float32 if kind == "f32" else torch.bfloat16).cuda()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", [(9, 32, 4), (5, 300, 10), (3, 200, 80)])
def test_renormalised_gradient_of_low_logits(T, E, k, kind):
    """Scores that float32 does not hold: their ratios count, and gates and gradient agree."""
    torch, moe = torch_cuda(), lib()
    rng = np.random.default_rng(E)
    for level in (-60.0, -64.0, -80.0, -87.5, -88.0, -88.6, -89.0, -92.0, -104.0, -120.0, -300.0, -690.0):
        x = typed(level + 2 * rng.standard_normal((T, E)), kind)
        idx, gates = check(x, None, k, scale=2.5)
        d = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
        got = check_gradient(x, idx, d, True, f"{T}x{E}x{k} at {level}")
        assert (got != 0).any()
    # some that are off beside them; and scores that 64 bits do not hold either: gates and gradient are 0
    x = typed(-90 + 2 * rng.standard_normal((T, E)), kind)
    x[:, 2:] = -float("inf")
    idx, gates = check(x, None, k, scale=2.5)
    check_gradient(x, idx, torch.ones((T, k), device="cuda") * torch.arange(k, device="cuda"), True, "few left")
    x = torch.full_like(x, -800.0)
    idx, gates = check(x, None, k, scale=2.5)
    assert (gates == 0).all() and (moe.route_scores_backward(x, idx, gates + 1, scale=2.5) == 0).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("k", [4, 12, 70])
def test_renormalised_shares_below_the_normal_numbers(k, score, kind):
    """A score under 2^-126 beside others under 1/2 is a share of their sum all the same. (exp(l - most): the difference's
    rounding is |l - most| 2^-24 of the share at most, which the gradient's bound has besides.)"""
    torch, moe = torch_cuda(), lib()
    rng = np.random.default_rng(k)
    for most, deep in ((-2.0, 110.0), (-20.0, 110.0), (-48.0, 89.5), (-61.0, 130.0), (-2.0, 300.0)):
        x = rng.uniform(-deep, most, (6, 80))
        x[:, 0] = most
        x[0, 5:9] = np.finfo(np.float32).min  # the lowest value: a share of 0
        if score == "softmax":
            x = np.concatenate([x, np.full((6, 80), 20.0)], 1)  # a group that is not chosen has the row's largest
            bias = torch.from_numpy(np.repeat([1.0, -1.0], 80).astype(np.float32)).cuda()
            x = typed(x, kind)
            check(x, bias, k, score=score, scale=2.5, groups=2, keep_groups=1, group_top=1)
            continue
        x = typed(x, kind)
        idx, _ = check(x, None, k, scale=2.5)
        ids = torch.from_numpy(np.argsort(rng.random((6, 80)), axis=1)[:, :k].astype(np.int32)).cuda().contiguous()
        d = torch.from_numpy(rng.standard_normal((6, k)).astype(np.float32)).cuda()
        for ids in (idx, ids):
            got = as64(moe.route_scores_backward(x, ids, d, renormalize=True, scale=2.5))
            want, size = gradient(as64(x), ids.cpu().numpy(), as64(d), True, 2.5)
            far = np.abs(as64(x) - np.take_along_axis(as64(x), ids.cpu().numpy().astype(np.int64), 1).max(1, keepdims=True))
            err = (80 + k + 24 + np.minimum(far, 1000)) * U * size
            half = torch.finfo(x.dtype).eps / 2
            assert np.all(np.abs(got - want) <= err + half * (np.abs(want) + err) + 1e-37)


def test_renormalised_gradient_at_the_least_normal_score():
    """Four logits around exp's last normal result: the formula gives 1.04, -0.97, 2.44, -2.50 and what goes with them."""
    torch = torch_cuda()
    idx = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    d = torch.tensor([[1.0, -2.0, 3.0, -6.0]], device="cuda")
    for level in (-87.0, -88.0, -88.6, -89.0, -95.0):
        x = torch.tensor([[level, level - 0.1, level + 0.05, level - 0.4]], device="cuda")
        check_gradient(x, idx, d, True, f"at {level}")


def test_renormalised_gradient_of_large_gradients():
    """Small scores and large gradients of the gates: no product of the two leaves float32's range on the way."""
    torch = torch_cuda()
    rng = np.random.default_rng(3)
    for k in (6, 70):
        x = typed(-55 + rng.standard_normal((4, 100)), "f32")
        idx = torch.from_numpy(np.argsort(-x.cpu().numpy(), axis=1)[:, :k].astype(np.int32)).cuda().contiguous()
        d = torch.from_numpy((1e25 * rng.standard_normal((4, k))).astype(np.float32)).cuda()
        check_gradient(x, idx, d, True, f"large, k {k}")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(40, 32, 4), (7, 300, 10), (3, 200, 80)])
def test_gradient_of_high_logits(T, E, k, renorm, kind):
    """1 - s of a score near 1 keeps its bits."""
    torch = torch_cuda()
    rng = np.random.default_rng(E + 1)
    for lo, hi in ((8, 30), (15, 18), (60, 80), (-30, 30)):
        x = typed(rng.uniform(lo, hi, (T, E)), kind)
        idx = torch.from_numpy(np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)).cuda().contiguous()
        d = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
        got = check_gradient(x, idx, d, renorm, f"{T}x{E}x{k} {renorm} {kind} in {lo} .. {hi}")
        # (not where one score may outweigh the others 2^24 times: its d - sum d s / S is then 0 in 32 bits, within the bound)
        assert lo < 0 or (got.gather(1, idx.long()) != 0).all()


def near_groups(rng, T, groups, size):
    """Logits whose groups' best two sigmoid scores add up to nearly the same, apart by 1e-6 to 1e-3."""
    s = rng.uniform(0.05, 0.3, (T, groups, size))
    s[..., 0] = rng.uniform(0.5, 0.6, (T, groups))
    apart = rng.choice([-1, 1], (T, groups)) * 10 ** rng.uniform(-6, -3, (T, groups))
    s[..., 1] = 1.0 - s[..., 0] + apart
    return np.log(s / (1 - s)).reshape(T, groups * size).astype(np.float32)


@pytest.mark.parametrize("size", [2, 3, 4])
@pytest.mark.parametrize("groups,keep", [(2, 1), (8, 3), (16, 5)])
@pytest.mark.parametrize("B", [1.0, 200.0, 1e3, 1e4, 1e5, 3e7])
def test_groups_of_opposite_biases(B, groups, keep, size):
    """A group's value is small, its two terms are not: what 32 bits lose of them is not relative to the sum."""
    torch = torch_cuda()
    rng = np.random.default_rng(int(B) + groups)
    x = torch.from_numpy(near_groups(rng, 300, groups, size)).cuda()
    bias = np.full((groups, size), -4 * B, np.float32)
    bias[:, 0], bias[:, 1] = B, -B
    check(x, torch.from_numpy(bias.reshape(-1)).cuda(), min(4, keep * size), groups=groups, keep_groups=keep, group_top=2)
    # (each group with a size of its own)
    own = (np.float32(B) * rng.uniform(0.5, 1.5, (groups, 1))).astype(np.float32)
    bias[:, :1], bias[:, 1:2] = own, -own
    check(x, torch.from_numpy(bias.reshape(-1)).cuda(), min(4, keep * size), groups=groups, keep_groups=keep, group_top=2)


def test_groups_of_opposite_biases_by_hand():
    """32 bits: 0.68555 and 0.68549; exactly: 0.68550 and 0.68554."""
    torch = torch_cuda()
    x = torch.tensor([[-.20984702, -1.1649512, .28798392, -2.0501812]], device="cuda")
    b = torch.tensor([1e3, -1e3, 1e3, -1e3], device="cuda")
    idx, _ = check(x, b, 2, groups=2, keep_groups=1, group_top=2)
    assert idx.tolist() == [[2, 3]]


def test_groups_whose_sums_pass_float32():
    """Sums of two below -2^128 are values, in their order, and come before groups that are off."""
    torch = torch_cuda()
    inf, least = float("inf"), torch.finfo(torch.float32).min
    x = torch.from_numpy(np.random.default_rng(5).standard_normal((20, 10)).astype(np.float32)).cuda()
    for b in ([-3e38, -3e38, -inf, -inf, -2e38, -2e38, 0, 0, -3.2e38, -3e38],
              [-inf, -inf, least, least, -2e38, -2e38, 1, 0, least, -3e38],
              [-inf, -inf, -inf, -inf, -inf, -inf, least, least, -3e38, -3e38],
              [3e38, 3e38, 2e38, 3e38, 3e38, 0, inf, least, -inf, 3e38],
              [-3e38, -3e38, -2.5e38, -inf, -3e38, 3e38, 0, least, -1, -1]):
        bias = torch.tensor(b, device="cuda")
        for keep in (1, 2, 3, 4, 5):
            for top in (1, 2):
                for k in (1, 2 * keep):
                    check(x, bias, k, groups=5, keep_groups=keep, group_top=top)
    # with logits that are off, too
    x[:, 6] = -inf
    x[::2, 2:4] = -inf
    bias = torch.tensor([-3e38, -3e38, -inf, -inf, -2e38, -2e38, 0, 0, -3.2e38, -3e38], device="cuda")
    for keep in (1, 2, 3, 4):
        check(x, bias, keep, groups=5, keep_groups=keep, group_top=2)


@pytest.mark.parametrize("E,groups", [(65, 13), (66, 33), (100, 50), (63, 63), (129, 43), (520, 52), (640, 64), (2046, 62)])
def test_groups_that_fit_no_wave(E, groups):
    """Lanes past the experts belong to no group."""
    rng = np.random.default_rng(E)
    x = typed(rng.standard_normal((50, E)), "f32")
    b = typed(0.2 * rng.standard_normal(E), "f32")
    for keep in (1, groups // 3, groups - 1):
        for top in (1, 2):
            k = min(10, keep * (E // groups))
            check(x, b, k, groups=groups, keep_groups=keep, group_top=top)
            check(x, None, k, groups=groups, keep_groups=keep, group_top=top)


def test_refusals_of_what_is_no_tensor():
    torch, moe = torch_cuda(), lib()
    x = torch.zeros((4, 16), device="cuda")
    d = torch.zeros((4, 2), device="cuda")
    for call in (lambda: moe.route_scores_backward(x, None, d), lambda: moe.route_scores_backward(x, [[0, 1]] * 4, d),
                 lambda: moe.route_scores(x, 2, out=(None, d))):
        with pytest.raises((ValueError, TypeError)):
            call()
