"""Counts, balance loss, z loss and their gradient on the GPU against float64.

Tolerances, u = 2^-24. A logit's distance to its row's largest, r = |x - top|, is rounded once and goes through an
exponential good to 2 units: exp(x - top) is within (r + 4) u of itself, the row's sum of E of them within E u more,
so p is within d = (R + E + 12) u of itself (R the largest r of a p that counts; below e^-104 p is 0 in float32 and
at most 2^-149 off). lse is within d + 2 |lse| u. Sums of positive terms add (E + T) u relative.
"""
import numpy as np
import pytest

import mx4_ref
from gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def check_case(logits, idx, mask, d=(0.7, 0.3)):
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    T, E = logits.shape
    keep = np.ones(T, bool) if mask is None else mask.cpu().numpy().astype(bool)
    x = logits.double().cpu().numpy()
    losses, counts, n, dx, p, lse = mx4_ref.balance(x, idx.cpu().numpy(), keep, d)
    dl = torch.tensor(d, dtype=torch.float32, device="cuda")
    d = dl.double().cpu().numpy()
    out = moe.balance_loss(logits, idx, mask)
    got = moe.balance_loss_backward(logits, out, dl, mask)
    again = moe.balance_loss(logits, idx, mask)
    assert torch.equal(again.losses, out.losses) and torch.equal(moe.balance_loss_backward(logits, out, dl, mask), got)
    assert np.array_equal(out.counts.cpu().numpy(), counts) and int(out.kept) == n
    live = x[keep]
    top = live.max(1, initial=-np.inf) if n else np.zeros(0)
    fin = np.isfinite(live) & np.isfinite(top)[:, None] if n else np.zeros((0, E), bool)
    R = min(104.0, float(np.max(np.where(fin, np.where(np.isfinite(top), top, 0)[:, None] - np.where(fin, live, 0), 0), initial=0.0)))
    e = (R + E + 12) * U
    lo = out.losses.double().cpu().numpy()
    el = np.abs(lse) * 2 * U + e
    tol = np.array([losses[0] * (2 * e + (E + T + 8) * U),
                    ((2 * np.abs(lse) + el) * el)[keep].sum() / max(n, 1) + losses[1] * (T + 8) * U])
    assert (np.abs(lo - losses) <= tol + 1e-37).all(), (lo, losses, tol)
    f = counts / max(n * idx.shape[1], 1)
    cb, cz = d[0] * E / max(n, 1), d[1] * 2 / max(n, 1)
    part = np.abs(cb) * (f + (p @ f)[:, None]) + np.abs(cz * lse)[:, None]
    half = torch.finfo(logits.dtype).eps / 2
    bound = p * ((3 * e + 12 * U) * part + np.abs(cz) * el[:, None]) + half * np.abs(dx if dx is not None else 0) * 1.001 \
        + 2.0 ** -140 * (1 + np.abs(cb) * 2 + np.abs(cz * lse)[:, None])
    g = got.double().cpu().numpy()
    want = dx if dx is not None else np.zeros_like(x)
    assert got.dtype == logits.dtype and np.isfinite(g).all()
    worst = np.max(np.abs(g - want) / bound, initial=0.0)
    log(f"[balance] T={T} E={E} {logits.dtype}: losses {lo}, gradient error / bound {worst:.3f}")
    assert worst <= 1
    assert not g[~keep].any()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 512, 10), (3, 5, 5), (4, 64, 2), (7, 65, 1), (64, 512, 10), (100, 100, 8),
                                   (257, 129, 3), (1000, 256, 8), (33, 2048, 16), (20, 1030, 4), (5000, 48, 2)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
def test_balance(T, E, k, kind, masked):
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(T + E)
    wide = torch.randn((T, E + 3), generator=g, device="cuda") * 3
    if E > 2 * k:
        wide[:, 2] = -float("inf")
    logits = wide.to(torch.float32 if kind == "f32" else torch.bfloat16)
    idx = torch.topk(logits[:, :E].float(), k).indices.int()
    mask = torch.rand(T, generator=g, device="cuda") < 0.7 if masked else None
    check_case(logits[:, :E].contiguous(), idx, mask)
    check_case(logits[:, :E], idx, None if mask is None else mask.to(torch.uint8))


def test_nothing_kept_and_no_tokens():
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    x = torch.full((6, 20), float("nan"), device="cuda")
    idx = torch.zeros((6, 2), dtype=torch.int32, device="cuda")
    none = torch.zeros(6, dtype=torch.bool, device="cuda")
    d = torch.ones(2, device="cuda")
    out = moe.balance_loss(x, idx, none)
    assert out.losses.tolist() == [0, 0] and not out.counts.any() and int(out.kept) == 0
    assert not moe.balance_loss_backward(x, out, d, none).any()
    out = moe.balance_loss(x[:0], idx[:0])
    assert out.losses.tolist() == [0, 0] and not out.counts.any() and int(out.kept) == 0
    assert moe.balance_loss_backward(x[:0], out, d).shape == (0, 20)


def test_rows_without_a_distribution_and_wild_values():
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((12, 70), generator=g, device="cuda")
    x[2] = -float("inf")                     # no distribution
    x[3, 1:] = -float("inf")                 # one expert left
    x[4] = torch.finfo(torch.float32).min    # all at the type's lowest: an even distribution
    x[4] /= 2.0 ** 66                        # (its square still fits float32)
    x[5] = 88.0                              # exp alone would overflow
    x[6] = -90.0
    idx = torch.topk(x, 3).indices.int()
    idx[7, 1], idx[8, 0], idx[9] = -1, 70, 5   # no expert; no expert; one expert three times
    check_case(x, idx, None)
    mask = torch.ones(12, dtype=torch.bool, device="cuda")
    x[10, 3], x[11, 4], mask[10], mask[11] = float("nan"), float("inf"), False, False
    check_case(torch.where(mask[:, None], x, 0.0), idx, mask)
    out = moe.balance_loss(x, idx, mask)
    same = moe.balance_loss(torch.where(mask[:, None], x, 0.0), idx, mask)
    assert torch.equal(out.losses, same.losses)
    mask[10] = True
    assert moe.balance_loss(x, idx, mask).losses.isnan().all()
    assert moe.balance_loss_backward(x, out, torch.ones(2, device="cuda"), mask)[10].isnan().all()


def test_gradient_against_differences():
    """Central differences of the loss in float64, counts held, agree with the kernel's gradient to the difference's own
    error: h^2 / 6 times a third derivative that is below 20 (E / n + 4 |lse| / n), and the gradient's float32."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    g = torch.Generator(device="cuda").manual_seed(3)
    T, E, k, h = 9, 21, 3, 1e-4
    x = torch.randn((T, E), generator=g, device="cuda")
    idx = torch.topk(x, k).indices.int()
    d = torch.tensor([0.5, 0.25], device="cuda")
    got = moe.balance_loss_backward(x, moe.balance_loss(x, idx), d).double().cpu().numpy()
    xv, iv, keep = x.double().cpu().numpy(), idx.cpu().numpy(), np.ones(T, bool)
    for t in range(0, T, 2):
        for e in range(0, E, 5):
            side = []
            for s in (h, -h):
                v = xv.copy()
                v[t, e] += s
                side.append(mx4_ref.balance(v, iv, keep)[0] @ np.array([0.5, 0.25]))
            assert abs((side[0] - side[1]) / (2 * h) - got[t, e]) <= 20 * (E + 16) / T * h * h / 6 + 1e-6


def test_balance_refusals():
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    x = torch.zeros((4, 20), device="cuda")
    idx = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    out = moe.balance_loss(x, idx)
    d = torch.ones(2, device="cuda")
    for f in (lambda: moe.balance_loss(x, idx[:3]), lambda: moe.balance_loss(x[:, ::2], idx), lambda: moe.balance_loss(x[0], idx),
              lambda: moe.balance_loss(x, idx, torch.ones(3, dtype=torch.bool, device="cuda")),
              lambda: moe.balance_loss(x, idx.cpu()), lambda: moe.balance_loss_backward(x[:, :10], out, d),
              lambda: moe.balance_loss_backward(x, out, d[:1]), lambda: moe.balance_loss_backward(x, out, d.cpu())):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: moe.balance_loss(x.half(), idx), lambda: moe.balance_loss(x, idx.long()),
              lambda: moe.balance_loss(x, idx, torch.ones(4, device="cuda"))):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(moe.MoeError):
        moe.balance_loss(x, idx, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
