"""The balance loss over many tokens and many experts together: the form of several launches, at every number of columns
a lane, against float64 with the tolerances of test_gpu_balance.py."""
import pytest

from gpu_util import torch_cuda
from test_gpu_balance import check_case

pytestmark = pytest.mark.gpu


def names_of(call):
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    moe.profile_begin(16)
    call()
    torch.cuda.synchronize()
    return set(moe.profile_end())


@pytest.mark.parametrize("T,E,k", [(129, 512, 10), (1000, 512, 10), (4100, 512, 10), (200, 300, 4), (300, 1024, 8), (130, 1030, 3),
                                   (500, 2048, 16), (257, 2047, 5), (2, 2048, 2048), (1500, 260, 3), (5000, 128, 8)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
def test_many_tokens_and_experts(T, E, k, kind, masked):
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    g = torch.Generator(device="cuda").manual_seed(T + E)
    wide = torch.randn((T, E + 3), generator=g, device="cuda") * 3
    if E > k:
        wide[:, 2] = -float("inf")
    logits = wide.to(torch.float32 if kind == "f32" else torch.bfloat16)
    idx = torch.topk(logits[:, :E].float(), k).indices.int()
    mask = torch.rand(T, generator=g, device="cuda") < 0.7 if masked else None
    if masked:  # tokens left out are not looked at
        mask[0], mask[T // 2] = True, False
    whole = logits[:, :E].contiguous()
    assert names_of(lambda: moe.balance_loss(whole, idx, mask)) == (
        {"balance_small"} if T <= 128 and T * k <= 4096 else {"balance_count", "balance_rows"})
    check_case(whole, idx, mask)
    check_case(logits[:, :E], idx, mask)


@pytest.mark.parametrize("E", [100, 512, 2048])
def test_odd_rows_among_many(E):
    """Rows without a distribution, with one expert left, at large values, ids of no expert; NaN in tokens left out."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    g = torch.Generator(device="cuda").manual_seed(E)
    x = torch.randn((700, E), generator=g, device="cuda")
    x[2] = -float("inf")
    x[3, 1:] = -float("inf")
    x[5], x[6] = 88.0, -90.0
    idx = torch.topk(x, 3).indices.int()
    idx[7, 1], idx[8, 0], idx[9] = -1, E, 5
    check_case(x, idx, None)
    mask = torch.ones(700, dtype=torch.bool, device="cuda")
    y = x.clone()
    y[100], y[699, E - 1], mask[100], mask[699] = float("nan"), float("inf"), False, False
    out, same = moe.balance_loss(y, idx, mask), moe.balance_loss(x, idx, mask)
    assert torch.equal(out.losses, same.losses) and torch.equal(out.counts, same.counts) and int(out.kept) == 698
    d = torch.tensor([0.3, 0.7], device="cuda")
    assert torch.equal(moe.balance_loss_backward(y, out, d, mask), moe.balance_loss_backward(x, same, d, mask))
    mask[100] = True
    assert moe.balance_loss(y, idx, mask).losses.isnan().all()


def test_gradient_over_the_logits():
    """The gradient may take the logits' place: every row is read by the wave that writes it, before it does."""
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    g = torch.Generator(device="cuda").manual_seed(1)
    for T, E in ((9000, 512), (9000, 100), (20, 33)):
        x = torch.randn((T, E), generator=g, device="cuda")
        idx = torch.topk(x, 2).indices.int()
        loss, d = moe.balance_loss(x, idx), torch.ones(2, device="cuda")
        want = moe.balance_loss_backward(x, loss, d)
        y = x.clone()
        assert torch.equal(moe.balance_loss_backward(y, loss, d, out=y), want)


@pytest.mark.parametrize("T,E,k,one", [(64, 512, 10, True), (65, 512, 10, False), (128, 256, 8, True), (128, 257, 8, False),
                                       (16, 2048, 16, True), (17, 2048, 3, False), (15, 2047, 4, True), (128, 100, 32, True),
                                       (128, 100, 33, False), (1, 2048, 2048, True)])
def test_either_side_of_the_one_launch_form(T, E, k, one):
    torch = torch_cuda()
    import bit_quantized_moe_topk_amd as moe
    g = torch.Generator(device="cuda").manual_seed(T + E)
    x = torch.randn((T, E), generator=g, device="cuda") * 2
    idx = torch.topk(x, k).indices.int()
    assert names_of(lambda: moe.balance_loss(x, idx)) == ({"balance_small"} if one else {"balance_count", "balance_rows"})
    check_case(x, idx, None)
    check_case(x.bfloat16(), idx, torch.arange(T, device="cuda") % 3 < 2)
