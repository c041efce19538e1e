"""The balance loss at probabilities next to nothing, and its gradient's zeros."""
import pytest
import torch

import tiled_tensor_core_persistent_gb300 as tcg

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tiled_tensor_core_persistent_gb300 import _build
    _build.build()


def call(T, E, k, logits, topk, mask=None, coef=1.0):
    counts = torch.empty(E, dtype=torch.int32, device="cuda")
    valid = torch.empty(1, dtype=torch.int32, device="cuda")
    loss = torch.empty(1, device="cuda")
    n = tcg.moe_balance_workspace_size()
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    tcg.moe_balance(T, E, k, logits, E, "f32", topk, k, mask, coef, counts, None, valid, loss, workspace=ws, workspace_bytes=n)
    return loss, counts, valid


@pytest.mark.parametrize("below", [4.0, 20.0, 30.0, 50.0, 60.0, 80.0])
@pytest.mark.parametrize("T,E", [(20, 32), (3000, 32), (20000, 200)])
def test_experts_of_next_to_no_probability(T, E, below):
    """All assignments fall on experts to which the router gives e^-below of
    the rest: the loss is as exact, relatively, as any other, whatever number
    of tokens.  Tolerance as in the other tests of the loss (sums of positive
    terms), the exponential's argument exact to a unit of its size more."""
    g = torch.Generator(device="cuda").manual_seed(int(below) + T)
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits[:, :3] -= below
    topk = torch.randint(0, 3, (T, 2), generator=g, device="cuda", dtype=torch.int32)
    loss, counts, valid = call(T, E, 2, logits, topk)
    p = torch.softmax(logits.double(), -1).sum(0)
    f = torch.bincount(topk.view(-1).long(), minlength=E).double() * E / (2 * T)
    want = float((f * p).sum() / T)
    units = E / 8 + 16 + T / 100 + E / 16 + 232 + 2 * (below + 10)
    assert abs(float(loss) - want) <= units * 2.0 ** -24 * want, (float(loss), want)


@pytest.mark.parametrize("grad", [float("inf"), float("nan"), 1e38])
@pytest.mark.parametrize("E", [7, 64, 200])
def test_tokens_that_do_not_count_have_gradient_zero_whatever_the_loss_scale(E, grad):
    T, k = 50, 2
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits[3] = -float("inf")
    topk = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    for mask in ((torch.arange(T, device="cuda") % 3 != 0).to(torch.uint8), torch.zeros(T, dtype=torch.uint8, device="cuda")):
        loss, counts, valid = call(T, E, k, logits, topk, mask)
        d = torch.full((T, E), 5.0, device="cuda")
        tcg.moe_balance_backward(T, E, k, logits, E, "f32", mask, 1.0, counts, valid, torch.tensor([grad], device="cuda"), d, E, "f32")
        assert not bool(d[mask == 0].any()) and not bool(d[3].any())
        assert bool(d[1].isfinite().all()) == (grad == 1e38 or not bool(mask.any()))


def test_a_logit_that_is_not_a_number_shows_in_the_loss_and_only_there():
    """Over several CTAs the sums meet in integers: NaN passes through them,
    and nothing of it stays for the next call on the workspace."""
    T, E, k = 3000, 32, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn(T, E, generator=g, device="cuda")
    topk = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    n = tcg.moe_balance_workspace_size()
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    counts = torch.empty(E, dtype=torch.int32, device="cuda")
    valid = torch.empty(1, dtype=torch.int32, device="cuda")
    losses = []
    for bad in (None, float("nan"), float("inf"), None):
        x = logits.clone()
        if bad is not None:
            x[1234, 5] = bad
        loss = torch.empty(1, device="cuda")
        tcg.moe_balance(T, E, k, x, E, "f32", topk, k, None, 1.0, counts, None, valid, loss, workspace=ws, workspace_bytes=n)
        assert torch.equal(counts.long(), torch.bincount(topk.view(-1).long(), minlength=E))
        assert not bool(ws.any())
        losses.append(float(loss))
    assert losses[1] != losses[1] and losses[2] != losses[2] and losses[0] == losses[3] == losses[0]
