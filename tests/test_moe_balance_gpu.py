"""The router's balance loss, its counts and its gradient on the GPU against
the formula in 64 bits, and the gradient against differences.

Tolerances (u = 2^-24).  A probability is one exp (2 units), a sum of E terms
(E / 8 additions in a lane, 8 more across lanes and chunks) and a product: at
most (E / 8 + 16) u of its value; the loss adds sums over the tokens (at most
T / CTAs + 200 additions in line, all of positive terms) and over the experts.
The gradient is a difference of terms at most max f, each that exact.
"""
import pytest
import torch

import tiled_tensor_core_persistent_gb300 as tcg

from block128 import TYPE, within

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tiled_tensor_core_persistent_gb300 import _build
    _build.build()


class Case:
    def __init__(self, T, E, k, dtype="f32", pad=0, shift=0, mask="none", dropped=True, seed=1, hide=False):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.T, self.E, self.k, self.dtype, self.ld = T, E, k, dtype, E + pad
        flat = torch.full((shift + T * self.ld,), float("nan"), dtype=TYPE[dtype], device="cuda")
        self.logits = flat[shift:].view(T, self.ld)
        x = 2.0 * torch.randn(T, E, generator=g, device="cuda")
        if hide:   # experts that are switched off, and a token without any
            x[:, torch.rand(E, generator=g, device="cuda") < 0.4] = -float("inf")
            if T > 1:
                x[1] = -float("inf")
        self.logits[:, :E] = x.to(TYPE[dtype])
        low = -1 if dropped else 0
        self.topk = torch.randint(low, E + (1 if dropped else 0), (T, k + pad), generator=g, device="cuda", dtype=torch.int32)
        self.mask = None
        if mask == "some":
            self.mask = (torch.rand(T, generator=g, device="cuda") < 0.6).to(torch.uint8) * 3
            self.logits[self.mask == 0] = float("nan")       # padding holds anything
            self.topk[self.mask == 0] = 0
        elif mask == "all":
            self.mask = torch.zeros(T, dtype=torch.uint8, device="cuda")
        self.coef = 0.37
        self.counts = torch.full((E,), -5, dtype=torch.int32, device="cuda")
        self.offsets = torch.full((E + 1,), -5, dtype=torch.int32, device="cuda")
        self.valid = torch.full((1,), -5, dtype=torch.int32, device="cuda")
        self.loss = torch.full((1,), 9.0, device="cuda")
        self.n = tcg.moe_balance_workspace_size()
        self.ws = torch.zeros(self.n, dtype=torch.uint8, device="cuda")

    def forward(self, offsets=True, stream=None):
        tcg.moe_balance(self.T, self.E, self.k, self.logits, self.ld, self.dtype, self.topk, self.topk.shape[1], self.mask, self.coef,
                        self.counts, self.offsets if offsets else None, self.valid, self.loss, workspace=self.ws,
                        workspace_bytes=self.n, stream=stream)

    def backward(self, d="f32", pad=0, grad=1.5):
        out = torch.full((self.T + 2, self.E + pad), 5.0, dtype=TYPE[d], device="cuda")
        tcg.moe_balance_backward(self.T, self.E, self.k, self.logits, self.ld, self.dtype, self.mask, self.coef, self.counts, self.valid,
                                 torch.tensor([grad], device="cuda"), out[1:], self.E + pad, d)
        return out

    def exact(self, logits=None):
        x = (self.logits[:, :self.E] if logits is None else logits).double()
        ok = torch.ones(self.T, dtype=torch.bool, device="cuda") if self.mask is None else self.mask != 0
        p = torch.softmax(x, -1)
        p = torch.where((x == -float("inf")).all(-1, keepdim=True) | ~ok[:, None], 0.0, p)
        picked = self.topk[:, :self.k][ok].reshape(-1).long()
        counts = torch.bincount(picked[(picked >= 0) & (picked < self.E)], minlength=self.E)
        n = int(ok.sum())
        f = counts.double() * self.E / (self.k * max(n, 1))
        loss = self.coef * (f * p.sum(0)).sum() / max(n, 1)
        grad = p * (f - p @ f[:, None]) * self.coef / max(n, 1)
        return loss, counts, n, grad, f


SIZES = [(1, 1, 1), (1, 2, 1), (1, 64, 8), (2, 3, 2), (64, 16, 2), (7, 17, 3), (100, 8, 1), (333, 130, 8), (1000, 256, 8), (50, 300, 4),
         (60, 512, 2), (40, 1000, 6), (30, 1024, 1), (5000, 60, 6), (40000, 64, 2)]


@pytest.mark.parametrize("mask,hide", [("none", False), ("some", False), ("all", False), ("none", True)])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_loss_counts_and_gradient(T, E, k, mask, hide):
    for dtype, pad, shift, d in (("f32", 0, 0, "f32"), ("bf16", 0, 0, "bf16"), ("f16", 3, 1, "f32"), ("bf16", 8, 0, "f16")):
        c = Case(T, E, k, dtype, pad, shift, mask, hide=hide, seed=T + E)
        c.forward(offsets=pad != 3)
        loss, counts, n, grad, f = c.exact()
        assert torch.equal(c.counts.long(), counts) and int(c.valid) == n
        if pad != 3:
            assert torch.equal(c.offsets.long(), torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0)))
        else:
            assert bool((c.offsets == -5).all())
        rel = (E / 8 + 16) * U
        assert abs(float(c.loss) - float(loss)) <= (rel + (T / 100 + 200 + E / 16 + 32) * U) * abs(float(loss))
        out = c.backward(d, pad)
        got = out[1:T + 1, :E].double()
        ref = 1.5 * grad
        bound = 1.5 * c.coef / max(n, 1) * float(f.max()) * (2 * rel + (E / 8 + 24) * U) + 2.0 ** -120
        assert within(out[1:T + 1, :E], ref, bound), float(((got - ref).abs() - bound).max())
        five = torch.tensor(5.0, dtype=out.dtype, device="cuda")
        assert bool((out[0] == five).all()) and bool((out[T + 1] == five).all()) and bool((out[1:T + 1, E:] == five).all())
        if mask == "all":
            assert float(c.loss) == 0.0 and not bool(got.any())
        elif mask == "some":
            assert not bool(got[c.mask == 0].any())


def test_no_tokens():
    c = Case(1, 40, 2)
    tcg.moe_balance(0, 40, 2, None, 40, "f32", None, 2, None, 1.0, c.counts, c.offsets, c.valid, c.loss, workspace=c.ws, workspace_bytes=c.n)
    assert not bool(c.counts.any()) and not bool(c.offsets.any()) and int(c.valid) == 0 and float(c.loss) == 0.0


def test_gradient_against_differences():
    """Central differences of the 64-bit loss (step 1e-5: error 1e-10 of its
    third derivative, below the fp32 gradient's own), for every logit."""
    c = Case(5, 7, 2, "f32", dropped=False, seed=4)
    c.forward()
    got = c.backward(grad=1.0)[1:6, :7].double()
    base = c.logits[:, :7].double()
    h = 1e-5
    for t in range(5):
        for e in range(7):
            up, down = base.clone(), base.clone()
            up[t, e] += h
            down[t, e] -= h
            slope = (float(c.exact(up)[0]) - float(c.exact(down)[0])) / (2 * h)
            assert abs(float(got[t, e]) - slope) <= 1e-6
    # and the loss itself moves along the gradient: fp32 losses, a step of 1e-2, error of the
    # quadratic term at most coef * max f * |step|^2
    moved = Case(5, 7, 2, "f32", dropped=False, seed=4)
    step = 1e-2 * torch.randn(5, 7, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    moved.logits[:, :7] += step
    moved.forward()
    predicted = float((got * step.double()).sum())
    f = c.exact()[4]
    assert abs(float(moved.loss) - float(c.loss) - predicted) <= c.coef * float(f.max()) * float((step ** 2).sum()) / 5 + 8 * U


def test_the_same_every_time_and_in_place():
    c = Case(3000, 100, 4, "f32", mask="some")
    c.forward()
    first = c.loss.clone()
    for _ in range(5):
        c.loss.zero_()
        c.forward()
        assert torch.equal(c.loss, first)
    want = c.backward()[1:3001, :100].clone()
    tcg.moe_balance_backward(c.T, c.E, c.k, c.logits, c.ld, "f32", c.mask, c.coef, c.counts, c.valid, torch.tensor([1.5], device="cuda"),
                             c.logits, c.ld, "f32")
    assert torch.equal(c.logits[:, :100], want)


def test_a_missing_workspace_is_refused():
    c = Case(10, 8, 2)
    for ws, n in ((None, 0), (c.ws, c.n - 1), (c.ws[4:], c.n)):
        c.ws_given = ws
        with pytest.raises(tcg.TcgError) as e:
            tcg.moe_balance(c.T, c.E, c.k, c.logits, c.ld, c.dtype, c.topk, 2, None, 1.0, c.counts, None, c.valid, c.loss, workspace=ws,
                            workspace_bytes=n)
        assert e.value.code == 5


def test_another_stream_and_a_graph():
    c = Case(200, 32, 2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    c.forward(stream=side)
    side.synchronize()
    want = float(c.loss)
    assert abs(want - float(c.exact()[0])) <= 1e-5 * abs(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.forward(stream=torch.cuda.current_stream())
    for _ in range(3):
        c.loss.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert float(c.loss) == want
