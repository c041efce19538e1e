"""The router's choice, its weights and the logits' gradient on the GPU against
the definition in 64 bits.

Tolerances (u = 2^-24).  x - m is rounded (a relative u, so exp is off by
|x - m| u), exp by two units, a sum of E terms by at most E / 32 + 5 additions
in line, a quotient by one: a weight is within (2 D + E / 32 + 16) u of itself, D
the widest finite distance from the maximum.  The gradient is a sum of at most
k + 2 products of such numbers; where it is rounded to 16 bits, half a step more.
"""
import math

import pytest
import torch

import tiled_tensor_core_persistent_gb300 as tcg

from block128 import TYPE

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF = math.inf


@pytest.fixture(autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tiled_tensor_core_persistent_gb300 import _build
    _build.build()


def reference(x, k, renormalize, ok):
    """(topk, weights in 64 bits): k times the first of the largest that is left."""
    T, E = x.shape
    left = torch.where(ok[:, None], x.double(), -INF)
    left = torch.where(left == 0, 0.0, left)
    order = torch.where(left.isnan(), INF, left)
    nan = left.isnan()
    topk = torch.full((T, k), -1, dtype=torch.long, device=x.device)
    rows = torch.arange(T, device=x.device)
    rank = order.clone()
    for j in range(k):
        best = rank.max(1).values
        # (a NaN stands above an infinity)
        first_nan = torch.where(nan, torch.arange(E, device=x.device), E).min(1).values
        first = torch.where(rank == best[:, None], torch.arange(E, device=x.device), E).min(1).values
        pick = torch.where(first_nan < E, first_nan, first)
        real = (best > -INF) | (first_nan < E)
        topk[:, j] = torch.where(real, pick, -1)
        rank[rows, pick] = -INF
        nan[rows, pick] = False
    z = torch.where(ok[:, None], x.double(), -INF)
    live = topk >= 0
    chosen = torch.where(live, z.gather(1, topk.clamp(min=0)), -INF)
    if renormalize:
        w = torch.softmax(chosen, 1)
    else:
        w = torch.exp(chosen - torch.logsumexp(z, 1, keepdim=True))
    return topk, torch.where(live, w, 0.0)


def reference_grad(x, topk, w, g, renormalize):
    T, E = x.shape
    live = (topk >= 0) & (topk < E)
    g = torch.where(live, g.double(), 0.0)
    inner = (w * g).sum(1, keepdim=True)
    size = torch.zeros(T, E, dtype=torch.float64, device=x.device)
    d = torch.zeros_like(size)
    at = topk.clamp(0, E - 1)
    if renormalize:
        part = torch.where(live, w * (g - inner), 0.0)
        d.scatter_add_(1, at, part)
        size.scatter_add_(1, at, torch.where(live, w * (g.abs() + (w * g).abs().sum(1, keepdim=True)), 0.0))
    else:
        p = torch.nan_to_num(torch.softmax(x.double(), 1), nan=0.0)
        direct = torch.zeros_like(d).scatter_add_(1, at, g)
        d = p * (direct - inner)
        size = p * (torch.zeros_like(d).scatter_add_(1, at, g.abs()) + (w * g).abs().sum(1, keepdim=True))
        none = ~live.any(1)
        d[none], size[none] = 0.0, 0.0
    return d, size


class Case:
    def __init__(self, T, E, k, dtype="f32", pad=0, shift=0, mask=False, off=0.0, ties=False, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed + T + 7 * E + k)
        self.T, self.E, self.k, self.dtype, self.ld = T, E, k, dtype, E + pad
        flat = torch.full((shift + T * self.ld,), float("nan"), dtype=TYPE[dtype], device="cuda")
        self.logits = flat[shift:].view(T, self.ld)
        x = 2.0 * torch.randn(T, E, generator=g, device="cuda")
        if ties:
            x = torch.round(x)
            x = torch.where((x == 0) & (torch.rand(T, E, generator=g, device="cuda") < 0.5), -0.0, x)
        if off:
            x[torch.rand(T, E, generator=g, device="cuda") < off] = -INF
        self.logits[:, :E] = x.to(TYPE[dtype])
        self.mask = None
        if mask:
            self.mask = (torch.rand(T, generator=g, device="cuda") < 0.6).to(torch.uint8) * 5
            self.logits[self.mask == 0] = float("nan")
        self.ok = torch.ones(T, dtype=torch.bool, device="cuda") if self.mask is None else self.mask != 0
        self.g = torch.randn(T, k + pad, generator=g, device="cuda")

    def route(self, renormalize, stream=None):
        p = 3 if self.ld != self.E else 0
        topk = torch.full((self.T + 1, self.k + p), -7, dtype=torch.int32, device="cuda")
        w = torch.full((self.T + 1, self.k + p), 9.0, device="cuda")
        tcg.moe_route(self.T, self.E, self.k, self.logits, self.ld, self.dtype, self.mask, renormalize, topk, self.k + p, w, self.k + p,
                      stream=stream)
        assert bool((topk[self.T] == -7).all()) and bool((w[self.T] == 9).all())
        assert bool((topk[:, self.k:] == -7).all()) and bool((w[:, self.k:] == 9).all())
        return topk[:self.T, :self.k], w[:self.T, :self.k]

    def backward(self, topk, renormalize, d="f32", pad=0, accumulate=None):
        out = torch.full((self.T + 1, self.E + pad), 5.0, dtype=TYPE[d], device="cuda")
        if accumulate is not None:
            out[:self.T, :self.E] = accumulate.to(TYPE[d])
        topk = topk.contiguous()
        tcg.moe_route_backward(self.T, self.E, self.k, self.logits, self.ld, self.dtype, topk, self.k, renormalize, self.g, self.g.shape[1],
                               accumulate is not None, out, self.E + pad, d)
        assert bool((out[self.T] == 5).all()) and bool((out[:, self.E:] == 5).all())
        return out[:self.T, :self.E]

    def units(self):
        x = self.logits[:, :self.E].double()
        far = torch.where(x.isfinite() & self.ok[:, None], x, 0.0)
        return (4 * float(far.abs().max()) + self.E / 32 + 16) * U


SIZES = [(1, 1, 1), (1, 2, 2), (3, 5, 3), (64, 16, 2), (7, 33, 8), (100, 64, 6), (50, 100, 32), (1000, 256, 8), (33, 257, 5), (40, 512, 8),
         (30, 1000, 16), (20, 1024, 32), (5000, 60, 1), (20000, 128, 4)]


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_choice_weights_and_gradient(T, E, k, renormalize):
    for dtype, pad, shift, mask, off, ties, d in (("f32", 0, 0, False, 0.0, False, "f32"), ("bf16", 0, 0, True, 0.0, False, "bf16"),
                                                  ("f16", 3, 1, False, 0.3, False, "f32"), ("bf16", 8, 0, False, 0.0, True, "f16"),
                                                  ("f32", 1, 1, True, 0.5, True, "f32")):
        c = Case(T, E, k, dtype, pad, shift, mask, off, ties)
        x = c.logits[:, :E]
        topk, w = c.route(renormalize)
        want, exact = reference(x, k, renormalize, c.ok)
        assert torch.equal(topk.long(), want), (dtype, ties)
        rel = c.units()
        assert bool(((w.double() - exact).abs() <= rel * exact + 2.0 ** -140).all()), (dtype, float(((w.double() - exact).abs() / exact.clamp(min=1e-30)).max()))
        safe = torch.where(c.ok[:, None], x.double(), 0.0)
        ref, size = reference_grad(safe, want, exact, c.g[:, :k], renormalize)
        half = torch.finfo(TYPE[d]).eps / 2 if d != "f32" else U
        tiny = 2.0 ** -25 if d == "f16" else 2.0 ** -120
        bound = (3 * rel + (k + 8) * U) * size + half * ref.abs() * 1.01 + tiny
        got = c.backward(topk, renormalize, d, pad)
        assert bool(((got.double() - ref).abs() <= bound).all()), (dtype, d, float(((got.double() - ref).abs() - bound).max()))
        if mask:
            assert not bool(got[~c.ok].any())
        # added to another gradient, rounded once
        other = torch.randn(T, E, device="cuda").to(TYPE[d])
        got = c.backward(topk, renormalize, d, pad, other)
        total = other.double() + ref
        bound = (3 * rel + (k + 8) * U) * size + (half + U) * total.abs() * 1.01 + U * other.double().abs() + tiny
        assert bool(((got.double() - total).abs() <= bound).all())


@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_against_differences(renormalize):
    T, E, k = 6, 24, 4
    c = Case(T, E, k, "f32")
    topk, w = c.route(renormalize)
    got = c.backward(topk, renormalize).double()
    x, at, g = c.logits.double(), topk.long(), c.g[:, :k].double()

    def total(x):
        if renormalize:
            return (torch.softmax(x.gather(1, at), 1) * g).sum()
        return (torch.softmax(x, 1).gather(1, at) * g).sum()

    h = 1e-5
    for t in range(T):
        for e in range(E):
            step = torch.zeros_like(x)
            step[t, e] = h
            slope = (total(x + step) - total(x - step)) / (2 * h)
            # differences are off by h^2 and by 64-bit rounding over h, the kernel by its units
            assert abs(float(slope - got[t, e])) <= 1e-9 + 40 * U * float(g[t].abs().sum())


def test_an_expert_named_twice_and_entries_out_of_range():
    T, E, k = 5, 20, 6
    c = Case(T, E, k, "f32")
    topk = torch.tensor([[3, 3, 3, 4, -1, 20], [0, 19, 0, 19, 0, 19], [-1] * 6, [25, -5, 7, 100, 7, -1], [1, 2, 3, 4, 5, 6]],
                        dtype=torch.int32, device="cuda")
    for renormalize in (True, False):
        x = c.logits.double()
        live = (topk >= 0) & (topk < E)
        chosen = torch.where(live, x.gather(1, topk.long().clamp(0, E - 1)), -INF)
        w = torch.nan_to_num(torch.softmax(chosen, 1), nan=0.0) if renormalize else torch.where(
            live, torch.softmax(x, 1).gather(1, topk.long().clamp(0, E - 1)), 0.0)
        ref, size = reference_grad(x, topk.long(), w, c.g, renormalize)
        got = c.backward(topk, renormalize).double()
        assert bool(((got - ref).abs() <= 3 * (c.units() + 16 * U) * size + 2.0 ** -120).all())
        assert not bool(got[2].any())
        again = c.backward(topk, renormalize).double()
        assert torch.equal(got, again)


def test_infinities_and_nan():
    """A NaN is chosen first and shows in the token's weights alone; a token
    whose experts are all switched off has none."""
    for dtype in ("f32", "bf16", "f16"):
        x = torch.zeros(6, 40, device="cuda")
        x[0, 17] = float("nan")
        x[1] = -INF
        x[2, 5], x[2, 30] = INF, -INF
        x[3, :39] = -INF
        x[4] = -torch.arange(40.0, device="cuda")
        logits = x.to(TYPE[dtype])
        if dtype == "f32":     # a NaN with its sign set
            logits[5] = torch.tensor([-1], dtype=torch.int32, device="cuda").view(torch.float32)
        else:
            logits[5] = torch.tensor([-1], dtype=torch.int16, device="cuda").view(TYPE[dtype])
        for renormalize in (True, False):
            topk = torch.empty(6, 3, dtype=torch.int32, device="cuda")
            w = torch.empty(6, 3, device="cuda")
            tcg.moe_route(6, 40, 3, logits, 40, dtype, None, renormalize, topk, 3, w, 3)
            assert topk.tolist() == [[17, 0, 1], [-1, -1, -1], [5, 0, 1], [39, -1, -1], [0, 1, 2], [0, 1, 2]]
            assert bool(w[0].isnan().all()) and not bool(w[1].any()) and bool(w[2].isnan().any()) and bool(w[5].isnan().all())
            assert w[3].tolist() == [1.0, 0.0, 0.0] and bool(w[4].isfinite().all())


def test_subnormal_and_largest_logits_keep_their_order():
    for dtype in ("f32", "bf16", "f16"):
        f = torch.finfo(TYPE[dtype])
        v = torch.tensor([f.min, -1.0, -f.tiny, -f.smallest_normal / 4, -0.0, 0.0, f.smallest_normal / 4, f.smallest_normal / 2, f.tiny, 1.0, f.max],
                         dtype=torch.float64).to(TYPE[dtype]).cuda()
        logits = v[torch.randperm(11, generator=torch.Generator().manual_seed(1)).cuda()].view(1, 11).contiguous()
        topk = torch.empty(1, 11, dtype=torch.int32, device="cuda")
        w = torch.empty(1, 11, device="cuda")
        tcg.moe_route(1, 11, 11, logits, 11, dtype, None, True, topk, 11, w, 11)
        order, _ = reference(logits, 11, True, torch.ones(1, dtype=torch.bool, device="cuda"))
        assert torch.equal(topk.long(), order)


def test_gradient_in_place_on_another_stream_and_replayed():
    T, E, k = 300, 96, 4
    c = Case(T, E, k, "bf16", mask=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    topk, w = c.route(False, stream=s)
    s.synchronize()
    want, _ = reference(c.logits, k, False, c.ok)
    assert torch.equal(topk.long(), want)
    ref = c.backward(topk, False, "bf16").clone()
    saved = c.logits.clone()
    topk = topk.contiguous()
    tcg.moe_route_backward(T, E, k, c.logits, E, "bf16", topk, k, False, c.g, k, False, c.logits, E, "bf16")
    assert torch.equal(c.logits, ref)
    c.logits.copy_(saved)
    out = torch.empty(T, E, device="cuda")
    topk2, w2 = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")

    def step():
        st = torch.cuda.current_stream()
        tcg.moe_route(T, E, k, c.logits, E, "bf16", c.mask, True, topk2, k, w2, k, stream=st)
        tcg.moe_route_backward(T, E, k, c.logits, E, "bf16", topk2, k, True, c.g, k, False, out, E, "f32", stream=st)

    torch.cuda.synchronize()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    c.logits.copy_(torch.where(c.ok[:, None], torch.randn(T, E, device="cuda"), saved.float()).to(torch.bfloat16))
    graph.replay()
    got = out.clone()
    want, exact = reference(c.logits, k, True, c.ok)
    assert torch.equal(topk2.long(), want)
    ref, size = reference_grad(torch.where(c.ok[:, None], c.logits.double(), 0.0), want, exact, c.g, True)
    assert bool(((got.double() - ref).abs() <= (3 * c.units() + 20 * U) * size + U * ref.abs() + 2.0 ** -120).all())
