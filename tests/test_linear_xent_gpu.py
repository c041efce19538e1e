"""Softmax cross entropy of a linear layer on the GPU against the formula in 64
bits, and its gradients against the formula and against differences.

Tolerances (u = 2^-24).  A logit is a sum of exact products that the tensor cores
cut to 24 bits after every 16 k (at most 2^-22 of the sum of magnitudes a step,
which counts the terms cut on the way as well): |dz| <= (H / 16 + 3) 2^-22 S, S
the sum of |x w|.  lse moves by no more than the largest |dz|; its exponentials
are good to 2^-22 and their arguments to 2 u of the distance from the maximum,
its sums are 40 additions in line in a thread and 8 + V / 4096 between them.
The gradients sum dz over words or tokens in the same way, dz being off by half
a step of its type, by the relative error of p, by 4 u, and by u of grad_mean / n
where grad_loss is added to that; fp16 adds half a step of its smallest numbers
(2^-25 of 2^14 times the largest weight).
"""
import pytest
import torch

import tiled_tensor_core_persistent_gb300 as tcg

from block128 import TYPE

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tiled_tensor_core_persistent_gb300 import _build
    _build.build()
    tcg.debug_set()
    yield
    tcg.debug_set()


def half_step(t):
    return torch.finfo(TYPE[t]).eps / 2


class Case:
    def __init__(self, T, V, H, dtype="bf16", pad=0, ignored=0.2, seed=0, spread=2.0):
        g = torch.Generator(device="cuda").manual_seed(seed + T + V + H)
        self.T, self.V, self.H, self.dtype = T, V, H, dtype
        self.ld = -(-H // 8) * 8 + 8 * pad
        w = torch.randn(V, H, generator=g, device="cuda") * (spread / H ** 0.5)
        target = torch.randint(0, V, (T,), generator=g, device="cuda")
        x = torch.randn(T, H, generator=g, device="cuda") + 2.0 * torch.rand(T, 1, generator=g, device="cuda") * w[target]
        self.x, self.w = self.held(x), self.held(w)
        drop = torch.rand(T, generator=g, device="cuda")
        target = torch.where(drop < ignored / 2, -100, torch.where(drop < ignored, V + 3, target))
        self.target = target.to(torch.int32)
        self.live = (target >= 0) & (target < V)
        self.lse, self.loss = torch.full((T + 1,), 9.0, device="cuda"), torch.full((T + 1,), 9.0, device="cuda")
        self.mean, self.valid = torch.full((1,), 9.0, device="cuda"), torch.full((1,), -9, dtype=torch.int32, device="cuda")
        self.bytes = tcg.linear_xent_workspace_size(T, V, H, True)
        self.ws = torch.zeros(self.bytes, dtype=torch.uint8, device="cuda")
        self.gen = g

    def held(self, m):
        out = torch.full((m.shape[0], self.ld), float("nan"), dtype=TYPE[self.dtype], device="cuda")
        out[:, :self.H] = m.to(TYPE[self.dtype])
        return out

    def forward(self, loss=True, stream=None):
        tcg.linear_xent(self.T, self.V, self.H, self.dtype, self.x, self.ld, self.w, self.ld, self.target, self.lse,
                        self.loss if loss else None, self.mean, self.valid, workspace=self.ws, workspace_bytes=self.bytes, stream=stream)

    def backward(self, dx_type, dw_type, grad_mean=None, grad_loss=None, beta=0.0, old=None, dx=True, dw=True, pad=0):
        ld = self.H + pad
        gx = torch.full((self.T + 1, ld), 5.0, dtype=TYPE[dx_type], device="cuda")
        gw = torch.full((self.V + 1, ld), 5.0, dtype=TYPE[dw_type], device="cuda")
        if old is not None:
            gw[:self.V, :self.H] = old.to(TYPE[dw_type])
        tcg.linear_xent_backward(self.T, self.V, self.H, self.dtype, self.x, self.ld, self.w, self.ld, self.target, self.lse, self.valid,
                                 grad_mean, grad_loss, gx if dx else None, ld, dx_type, beta, gw if dw else None, ld, dw_type,
                                 workspace=self.ws, workspace_bytes=self.bytes)
        assert tcg.device_status(self.ws) == 0
        assert bool((gx[self.T] == 5).all()) and bool((gw[self.V] == 5).all())
        assert bool((gx[:, self.H:] == 5).all()) and bool((gw[:, self.H:] == 5).all())
        return gx[:self.T, :self.H], gw[:self.V, :self.H]

    def exact(self):
        x, w = self.x[:, :self.H].double(), self.w[:, :self.H].double()
        z = x @ w.t()
        S = float((x.abs() @ w.abs().t()).max()) if z.numel() else 0.0
        lse = torch.logsumexp(z, 1)
        n = int(self.live.sum())
        at = self.target.long().clamp(0, self.V - 1)[:, None]
        loss = torch.where(self.live, lse - z.gather(1, at)[:, 0], 0.0)
        return z, lse, loss, n, S

    def z_error(self, S):
        return (self.H / 16 + 3) * 2.0 ** -22 * S

    def lse_error(self, z, lse, S):
        far = float((z.max() - z.min()).abs()) if z.numel() else 0.0
        return self.z_error(S) + 2.0 ** -22 + (4 * far + 60 + self.V / 4096) * U + U * lse.abs()

    def check_forward(self):
        z, lse, loss, n, S = self.exact()
        err = self.lse_error(z, lse, S)
        assert bool(((self.lse[:self.T].double() - lse).abs() <= err).all()), float(((self.lse[:self.T].double() - lse).abs() - err).max())
        assert bool(((self.loss[:self.T].double() - loss).abs() <= err + self.z_error(S) + U * loss.abs())[self.live].all())
        assert not bool(self.loss[:self.T][~self.live].any())
        assert float(self.lse[self.T]) == 9.0 and float(self.loss[self.T]) == 9.0
        assert int(self.valid) == n
        want = float(loss.sum() / max(n, 1))
        assert abs(float(self.mean) - want) <= float(err.max() if self.T else 0) + self.z_error(S) + 2 * U * abs(want)
        assert tcg.device_status(self.ws) == 0

    def weights(self, grad_mean, grad_loss):
        n = max(int(self.live.sum()), 1)
        r = torch.zeros(self.T, dtype=torch.float64, device="cuda")
        if grad_mean is not None:
            r += float(grad_mean) / n
        if grad_loss is not None:
            r += grad_loss.double()
        return torch.where(self.live, r, 0.0)

    def check_backward(self, gx, gw, grad_mean, grad_loss, beta=0.0, old=None):
        z, lse, _, n, S = self.exact()
        p = torch.exp(z - lse[:, None])
        r = self.weights(grad_mean, grad_loss)
        at = self.target.long().clamp(0, self.V - 1)
        hit = torch.zeros_like(p)
        hit[torch.arange(self.T, device="cuda"), at] = self.live.double()
        dz = r[:, None] * (p - hit)
        rel = float(self.lse_error(z, lse, S).max()) + self.z_error(S) + 8 * U + 2.0 ** -22   # of p
        off = half_step(self.dtype) * dz.abs() * 1.01 + r.abs()[:, None] * (p * rel * 1.01 + 4 * U * (p + hit))
        if grad_mean is not None:
            # r = fl(fl(g / n) + l): the quotient's rounding is u |g / n| whatever the sum is, which may be far smaller
            # than both where l is about -g / n; the sum's own and what follows are the 4 u of r above
            off += torch.where(self.live, U * abs(float(grad_mean)) / max(n, 1), 0.0)[:, None] * (p + hit)
        if self.dtype == "f16":
            off += float(r.abs().max()) * 2.0 ** -39
        size = dz.abs() + off
        x, w = self.x[:, :self.H].double(), self.w[:, :self.H].double()
        for got, ref, bound, add in ((gx, dz @ w, off @ w.abs() + (self.V / 16 + 40) * 2.0 ** -22 * (size @ w.abs()), None),
                                     (gw, dz.t() @ x, off.t() @ x.abs() + (self.T / 16 + 40) * 2.0 ** -22 * (size.t() @ x.abs()), old)):
            if got is None:
                continue
            half = U if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
            if add is not None and beta:
                ref = ref + beta * add.to(got.dtype).double()
                bound = bound + 2 * U * (beta * add.double()).abs()
            bound = bound + 4 * U * ref.abs() + half * (ref.abs() + bound) * 1.01 + (2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -120)
            assert bool(((got.double() - ref).abs() <= bound).all()), float(((got.double() - ref).abs() - bound).max())
            # most of that is the worst case: in the 2-norm the roundings of dz and of the output meet at random
            norm = float(ref.norm())
            if norm > 0 and got.dtype == TYPE[self.dtype] == torch.bfloat16 and self.H <= 2048:
                assert float((got.double() - ref).norm()) <= 2 * half_step("bf16") * norm


SIZES = [(1, 1, 8), (1, 100, 64), (3, 7, 5), (2, 300, 72), (64, 1000, 200), (128, 257, 96), (129, 500, 136), (257, 1030, 72), (256, 256, 64),
         (300, 5000, 1100), (40, 700, 1600), (130, 513, 4104), (700, 3001, 1537), (5, 40000, 256), (64, 40000, 1290)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,V,H", SIZES)
def test_loss_and_gradients(T, V, H, dtype):
    for pad, ignored, dx_type, dw_type, beta in ((0, 0.0, dtype, dtype, 0.0), (1, 0.3, "f32", "f32", 1.0), (0, 0.3, "bf16", "f16", 0.5)):
        c = Case(T, V, H, dtype, pad, ignored)
        c.forward()
        c.check_forward()
        gm = torch.rand(1, generator=c.gen, device="cuda") + 0.5
        gl = torch.randn(T, generator=c.gen, device="cuda") * 0.1 if pad else None
        old = torch.randn(V, H, generator=c.gen, device="cuda").to(TYPE[dw_type]).float() if beta else None
        gx, gw = c.backward(dx_type, dw_type, gm, gl, beta, old, pad=3 * pad)
        c.check_backward(gx, gw, gm, gl, beta, old)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_vocabulary_in_several_pieces(dtype):
    """2048 x 140000 words of dz are more than a piece holds (two and more, the last one shorter)."""
    c = Case(2048, 140011, 64, dtype, ignored=0.1)
    c.forward()
    c.check_forward()
    gm = torch.full((1,), 3.0, device="cuda")
    gx, gw = c.backward(dtype, dtype, gm)
    c.check_backward(gx, gw, gm, None)
    a, b = c.backward("f32", "f32", gm, beta=1.0, old=torch.ones(140011, 64, device="cuda"))
    c.check_backward(a, b, gm, None, 1.0, torch.ones(140011, 64, device="cuda"))


def test_a_vocabulary_in_many_pieces():
    c = Case(5000, 160011, 72, ignored=0.1)
    c.forward()
    c.check_forward()
    gm = torch.ones(1, device="cuda")
    gx, gw = c.backward("bf16", "bf16", gm, pad=8)
    c.check_backward(gx, gw, gm, None)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [1e-12, 1e-4, 1.0, 65536.0, 1e12])
def test_loss_scales(scale, dtype):
    """fp16 holds the gradients of any loss scale (fp32 outputs show them)."""
    c = Case(200, 900, 128, dtype)
    c.forward()
    gm, gl = torch.full((1,), scale, device="cuda"), torch.randn(200, device="cuda") * scale * 0.01
    gx, gw = c.backward("f32", "f32", gm, gl)
    c.check_backward(gx, gw, gm, gl)


@pytest.mark.parametrize("T,V,H", [(70000, 300, 72), (33, 30000, 1032), (5000, 40, 2056)])
def test_many_tokens_many_words_long_rows(T, V, H):
    """More row tiles than CTAs, a long sum in few tiles of dX (split among CTAs), few words."""
    c = Case(T, V, H, "bf16", ignored=0.1)
    c.forward()
    c.check_forward()
    gm, gl = torch.ones(1, device="cuda"), torch.randn(T, device="cuda") / T
    gx, gw = c.backward("bf16", "bf16", gm, gl)
    c.check_backward(gx, gw, gm, gl)
    again = c.backward("bf16", "bf16", gm, gl)
    assert torch.equal(gx, again[0]) and torch.equal(gw, again[1])


def test_weights_past_31_bits():
    """W and dW whose elements reach past 2^31; the last words are looked at."""
    T, V, H = 24, 270000, 8192
    if torch.cuda.get_device_properties(0).total_memory < 64 << 30:
        pytest.skip("needs 20 GB")
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.empty(V, H, dtype=torch.bfloat16, device="cuda")
    for a in range(0, V, 30000):
        w[a:a + 30000] = (torch.randn(min(30000, V - a), H, generator=g, device="cuda") * (2.0 / H ** 0.5)).to(torch.bfloat16)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    target = torch.randint(V - 100, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    lse, loss, mean = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty(1, device="cuda")
    n = torch.empty(1, dtype=torch.int32, device="cuda")
    size = tcg.linear_xent_workspace_size(T, V, H, True)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    tcg.linear_xent(T, V, H, "bf16", x, H, w, H, target, lse, loss, mean, n, workspace=ws, workspace_bytes=size)
    z = torch.cat([x.double() @ w[a:a + 10000].double().t() for a in range(0, V, 10000)], 1)
    ref = torch.logsumexp(z, 1)
    S = float((x.double().abs() @ w[:4000].double().abs().t()).max()) * 1.1
    err = (H / 16 + 3) * 2.0 ** -22 * S + 200 * U + U * ref.abs()
    assert bool(((lse.double() - ref).abs() <= err).all())
    dw = torch.full((V + 1, H), 5.0, dtype=torch.bfloat16, device="cuda")
    dx = torch.empty_like(x)
    gm = torch.ones(1, device="cuda")
    tcg.linear_xent_backward(T, V, H, "bf16", x, H, w, H, target, lse, n, gm, None, dx, H, "bf16", 0.0, dw, H, "bf16", workspace=ws,
                             workspace_bytes=size)
    p = torch.exp(z - ref[:, None]) / T
    p[torch.arange(T, device="cuda"), target.long()] -= 1.0 / T
    for rows in (slice(0, 200), slice(V // 2, V // 2 + 200), slice(V - 200, V)):
        want = p[:, rows].t() @ x.double()
        # half a step of dz and half a step of the output, and p's own error
        bound = (p[:, rows].abs().t() @ x.double().abs()) * (half_step("bf16") * 1.01 + 2 * float(err.max())) + half_step("bf16") * 1.02 * want.abs() + 1e-30
        assert bool(((dw[rows].double() - want).abs() <= bound).all())
    assert bool((dw[V] == 5).all())
    want, bound = torch.zeros(T, H, dtype=torch.float64, device="cuda"), torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for a in range(0, V, 10000):
        want += p[:, a:a + 10000] @ w[a:a + 10000].double()
        bound += p[:, a:a + 10000].abs() @ w[a:a + 10000].double().abs()
    bound = bound * (half_step("bf16") * 1.01 + 2 * float(err.max()) + (8192 / 16 + 40) * 2.0 ** -22) + half_step("bf16") * 1.02 * want.abs()
    assert bool(((dx.double() - want).abs() <= bound).all())


def test_which_gradients_and_outputs():
    c = Case(150, 600, 96)
    c.forward(loss=False)
    assert bool((c.loss == 9).all())
    full = c.loss.clone()
    c.forward()
    c.check_forward()
    del full
    gm, gl = torch.full((1,), 2.0, device="cuda"), torch.randn(150, device="cuda")
    both = c.backward("bf16", "bf16", gm, gl)
    a, untouched = c.backward("bf16", "bf16", gm, gl, dw=False)
    assert torch.equal(a, both[0]) and bool((untouched == 5).all())
    untouched, b = c.backward("bf16", "bf16", gm, gl, dx=False)
    assert torch.equal(b, both[1]) and bool((untouched == 5).all())
    c.backward("bf16", "bf16", gm, gl, dx=False, dw=False)
    for given in ((gm, None), (None, gl)):
        gx, gw = c.backward("bf16", "bf16", *given)
        c.check_backward(gx, gw, *given)
    gx, gw = c.backward("bf16", "f32")           # no gradient of either
    assert not bool(gx.any()) and not bool(gw.any())


def test_no_tokens_and_none_that_count():
    H, V = 40, 70
    for T in (0, 5, 200):
        c = Case(max(T, 1), V, H, ignored=1.1)
        c.T = T
        c.bytes = tcg.linear_xent_workspace_size(T, V, H, True)
        c.forward()
        assert float(c.mean) == 0.0 and int(c.valid) == 0 and not bool(c.loss[:T].any())
        gm = torch.full((1,), float("inf"), device="cuda")       # of a mean of nothing
        old = torch.randn(V, H, device="cuda").to(torch.bfloat16).float()
        gx, gw = c.backward("bf16", "bf16", gm, None, 1.0, old)
        assert not bool(gx.any()) and torch.equal(gw.float(), old)


def test_gradients_against_differences():
    """The slope of the 64-bit loss along random directions against the kernel's gradients."""
    c = Case(33, 150, 64, ignored=0.2, spread=1.0)
    c.forward()
    gm, gl = torch.full((1,), 1.5, device="cuda"), torch.randn(33, device="cuda")
    gx, gw = c.backward("f32", "f32", gm, gl)
    r = c.weights(gm, gl)
    x, w = c.x[:, :64].double(), c.w[:, :64].double()
    at = c.target.long().clamp(0, 149)[:, None]

    def total(x, w):
        z = x @ w.t()
        return (r * (torch.logsumexp(z, 1) - z.gather(1, at)[:, 0])).sum()

    h = 1e-4
    for _ in range(10):
        a = torch.randn(33, 64, generator=c.gen, device="cuda", dtype=torch.float64)
        b = torch.randn(150, 64, generator=c.gen, device="cuda", dtype=torch.float64)
        for slope, grad, step in (((total(x + h * a, w) - total(x - h * a, w)) / (2 * h), gx, a), ((total(x, w + h * b) - total(x, w - h * b)) / (2 * h), gw, b)):
            # half a step of bf16 in every dz at worst; differences are off by h^2 times third derivatives (below 1e3 here)
            assert abs(float(slope - (grad.double() * step).sum())) <= 2 * half_step("bf16") * float((grad.double() * step).abs().sum()) + 1e-5


def test_a_token_that_is_not_a_number():
    c = Case(300, 500, 64, ignored=0.0)
    c.forward()
    before = c.lse.clone()
    c.x[77, 3] = float("nan")
    c.forward()
    assert bool(c.lse[77].isnan()) and bool(c.loss[77].isnan()) and bool(c.mean.isnan())
    c.lse[77] = before[77]
    assert torch.equal(c.lse, before)
    # one that does not count leaves the mean alone
    c.target[77] = -1
    c.forward()
    assert bool(c.lse[77].isnan()) and float(c.loss[77]) == 0.0 and bool(c.mean.isfinite()) and int(c.valid) == 299


def test_words_that_are_nearly_impossible():
    """Logits hundreds below the largest: probabilities of 0, a loss of hundreds."""
    c = Case(70, 300, 64, ignored=0.0)
    c.x[:, :64] = 0.0
    c.x[:, 0] = 16.0
    c.w[:, :64] = 0.0
    c.w[:, 0] = torch.linspace(-40, 40, 300, device="cuda").to(torch.bfloat16)
    c.forward()
    c.check_forward()
    gm = torch.ones(1, device="cuda")
    gx, gw = c.backward("bf16", "bf16", gm)
    c.check_backward(gx, gw, gm, None)


def test_results_are_the_same_every_time_and_leave_the_counters_zero():
    c = Case(777, 5001, 328)
    c.forward()
    first = [v.clone() for v in (c.lse, c.loss, c.mean)]
    gm = torch.ones(1, device="cuda")
    gx, gw = c.backward("bf16", "bf16", gm)
    for _ in range(5):
        c.forward()
        assert all(torch.equal(a, b) for a, b in zip(first, (c.lse, c.loss, c.mean)))
        a, b = c.backward("bf16", "bf16", gm)
        assert torch.equal(a, gx) and torch.equal(b, gw)
        assert not bool(c.ws[:256 + 8192].any())


def test_replayed_graph_and_two_streams():
    cases = [Case(500, 3000, 256, seed=s) for s in (0, 1)]
    gm = torch.ones(1, device="cuda")
    outs = [(torch.zeros(500, 256, device="cuda", dtype=torch.bfloat16), torch.zeros(3000, 256, device="cuda")) for _ in cases]

    def step(c, out):
        st = torch.cuda.current_stream()
        c.forward(stream=st)
        tcg.linear_xent_backward(c.T, c.V, c.H, c.dtype, c.x, c.ld, c.w, c.ld, c.target, c.lse, c.valid, gm, None, out[0], 256, "bf16", 0.0,
                                 out[1], 256, "f32", workspace=c.ws, workspace_bytes=c.bytes, stream=st)

    def check():
        torch.cuda.synchronize()
        for c, out in zip(cases, outs):
            c.check_forward()
            c.check_backward(*out, gm, None)

    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, out, s in zip(cases, outs, streams):
            with torch.cuda.stream(s):
                step(c, out)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cases[0], outs[0])
    cases[0].x[:, :256] = torch.randn(500, 256, device="cuda").to(torch.bfloat16)
    outs[0][0].zero_()
    graph.replay()
    check()


@pytest.mark.parametrize("T", [40, 600])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_exact(T):
    c = Case(T, 3000, 128)
    c.forward()
    torch.cuda.synchronize()
    tcg.debug_set(fault_inject=1, wait_timeout_ns=20_000_000)
    c.forward()
    assert tcg.device_status(c.ws) == 7
    tcg.debug_set()
    c.forward()
    c.check_forward()


@pytest.mark.parametrize("V", [600, 150003])
def test_a_workspace_that_starts_on_any_16_bytes(V):
    c = Case(70 if V < 1000 else 2000, V, 72)
    want = []
    for shift in (0, 16):
        c.ws = torch.zeros(c.bytes + shift + 16, dtype=torch.uint8, device="cuda")[shift:shift + c.bytes]
        assert c.ws.data_ptr() % 32 == shift
        c.forward()
        one = torch.ones(1, device="cuda")
        gx, gw = c.backward("bf16", "f32", one)
        want.append([c.lse.clone(), c.loss.clone(), gx, gw])
    for a, b in zip(*want):
        assert torch.equal(a, b)


def test_a_workspace_that_does_not_do():
    c = Case(10, 50, 64)
    gm = torch.ones(1, device="cuda")
    c.forward()
    for ws, n in ((None, c.bytes), (c.ws, tcg.linear_xent_workspace_size(10, 50, 64, False) - 1), (c.ws[8:], c.bytes)):
        with pytest.raises(tcg.TcgError) as e:
            tcg.linear_xent(10, 50, 64, "bf16", c.x, c.ld, c.w, c.ld, c.target, c.lse, c.loss, c.mean, c.valid, workspace=ws, workspace_bytes=n)
        assert e.value.code == 5
        with pytest.raises(tcg.TcgError) as e:
            tcg.linear_xent_backward(10, 50, 64, "bf16", c.x, c.ld, c.w, c.ld, c.target, c.lse, c.valid, gm, None, torch.empty_like(c.x), c.ld,
                                     "bf16", 0.0, None, 64, "bf16", workspace=ws, workspace_bytes=min(n, c.bytes - 1) if ws is c.ws else n)
        assert e.value.code == 5
