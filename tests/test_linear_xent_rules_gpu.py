"""Softmax cross entropy of a linear layer: what its gradients take from the
forward call, tokens' weights that are not finite, and very long sums.

Tolerances as in test_linear_xent_gpu.py (u = 2^-24).  The logits' sums are taken
in parts of at most 1536 k, cut after every 16 (at most 2^-22 of the part's
magnitudes a step), and the parts are added with a rounding each: a logit is off by
no more than ((1536 + 128) / 16 2^-22 + (H / 1024 + 2) u) S.
"""
import copy

import pytest
import torch

import tiled_tensor_core_persistent_gb300 as tcg

from test_linear_xent_gpu import U, Case, half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tiled_tensor_core_persistent_gb300 import _build
    _build.build()
    tcg.debug_set()
    yield
    tcg.debug_set()


def sure(T, V, H, dtype, unlikely=1e-4):
    """Every token's hidden state lies along its target's weights, so that all other words together have about
    `unlikely`; the products of the target's logit are all of one sign.  W's first column is 1 (and X's 0): the first
    column of dX is the sum of dz over the words, which is 0."""
    c = Case(T, V, H, dtype, ignored=0.0)
    w = torch.randn(V, H, generator=c.gen, device="cuda") * (2.0 / H ** 0.5)
    w[:, 0] = 1.0
    c.w = c.held(w)
    at = c.w[c.target.long(), :H].float()
    at[:, 0] = 0.0
    z = torch.log(torch.tensor(V / unlikely))
    c.x = c.held(at * (z.cuda() / (at * at).sum(1, keepdim=True)))
    return c


def sum_error(H, S):
    return ((1536 + 128) / 16 * 2.0 ** -22 + (H / 1024 + 2) * U) * S


LONG = [(100, 300, 131080), (200, 300, 131080)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,V,H", LONG)
def test_long_sums_of_one_sign(T, V, H, dtype):
    """Sums of 131080 products in one go are about five times this bound too near zero."""
    c = sure(T, V, H, dtype)
    c.forward()
    _, lse, loss, _, S = c.exact()
    # (exponentials, their sums and the join: a probability that is all but 1)
    err = sum_error(H, S) + 2.0 ** -22 + 60 * U + U * lse.abs()
    assert bool(((c.lse[:T].double() - lse).abs() <= err).all()), float(((c.lse[:T].double() - lse).abs() - err).max())
    # the loss is lse less the target's logit, which are off together
    assert bool(((c.loss[:T].double() - loss).abs() <= 2 * sum_error(H, S) * loss + 2.0 ** -22 + 60 * U + 2 * U * lse.abs()).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,V,H", LONG)
def test_gradients_of_what_is_all_but_certain(T, V, H, dtype):
    """exp(z - lse) of a target of probability p is off by (1 - p) times what z is off, as lse is off with it, plus
    roundings of lse (here and times log2 e): the gradient takes the same sums as the loss."""
    c = sure(T, V, H, dtype)
    c.forward()
    z, lse, _, n, S = c.exact()
    gm = torch.full((1,), float(n), device="cuda")      # every token's weight is 1
    gx, gw = c.backward("f32", "f32", gm)
    p = torch.exp(z - lse[:, None])
    rows, y = torch.arange(T, device="cuda"), c.target.long()
    rest = p.clone()
    rest[rows, y] = 0.0
    rest = rest.sum(1)                                  # 1 - p of the target
    assert 1e-5 < float(rest.min()) and float(rest.max()) < 1e-3
    dz = p.clone()
    dz[rows, y] = -rest
    arg = 2 * U * lse.abs() + 2 * 2.0 ** -22 + 16 * U   # roundings of lse and of its multiple, the exponentials here and there
    off = p * (2 * sum_error(H, S) + arg[:, None])
    off[rows, y] = rest * 2 * sum_error(H, S) + arg + 4 * U
    off = off * 1.01 + half_step(dtype) * (dz.abs() + off) * 1.01 + (2.0 ** -39 if dtype == "f16" else 0.0)
    x, w = c.x[:, :H].double(), c.w[:, :H].double()
    size = dz.abs() + off
    for got, ref, bound in ((gx, dz @ w, off @ w.abs() + (V / 16 + 40) * 2.0 ** -22 * (size @ w.abs())),
                            (gw, dz.t() @ x, off.t() @ x.abs() + (T / 16 + 40) * 2.0 ** -22 * (size.t() @ x.abs()))):
        bound = bound + 5 * U * ref.abs() + 2.0 ** -120
        assert bool(((got.double() - ref).abs() <= bound).all()), float(((got.double() - ref).abs() / bound).max())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("weight", [float("inf"), float("-inf"), float("nan")])
def test_a_weight_that_is_not_finite_leaves_other_tokens_alone(weight, dtype):
    """dz is held over the largest weight that is finite: the others' gradients are as without that token."""
    c = Case(260, 700, 72, dtype, ignored=0.1)
    c.target[131] = 5
    c.live[131] = True
    c.forward()
    for size in (1e-9, 20.0):
        gl = torch.randn(260, generator=c.gen, device="cuda") * size
        gl[131] = 0.0
        want, _ = c.backward("f32", "f32", None, gl)
        want = want.clone()
        gl[131] = weight
        got, gw = c.backward("f32", "f32", None, gl)
        others = torch.arange(260, device="cuda") != 131
        assert torch.equal(got[others], want[others]) and bool(want[others].isfinite().all())
        assert not bool(got[131].isfinite().any())
        gl[~c.live] = weight                            # of tokens that do not count: nothing
        gl[131] = 0.0
        again, _ = c.backward("f32", "f32", None, gl)
        assert torch.equal(again, want)


class Spread(Case):
    """A case of 64 hidden values that stand in `hidden` columns, all others 0 (the first and the last are among them)."""

    def __init__(self, T, V, hidden):
        super().__init__(T, V, 64, ignored=0.2)
        self.hidden = hidden
        at = torch.randint(1, hidden - 1, (64,), generator=self.gen, device="cuda").unique()
        assert at.numel() == 64
        at[0], at[-1] = 0, hidden - 1
        self.at = at
        self.wide = [torch.zeros(m.shape[0], -(-hidden // 8) * 8, dtype=m.dtype, device="cuda") for m in (self.x, self.w)]
        for big, m in zip(self.wide, (self.x, self.w)):
            big[:, at] = m[:, :64]
        self.bytes = tcg.linear_xent_workspace_size(T, V, hidden, True)
        self.ws = torch.zeros(self.bytes, dtype=torch.uint8, device="cuda")

    def z_error(self, S):
        return (64 + 3) * 2.0 ** -22 * S + 64 * U * S     # zeros cut nothing


@pytest.mark.parametrize("T,V,H", [(3, 5, 12_000_008), (130, 6, 16_800_001)])
def test_hidden_sizes_of_many_millions(T, V, H):
    """Stages of K times parts of K pass 2^31; one CTA a tile, and a pair."""
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 20 GB")
    c = Spread(T, V, H)
    x, w = c.wide
    ld = x.shape[1]
    tcg.linear_xent(T, V, H, "bf16", x, ld, w, ld, c.target, c.lse, c.loss, c.mean, c.valid, workspace=c.ws, workspace_bytes=c.bytes)
    c.check_forward()
    gm = torch.ones(1, device="cuda")
    gx, gw = torch.full_like(x, 5.0), torch.full_like(w, 5.0)
    tcg.linear_xent_backward(T, V, H, "bf16", x, ld, w, ld, c.target, c.lse, c.valid, gm, None, gx, ld, "bf16", 0.0, gw, ld, "bf16",
                             workspace=c.ws, workspace_bytes=c.bytes)
    assert tcg.device_status(c.ws) == 0
    c.check_backward(gx[:, c.at], gw[:, c.at], gm, None)
    for g in (gx, gw):
        assert bool((g[:, H:] == 5).all())
        g[:, c.at] = 0
        assert not bool(g[:, :H].any())


@pytest.mark.parametrize("T,V,H,split", [(40, 3000, 128, True), (600, 3000, 128, True), (33, 30000, 1032, True), (2048, 140011, 64, False)])
def test_a_wait_of_the_gradient_that_runs_out_is_reported_and_the_next_call_is_exact(T, V, H, split):
    """In the kernel of dz and in that of the products, whose split tiles are left with counters that count; one piece of
    the vocabulary and two."""
    c = Case(T, V, H)
    c.forward()
    gm = torch.ones(1, device="cuda")
    want = [g.clone() for g in c.backward("bf16", "bf16", gm)]
    gx, gw = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(V, H, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    tcg.debug_set(fault_inject=1, wait_timeout_ns=20_000_000)
    tcg.linear_xent_backward(T, V, H, "bf16", c.x, c.ld, c.w, c.ld, c.target, c.lse, c.valid, gm, None, gx, H, "bf16", 0.0, gw, H, "bf16",
                             workspace=c.ws, workspace_bytes=c.bytes)
    torch.cuda.synchronize()
    counters = c.ws[256:256 + 8192]
    assert bool(counters.any()) or not split
    assert tcg.device_status(c.ws) == 7
    tcg.debug_set()
    assert not bool(counters.any())
    got = c.backward("bf16", "bf16", gm)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    c.forward()
    c.check_forward()
    c.check_backward(*got, gm, None)


@pytest.mark.parametrize("dx_type", ["bf16", "f32"])
def test_nine_pieces_of_a_vocabulary(dx_type):
    """262144 tokens leave a piece 1024 words; looked at in 64 bits, 16384 tokens at a time."""
    T, V, H, step = 262144, 9000, 64, 16384
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 20 GB")
    c = Case(T, V, H, ignored=0.1)
    assert c.bytes < (512 << 20) + T * H * 4 + (300 << 20)      # not of the whole vocabulary (4.7 GB)
    c.forward()
    n = int(c.live.sum())
    assert int(c.valid) == n
    gm = torch.full((1,), 3.0 * n, device="cuda")
    gx, gw = c.backward(dx_type, "f32", gm)
    each = torch.full((T,), float(gm / c.valid.float()), device="cuda")     # every token's weight
    want, bound = (torch.zeros(V, H, dtype=torch.double, device="cuda") for _ in range(2))
    for a in range(0, T, step):
        s = copy.copy(c)
        s.T = step
        s.x, s.target, s.live, s.lse = c.x[a:a + step], c.target[a:a + step], c.live[a:a + step], c.lse[a:a + step]
        s.check_backward(gx[a:a + step], None, None, each[a:a + step])
        z, lse, _, _, S = s.exact()
        err = s.lse_error(z, lse, S)
        assert bool(((s.lse.double() - lse).abs() <= err).all())
        p = torch.exp(z - lse[:, None])
        hit = torch.zeros_like(p)
        hit[torch.arange(step, device="cuda"), s.target.long().clamp(0, V - 1)] = s.live.double()
        r = torch.where(s.live, each[a:a + step].double(), 0.0)[:, None]
        dz = r * (p - hit)
        off = half_step("bf16") * dz.abs() * 1.01 + r * (p * (float(err.max()) + s.z_error(S) + 8 * U + 2.0 ** -22) * 1.01 + 4 * U * (p + hit))
        x = s.x[:, :H].double()
        want += dz.t() @ x
        bound += off.t() @ x.abs() + (8192 / 16 + T / 8192 + 40) * 2.0 ** -22 * ((dz.abs() + off).t() @ x.abs())
    assert bool(((gw.double() - want).abs() <= bound + 4 * U * want.abs()).all())
