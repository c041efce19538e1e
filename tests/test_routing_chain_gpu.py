"""A mixture-of-experts layer's routing and the loss behind it as they are used
together: choice, sort, dispatch, experts' product, combine, loss, and all
gradients, with the same buffers and one workspace in every step and nothing of
another library in between.  Blocks of a call start while the call before still
runs, so a read that came too early, or zeros that a call found spoilt, would
show; each step's results are compared, bit for bit, with the step run alone, and
the first step's with the layer in 64 bits.
"""
import threading

import pytest
import torch

import tiled_tensor_core_persistent_gb300 as tcg

from block128 import wide64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tiled_tensor_core_persistent_gb300 import _build
    _build.build()
    tcg.debug_set()


def blocks(n):
    return -(-n // 128)


class Model:
    """logits -> experts; y = sum of the experts' products of quantised rows; loss of y over a vocabulary."""

    def __init__(self, T, E, k, H, V, steps, seed, renormalize=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.size, self.renormalize = (T, E, k, H, V), renormalize
        self.logits = rand(steps, T, E) + rand(E)
        self.mask = (torch.rand(steps, T, generator=g, device="cuda") < 0.9).to(torch.uint8)
        self.x = rand(steps, T, H).to(torch.bfloat16)
        self.target = torch.randint(-V // 10, V, (steps, T), generator=g, device="cuda", dtype=torch.int32)
        self.words = (rand(V, H) * (2.0 / H ** 0.5)).to(torch.bfloat16)
        w = (rand(E * H, H) / H ** 0.5).to(torch.bfloat16)
        self.wq, self.ws = torch.empty(E * H, H, dtype=torch.uint8, device="cuda"), torch.empty(E, blocks(H), blocks(H), device="cuda")
        tcg.quantize_tiles128(E, H, H, w, H, "bf16", self.wq, H, None, 0, "e4m3", self.ws, stream=torch.cuda.current_stream())
        n = T * k
        ints = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        # the same in every step
        self.topk, self.weights, self.offsets, self.row_token, self.row_of = ints(T, k), f32(T, k), ints(E + 1), ints(n), ints(T, k)
        self.counts, self.valid, self.balance = ints(E), ints(1), f32(1)
        self.xq, self.xs = torch.empty(n, H, dtype=torch.uint8, device="cuda"), f32(blocks(H), n)
        self.out, self.rows, self.y, self.lse = bf(n, H), bf(n, H), bf(T, H), f32(T)
        self.num, self.one = ints(1), torch.ones(1, device="cuda")
        self.dy, self.dout = bf(T, H), bf(n, H)
        self.dweights = f32(T, k)
        # a place for each step
        self.kept = dict(mean=f32(steps, 1), loss=f32(steps, T), dlogits=f32(steps, T, E), dx=bf(steps, T, H), dwords=bf(steps, V, H))
        need = max(tcg.moe_balance_workspace_size(), tcg.moe_sort_workspace_size(T, E, k), tcg.block128_workspace_size(E, n, H, H),
                   tcg.linear_xent_workspace_size(T, V, H, True))
        self.work = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def clear(self):
        for v in self.kept.values():
            v.fill_(-77)
        for v in (self.out, self.rows, self.dout):
            v.zero_()

    def step(self, i, stream):
        T, E, k, H, V = self.size
        n, on, kept = T * k, dict(workspace=self.work, workspace_bytes=self.work.numel(), stream=stream), self.kept
        tcg.moe_route(T, E, k, self.logits[i], E, "f32", self.mask[i], self.renormalize, self.topk, k, self.weights, k, stream=stream)
        tcg.moe_balance(T, E, k, self.logits[i], E, "f32", self.topk, k, self.mask[i], 0.01, self.counts, None, self.valid, self.balance, **on)
        tcg.moe_sort(T, E, k, self.topk, k, self.mask[i], self.offsets, self.row_token, self.row_of, k, **on)
        tcg.moe_dispatch(T, k, H, n, self.x[i], H, "bf16", self.row_of, k, self.rows, H, "bf16", stream=stream)
        tcg.quantize_rows128(n, H, self.rows, H, "bf16", self.xq, H, "e4m3", self.xs, n, stream=stream)
        tcg.gemm_block128_grouped(E, self.offsets, n, H, H, tcg.block_operand(self.xq, H, self.xs, 1, 1, n),
                                  tcg.block_operand(self.wq, H, self.ws, 128, blocks(H), 1, blocks(H) ** 2), self.out, H, "bf16", **on)
        tcg.moe_combine(T, k, H, n, self.out, H, "bf16", self.row_of, k, self.weights, k, self.y, H, "bf16", stream=stream)
        tcg.linear_xent(T, V, H, "bf16", self.y, H, self.words, H, self.target[i], self.lse, kept["loss"][i], kept["mean"][i], self.num, **on)
        tcg.linear_xent_backward(T, V, H, "bf16", self.y, H, self.words, H, self.target[i], self.lse, self.num, self.one, None, self.dy, H, "bf16",
                                 0.0, kept["dwords"][i], H, "bf16", **on)
        tcg.moe_combine_backward(T, k, H, n, self.out, H, "bf16", self.row_of, k, self.weights, k, self.dy, H, "bf16", self.dout, H,
                                 self.dweights, k, stream=stream)
        tcg.moe_balance_backward(T, E, k, self.logits[i], E, "f32", self.mask[i], 0.01, self.counts, self.valid, self.one, kept["dlogits"][i], E,
                                 "f32", stream=stream)
        tcg.moe_route_backward(T, E, k, self.logits[i], E, "f32", self.topk, k, self.renormalize, self.dweights, k, True, kept["dlogits"][i], E,
                               "f32", stream=stream)
        tcg.moe_combine(T, k, H, n, self.dout, H, "bf16", self.row_of, k, None, k, kept["dx"][i], H, "bf16", stream=stream)


SIZES = {"few tokens": (40, 8, 2, 256, 1000), "many": (3000, 24, 4, 384, 2050), "one expert each": (700, 200, 1, 128, 5000)}


def results(m, steps):
    return {k: v[:steps].clone() for k, v in m.kept.items()}


def alone(m, steps):
    m.clear()
    for i in range(steps):
        torch.cuda.synchronize()
        m.step(i, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert tcg.device_status(m.work) == 0
    return results(m, steps)


@pytest.mark.parametrize("which", list(SIZES))
def test_steps_in_a_row_equal_steps_alone(which):
    steps = 6
    m = Model(*SIZES[which], steps, 1)
    want = alone(m, steps)
    stream = torch.cuda.Stream()
    for _ in range(4):
        m.clear()
        torch.cuda.synchronize()
        for i in range(steps):
            m.step(i, stream)
        torch.cuda.synchronize()
        assert tcg.device_status(m.work) == 0
        for name, v in results(m, steps).items():
            assert torch.equal(v, want[name]), name
        # counters and totals are as the calls found them
        assert not bool(m.work[:256 + 8192].any())


def test_streams_and_threads_at_once():
    steps = 6
    models = [Model(*size, steps, 3 + i) for i, size in enumerate(SIZES.values())]
    want = [alone(m, steps) for m in models]
    for m in models:
        m.clear()
    torch.cuda.synchronize()
    errors = []

    def work(m):
        try:
            stream = torch.cuda.Stream()
            for _ in range(4):
                for i in range(steps):
                    m.step(i, stream)
            stream.synchronize()
        except Exception as e:   # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(m,)) for m in models]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    for m, ref in zip(models, want):
        for name, v in results(m, steps).items():
            assert torch.equal(v, ref[name]), name


@pytest.mark.parametrize("which", list(SIZES))
def test_the_layer_and_its_loss_in_64_bits(which):
    """y, the loss and the weights' gradient of one step against the formulas on
    the same codes.  y is rounded twice (the experts' rows and the sum: 2^-8 of
    each term), which moves the loss by |dy . (W_target - mean W)|."""
    m = Model(*SIZES[which], 1, 8)
    alone(m, 1)
    T, E, k, H, V = m.size
    ok = m.mask[0] != 0
    value, index = torch.topk(m.logits[0].double(), k, -1)
    assert torch.equal(m.topk[ok].long(), index[ok])
    w = torch.softmax(value, -1) * ok[:, None]
    assert bool(((m.weights.double() - w).abs() <= 200 * U * w).all())
    live = int(m.offsets[-1])
    token, rows = m.row_token[:live].long(), wide64(m.xq[:live].view(torch.float8_e4m3fn), m.xs[:, :live], 1)
    out = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        a, b = int(m.offsets[e]), int(m.offsets[e + 1])
        if b > a:
            assert bool((m.topk[token[a:b]] == e).any(1).all())
            out[a:b] = rows[a:b] @ wide64(m.wq[e * H:(e + 1) * H].view(torch.float8_e4m3fn), m.ws[e], 128).t()
    at = m.row_of.long()
    picked = torch.where((at >= 0)[..., None], out[at.clamp(min=0)], 0.0)
    y = (picked * w[..., None]).sum(1)
    size = (picked * w[..., None]).abs().sum(1)
    assert bool(((m.y.double() - y).abs() <= 2.02 * 2.0 ** -8 * size + 2.0 ** -30).all())
    z = m.y.double() @ m.words.double().t()
    lse = torch.logsumexp(z, 1)
    t = m.target[0].long()
    counted = t >= 0
    loss = torch.where(counted, lse - z.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    assert bool(((m.kept["loss"][0].double() - loss).abs() <= (H / 16 + 3) * 2.0 ** -21 * float((m.y.double().abs() @ m.words.double().abs().t()).max())
                 + 300 * U * (1 + lse.abs())).all())
    # the weights' gradient of the loss, from the kernel's own dy
    dw = (picked * m.dy.double()[:, None, :]).sum(-1)
    bound = 1.01 * 2.0 ** -8 * (picked * m.dy.double()[:, None, :]).abs().sum(-1)
    assert bool(((m.dweights.double() - dw).abs() <= bound + 2.0 ** -60).all())
