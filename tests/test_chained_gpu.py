"""One operator feeding the next with nothing of another library in between,
and calls in flight on several streams and from several host threads.

Blocks of a call are launched while the call before still runs, and wait for
it before they read.  The buffers that carry codes, scales, offsets and
workspace from call to call are the same in every step, so a read that came
too early, or from a cache that the step before filled, would show the step
before's values.  Each step's results are kept and compared, bit for bit, with
the same step run alone.
"""
import threading

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
    tcg.debug_set()


def blocks(n):
    return -(-n // 128)


class Linear:
    """x by rows and w by tiles, quantised into the same buffers every step, and their product."""

    def __init__(self, M, N, K, steps, seed, pow2=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.size, self.pow2 = (M, N, K), pow2
        self.x = torch.randn(steps, M, K, generator=g, device="cuda").to(torch.bfloat16)
        self.x *= torch.exp2(torch.randint(-9, 9, (steps, M, 1), generator=g, device="cuda").float()).to(torch.bfloat16)
        self.w = torch.randn(2, N, K, generator=g, device="cuda").to(torch.bfloat16)
        self.xq = torch.empty(M, K, dtype=torch.uint8, device="cuda")
        self.xs = torch.empty(blocks(K), M, device="cuda")
        self.wq = torch.empty(N, K, dtype=torch.uint8, device="cuda")
        self.ws = torch.empty(blocks(N), blocks(K), device="cuda")
        self.work = torch.zeros(tcg.block128_workspace_size(0, M, N, K), dtype=torch.uint8, device="cuda")
        self.out = torch.empty(steps, M, N, device="cuda")

    def step(self, i, stream):
        M, N, K = self.size
        tcg.quantize_tiles128(1, N, K, self.w[i % 2], K, "bf16", self.wq, K, None, 0, "e4m3", self.ws, pow2=self.pow2, stream=stream)
        tcg.quantize_rows128(M, K, self.x[i], K, "bf16", self.xq, K, "e4m3", self.xs, M, pow2=self.pow2, stream=stream)
        tcg.gemm_block128(M, N, K, tcg.block_operand(self.xq, K, self.xs, 1, 1, M),
                          tcg.block_operand(self.wq, K, self.ws, 128, blocks(K), 1), 0.0, None, 0, "f32", self.out[i], N, "f32",
                          workspace=self.work, workspace_bytes=self.work.numel(), stream=stream)


class Routed:
    """The router's counts and offsets, the grouped product that reads them, and its weight gradient."""

    def __init__(self, T, E, N, K, steps, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.size = (T, E, N, K)
        self.logits = torch.randn(T, E, generator=g, device="cuda")
        self.topk = torch.randint(0, E, (steps, T, 1), generator=g, device="cuda", dtype=torch.int32)
        self.topk = torch.minimum(self.topk, torch.randint(0, E, (steps, 1, 1), generator=g, device="cuda", dtype=torch.int32))   # skewed
        self.x = torch.randn(steps, T, K, generator=g, device="cuda")
        self.xq = torch.empty(T, K, dtype=torch.uint8, device="cuda")
        self.xs = torch.empty(blocks(K), T, device="cuda")
        self.places = (T // 128 + E) * 128
        self.xt = torch.empty(K, self.places, dtype=torch.uint8, device="cuda")
        self.xts = torch.empty(self.places // 128, K, device="cuda")
        w = torch.randn(E * N, K, generator=g, device="cuda").to(torch.bfloat16)
        self.wq = torch.empty(E * N, K, dtype=torch.uint8, device="cuda")
        self.ws = torch.empty(E, blocks(N), blocks(K), device="cuda")
        tcg.quantize_tiles128(E, N, K, w, K, "bf16", self.wq, K, None, 0, "e4m3", self.ws, stream=torch.cuda.current_stream())
        self.counts = torch.empty(steps, E, dtype=torch.int32, device="cuda")
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        self.valid = torch.empty(1, dtype=torch.int32, device="cuda")
        self.loss = torch.empty(steps, 1, device="cuda")
        need = max(tcg.moe_balance_workspace_size(), tcg.block128_workspace_size(E, T, N, K))
        self.work = torch.zeros(need, dtype=torch.uint8, device="cuda")
        self.out = torch.empty(steps, T, N, device="cuda")
        self.grad = torch.empty(steps, E, K, K, device="cuda")

    def step(self, i, stream):
        T, E, N, K = self.size
        on = dict(workspace=self.work, workspace_bytes=self.work.numel(), stream=stream)
        tcg.moe_balance(T, E, 1, self.logits, E, "f32", self.topk[i], 1, None, 1.0, self.counts[i], self.offsets, self.valid, self.loss[i], **on)
        tcg.quantize_rows128(T, K, self.x[i], K, "f32", self.xq, K, "e4m3", self.xs, T, stream=stream)
        tcg.quantize_cols128(T, K, self.x[i], K, "f32", self.xt, self.places, "e4m3", self.xts, K, padded_rows=self.places, num_groups=E,
                             offsets=self.offsets, stream=stream)
        tcg.gemm_block128_grouped(E, self.offsets, T, N, K, tcg.block_operand(self.xq, K, self.xs, 1, 1, T),
                                  tcg.block_operand(self.wq, K, self.ws, 128, blocks(K), 1, blocks(N) * blocks(K)), self.out[i], N, "f32", **on)
        a = tcg.block_operand(self.xt, self.places, self.xts, 1, 1, K)
        tcg.gemm_block128_grouped_k(E, self.offsets, K, K, self.places, a, a, 0.0, None, K, "f32", self.grad[i], K, "f32", **on)


MAKE = {
    "few rows": lambda steps, seed: Linear(8, 1024, 4096, steps, seed),
    "single tiles": lambda steps, seed: Linear(96, 640, 2048, steps, seed),
    "pairs": lambda steps, seed: Linear(2048, 2560, 512, steps, seed),
    "few rows routed": lambda steps, seed: Routed(64, 8, 512, 256, steps, seed),
    "many rows routed": lambda steps, seed: Routed(3000, 6, 768, 512, steps, seed),
}


def results(job):
    return [t.clone() for t in (job.out, *([job.counts, job.loss, job.grad] if isinstance(job, Routed) else []))]


def alone(job, steps):
    stream = torch.cuda.current_stream()
    for i in range(steps):
        torch.cuda.synchronize()
        job.step(i, stream)
    torch.cuda.synchronize()
    return results(job)


@pytest.mark.parametrize("which", list(MAKE))
def test_steps_in_a_row_equal_steps_alone(which):
    steps = 12
    job = MAKE[which](steps, 1)
    want = alone(job, steps)
    stream = torch.cuda.Stream()
    for _ in range(5):
        job.out.fill_(float("nan"))
        torch.cuda.synchronize()
        for i in range(steps):
            job.step(i, stream)
        torch.cuda.synchronize()
        assert tcg.device_status(job.work) == 0
        for a, b in zip(results(job), want):
            assert torch.equal(a, b)


def test_streams_and_threads_at_once():
    """Every kind of step on a stream and from a host thread of its own, at the same time."""
    steps = 12
    jobs = [make(steps, 10 + i) for i, make in enumerate(MAKE.values())]
    want = [alone(job, steps) for job in jobs]
    for job in jobs:
        job.out.fill_(float("nan"))
    torch.cuda.synchronize()
    errors = []

    def work(job):
        try:
            stream = torch.cuda.Stream()
            for _ in range(5):
                for i in range(steps):
                    job.step(i, stream)
            stream.synchronize()
        except Exception as e:   # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(job,)) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    for job, ref in zip(jobs, want):
        assert tcg.device_status(job.work) == 0
        for a, b in zip(results(job), ref):
            assert torch.equal(a, b)
