"""One workspace, zero-filled once, serves every entry point in any order, and
a call whose waits ran out leaves nothing behind that a later call trips over.

Operands are integers with power-of-two scales, so every product is exact and
results are compared for equality; counts and offsets are integers.
"""
import pytest
import torch

import tiled_tensor_core_persistent_gb300 as tcg

from block128 import operand, wide64
from test_block128_gpu import int_operand, stacked

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


class Block:
    """gemm_block128 with K shared among the SMs (or, M large, whole pair tiles)."""

    def __init__(self, M, N, K, seed, scale_rows=128):
        a, b = int_operand(M, K, 1, seed), int_operand(N, K, scale_rows, seed + 1)
        self.size = (M, N, K)
        self.A, self.ka = operand(*a, 1)
        self.B, self.kb = operand(*b, scale_rows)
        self.want = wide64(*a, 1) @ wide64(*b, scale_rows).t()
        self.D = torch.empty(M, N, device="cuda")

    def need(self):
        return tcg.block128_workspace_size(0, *self.size)

    def run(self, ws):
        M, N, K = self.size
        self.D.fill_(9.0)
        tcg.gemm_block128(M, N, K, self.A, self.B, 0.0, None, 0, "f32", self.D, N, "f32", workspace=ws, workspace_bytes=ws.numel())

    def check(self):
        assert torch.equal(self.D.double(), self.want)


class Grouped:
    """gemm_block128_grouped, few rows a group."""

    def __init__(self, lens, N, K, seed):
        self.G, self.N, self.K, self.rows = len(lens), N, K, sum(lens)
        a = int_operand(self.rows, K, 1, seed)
        self.A, self.ka = operand(*a, 1)
        self.B, values, self.kb = stacked(self.G, N, K, 128, seed + 1)
        at = [sum(lens[:g]) for g in range(self.G + 1)]
        self.offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
        a64 = wide64(*a, 1)
        self.want = torch.cat([a64[at[g]:at[g + 1]] @ values[g].t() for g in range(self.G)])
        self.D = torch.empty(self.rows, N, device="cuda")

    def need(self):
        return tcg.block128_workspace_size(self.G, self.rows, self.N, self.K)

    def run(self, ws):
        self.D.fill_(9.0)
        tcg.gemm_block128_grouped(self.G, self.offsets, self.rows, self.N, self.K, self.A, self.B, self.D, self.N, "f32", workspace=ws,
                                  workspace_bytes=ws.numel())

    def check(self):
        assert torch.equal(self.D.double(), self.want)


class Balance:
    """moe_balance over several CTAs."""

    def __init__(self, T, E, k, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.size = (T, E, k)
        self.logits = torch.randn(T, E, generator=g, device="cuda")
        self.topk = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
        self.counts = torch.empty(E, dtype=torch.int32, device="cuda")
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        self.valid = torch.empty(1, dtype=torch.int32, device="cuda")
        self.loss = torch.empty(1, device="cuda")

    def need(self):
        return tcg.moe_balance_workspace_size()

    def run(self, ws):
        T, E, k = self.size
        tcg.moe_balance(T, E, k, self.logits, E, "f32", self.topk, k, None, 1.0, self.counts, self.offsets, self.valid, self.loss,
                        workspace=ws, workspace_bytes=ws.numel())

    def check(self):
        T, E, k = self.size
        counts = torch.bincount(self.topk.view(-1).long(), minlength=E)
        assert torch.equal(self.counts.long(), counts) and int(self.valid) == T
        assert torch.equal(self.offsets.long(), torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0)))
        p = torch.softmax(self.logits.double(), -1).sum(0)
        want = float((counts.double() * E / (k * T) * p).sum() / T)
        # positive terms: a probability within (E / 8 + 16) units, the sums within T / 100 + E / 16 + 232
        assert abs(float(self.loss) - want) <= (E / 8 + 16 + T / 100 + E / 16 + 232) * 2.0 ** -24 * want


class Dense:
    """tcg_gemm in bf16: K split (few tiles), whole tiles, or operands that are packed first."""

    def __init__(self, M, N, K, seed, lda=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.size, self.lda = (M, N, K), lda or K
        A = torch.zeros(M, self.lda, dtype=torch.bfloat16, device="cuda")
        A[:, :K] = torch.randint(-4, 5, (M, K), generator=g, device="cuda")
        B = torch.randint(-4, 5, (N, K), generator=g, device="cuda").to(torch.bfloat16)
        self.A, self.B = A, B
        self.want = A[:, :K].double() @ B.double().t()
        self.D = torch.empty(M, N, device="cuda")

    def need(self):
        M, N, K = self.size
        return tcg.workspace_size_for(M, N, K, "bf16", self.A, self.lda, "row", self.B, K, "col")

    def run(self, ws):
        M, N, K = self.size
        self.D.fill_(9.0)
        tcg.gemm(M, N, K, 1.0, self.A, self.lda, "row", self.B, K, "col", 0.0, None, N, "f32", self.D, N, "f32", workspace=ws,
                 workspace_bytes=ws.numel())

    def check(self):
        assert torch.equal(self.D.double(), self.want)


class DenseGrouped:
    """tcg_gemm_grouped: its table of problems lives in the workspace."""

    def __init__(self, sizes, seed):
        self.parts = [Dense(*s, seed + i) for i, s in enumerate(sizes)]

    def need(self):
        return tcg.grouped_workspace_size(len(self.parts))

    def run(self, ws):
        problems = []
        for d in self.parts:
            M, N, K = d.size
            d.D.fill_(9.0)
            problems.append(dict(M=M, N=N, K=K, A=d.A, lda=K, B=d.B, ldb=K, D=d.D, ldd=N))
        tcg.gemm_grouped(problems, "row", "col", 0.0, "f32", "f32", workspace=ws, workspace_bytes=ws.numel())

    def check(self):
        for d in self.parts:
            d.check()


def share(calls):
    """Every ordered pair of the calls on one workspace that is zero-filled once."""
    ws = torch.zeros(max(c.need() for c in calls), dtype=torch.uint8, device="cuda")
    for first in calls:
        for second in calls:
            first.run(ws)
            second.run(ws)
            assert tcg.device_status(ws) == 0
            first.check()
            second.check()


def test_block_scaled_products_and_the_balance_loss_share_a_workspace():
    share([Block(16, 1500, 8192, 1), Block(120, 300, 9000, 3, 1), Grouped([3, 0, 1, 9, 2], 700, 4096, 5), Balance(4000, 100, 4, 7),
           Balance(20, 9, 2, 8), Block(2048, 2560, 512, 9)])


def test_every_entry_point_shares_a_workspace():
    share([Dense(16, 4096, 8192, 11), Dense(500, 300, 4096, 12), Dense(333, 290, 201, 13, lda=202), Dense(300, 2000, 2500, 14, lda=2501),
           DenseGrouped([(100, 300, 128), (7, 260, 512), (64, 128, 256)], 15), Block(16, 1500, 8192, 1), Grouped([3, 0, 1, 9, 2], 700, 4096, 5),
           Balance(4000, 100, 4, 7)])


@pytest.mark.parametrize("which", ["dense", "few rows", "one tile", "grouped"])
def test_a_call_after_one_whose_waits_ran_out_is_exact(which):
    """The test knob lets the first CTA's producer skip its first stage, so
    some tiles' pieces arrive and others do not; reading the status makes the
    workspace ready again without another zero-fill, its counters included
    (the first 8448 bytes hold the status words and the counters)."""
    make = dict(dense=lambda s: Dense(16, 4096, 8192, s), **{
        "few rows": lambda s: Block(4, 900, 8192, s), "one tile": lambda s: Block(120, 300, 9000, s),
        "grouped": lambda s: Grouped([3, 0, 1, 9, 2], 700, 4096, s)})[which]
    calls = [make(s) for s in (1, 11, 21)]      # other operands: sums left over from one call are wrong for the next
    ws = torch.zeros(calls[0].need(), dtype=torch.uint8, device="cuda")
    tcg.debug_set(fault_inject=1, wait_timeout_ns=200_000_000)
    calls[0].run(ws)
    assert tcg.device_status(ws) == 7
    tcg.debug_set()
    assert not bool(ws[:256 + 8192].any())
    for call in calls[1:] + calls:
        call.run(ws)
        assert tcg.device_status(ws) == 0
        call.check()
