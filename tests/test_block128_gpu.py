"""The block-scaled 8-bit products on the GPU against 64-bit products of the
same operands.

Tolerances.  Integers with power-of-two scales: every partial sum is a number
fp32 holds, so the results are equal.  Otherwise, with S = |A| |B|^T the sum of
the terms' magnitudes and u = 2^-24: a sum of 128 products in any order loses at
most 128 u S, its scaling and the sum over the k-blocks (kb + 4) u S more, bias
and beta C two roundings of the result; bf16 results half a unit, 2^-9 of the
value.  GELU changes errors by at most 1.13 and its erf adds 1.5e-7 |x| / 2 + the
rounding of its fp32 steps, 16 u |x|.
"""
import pytest
import torch

import tiled_tensor_core_persistent_gb300 as tcg

from block128 import CODE, ceil_div, operand, padded_places, quantize_rows, quantize_tiles, wide64, within, workspace

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SENTINEL = 777.0


@pytest.fixture(autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tiled_tensor_core_persistent_gb300 import _build
    _build.build()
    tcg.debug_set()
    yield
    tcg.debug_set()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def int_operand(r, k, scale_rows, seed, q="e4m3"):
    """Codes of integers in [-4, 4], scales 1/2, 1 or 2."""
    g = gen(seed)
    codes = torch.randint(-4, 5, (r, k), generator=g, device="cuda").float().to(CODE[q])
    kb = ceil_div(k, 128)
    shape = (kb, r) if scale_rows == 1 else (ceil_div(r, 128), kb)
    scales = torch.exp2(torch.randint(-1, 2, shape, generator=g, device="cuda").float())
    return codes, scales


def real_operand(r, k, scale_rows, seed, q="e4m3"):
    g = gen(seed)
    x = torch.randn(r, k, generator=g, device="cuda") * torch.exp(torch.randn(1, k, generator=g, device="cuda"))
    return quantize_rows(x, q) if scale_rows == 1 else quantize_tiles(x, q)


class Out:
    """D (and C) with a border of sentinels and a chosen pitch and offset."""

    def __init__(self, rows, cols, dtype, pad=0, shift=0):
        self.rows, self.cols, self.ld, self.shift = rows, cols, cols + pad, shift
        self.flat = torch.full((shift + (rows + 2) * self.ld,), SENTINEL, dtype=dtype, device="cuda")
        self.full = self.flat[shift:].view(rows + 2, self.ld)
        self.view = self.full[1:rows + 1, :cols]
        self.start = self.full[1:]

    def clean(self):
        mark = torch.tensor(SENTINEL, dtype=self.flat.dtype, device="cuda")
        inner = self.full.clone()
        inner[1:self.rows + 1, :self.cols] = mark
        return bool((inner == mark).all()) and bool((self.flat[:self.shift] == mark).all())


def ws_header_clean(ws):
    return not ws[:256 + 8192].any()


SHAPES = [(1, 1, 1), (1, 128, 128), (1, 4096, 8192), (2, 300, 129), (3, 130, 257), (16, 512, 1024), (17, 129, 2048), (33, 200, 384),
          (64, 1000, 640), (65, 129, 130), (128, 256, 128), (129, 257, 1000), (300, 520, 1100), (256, 4096, 512), (700, 96, 5000),
          (1000, 3000, 1000), (2049, 2310, 384), (2560, 2500, 127), (4100, 1100, 129)]


@pytest.mark.parametrize("scale_rows", [1, 128])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_integers_are_exact(M, N, K, scale_rows):
    """Every tile shape, ragged in every direction, both scale forms of B, both orders of the scales."""
    seed = M * 7 + N * 3 + K + scale_rows
    a, b = int_operand(M, K, 1, seed), int_operand(N, K, scale_rows, seed + 1)
    want = wide64(*a, 1) @ wide64(*b, scale_rows).t()
    A, ka = operand(*a, 1, k_minor=bool(seed & 1))
    B, kb = operand(*b, scale_rows, extra=1, k_minor=bool(seed & 2))
    n = tcg.block128_workspace_size(0, M, N, K)
    ws = workspace(n)
    for d, pad, shift in (("f32", 0, 0), ("f32", 3, 1), ("bf16", 5, 1), ("bf16", (-N) % 16 + 16, 0)):
        out = Out(M, N, torch.float32 if d == "f32" else torch.bfloat16, pad, shift)
        tcg.gemm_block128(M, N, K, A, B, 0.0, None, 0, "f32", out.start, out.ld, d, workspace=ws, workspace_bytes=n)
        assert tcg.device_status(ws) == 0
        assert ws_header_clean(ws)
        got = out.view
        assert torch.equal(got, want.to(got.dtype)), (d, pad, shift, (got.double() - want).abs().max())
        assert out.clean()


@pytest.mark.parametrize("q", ["e4m3", "e5m2"])
@pytest.mark.parametrize("scale_rows", [1, 128])
@pytest.mark.parametrize("M,N,K", [(5, 700, 3000), (40, 300, 1000), (200, 333, 1500), (1500, 2100, 900)])
def test_real_values_and_epilogue(M, N, K, scale_rows, q):
    a, b = real_operand(M, K, 1, 1, q), real_operand(N, K, scale_rows, 2, q)
    a64, b64 = wide64(*a, 1), wide64(*b, scale_rows)
    prod, mass = a64 @ b64.t(), a64.abs() @ b64.abs().t()
    kb = ceil_div(K, 128)
    for d, beta, cdt, bias_dt, act in (("f32", 0.0, None, None, "none"), ("bf16", 0.0, None, torch.bfloat16, "gelu"),
                                       ("f32", 1.0, torch.float32, None, "none"), ("f32", -0.5, torch.bfloat16, torch.float32, "relu"),
                                       ("bf16", 0.5, torch.bfloat16, torch.float32, "gelu")):
        g = gen(3)
        C = torch.randn(M, N + 3, generator=g, device="cuda").to(cdt) if cdt else None
        bias = torch.randn(N, generator=g, device="cuda").to(bias_dt) if bias_dt else None
        A, ka = operand(*a, 1)
        B, kb_ = operand(*b, scale_rows)
        out = Out(M, N, torch.float32 if d == "f32" else torch.bfloat16, 1)
        n = tcg.block128_workspace_size(0, M, N, K)
        ws = workspace(n)
        tcg.gemm_block128(M, N, K, A, B, beta, C, N + 3, "f32" if cdt == torch.float32 else "bf16", out.start, out.ld, d, ab_dtype=q,
                          bias=bias, bias_dtype="f32" if bias_dt == torch.float32 else "bf16", act=act, workspace=ws, workspace_bytes=n)
        assert tcg.device_status(ws) == 0
        x = prod.clone()
        size = mass.clone()
        if C is not None:
            x += beta * C[:, :N].double()
            size += abs(beta) * C[:, :N].double().abs()
        if bias is not None:
            x += bias.double()
            size += bias.double().abs()
        tol = (128 + kb + 8) * U * size
        if act == "relu":
            ref = x.clamp(min=0)
        elif act == "gelu":
            ref = x * torch.special.ndtr(x)
            tol = 1.13 * tol + (0.75e-7 + 16 * U) * x.abs()
        else:
            ref = x
        assert within(out.view, ref, tol), (d, act)
        assert out.clean()


def test_k_zero_is_the_epilogue_alone():
    for M, N in ((3, 40), (100, 200), (3000, 2600)):
        C = torch.randn(M, N, device="cuda")
        bias = torch.randn(N, device="cuda")
        out = Out(M, N, torch.float32)
        n = tcg.block128_workspace_size(0, M, N, 0)
        ws = workspace(n)
        none = tcg.block_operand(None, 0, None, 1, 0, 0)
        tcg.gemm_block128(M, N, 0, none, none, 2.0, C, N, "f32", out.start, out.ld, "f32", bias=bias, bias_dtype="f32", act="relu",
                          workspace=ws, workspace_bytes=n)
        assert torch.equal(out.view, torch.clamp(2.0 * C + bias, min=0.0))


def test_accumulating_in_place_and_the_same_every_time():
    """D == C, and a K split over the SMs gives the same bits in every run."""
    for M, N, K, scale_rows in ((4, 900, 8192, 128), (120, 300, 9000, 1), (2048, 2560, 512, 1)):
        a, b = real_operand(M, K, 1, 5), real_operand(N, K, scale_rows, 6)
        A, ka = operand(*a, 1)
        B, kb = operand(*b, scale_rows)
        n = tcg.block128_workspace_size(0, M, N, K)
        ws = workspace(n)
        start = torch.randn(M, N, device="cuda")
        first = None
        for _ in range(6):
            D = start.clone()
            tcg.gemm_block128(M, N, K, A, B, 1.0, D, N, "f32", D, N, "f32", workspace=ws, workspace_bytes=n)
            E = torch.empty_like(D)
            tcg.gemm_block128(M, N, K, A, B, 1.0, start, N, "f32", E, N, "f32", workspace=ws, workspace_bytes=n)
            assert torch.equal(D, E)
            first = D if first is None else first
            assert torch.equal(D, first)
        assert tcg.device_status(ws) == 0


def test_nan_and_infinity_stay_in_their_row():
    M, N, K = 300, 400, 512
    for rows in (M, 7):
        codes, scales = int_operand(rows, K, 1, 1)
        b = int_operand(N, K, 128, 2)
        codes.view(torch.uint8)[3, 200] = 0x7F      # a NaN code
        scales[1, 5] = float("inf")                  # and an infinite scale
        scales[2, 6] = float("nan")
        A, ka = operand(codes, scales, 1)
        B, kb = operand(*b, 128)
        D = torch.empty(rows, N, device="cuda")
        n = tcg.block128_workspace_size(0, rows, N, K)
        ws = workspace(n)
        tcg.gemm_block128(rows, N, K, A, B, 0.0, None, 0, "f32", D, N, "f32", workspace=ws, workspace_bytes=n)
        keep = [r for r in range(rows) if r not in (3, 5, 6)]
        want = wide64(codes, scales, 1)[keep] @ wide64(*b, 128).t()
        assert torch.equal(D[keep].double(), want)
        assert bool(torch.isnan(D[3]).all()) and bool(torch.isnan(D[6]).all()) and not bool(torch.isfinite(D[5]).any())


def test_gradients_of_a_linear_layer():
    """y = x W^T with x by rows and W by tiles.  The input gradient (W's
    transposed codes, scale strides exchanged) and the weight gradient (both
    operands by 128 tokens) against the formula and against differences of the
    forward product: it is linear, so with integers they are equal."""
    T, I, O = 260, 400, 300
    w = int_operand(O, I, 128, 1)
    g = gen(9)
    x = torch.randint(-4, 5, (T, I), generator=g, device="cuda").float()
    dy = torch.randint(-2, 3, (T, O), generator=g, device="cuda").float()
    ones = lambda r, k: torch.ones(ceil_div(k, 128), r, device="cuda")   # noqa: E731

    def forward(xv, codes_w, scales_w):
        A, ka = operand(xv.to(CODE["e4m3"]), ones(T, I), 1)
        B, kb = operand(codes_w, scales_w, 128)
        y = torch.empty(T, O, device="cuda")
        n = tcg.block128_workspace_size(0, T, O, I)
        tcg.gemm_block128(T, O, I, A, B, 0.0, None, 0, "f32", y, O, "f32", workspace=workspace(n), workspace_bytes=n)
        return y

    # dx = dy W
    wt = w[0].view(torch.uint8).t().contiguous().view(CODE["e4m3"])
    data, ld = torch.zeros(I, 304, dtype=torch.uint8, device="cuda"), 304
    data[:, :O] = wt.view(torch.uint8)
    cb = ceil_div(I, 128)
    A, ka = operand(dy.to(CODE["e4m3"]), ones(T, O), 1)
    B = tcg.block_operand(data, ld, w[1], 128, 1, cb)
    dx = torch.empty(T, I, device="cuda")
    n = tcg.block128_workspace_size(0, T, I, O)
    tcg.gemm_block128(T, I, O, A, B, 0.0, None, 0, "f32", dx, I, "f32", workspace=workspace(n), workspace_bytes=n)
    assert torch.equal(dx.double(), dy.double() @ wide64(*w, 128))
    step = torch.randint(-2, 3, (T, I), generator=g, device="cuda").float()
    diff = (forward((x + step).clamp(-8, 8), *w) - forward(x, *w)).double()
    moved = ((x + step).clamp(-8, 8) - x).double()
    assert float((dy.double() * diff).sum()) == float((dx.double() * moved).sum())

    # dW = dy^T x
    A, ka = operand(dy.t().contiguous().to(CODE["e4m3"]), ones(O, T), 1)
    B, kb = operand(x.t().contiguous().to(CODE["e4m3"]), ones(I, T), 1)
    dw = torch.empty(O, I, device="cuda")
    n = tcg.block128_workspace_size(0, O, I, T)
    tcg.gemm_block128(O, I, T, A, B, 0.0, None, 0, "f32", dw, I, "f32", workspace=workspace(n), workspace_bytes=n)
    assert torch.equal(dw.double(), dy.double().t() @ x.double())
    other = int_operand(O, I, 128, 1)[0].float().roll(1, 0).to(CODE["e4m3"])
    diff = (forward(x, other, torch.ones_like(w[1])) - forward(x, w[0], torch.ones_like(w[1]))).double()
    assert float((dy.double() * diff).sum()) == float((dw.double() * (other.float() - w[0].float()).double()).sum())


def test_output_past_two_to_the_31_elements():
    M, N, K = 70000, 32768, 128
    a, b = int_operand(M, K, 1, 1), int_operand(N, K, 128, 2)
    A, ka = operand(*a, 1)
    B, kb = operand(*b, 128)
    D = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    n = tcg.block128_workspace_size(0, M, N, K)
    tcg.gemm_block128(M, N, K, A, B, 0.0, None, 0, "f32", D, N, "bf16", workspace=workspace(n), workspace_bytes=n)
    at = torch.tensor([0, 1, 65535, 65536, 65537, 69998, 69999], device="cuda")
    want = wide64(a[0].float()[at].to(CODE["e4m3"]), a[1][:, at], 1) @ wide64(*b, 128).t()
    assert torch.equal(D[at], want.to(torch.bfloat16))


def test_another_stream_and_a_graph():
    M, N, K = 24, 700, 2000
    a, b = int_operand(M, K, 1, 1), int_operand(N, K, 128, 2)
    A, ka = operand(*a, 1)
    B, kb = operand(*b, 128)
    want = (wide64(*a, 1) @ wide64(*b, 128).t()).float()
    n = tcg.block128_workspace_size(0, M, N, K)
    ws = workspace(n)
    D = torch.zeros(M, N, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    tcg.gemm_block128(M, N, K, A, B, 0.0, None, 0, "f32", D, N, "f32", workspace=ws, workspace_bytes=n, stream=side)
    side.synchronize()
    assert torch.equal(D, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        tcg.gemm_block128(M, N, K, A, B, 0.0, None, 0, "f32", D, N, "f32", workspace=ws, workspace_bytes=n,
                          stream=torch.cuda.current_stream())
    for _ in range(3):
        D.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(D, want)


def test_a_small_or_missing_workspace_is_refused():
    M, N, K = 4, 700, 8192
    A, ka = operand(*int_operand(M, K, 1, 1), 1)
    B, kb = operand(*int_operand(N, K, 128, 2), 128)
    D = torch.empty(M, N, device="cuda")
    n = tcg.block128_workspace_size(0, M, N, K)
    ws = workspace(n)
    for w, size in ((None, 0), (ws, n - 1), (ws[1:], n)):
        with pytest.raises(tcg.TcgError) as e:
            tcg.gemm_block128(M, N, K, A, B, 0.0, None, 0, "f32", D, N, "f32", workspace=w, workspace_bytes=size)
        assert e.value.code == 5


@pytest.mark.parametrize("M,N,K", [(4, 900, 4096), (300, 520, 1100), (4096, 4096, 512)])
def test_a_wait_that_runs_out_is_reported(M, N, K):
    """The test knob lets the first CTA's producer skip its first stage: the
    bounded waits run out, the status word says so, the next call is exact."""
    a, b = int_operand(M, K, 1, 1), int_operand(N, K, 128, 2)
    A, ka = operand(*a, 1)
    B, kb = operand(*b, 128)
    D = torch.empty(M, N, device="cuda")
    n = tcg.block128_workspace_size(0, M, N, K)
    ws = workspace(n)
    tcg.debug_set(fault_inject=1, wait_timeout_ns=200_000_000)
    tcg.gemm_block128(M, N, K, A, B, 0.0, None, 0, "f32", D, N, "f32", workspace=ws, workspace_bytes=n)
    assert tcg.device_status(ws) == 7
    tcg.debug_set()
    ws.zero_()   # a call that ended so may leave counters behind
    tcg.gemm_block128(M, N, K, A, B, 0.0, None, 0, "f32", D, N, "f32", workspace=ws, workspace_bytes=n)
    assert tcg.device_status(ws) == 0
    assert torch.equal(D.double(), wide64(*a, 1) @ wide64(*b, 128).t())


# -------------------------------------------------------------------- grouped

def stacked(G, N, K, scale_rows, seed):
    """G weights as one operand, and their values."""
    codes, scales = zip(*(int_operand(N, K, scale_rows, seed + g) for g in range(G)))
    values = [wide64(c, s, scale_rows) for c, s in zip(codes, scales)]
    data = torch.cat([c.view(torch.uint8) for c in codes])
    ld = ceil_div(K, 16) * 16
    buf = torch.zeros(G * N, ld, dtype=torch.uint8, device="cuda")
    buf[:, :K] = data
    s = torch.stack(scales).contiguous()
    rs, ks = (1, s.shape[2]) if scale_rows == 1 else (s.shape[2], 1)
    return tcg.block_operand(buf, ld, s, scale_rows, rs, ks, s.shape[1] * s.shape[2]), values, (buf, s)


LENS = {
    "one": [37],
    "empty ends": [0, 5, 0, 0, 130, 1, 0],
    "all in one": [0, 0, 400, 0],
    "nothing": [0, 0, 0],
    "single rows": [1] * 9,
    "ragged": [3, 129, 64, 0, 255, 128, 17, 1, 90],
    "long": [700, 0, 513, 1200, 256, 300],
    "many": [g % 5 for g in range(300)],
}


@pytest.mark.parametrize("scale_rows", [1, 128])
@pytest.mark.parametrize("N,K", [(200, 300), (384, 1024), (1030, 128)])
@pytest.mark.parametrize("which", list(LENS))
def test_grouped_rows_are_exact(which, N, K, scale_rows):
    lens = LENS[which]
    G, before, after = len(lens), 2, 3       # rows outside every group stay as they are
    at = [before]
    for n in lens:
        at.append(at[-1] + n)
    rows = at[-1] + after
    a = int_operand(rows, K, 1, 11)
    A, ka = operand(*a, 1)
    B, values, kb = stacked(G, N, K, scale_rows, 20)
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    n = tcg.block128_workspace_size(G, rows, N, K)
    ws = workspace(n)
    a64 = wide64(*a, 1)
    for d, pad in (("f32", 0), ("bf16", 3)):
        out = Out(rows, N, torch.float32 if d == "f32" else torch.bfloat16, pad)
        tcg.gemm_block128_grouped(G, offsets, rows, N, K, A, B, out.start, out.ld, d, workspace=ws, workspace_bytes=n)
        assert tcg.device_status(ws) == 0
        assert out.clean() and ws_header_clean(ws)
        want = torch.full((rows, N), SENTINEL, dtype=torch.float64, device="cuda")
        for g in range(G):
            want[at[g]:at[g + 1]] = a64[at[g]:at[g + 1]] @ values[g].t()
        assert torch.equal(out.view, want.to(out.view.dtype))


def test_grouped_offsets_past_the_rows_are_clamped():
    G, rows, N, K = 3, 50, 130, 256
    a = int_operand(rows, K, 1, 1)
    A, ka = operand(*a, 1)
    B, values, kb = stacked(G, N, K, 128, 5)
    offsets = torch.tensor([-7, 20, 1000, 2000], dtype=torch.int32, device="cuda")
    n = tcg.block128_workspace_size(G, rows, N, K)
    ws = workspace(n)
    out = Out(rows, N, torch.float32)
    tcg.gemm_block128_grouped(G, offsets, rows, N, K, A, B, out.start, out.ld, "f32", workspace=ws, workspace_bytes=n)
    assert tcg.device_status(ws) == 0 and out.clean()
    a64 = wide64(*a, 1)
    assert torch.equal(out.view.double(), torch.cat([a64[:20] @ values[0].t(), a64[20:] @ values[1].t()]))


def test_grouped_k_zero_is_zero():
    offsets = torch.tensor([0, 3, 10], dtype=torch.int32, device="cuda")
    D = torch.full((10, 40), 5.0, device="cuda")
    none = tcg.block_operand(None, 0, None, 1, 0, 0)
    n = tcg.block128_workspace_size(2, 10, 40, 0)
    tcg.gemm_block128_grouped(2, offsets, 10, 40, 0, none, none, D, 40, "f32", workspace=workspace(n), workspace_bytes=n)
    assert not bool(D.any())


@pytest.mark.parametrize("M,N", [(64, 200), (300, 130), (512, 1040)])
@pytest.mark.parametrize("which", ["one", "empty ends", "nothing", "ragged", "long", "many"])
def test_grouped_k_is_exact(which, M, N):
    lens = LENS[which]
    G = len(lens)
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    padded = sum(ceil_div(n, 128) for n in lens) * 128 + 128
    places = torch.tensor(padded_places(at, padded), device="cuda")
    a, b = int_operand(M, padded, 1, 1), int_operand(N, padded, 1, 2)
    for codes, _ in (a, b):
        codes.view(torch.uint8)[:, places < 0] = 0
    A, ka = operand(*a, 1)
    B, kb = operand(*b, 1)
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    ws = workspace(256)
    a64, b64 = wide64(*a, 1), wide64(*b, 1)
    want = torch.zeros(G, M, N, dtype=torch.float64, device="cuda")
    place = 0
    for g in range(G):
        n = ceil_div(lens[g], 128) * 128
        want[g] = a64[:, place:place + n] @ b64[:, place:place + n].t()
        place += n
    for d, beta, cdt, pad in (("f32", 0.0, None, 0), ("f32", 1.0, torch.float32, 1), ("bf16", 1.0, torch.bfloat16, 0)):
        out = Out(G * M, N, torch.float32 if d == "f32" else torch.bfloat16, pad)
        C = torch.randint(-8, 9, (G * M, N), generator=gen(4), device="cuda").to(cdt) if cdt else None
        tcg.gemm_block128_grouped_k(G, offsets, M, N, padded, A, B, beta, C, N, "bf16" if cdt == torch.bfloat16 else "f32", out.start,
                                    out.ld, d, workspace=ws, workspace_bytes=256)
        assert tcg.device_status(ws) == 0 and out.clean()
        ref = want.view(G * M, N) + (beta * C.double() if cdt else 0.0)
        assert torch.equal(out.view, ref.to(out.view.dtype))
