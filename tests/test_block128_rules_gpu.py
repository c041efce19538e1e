"""Rules of the block-scaled operators that only unusual arguments show."""
import pytest
import torch

import tiled_tensor_core_persistent_gb300 as tcg

from block128 import ceil_div, operand, pitched, quantize_rows, wide64, workspace
from test_block128_gpu import int_operand, stacked

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tiled_tensor_core_persistent_gb300 import _build
    _build.build()
    tcg.debug_set()


@pytest.mark.parametrize("lens,N,K", [([2, 0, 3, 1], 200, 300), ([40, 90, 0, 33], 300, 512), ([300, 700, 256], 2100, 384)])
def test_group_stride_of_the_rows_operand(lens, N, K):
    """Every group has a scale matrix of its own for A (a group's rows at
    their own row numbers in it); what it holds for the other groups' rows is NaN."""
    G, rows, kb = len(lens), sum(lens), ceil_div(K, 128)
    codes, scales = int_operand(rows, K, 1, 3)
    at = [sum(lens[:g]) for g in range(G + 1)]
    per_group = torch.full((G, kb, rows), float("nan"), device="cuda")
    for g in range(G):
        per_group[g, :, at[g]:at[g + 1]] = scales[:, at[g]:at[g + 1]]
    data, ld = pitched(codes)
    A = tcg.block_operand(data, ld, per_group, 1, 1, rows, kb * rows)
    B, values, keep = stacked(G, N, K, 128, 9)
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    D = torch.empty(rows, N, device="cuda")
    n = tcg.block128_workspace_size(G, rows, N, K)
    ws = workspace(n)
    tcg.gemm_block128_grouped(G, offsets, rows, N, K, A, B, D, N, "f32", workspace=ws, workspace_bytes=n)
    assert tcg.device_status(ws) == 0
    a64 = wide64(codes, scales, 1)
    assert torch.equal(D.double(), torch.cat([a64[at[g]:at[g + 1]] @ values[g].t() for g in range(G)]))


@pytest.mark.parametrize("which", ["A", "B"])
def test_group_stride_of_weight_gradients(which):
    lens, M, N = [100, 0, 300], 200, 130
    G, at = len(lens), [0, 100, 100, 400]
    padded = sum(ceil_div(n, 128) for n in lens) * 128
    kb = padded // 128
    ops = {"A": int_operand(M, padded, 1, 1), "B": int_operand(N, padded, 1, 2)}
    want = [wide64(*ops[k], 1) for k in "AB"]
    held, keep = {}, []
    for name, (codes, scales) in ops.items():
        r = codes.shape[0]
        data, ld = pitched(codes)
        if name == which:
            factor = torch.tensor([1.0, 2.0, 4.0], device="cuda")[:, None, None]
            scales = (scales[None] * factor).contiguous()
            held[name] = tcg.block_operand(data, ld, scales, 1, 1, r, kb * r)
        else:
            held[name] = tcg.block_operand(data, ld, scales, 1, 1, r)
        keep += [data, scales]
    D = torch.empty(G, M, N, device="cuda")
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    ws = workspace(256)
    tcg.gemm_block128_grouped_k(G, offsets, M, N, padded, held["A"], held["B"], 0.0, None, N, "f32", D, N, "f32", workspace=ws,
                                workspace_bytes=256)
    assert tcg.device_status(ws) == 0
    place = 0
    for g in range(G):
        n = ceil_div(lens[g], 128) * 128
        ref = (want[0][:, place:place + n] @ want[1][:, place:place + n].t()) * 2.0 ** g
        assert torch.equal(D[g].double(), ref)
        place += n


# offsets that go back: what they stand for (an offset below an earlier one counts as that one)
TABLES = [([0, 30, 10, 50], [0, 30, 30, 50]), ([5, 3, 60, 60, 2, 70], [5, 5, 60, 60, 60, 70]), ([80, 10, 20, 30], [80, 80, 80, 80])]


@pytest.mark.parametrize("given,meant", TABLES)
def test_offsets_that_go_back(given, meant):
    G, rows, N, K = len(given) - 1, 80, 200, 256
    a = int_operand(rows, K, 1, 1)
    A, ka = operand(*a, 1)
    B, values, kb = stacked(G, N, K, 128, 5)
    offsets = torch.tensor(given, dtype=torch.int32, device="cuda")
    n = tcg.block128_workspace_size(G, rows, N, K)
    ws = workspace(n)
    D = torch.full((rows, N), 777.0, device="cuda")
    tcg.gemm_block128_grouped(G, offsets, rows, N, K, A, B, D, N, "f32", workspace=ws, workspace_bytes=n)
    assert tcg.device_status(ws) == 0
    want = torch.full((rows, N), 777.0, dtype=torch.float64, device="cuda")
    a64 = wide64(*a, 1)
    for g in range(G):
        want[meant[g]:meant[g + 1]] = a64[meant[g]:meant[g + 1]] @ values[g].t()
    assert torch.equal(D.double(), want)


@pytest.mark.parametrize("given,meant", TABLES)
def test_offsets_that_go_back_by_columns(given, meant):
    """The column quantiser and the weight gradients read such a table the same way."""
    G, rows, M, N = len(given) - 1, 80, 150, 70
    padded = 128 * G
    xa, xb = torch.randn(rows, M, device="cuda"), torch.randn(rows, N, device="cuda")
    offsets = torch.tensor(given, dtype=torch.int32, device="cuda")
    ops, keep, wide = [], [], []
    for x in (xa, xb):
        c = x.shape[1]
        q, s = torch.empty(c, padded, dtype=torch.uint8, device="cuda"), torch.empty(G, c, device="cuda")
        tcg.quantize_cols128(rows, c, x, c, "f32", q, padded, "e4m3", s, c, padded_rows=padded, num_groups=G, offsets=offsets)
        y = torch.zeros(padded, c, device="cuda")
        place = 0
        for g in range(G):
            n = meant[g + 1] - meant[g]
            y[place:place + n] = x[meant[g]:meant[g + 1]]
            place += ceil_div(n, 128) * 128
        want_q, want_s = quantize_rows(y.t().contiguous())
        assert torch.equal(s, want_s) and torch.equal(q, want_q.view(torch.uint8))
        wide.append(wide64(want_q, want_s, 1))
        ops.append(tcg.block_operand(q, padded, s, 1, 1, c))
        keep += [q, s]
    D = torch.empty(G, M, N, device="cuda")
    ws = workspace(256)
    tcg.gemm_block128_grouped_k(G, offsets, M, N, padded, ops[0], ops[1], 0.0, None, N, "f32", D, N, "f32", workspace=ws, workspace_bytes=256)
    assert tcg.device_status(ws) == 0
    place = 0
    for g in range(G):
        n = ceil_div(meant[g + 1] - meant[g], 128) * 128
        a, b = wide[0][:, place:place + n], wide[1][:, place:place + n]
        # 128 products and their scaling (132 units of the terms' magnitudes), one k-block
        assert bool(((D[g].double() - a @ b.t()).abs() <= 136 * 2.0 ** -24 * (a.abs() @ b.abs().t())).all())
        place += n


@pytest.mark.parametrize("scale_rows", [1, 128])
@pytest.mark.parametrize("G,rows,N", [(1024, 1500, 40), (1000, 50000, 136), (800, 4000, 300)])
def test_as_many_groups_as_the_tables_hold(G, rows, N, scale_rows):
    """Few-row, single and pair tiles next to the tables of many groups: every
    row of D, and the weight gradients, exact."""
    K = 128
    g = torch.Generator().manual_seed(G)
    cuts = torch.sort(torch.randint(0, rows + 1, (G - 1,), generator=g)).values.tolist()
    at = [0] + cuts + [rows]
    a, (bc, bs) = int_operand(rows, K, 1, 1), int_operand(G * N, K, 1, 2)
    A, ka = operand(*a, 1)
    data, ld = pitched(bc)
    if scale_rows == 1:
        B = tcg.block_operand(data, ld, bs, 1, 1, G * N, N)
        wide = wide64(bc, bs, 1)
    else:
        nb = ceil_div(N, 128)
        tiles = torch.exp2(torch.randint(-1, 2, (G, nb), generator=g).float()).cuda()
        B = tcg.block_operand(data, ld, tiles, 128, 1, 1, nb)
        wide = wide64(bc, tiles.repeat_interleave(128, 1)[:, :N].reshape(1, G * N), 1)
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    n = tcg.block128_workspace_size(G, rows, N, K)
    ws = workspace(n)
    D = torch.full((rows, N), 777.0, device="cuda")
    tcg.gemm_block128_grouped(G, offsets, rows, N, K, A, B, D, N, "f32", workspace=ws, workspace_bytes=n)
    assert tcg.device_status(ws) == 0
    owner = torch.searchsorted(offsets[1:].contiguous(), torch.arange(rows, device="cuda", dtype=torch.int32), right=True)
    a64, wide = wide64(*a, 1), wide.view(G, N, K)
    for r0 in range(0, rows, 2000):
        r = slice(r0, min(rows, r0 + 2000))
        assert torch.equal(D[r].double(), torch.einsum("rk,rnk->rn", a64[r], wide[owner[r]]))


@pytest.mark.parametrize("G,M,N", [(1024, 130, 140), (300, 300, 520), (1024, 40, 20)])
def test_weight_gradients_of_as_many_groups_as_the_tables_hold(G, M, N):
    g = torch.Generator().manual_seed(G + M)
    lens = torch.randint(0, 3, (G,), generator=g).tolist()
    at = [sum(lens[:i]) for i in range(G + 1)]
    padded = sum(ceil_div(n, 128) for n in lens) * 128
    a, b = int_operand(M, padded, 1, 1), int_operand(N, padded, 1, 2)
    A, ka = operand(*a, 1)
    B, kb = operand(*b, 1)
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    D = torch.empty(G, M, N, device="cuda")
    ws = workspace(256)
    tcg.gemm_block128_grouped_k(G, offsets, M, N, padded, A, B, 0.0, None, N, "f32", D, N, "f32", workspace=ws, workspace_bytes=256)
    assert tcg.device_status(ws) == 0
    a64, b64 = wide64(*a, 1), wide64(*b, 1)
    place = 0
    for i in range(G):
        n = ceil_div(lens[i], 128) * 128
        assert torch.equal(D[i].double(), a64[:, place:place + n] @ b64[:, place:place + n].t())
        place += n
