"""Rows, sorts and vocabularies of the largest sizes that are taken, where every
index that is kept in 32 bits comes near its end."""
import pytest
import torch

import tiled_tensor_core_persistent_gb300 as tcg

pytestmark = pytest.mark.gpu

EXTENT = 2 ** 31 - 4096
STEP = 1 << 28


@pytest.fixture(autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 60 GB")
    from tiled_tensor_core_persistent_gb300 import _build
    _build.build()
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def whole_numbers(n):
    x = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    for a in range(0, n, STEP):
        x[a:a + STEP] = torch.randint(-100, 100, (min(STEP, n - a),), device="cuda", dtype=torch.int8).to(torch.bfloat16)
    return x


@pytest.mark.parametrize("shift", [0, 1])
def test_a_row_of_the_most_columns(shift):
    cols = 65535 * 2048 - 8
    src = whole_numbers(cols + 8)[shift:shift + cols]
    row_of = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for what in ("dispatch", "combine", "gradient"):
        out = torch.zeros(cols + 8, dtype=torch.bfloat16, device="cuda")
        at = out[shift:]
        if what == "dispatch":
            tcg.moe_dispatch(1, 1, cols, 1, src, cols, "bf16", row_of, 1, at, cols, "bf16")
        elif what == "combine":
            tcg.moe_combine(1, 1, cols, 1, src, cols, "bf16", row_of, 1, None, 1, at, cols, "bf16")
        else:
            dw = torch.zeros(1, 1, device="cuda")
            tcg.moe_combine_backward(1, 1, cols, 1, src, cols, "bf16", row_of, 1, None, 1, src, cols, "bf16", at, cols, dw, 1)
            want = float((src.double() ** 2).sum())
            # additions in line of a thread of 256, of terms that are all positive: half a step of the sum each at most
            assert abs(float(dw) - want) <= (cols / 256 + 48) * 2.0 ** -24 * want
        assert torch.equal(at[:cols], src) and not bool(out[:shift].any()) and not bool(out[shift + cols:].any())


def test_the_most_tokens_and_rows():
    n = EXTENT
    x, y = whole_numbers(n), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    row_of = torch.arange(n - 1, -1, -1, device="cuda", dtype=torch.int32)
    tcg.moe_dispatch(n, 1, 1, n, x, 1, "bf16", row_of, 1, y, 1, "bf16")
    for a in range(0, n, STEP):
        b = min(n, a + STEP)
        assert torch.equal(y[n - b:n - a], x[a:b].flip(0))
    back, dw = torch.zeros_like(x), torch.empty(n, device="cuda")
    tcg.moe_combine(n, 1, 1, n, y, 1, "bf16", row_of, 1, None, 1, back, 1, "bf16")
    assert torch.equal(x, back)
    back.zero_()
    tcg.moe_combine_backward(n, 1, 1, n, y, 1, "bf16", row_of, 1, None, 1, x, 1, "bf16", back, 1, dw, 1)
    assert torch.equal(back, y)
    for a in range(0, n, STEP):
        assert torch.equal(dw[a:a + STEP], x[a:a + STEP].float() ** 2)


@pytest.mark.parametrize("E,k", [(1000, 1), (3, 2 ** 31 - 2 ** 20 - 4096)])
def test_the_longest_sorts(E, k):
    n = 2 ** 31 - 2 ** 20 - 4096
    T = n // k
    topk = torch.empty(n, dtype=torch.int32, device="cuda")
    for a in range(0, n, STEP):
        topk[a:a + STEP] = torch.randint(-1, E + 1, (min(STEP, n - a),), device="cuda", dtype=torch.int32)
    size = tcg.moe_sort_workspace_size(T, E, k)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    offsets, row_token, row_of = (torch.empty(m, dtype=torch.int32, device="cuda") for m in (E + 1, n, n))
    tcg.moe_sort(T, E, k, topk, k, None, offsets, row_token, row_of, k, workspace=ws, workspace_bytes=size)
    count = torch.zeros(E, dtype=torch.long, device="cuda")
    last = torch.full((E,), -1, dtype=torch.long, device="cuda")
    for a in range(0, n, STEP // 4):
        e, r = topk[a:a + STEP // 4], row_of[a:a + STEP // 4]
        there = (e >= 0) & (e < E)
        assert torch.equal(r >= 0, there)
        token = torch.arange(a, a + e.numel(), device="cuda")[there] // k
        e, r = e[there].long(), r[there].long()
        assert bool((r >= offsets[e]).all()) and bool((r < offsets[e + 1]).all())
        assert torch.equal(row_token[r].long(), token)
        count += torch.bincount(e, minlength=E)
        for one in (0, E // 2, E - 1):      # an expert's rows rise with the assignments, one by one
            mine = r[e == one]
            if mine.numel():
                assert bool((mine[1:] == mine[:-1] + 1).all()) and (last[one] < 0 or int(mine[0]) == int(last[one]) + 1)
                last[one] = mine[-1]
    assert int(offsets[0]) == 0 and torch.equal(offsets[1:].long(), count.cumsum(0))
    assert bool((row_token[int(offsets[E]):] == -1).all())


def test_the_most_words():
    """One token, so that pieces of the vocabulary are of 2^28 words."""
    V, H = EXTENT // 2, 8
    w = torch.empty(V, H, dtype=torch.bfloat16, device="cuda")
    for a in range(0, V, STEP // 8):
        w[a:a + STEP // 8].normal_()
    x = torch.randn(1, H, device="cuda").to(torch.bfloat16)
    target = torch.tensor([V - 3], dtype=torch.int32, device="cuda")
    lse, loss, mean = (torch.empty(1, device="cuda") for _ in range(3))
    n = torch.empty(1, dtype=torch.int32, device="cuda")
    size = tcg.linear_xent_workspace_size(1, V, H, True)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    tcg.linear_xent(1, V, H, "bf16", x, H, w, H, target, lse, loss, mean, n, workspace=ws, workspace_bytes=size)
    dx, dw = torch.empty(1, H, device="cuda"), torch.empty_like(w)
    tcg.linear_xent_backward(1, V, H, "bf16", x, H, w, H, target, lse, n, torch.ones(1, device="cuda"), None, dx, H, "f32", 0.0, dw, H, "bf16",
                             workspace=ws, workspace_bytes=size)
    assert tcg.device_status(ws) == 0 and int(n) == 1
    at = x[0].double()
    parts = [torch.logsumexp(w[a:a + STEP // 8].double() @ at, 0) for a in range(0, V, STEP // 8)]
    ref = torch.logsumexp(torch.stack(parts), 0)
    z = (w[V - 3].double() * at).sum()
    # (tiles' sums of 128 in line in a thread, then 2^22 of them and more in batches of eight by 32 threads)
    off = (V / 256 / 32 / 8 + 200) * 2.0 ** -24
    assert abs(float(lse) - float(ref)) <= off and abs(float(loss) - float(ref - z)) <= off + 2.0 ** -22 and float(mean) == float(loss)
    want, size = torch.zeros(H, dtype=torch.double, device="cuda"), torch.zeros(H, dtype=torch.double, device="cuda")
    for a in range(0, V, STEP // 8):
        rows = w[a:a + STEP // 8].double()
        dz = torch.exp(rows @ at - ref)
        if a <= V - 3 < a + STEP // 8:
            dz[V - 3 - a] -= 1.0
        got, one = dw[a:a + STEP // 8].double(), dz[:, None] * at
        # half a step of dz and of dW, and p's own error
        assert bool(((got - one).abs() <= (2 * 2.0 ** -8 * 1.01 + 2 * off) * one.abs() + 1e-38).all())
        want += dz @ rows
        size += dz.abs() @ rows.abs()
    # sums of 8192 words in one go, and those added in fp32
    assert bool(((dx[0].double() - want).abs() <= (2.0 ** -8 * 1.01 + 2 * off + (8192 / 16 + 40) * 2.0 ** -22) * size).all())
