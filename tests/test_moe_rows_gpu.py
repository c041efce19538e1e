"""Tokens in expert order and back, on the GPU.  The sort is compared for
equality with one over the assignments on the host; copies for equality; sums in
64 bits, within u = 2^-24 for each of their additions and half a step of the
output's type.
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


def half_step(t):
    return torch.finfo(TYPE[t]).eps / 2


def sorted_reference(topk, mask, E):
    T, k = topk.shape
    key = topk.cpu().long().clone()
    key[(key < 0) | (key >= E)] = E
    if mask is not None:
        key[mask.cpu() == 0] = E
    key = key.view(-1)
    order = torch.sort(key, stable=True).indices
    n = int((key < E).sum())
    row_token = torch.full((T * k,), -1, dtype=torch.long)
    row_token[:n] = order[:n] // k
    row_of = torch.full((T * k,), -1, dtype=torch.long)
    row_of[order[:n]] = torch.arange(n)
    offsets = torch.zeros(E + 1, dtype=torch.long)
    offsets[1:] = torch.cumsum(torch.bincount(key[key < E], minlength=E), 0)
    return offsets, row_token, row_of.view(T, k)


def random_choice(T, E, k, gen, low=-1):
    return torch.randint(low, E + 1 if low < 0 else E, (T, k), generator=gen, device="cuda", dtype=torch.int32)


def sort(T, E, k, topk, mask, ws=None, offsets=True, pad=0, stream=None):
    n = tcg.moe_sort_workspace_size(T, E, k)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda") if ws is None else ws
    off = torch.full((E + 2,), -9, dtype=torch.int32, device="cuda")
    row_token = torch.full((T * k + 1,), -9, dtype=torch.int32, device="cuda")
    row_of = torch.full((T + 1, k + pad), -9, dtype=torch.int32, device="cuda")
    tcg.moe_sort(T, E, k, topk, topk.shape[1], mask, off if offsets else None, row_token, row_of, k + pad, workspace=ws,
                 workspace_bytes=ws.numel(), stream=stream)
    if stream is not None:
        stream.synchronize()
    assert int(off[E + 1]) == -9 and int(row_token[T * k]) == -9 and bool((row_of[T] == -9).all()) and bool((row_of[:, k:] == -9).all())
    if not offsets:
        assert bool((off == -9).all())
    return off[:E + 1], row_token[:T * k], row_of[:T, :k]


SIZES = [(1, 1, 1), (1, 1, 5), (2, 3, 2), (64, 16, 2), (17, 5, 3), (4096, 8, 1), (4097, 8, 1), (1000, 1024, 7), (1366, 40, 3), (700, 2, 6),
         (32768, 256, 8), (20001, 300, 13), (100000, 7, 4), (300000, 64, 2), (2, 9, 100000), (2048, 8, 1), (2049, 9, 1), (3000, 1021, 3), (1030, 513, 2)]


@pytest.mark.parametrize("T,E,k", SIZES)
def test_sort(T, E, k):
    gen = torch.Generator(device="cuda").manual_seed(T + E + k)
    for masked, pad, offsets in ((0, 0, True), (1, 2, True), (2, 0, False)):
        topk = random_choice(T, E, k + pad, gen)
        mask = None
        if masked == 1:
            mask = (torch.rand(T, generator=gen, device="cuda") < 0.7).to(torch.uint8) * 9
        elif masked == 2:
            topk[:, :] = E // 2          # all to one expert
        want = sorted_reference(topk[:, :k], mask, E)
        got = sort(T, E, k, topk, mask, offsets=offsets, pad=pad)
        for a, b, skip in zip(got, want, (not offsets, False, False)):
            assert skip or torch.equal(a.cpu().long(), b)


def test_sort_of_nothing():
    E = 12
    off = torch.full((E + 1,), -9, dtype=torch.int32, device="cuda")
    ws = torch.zeros(tcg.moe_sort_workspace_size(0, E, 2), dtype=torch.uint8, device="cuda")
    tcg.moe_sort(0, E, 2, None, 2, None, off, None, None, 2, workspace=ws, workspace_bytes=ws.numel())
    assert not bool(off.any())
    # every token masked, every entry out of range
    for T in (5, 5000):
        topk = torch.randint(0, E, (T, 2), device="cuda", dtype=torch.int32)
        off, row_token, row_of = sort(T, E, 2, topk, torch.zeros(T, dtype=torch.uint8, device="cuda"))
        assert not bool(off.any()) and bool((row_token == -1).all()) and bool((row_of == -1).all())
        off, row_token, row_of = sort(T, E, 2, topk + E, None)
        assert not bool(off.any()) and bool((row_token == -1).all()) and bool((row_of == -1).all())


def test_sort_offsets_are_the_balance_losss():
    T, E, k = 3000, 48, 4
    gen = torch.Generator(device="cuda").manual_seed(5)
    topk, mask = random_choice(T, E, k, gen), (torch.rand(T, generator=gen, device="cuda") < 0.8).to(torch.uint8)
    logits = torch.randn(T, E, generator=gen, device="cuda")
    n = max(tcg.moe_balance_workspace_size(), tcg.moe_sort_workspace_size(T, E, k))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    ints = [torch.empty(m, dtype=torch.int32, device="cuda") for m in (E, E + 1, 1)]
    loss = torch.empty(1, device="cuda")
    for _ in range(2):       # one workspace for both, in turn
        tcg.moe_balance(T, E, k, logits, E, "f32", topk, k, mask, 1.0, *ints, loss, workspace=ws, workspace_bytes=n)
        off, _, _ = sort(T, E, k, topk, mask, ws)
        assert torch.equal(off, ints[1])


def test_sorts_of_different_sizes_share_a_workspace_back_to_back():
    gen = torch.Generator(device="cuda").manual_seed(3)
    cases = [(T, E, 2, random_choice(T, E, 2, gen)) for T, E in ((9000, 100), (30, 8), (20000, 400), (9000, 100))]
    n = max(tcg.moe_sort_workspace_size(T, E, k) for T, E, k, _ in cases)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    outs = []
    for T, E, k, topk in cases * 3:
        out = [torch.empty(m, dtype=torch.int32, device="cuda") for m in (E + 1, T * k, T * k)]
        tcg.moe_sort(T, E, k, topk, k, None, *out, k, workspace=ws, workspace_bytes=n)
        outs.append(out)
    for (T, E, k, topk), out in zip(cases * 3, outs):
        want = sorted_reference(topk, None, E)
        assert all(torch.equal(a.cpu().long().view(-1), b.view(-1)) for a, b in zip(out, want))


class Rows:
    def __init__(self, T, E, k, cols, x="bf16", pad=0, shift=0, seed=0, masked=False):
        gen = torch.Generator(device="cuda").manual_seed(seed + T + cols)
        self.T, self.E, self.k, self.cols, self.x_type, self.ld, self.n = T, E, k, cols, x, cols + pad, T * k
        topk = random_choice(T, E, k, gen)
        if masked:
            topk[torch.rand(T, generator=gen, device="cuda") < 0.4] = -1
        _, self.row_token, self.row_of = (v.cuda() for v in sorted_reference(topk, None, E))
        self.row_of = self.row_of.to(torch.int32).contiguous()
        self.live = int((self.row_token >= 0).sum())
        self.shift = shift
        self.x = self.matrix(self.n, x, gen)
        self.w = torch.randn(T, k + 1, generator=gen, device="cuda")
        self.gen = gen

    def matrix(self, rows, t, gen=None):
        """rows x cols, rows ld apart, a few elements off 16 bytes; NaN between the rows."""
        flat = torch.full((self.shift + rows * self.ld,), float("nan"), dtype=TYPE[t], device="cuda")
        m = flat[self.shift:].view(rows, self.ld)
        if gen is not None:
            m[:, :self.cols] = torch.randn(rows, self.cols, generator=gen, device="cuda").to(TYPE[t])
            m[:, self.cols:] = float("nan")
        else:
            m.fill_(3.0)
        return m

    def untouched(self, m, rows):
        three = torch.tensor(3.0, dtype=m.dtype, device="cuda")
        return bool((m[:, self.cols:] == three).all()) and bool((m[rows:] == three).all())


SHAPES = [(1, 1, 1, 1), (1, 4, 2, 8), (3, 5, 3, 7), (64, 16, 2, 4096), (50, 8, 8, 100), (17, 9, 5, 1030), (300, 40, 4, 264), (5, 3, 2, 9000),
          (1, 2, 33, 16), (2000, 16, 2, 65), (900, 12, 5, 4100), (350, 12, 3, 2050)]
TYPES = [("bf16", "bf16", 0, 0), ("f16", "f32", 3, 1), ("f32", "bf16", 0, 0), ("bf16", "f16", 8, 0), ("f32", "f32", 1, 1)]


@pytest.mark.parametrize("x,y,pad,shift", TYPES)
@pytest.mark.parametrize("T,E,k,cols", SHAPES)
def test_dispatch(T, E, k, cols, x, y, pad, shift):
    c = Rows(T, E, k, cols, x, pad, shift)
    src = c.matrix(T, y, c.gen)
    out = c.matrix(c.n + 1, x)
    tcg.moe_dispatch(T, k, cols, c.n, src, c.ld, y, c.row_of, k, out, c.ld, x)
    assert torch.equal(out[:c.live, :cols], src[c.row_token[:c.live], :cols].to(TYPE[x]))
    assert c.untouched(out, c.live)


@pytest.mark.parametrize("x,y,pad,shift", TYPES)
@pytest.mark.parametrize("T,E,k,cols", SHAPES)
def test_combine(T, E, k, cols, x, y, pad, shift):
    for weighted in (True, False):
        c = Rows(T, E, k, cols, x, pad, shift, masked=True)
        c.x[c.live:, :] = float("nan")        # rows of nobody
        out = c.matrix(T + 1, y)
        tcg.moe_combine(T, k, cols, c.n, c.x, c.ld, x, c.row_of, k, c.w if weighted else None, k + 1, out, c.ld, y)
        ref = torch.zeros(T, cols, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(ref)
        for j in range(k):
            at = c.row_of[:, j].long()
            part = torch.where((at >= 0)[:, None], c.x[at.clamp(min=0), :cols].double(), 0.0) * (c.w[:, j, None].double() if weighted else 1.0)
            ref += part
            size += part.abs()
        bound = (k + 1) * U * size + half_step(y) * ref.abs() * 1.01 + (2.0 ** -25 if y == "f16" else 2.0 ** -140)
        assert bool(((out[:T, :cols].double() - ref).abs() <= bound).all())
        assert c.untouched(out, T)


@pytest.mark.parametrize("x,y,pad,shift", TYPES)
@pytest.mark.parametrize("T,E,k,cols", SHAPES)
def test_combine_backward(T, E, k, cols, x, y, pad, shift):
    for weighted, wanted in ((True, True), (False, True), (True, False)):
        c = Rows(T, E, k, cols, x, pad, shift, masked=True)
        c.x[c.live:, :] = float("nan")
        dy = c.matrix(T, y, c.gen)
        dx = c.matrix(c.n + 1, x)
        dw = torch.full((T + 1, k + 2), 3.0, device="cuda")
        tcg.moe_combine_backward(T, k, cols, c.n, c.x if wanted else None, c.ld, x, c.row_of, k, c.w if weighted else None, k + 1, dy, c.ld, y,
                                 dx, c.ld, dw if wanted else None, k + 2)
        ref = torch.zeros(c.n, cols, dtype=torch.float64, device="cuda")
        adds = cols / 256 + 48      # additions in line of a thread (32 lanes or more share a row), then across lanes and warps
        for j in range(k):
            at = c.row_of[:, j].long()
            live = at >= 0
            w = c.w[:, j, None].double() if weighted else torch.ones(T, 1, dtype=torch.float64, device="cuda")
            ref[at[live]] = (dy[:, :cols].double() * w)[live]
            part = torch.where(live[:, None], c.x[at.clamp(min=0), :cols].double(), 0.0) * dy[:, :cols].double()
            if wanted:
                assert bool(((dw[:T, j].double() - part.sum(1)).abs() <= (adds + 1) * U * part.abs().sum(1) + 2.0 ** -140).all())
                assert not bool(dw[:T, j][~live].any())
        bound = (half_step(x) * 1.01 + U) * ref.abs() + (2.0 ** -25 if x == "f16" else 2.0 ** -140)
        assert bool(((dx[:c.live, :cols].double() - ref[:c.live]).abs() <= bound[:c.live]).all())
        assert c.untouched(dx, c.live)
        assert bool((dw[T] == 3).all()) and bool((dw[:, k:] == 3).all()) and (wanted or bool((dw == 3).all()))


def test_combine_gradients_against_differences():
    T, E, k, cols = 5, 4, 3, 40
    c = Rows(T, E, k, cols, "f32")
    dy = c.matrix(T, "f32", c.gen)
    dx, dw = torch.zeros(c.n, cols, device="cuda"), torch.zeros(T, k, device="cuda")
    tcg.moe_combine_backward(T, k, cols, c.n, c.x, c.ld, "f32", c.row_of, k, c.w, k + 1, dy, c.ld, "f32", dx, cols, dw, k)
    at = c.row_of.long()

    def total(x, w):
        rows = torch.where((at >= 0)[..., None], x[at.clamp(min=0)], 0.0)
        return ((rows * w[..., None]).sum(1) * dy.double()).sum()

    x, w, h = c.x.double(), c.w[:, :k].double(), 1e-3
    gen = torch.Generator(device="cuda").manual_seed(9)
    for _ in range(20):
        a = torch.randn(c.n, cols, generator=gen, device="cuda", dtype=torch.float64)
        b = torch.randn(T, k, generator=gen, device="cuda", dtype=torch.float64)
        # (the sum is a product of the two at most, so central differences have no error but rounding)
        slope_x = (total(x + h * a, w) - total(x - h * a, w)) / (2 * h)
        slope_w = (total(x, w + h * b) - total(x, w - h * b)) / (2 * h)
        assert abs(float(slope_x - (dx.double() * a).sum())) <= 4 * U * float((dx.double() * a).abs().sum()) + 1e-8
        assert abs(float(slope_w - (dw.double() * b).sum())) <= 60 * U * float((c.w[:, :k].abs() + 1).sum() * cols)


def test_nothing_to_move():
    one = torch.full((4, 8), 2.0, device="cuda")
    row_of = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    dw = torch.full((4, 2), 7.0, device="cuda")
    tcg.moe_dispatch(0, 2, 8, 4, None, 8, "f32", None, 2, one, 8, "f32")
    tcg.moe_dispatch(4, 2, 8, 4, one.clone(), 8, "f32", row_of, 2, one, 8, "f32")
    tcg.moe_dispatch(4, 2, 0, 4, one, 8, "f32", row_of, 2, one, 8, "f32")
    tcg.moe_dispatch(4, 2, 8, 0, one, 8, "f32", row_of, 2, None, 8, "f32")
    assert bool((one == 2).all())
    y = torch.full((4, 8), 2.0, device="cuda")
    tcg.moe_combine(4, 2, 8, 0, None, 8, "f32", row_of, 2, None, 2, y, 8, "f32")
    assert not bool(y.any())
    # no columns, no rows: the weights' gradient is 0
    for cols, rows in ((0, 4), (8, 0)):
        dw.fill_(7.0)
        tcg.moe_combine_backward(4, 2, cols, rows, one, 8, "f32", row_of, 2, None, 2, y, 8, "f32", one, 8, dw, 2)
        assert not bool(dw.any())
    # rows past the end of x are nobody's
    row_of[:] = torch.tensor([[0, 4], [3, 100], [-2, 1], [2, -1]], dtype=torch.int32)
    x = torch.arange(32.0, device="cuda").view(4, 8)
    tcg.moe_combine(4, 2, 8, 4, x, 8, "f32", row_of, 2, None, 2, y, 8, "f32")
    assert torch.equal(y, x[[0, 3, 1, 2]])


def test_no_columns_at_addresses_that_are_not_whole_words():
    row_of = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    m = torch.full((4, 7), 2.0, dtype=torch.bfloat16, device="cuda")
    for shift in range(1, 7):
        at = m.view(-1)[shift:]
        dw = torch.full((4, 2), 7.0, device="cuda")
        tcg.moe_dispatch(4, 2, 0, 4, at, 7, "bf16", row_of, 2, at, 7, "bf16")
        tcg.moe_combine(4, 2, 0, 4, at, 7, "bf16", row_of, 2, None, 2, at, 7, "bf16")
        tcg.moe_combine_backward(4, 2, 0, 4, at, 7, "bf16", row_of, 2, None, 2, at, 7, "bf16", at, 7, dw, 2)
        assert not bool(dw.any())
    assert bool((m == 2).all())


@pytest.mark.parametrize("shift", [0, 1])
def test_the_same_row_twice(shift):
    """By two places of a token, and by two tokens: each value is one of theirs, sums and weights' gradients are exact."""
    cols, rows = 40, 3
    gen = torch.Generator(device="cuda").manual_seed(5)
    row_of = torch.tensor([[1, 1], [2, 0], [2, 1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, 2.0], [4.0, 8.0], [16.0, 32.0]], device="cuda")
    small = lambda n: torch.randint(-9, 10, (n, cols), generator=gen, device="cuda").float()
    room = lambda m: torch.cat([torch.zeros(shift, device="cuda"), m.flatten()])[shift:].view_as(m)
    x, y, dx, out = room(small(rows)), room(small(3)), room(torch.full((rows, cols), 500.0, device="cuda")), room(torch.zeros(rows, cols, device="cuda"))
    dw, got = torch.zeros(3, 2, device="cuda"), room(torch.zeros(3, cols, device="cuda"))
    tcg.moe_dispatch(3, 2, cols, rows, y, cols, "f32", row_of, 2, out, cols, "f32")
    tcg.moe_combine(3, 2, cols, rows, x, cols, "f32", row_of, 2, w, 2, got, cols, "f32")
    tcg.moe_combine_backward(3, 2, cols, rows, x, cols, "f32", row_of, 2, w, 2, y, cols, "f32", dx, cols, dw, 2)
    assert torch.equal(got, (w[:, :, None] * x[row_of.long()]).sum(1))
    assert torch.equal(dw, (y[:, None] * x[row_of.long()]).sum(2))
    for r in range(rows):
        named = (row_of == r).nonzero().tolist()
        assert bool(torch.stack([out[r] == y[t] for t, _ in named]).any(0).all())
        assert bool(torch.stack([dx[r] == w[t, j] * y[t] for t, j in named]).any(0).all())


def test_offsets_past_31_bits():
    """Rows whose elements start past 2^31."""
    T, k, cols = 600000, 1, 4096
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 15 GB")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(0, 100, (T, cols), generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    row_of = torch.randperm(T, generator=gen, device="cuda").to(torch.int32).view(T, 1)
    out = torch.empty(T, cols, dtype=torch.bfloat16, device="cuda")
    tcg.moe_dispatch(T, k, cols, T, x, cols, "bf16", row_of, 1, out, cols, "bf16")
    for at in range(0, T, 50000):
        assert torch.equal(out[row_of[at:at + 50000, 0].long()], x[at:at + 50000])
    y = torch.empty_like(x)
    tcg.moe_combine(T, k, cols, T, out, cols, "bf16", row_of, 1, None, 1, y, cols, "bf16")
    assert torch.equal(x, y)


def test_streams_and_a_replayed_graph():
    T, E, k, cols = 700, 24, 3, 200
    gen = torch.Generator(device="cuda").manual_seed(4)
    topk = random_choice(T, E, k, gen)
    x = torch.randn(T, cols, generator=gen, device="cuda")
    n = tcg.moe_sort_workspace_size(T, E, k)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    off, row_token, row_of = (torch.empty(m, dtype=torch.int32, device="cuda") for m in (E + 1, T * k, T * k))
    rows, y = torch.zeros(T * k, cols, device="cuda"), torch.empty(T, cols, device="cuda")

    def step():
        st = torch.cuda.current_stream()
        tcg.moe_sort(T, E, k, topk, k, None, off, row_token, row_of, k, workspace=ws, workspace_bytes=n, stream=st)
        tcg.moe_dispatch(T, k, cols, T * k, x, cols, "f32", row_of, k, rows, cols, "f32", stream=st)
        tcg.moe_combine(T, k, cols, T * k, rows, cols, "f32", row_of, k, None, k, y, cols, "f32", stream=st)

    def check():
        torch.cuda.synchronize()
        live = ((topk >= 0) & (topk < E)).sum(1, keepdim=True)
        want = x * live
        assert bool(((y - want).abs() <= 4 * U * want.abs()).all())
        assert torch.equal(row_of.view(T, k).cpu().long(), sorted_reference(topk, None, E)[2])

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        topk.copy_(random_choice(T, E, k, gen))
        x.normal_(generator=gen)
        graph.replay()
        check()
