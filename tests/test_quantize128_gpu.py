"""The quantisers of blocks of 128 on the GPU: codes and scales equal the
definition's fp32 arithmetic bit for bit, and the values they stand for lie
within the format's rounding of x."""
import pytest
import torch

import tiled_tensor_core_persistent_gb300 as tcg

from block128 import CODE, TYPE, ceil_div, padded_places, quantize_rows, quantize_tiles

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tiled_tensor_core_persistent_gb300 import _build
    _build.build()


def values(r, c, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(r, c, generator=g, device="cuda") * torch.exp(2.0 * torch.randn(r, 1, generator=g, device="cuda"))
    return torch.where(torch.rand(r, c, generator=g, device="cuda") < 0.05, 0.0, x).to(TYPE[dtype])


def held(x, pad, shift):
    """x in a buffer of another pitch that starts `shift` elements in; NaN around it."""
    r, c = x.shape
    flat = torch.full((shift + r * (c + pad),), float("nan"), dtype=x.dtype, device="cuda")
    view = flat[shift:].view(r, c + pad)
    view[:, :c] = x
    return view


def same(got, want):
    """Equal codes; any NaN code is a NaN."""
    g, w = got.view(torch.uint8), want.view(torch.uint8)
    nan = torch.isnan(want.float())
    return torch.equal(torch.isnan(got.float()), nan) and torch.equal(g[~nan], w[~nan])


class Codes:
    """A byte matrix with a border."""

    def __init__(self, rows, cols, pad=0, shift=0):
        self.rows, self.cols, self.ld, self.shift = rows, cols, cols + pad, shift
        self.flat = torch.full((shift + (rows + 2) * self.ld,), 0x55, dtype=torch.uint8, device="cuda")
        self.full = self.flat[shift:].view(rows + 2, self.ld)
        self.start = self.full[1:]

    def codes(self, q):
        return self.full[1:self.rows + 1, :self.cols].contiguous().view(CODE[q])

    def clean(self):
        inner = self.full.clone()
        inner[1:self.rows + 1, :self.cols] = 0x55
        return bool((inner == 0x55).all()) and bool((self.flat[:self.shift] == 0x55).all())


SHAPES = [(1, 1), (1, 128), (3, 127), (16, 8192), (5, 129), (33, 300), (130, 520), (257, 1024), (1000, 96), (4099, 2064)]
FORMS = [("bf16", "e4m3", False, 0, 0), ("f16", "e4m3", True, 3, 1), ("f32", "e5m2", False, 1, 1), ("bf16", "e5m2", True, 8, 0),
         ("f32", "e4m3", False, 0, 0), ("bf16", "e4m3", False, 8, 8)]


@pytest.mark.parametrize("xt,q,pow2,pad,shift", FORMS)
@pytest.mark.parametrize("r,c", SHAPES)
def test_rows(r, c, xt, q, pow2, pad, shift):
    x = values(r, c, xt, r + c)
    src = held(x, pad, shift)
    out = Codes(r, c, pad, shift)
    kb = ceil_div(c, 128)
    s = torch.full((kb, r + 2), -1.0, device="cuda")
    tcg.quantize_rows128(r, c, src, c + pad, xt, out.start, out.ld, q, s, r + 2, pow2=pow2)
    want_q, want_s = quantize_rows(x, q, pow2)
    assert torch.equal(s[:, :r], want_s) and bool((s[:, r:] == -1.0).all())
    assert same(out.codes(q), want_q) and out.clean()
    # within the format: half a unit of 3 (2) mantissa bits, or half the smallest step
    wide = want_s.t().repeat_interleave(128, 1)[:, :c].double()
    err = (out.codes(q).float().double() * wide - x.double()).abs()
    rel, low = (2.0 ** -4, 2.0 ** -10) if q == "e4m3" else (2.0 ** -3, 2.0 ** -17)
    assert bool((err <= torch.maximum(rel * x.double().abs(), low * wide) * (1 + 2.0 ** -20)).all())


@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_rows_gathered(xt):
    source, r, c = 50, 333, 700
    x = values(source, c, xt, 3)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    index = torch.randint(-3, source + 3, (r,), generator=g, device="cuda", dtype=torch.int32)
    out = Codes(r, c)
    s = torch.empty(ceil_div(c, 128), r, device="cuda")
    tcg.quantize_rows128(r, c, x, c, xt, out.start, out.ld, "e4m3", s, r, row_index=index, source_rows=source)
    real = (index >= 0) & (index < source)
    y = torch.where(real[:, None], x.float()[index.clamp(0, source - 1).long()], 0.0)
    want_q, want_s = quantize_rows(y)
    assert torch.equal(s, want_s) and same(out.codes("e4m3"), want_q) and out.clean()


def test_special_values():
    x = torch.randn(12, 256, device="cuda")
    x[0] = 0.0
    x[1, 3] = float("nan")
    x[2, 3] = float("inf")
    x[3, 3] = -float("inf")
    x[4] = 1e-40                       # subnormal
    x[5] = -0.0
    x[6] = 3e38
    x[7] = 448.0
    x[8, :128] = 2.0 ** -96
    x[9] = float("nan")
    want_q, want_s = quantize_rows(x)
    out = Codes(12, 256)
    s = torch.empty(2, 12, device="cuda")
    tcg.quantize_rows128(12, 256, x, 256, "f32", out.start, out.ld, "e4m3", s, 12)
    assert torch.equal(s, want_s)
    assert same(out.codes("e4m3"), want_q)
    v = out.codes("e4m3").float() * s.t().repeat_interleave(128, 1)
    assert bool(torch.isnan(v[1, 3])) and int(torch.isnan(v[1]).sum()) == 1
    assert int(torch.isnan(v[2]).sum()) == 128 and int(torch.isnan(v[3]).sum()) == 128
    assert bool((v[7] == 448.0).all()) and not bool(v[0].any())


GROUPS = {"one": [300], "short": [1], "exact": [128, 256], "ragged": [3, 129, 0, 64, 0, 255, 128, 17], "none": [0, 0], "many": [g % 3 for g in range(200)]}


@pytest.mark.parametrize("xt,q,pow2,pad,shift", FORMS)
@pytest.mark.parametrize("which", list(GROUPS))
def test_cols(which, xt, q, pow2, pad, shift):
    lens = GROUPS[which]
    G, c = len(lens), 210
    at = [1]
    for n in lens:
        at.append(at[-1] + n)
    rows = at[-1] + 2
    padded = (rows // 128 + G) * 128
    x = values(rows, c, xt, rows)
    out = Codes(c, padded, pad, shift)
    s = torch.full((padded // 128, c + 3), -1.0, device="cuda")
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    tcg.quantize_cols128(rows, c, held(x, pad, shift), c + pad, xt, out.start, out.ld, q, s, c + 3, padded_rows=padded, num_groups=G,
                         offsets=offsets, pow2=pow2)
    places = torch.tensor(padded_places(at, padded), device="cuda")
    y = torch.where((places >= 0)[:, None], x.float()[places.clamp(min=0)], 0.0)
    want_q, want_s = quantize_rows(y.t().contiguous(), q, pow2)
    assert torch.equal(s[:, :c], want_s) and bool((s[:, c:] == -1.0).all())
    assert same(out.codes(q), want_q) and out.clean()


@pytest.mark.parametrize("rows,c", [(0, 5), (1, 1), (127, 64), (128, 65), (1000, 4104)])
def test_cols_without_groups(rows, c):
    padded = ceil_div(rows, 128) * 128 + 128
    x = values(max(rows, 1), c, "bf16", 1)[:rows]
    out = Codes(c, padded)
    s = torch.empty(padded // 128, c, device="cuda")
    tcg.quantize_cols128(rows, c, x if rows else None, c, "bf16", out.start, out.ld, "e4m3", s, c, padded_rows=padded)
    y = torch.zeros(padded, c, device="cuda")
    y[:rows] = x.float()
    want_q, want_s = quantize_rows(y.t().contiguous())
    assert torch.equal(s, want_s) and same(out.codes("e4m3"), want_q) and out.clean()


def test_cols_gathered():
    source, lens, c = 40, [100, 0, 150], 130
    x = values(source, c, "bf16", 2)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    index = torch.randint(-2, source + 2, (250,), generator=g, device="cuda", dtype=torch.int32)
    offsets = torch.tensor([0, 100, 100, 250], dtype=torch.int32, device="cuda")
    padded = 512
    out = Codes(c, padded)
    s = torch.empty(4, c, device="cuda")
    tcg.quantize_cols128(250, c, x, c, "bf16", out.start, out.ld, "e4m3", s, c, padded_rows=padded, num_groups=3, offsets=offsets,
                         row_index=index, source_rows=source)
    real = (index >= 0) & (index < source)
    y = torch.where(real[:, None], x.float()[index.clamp(0, source - 1).long()], 0.0)
    places = torch.tensor(padded_places([0, 100, 100, 250], padded), device="cuda")
    y = torch.where((places >= 0)[:, None], y[places.clamp(min=0)], 0.0)
    want_q, want_s = quantize_rows(y.t().contiguous())
    assert torch.equal(s, want_s) and same(out.codes("e4m3"), want_q)


@pytest.mark.parametrize("xt,q,pow2,pad,shift", FORMS)
@pytest.mark.parametrize("b,r,c", [(1, 1, 1), (1, 128, 128), (3, 130, 257), (2, 127, 640), (1, 1000, 520)])
def test_tiles(b, r, c, xt, q, pow2, pad, shift):
    x = values(b * r, c, xt, r)
    src = held(x, pad, shift)
    rb, cb = ceil_div(r, 128), ceil_div(c, 128)
    for with_q, with_t in ((True, True), (True, False), (False, True)):
        out, outt = Codes(b * r, c, pad, shift), Codes(b * c, r, pad, shift)
        s = torch.empty(b, rb, cb, device="cuda")
        tcg.quantize_tiles128(b, r, c, src, c + pad, xt, out.start if with_q else None, out.ld if with_q else 0,
                              outt.start if with_t else None, outt.ld if with_t else 0, q, s, pow2=pow2)
        got, gott = out.codes(q).view(torch.uint8).view(b, r, c), outt.codes(q).view(torch.uint8).view(b, c, r)
        for i in range(b):
            want_q, want_s = quantize_tiles(x[i * r:(i + 1) * r], q, pow2)
            assert torch.equal(s[i], want_s)
            w = want_q.view(torch.uint8)
            if with_q:
                assert same(got[i].contiguous().view(CODE[q]), want_q)
            if with_t:
                assert same(gott[i].contiguous().view(CODE[q]), w.t().contiguous().view(CODE[q]))
        assert out.clean() and outt.clean()


def test_rows_past_two_to_the_31_elements():
    r, c = 262200, 8320
    x = torch.zeros(r, c, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 131071, 258110, 258111, 258112, 262199], device="cuda")
    x[at] = torch.randn(7, c, device="cuda").to(torch.bfloat16)
    q = torch.empty(r, c, dtype=torch.uint8, device="cuda")
    s = torch.empty(65, r, device="cuda")
    tcg.quantize_rows128(r, c, x, c, "bf16", q, c, "e4m3", s, r)
    want_q, want_s = quantize_rows(x[at])
    assert torch.equal(q[at], want_q.view(torch.uint8)) and torch.equal(s[:, at], want_s)


def test_another_stream():
    x = values(100, 300, "bf16", 1)
    q = torch.empty(100, 300, dtype=torch.uint8, device="cuda")
    s = torch.empty(3, 100, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    tcg.quantize_rows128(100, 300, x, 300, "bf16", q, 300, "e4m3", s, 100, stream=side)
    side.synchronize()
    want_q, want_s = quantize_rows(x)
    assert torch.equal(q, want_q.view(torch.uint8)) and torch.equal(s, want_s)
