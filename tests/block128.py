"""Plain forms of the block-scaled 8-bit operators (tests only): torch on
whatever device the inputs live on, fp32 where the definition says fp32, 64
bits for the products."""
from __future__ import annotations

import torch

import tiled_tensor_core_persistent_gb300 as tcg

TOP = {"e4m3": 448.0, "e5m2": 57344.0}
CODE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def ceil_div(a, b):
    return -(-a // b)


def scale_of(amax, q="e4m3", pow2=False):
    s = torch.clamp(amax, min=2.0 ** -96) * torch.tensor(1.0 / TOP[q], dtype=torch.float32, device=amax.device)
    return ((s.view(torch.int32) + 0x7FFFFF) & 0x7F800000).view(torch.float32) if pow2 else s


def codes_of(x, s, q="e4m3"):
    """x, s fp32 (broadcast): the codes, NaN where x / s is not a number."""
    v = x * (torch.ones_like(s) / s)
    return v.clamp(-TOP[q], TOP[q]).to(CODE[q])


def amax_last(x):
    """Largest magnitude along the last axis, NaN ignored."""
    return torch.nan_to_num(x.abs(), nan=0.0, posinf=float("inf")).amax(-1)


def quantize_rows(x, q="e4m3", pow2=False):
    """x R x C: codes R x C, scales blocks x R."""
    r, c = x.shape
    kb = ceil_div(c, 128)
    b = torch.zeros(r, kb * 128, device=x.device)
    b[:, :c] = x.float()
    b = b.view(r, kb, 128)
    s = scale_of(amax_last(b), q, pow2)
    return codes_of(b, s[..., None], q).view(r, -1)[:, :c].contiguous(), s.t().contiguous()


def quantize_tiles(x, q="e4m3", pow2=False):
    """x R x C: codes R x C, scales row blocks x column blocks."""
    r, c = x.shape
    rb, cb = ceil_div(r, 128), ceil_div(c, 128)
    b = torch.zeros(rb * 128, cb * 128, device=x.device)
    b[:r, :c] = x.float()
    t = b.view(rb, 128, cb, 128).permute(0, 2, 1, 3).reshape(rb, cb, -1)
    s = scale_of(amax_last(t), q, pow2)
    wide = s.repeat_interleave(128, 0).repeat_interleave(128, 1)
    return codes_of(b, wide, q)[:r, :c].contiguous(), s


def pitched(codes, extra=0):
    """The codes in rows of a 16-byte pitch (plus extra * 16 bytes)."""
    r, k = codes.shape
    ld = ceil_div(max(k, 1), 16) * 16 + 16 * extra
    out = torch.full((r, ld), 0x7F, dtype=torch.uint8, device=codes.device)   # NaN codes past K
    out[:, :k] = codes.view(torch.uint8)
    return out, ld


def wide64(codes, scales, scale_rows):
    """Values in 64 bits; scales (K blocks x rows) or (row blocks x K blocks)."""
    v = codes.to(torch.float32).double()
    s = scales.double().t() if scale_rows == 1 else scales.double().repeat_interleave(128, 0)[: v.shape[0]]
    return v * s.repeat_interleave(128, 1)[:, : v.shape[1]]


def operand(codes, scales, scale_rows, extra=0, k_minor=False):
    """(tcg operand, tensors to keep alive).  k_minor: the scales stored in the other order."""
    data, ld = pitched(codes, extra)
    if k_minor:
        scales = scales.t().contiguous()
    kb_first = (scale_rows == 1) != k_minor      # dimension 0 runs over K blocks
    rs, ks = (1, scales.shape[1]) if kb_first else (scales.shape[1], 1)
    return tcg.block_operand(data, ld, scales, scale_rows, rs, ks), (data, scales)


def workspace(nbytes):
    return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device="cuda")


def padded_places(offsets, rows_cap):
    """Host list: for each place of the padded order its row, or -1; the places are rows_cap many."""
    places = []
    for a, b in zip(offsets[:-1], offsets[1:]):
        places += list(range(a, b))
        places += [-1] * (-(b - a) % 128)
    places = places[:rows_cap]
    return places + [-1] * (rows_cap - len(places))


def within(got, ref, tol):
    """Whether got is what some value of [ref - tol, ref + tol] rounds to in got's type (rounding is
    monotonic, so the interval's ends bound it); ref and tol in 64 bits."""
    lo, hi = (ref - tol).to(got.dtype), (ref + tol).to(got.dtype)
    return bool(((got >= lo) & (got <= hi)).all())
