"""What is measured of the block-scaled 8-bit operators and the expert-balance operators.

Each case is one call (or one training step's calls) of a mixture-of-experts
layer that keeps its operands in 8 bits with one fp32 scale per 128 elements:

  quantize_rows   activations, one scale per 1 x 128 of a row, rows gathered
                  into expert order on the way (row_index, -1 = no token)
  quantize_cols   the same activations transposed for the weight gradient, one
                  scale per 128 rows of a column; every expert's rows start on
                  a multiple of 128 and the gaps hold zeros
  quantize_tiles  weights, one scale per 128 x 128, with the transposed copy
                  the input gradient reads
  gemm            D = act(A @ B^T + beta C + bias): a linear layer, its input
                  gradient, or (both operands scaled per 1 x 128) its weight
                  gradient added to what was there
  grouped         the rows of expert g times weight g
  grouped_k       the weight gradients of every expert
  balance         the balance loss of a router, the assignments per expert and
                  where each expert's rows start; with the logits' gradient
                  where the case trains

The scale of a block is max(largest |x|, 2^-96) / 448 (57344 for e5m2), held
in fp32, rounded up to a power of two where the case says so; the element is
x times the scale's fp32 reciprocal, rounded to nearest even.
"""
import math

import torch

own = False

BLOCK = 128
TINY = 2.0 ** -96
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
CODE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
# one workspace of a program that calls these operators one after the other, zeroed once
WORKSPACE_BYTES = 64 << 20


def listed():
    return [
        # the tokens of a small decode batch, before the layer's first product: latency
        dict(name="quantize_rows 16x8192", op="quantize_rows", rows=16, source=0, cols=8192, x="bf16", q="e4m3", pow2=False),
        # a prefill or training batch: every token goes to two experts, in expert order
        dict(name="quantize_rows 32768x4096", op="quantize_rows", rows=32768, source=16384, cols=4096, x="bf16", q="e4m3", pow2=False),
        # output gradients of a training batch for the weight gradient; ragged experts, one of them without a token
        dict(name="quantize_cols 20011x4104", op="quantize_cols", rows=20011, source=0, cols=4104, groups=16, empty=1, x="bf16", q="e4m3", pow2=False),
        # the experts' weights after an optimizer step, from the fp32 master copy's bf16 image
        dict(name="quantize_tiles 16x4096x4096", op="quantize_tiles", batch=16, rows=4096, cols=4096, x="bf16", q="e4m3", pow2=False),
        # one token through a square layer: the weights' bytes
        dict(name="gemm 1x8192x8192", op="gemm", M=1, N=8192, K=8192, per_row=False, beta=0.0, bias=False, act="none", d="bf16", q="e4m3"),
        # an ordinary batch of odd sizes with the fused epilogue
        dict(name="gemm 4095x3001x1537", op="gemm", M=4095, N=3001, K=1537, per_row=False, beta=0.0, bias=True, act="gelu", d="bf16", q="e4m3"),
        # the largest dense product
        dict(name="gemm 8192x8192x8192", op="gemm", M=8192, N=8192, K=8192, per_row=False, beta=0.0, bias=False, act="none", d="bf16", q="e4m3"),
        # a decode batch over 16 experts: a few rows each, two experts idle
        dict(name="grouped 32x4096x4096", op="grouped", groups=16, empty=2, rows=32, N=4096, K=4096, d="bf16", q="e4m3"),
        # a training batch over 16 ragged experts
        dict(name="grouped 32768x4096x4096", op="grouped", groups=16, empty=0, rows=32768, N=4096, K=4096, d="bf16", q="e4m3"),
        # its weight gradients, added to fp32 sums
        dict(name="grouped_k 4096x4096x16384", op="grouped_k", groups=16, empty=1, rows=16384, M=4096, N=4096, beta=1.0, d="f32", q="e4m3"),
        # the router of a decode batch: counts and starts only cost latency
        dict(name="balance 64x16", op="balance", tokens=64, experts=16, k=2, x="bf16", masked=0.0, train=False),
        # the router of a training batch with padding, loss and gradient
        dict(name="balance 32768x256 train", op="balance", tokens=32768, experts=256, k=8, x="bf16", masked=0.1, train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize_rows", "quantize_cols", "quantize_tiles", "gemm", "gemm", "grouped", "grouped_k", "balance", "balance"])
    q = rng.choice(["e4m3", "e4m3", "e4m3", "e5m2"])
    x = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quantize_rows":
        rows = _log(rng, 1, 32768)
        return dict(op=op, rows=rows, source=rng.choice([0, max(1, rows // 2)]), cols=_log(rng, 96, 8192), x=x, q=q, pow2=rng.random() < 0.3)
    if op == "quantize_cols":
        groups = _log(rng, 1, 64)
        return dict(op=op, rows=_log(rng, 1, 32768), source=0, cols=_log(rng, 96, 4200), groups=groups, empty=rng.randrange(0, groups), x=x, q=q,
                    pow2=rng.random() < 0.3)
    if op == "quantize_tiles":
        return dict(op=op, batch=_log(rng, 1, 16), rows=_log(rng, 96, 4096), cols=_log(rng, 96, 4096), x=x, q=q, pow2=rng.random() < 0.3)
    if op == "gemm":
        per_row = rng.random() < 0.4
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 96, 8192), K=_log(rng, 96, 8192), per_row=per_row, beta=1.0 if per_row else 0.0,
                    bias=not per_row and rng.random() < 0.5, act="none" if per_row else rng.choice(["none", "relu", "gelu"]),
                    d="f32" if per_row else "bf16", q=q)
    if op == "grouped":
        groups = _log(rng, 1, 64)
        return dict(op=op, groups=groups, empty=rng.randrange(0, groups), rows=_log(rng, 1, 16384), N=_log(rng, 96, 2048), K=_log(rng, 96, 4096),
                    d=rng.choice(["bf16", "f32"]), q=q)
    if op == "grouped_k":
        groups = _log(rng, 1, 16)
        return dict(op=op, groups=groups, empty=rng.randrange(0, groups), rows=_log(rng, 1, 16384), M=_log(rng, 96, 4096), N=_log(rng, 96, 2048),
                    beta=rng.choice([0.0, 1.0]), d="f32", q=q)
    experts = _log(rng, 2, 512)
    return dict(op=op, tokens=_log(rng, 1, 32768), experts=experts, k=rng.randrange(1, max(1, min(8, experts // 2)) + 1), x=x, masked=rng.choice([0.0, 0.1, 0.5]),
                train=rng.random() < 0.6)


# ------------------------------------------------------------------ shapes


def _blocks(n):
    return -(-n // BLOCK)


def _pitch(n):
    """Row pitch of an 8-bit operand: a multiple of 16 bytes."""
    return -(-n // 16) * 16


def _padded(rows, groups):
    """Room for `groups` runs of `rows` rows in all, each starting on a multiple of 128."""
    return (rows // BLOCK + groups) * BLOCK if groups > 1 else _blocks(rows) * BLOCK


def _lens(rows, groups, empty, gen):
    """Rows per expert: a routed batch's ragged counts, `empty` of them zero."""
    active = groups - empty
    share = torch.exp(0.5 * torch.randn(active, generator=gen))
    base = 1 if rows >= active else 0
    lens = base + torch.floor(share / share.sum() * (rows - base * active)).long()
    short = rows - int(lens.sum())
    lens[: short % active] += 1
    lens += short // active
    place = torch.zeros(groups, dtype=torch.long)
    place[torch.randperm(groups, generator=gen)[:active]] = lens
    return place


# ------------------------------------------------------------- plain form


def _scales(amax, q, pow2):
    s = torch.clamp(amax, min=TINY) * (1.0 / TOP[q])
    if pow2:
        s = ((s.view(torch.int32) + 0x7FFFFF) & 0x7F800000).view(torch.float32)
    return s


def _codes(x, scale, q):
    return (x * (torch.ones_like(scale) / scale)).clamp(-TOP[q], TOP[q]).to(CODE[q])


def _pad(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[-1], 0, rows - x.shape[-2]))


def _gathered(x, index):
    """Rows of x in the order of index, zeros where it holds -1."""
    return x if index is None else torch.where((index >= 0)[:, None], x[index.clamp(min=0).long()], 0.0)


def _rows_quantized(x, q, pow2):
    """x: R x C in fp32.  Codes R x C and scales blocks x R."""
    r, c = x.shape
    blocks = _pad(x, r, _blocks(c) * BLOCK).view(r, _blocks(c), BLOCK)
    s = _scales(blocks.abs().amax(-1), q, pow2)
    return _codes(blocks, s[..., None], q).view(r, -1)[:, :c].contiguous(), s.t().contiguous()


def _tiles_quantized(x, q, pow2):
    """x: B x R x C in fp32.  Codes B x R x C and scales B x row blocks x column blocks."""
    b, r, c = x.shape
    tiles = _pad(x, _blocks(r) * BLOCK, _blocks(c) * BLOCK).view(b, _blocks(r), BLOCK, _blocks(c), BLOCK)
    s = _scales(tiles.abs().amax((2, 4)), q, pow2)
    codes = _codes(tiles, s[:, :, None, :, None], q).view(b, _blocks(r) * BLOCK, _blocks(c) * BLOCK)
    return codes[:, :r, :c].contiguous(), s


def _padded_index(offsets, padded):
    """For each place of the padded order the row it holds, or -1."""
    lens = offsets[1:] - offsets[:-1]
    starts = torch.cumsum((lens + BLOCK - 1) // BLOCK * BLOCK, 0)
    at = torch.arange(padded, device=offsets.device)
    g = torch.searchsorted(starts, at, right=True)
    real = g.clamp(max=lens.numel() - 1)
    inside = at - torch.where(g > 0, starts[(g - 1).clamp(min=0)], 0)
    return torch.where((g < lens.numel()) & (inside < lens[real]), offsets[real] + inside, -1)


def _group_rows(offsets, cap):
    """(groups x cap) row numbers and which of them exist."""
    at = torch.arange(cap, device=offsets.device)
    rows = offsets[:-1, None] + at
    return rows, at < (offsets[1:] - offsets[:-1])[:, None]


def _wide(codes, scales, per_row):
    """The fp32 values of an operand: codes R x K, scales (K blocks x R) or tiles of 128 x 128."""
    v = codes.to(torch.float32)
    s = scales.t() if per_row else scales.repeat_interleave(BLOCK, -2)[..., : v.shape[-2], :]
    return v * s.repeat_interleave(BLOCK, -1)[..., : v.shape[-1]]


def _activated(y, act):
    if act == "relu":
        return y.clamp(min=0.0)
    if act == "gelu":
        return 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    return y


def _router(s, real):
    """(p, f, loss, counts, offsets, valid) of a router in the type `real`."""
    c = s["case"]
    e = c["experts"]
    valid = s["mask"].bool()
    x = torch.where(valid[:, None], s["logits"].to(real), 0.0)
    z = torch.exp(x - x.amax(-1, keepdim=True))
    p = torch.where(valid[:, None], z / z.sum(-1, keepdim=True), 0.0)
    picked = torch.where(valid[:, None], s["topk"], -1).reshape(-1, 1)
    counts = (picked == torch.arange(e, device=p.device)).sum(0)
    n = valid.sum()
    f = counts.to(real) * (e / c["k"]) / n.clamp(min=1).to(real)
    loss = s["coef"] * (f * (p.sum(0) / n.clamp(min=1).to(real))).sum()
    offsets = torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0))
    return p, f, loss, counts, offsets, n


def _router_grad(s, p, f, n, real):
    inner = (p * f).sum(-1, keepdim=True)
    return p * (f - inner) * (s["grad"].to(real) * s["coef"] / n.clamp(min=1).to(real))


# ----------------------------------------------------------------- states


def _activations(rows, cols, gen):
    """Hidden states: unit scale, a few channels ten times as large, rows of different norms."""
    dev = gen.device
    x = torch.randn(rows, cols, generator=gen, device=dev)
    channel = torch.exp(0.4 * torch.randn(cols, generator=gen, device=dev))
    channel = torch.where(torch.rand(cols, generator=gen, device=dev) < 0.01, 10.0 * channel, channel)
    return x * channel * torch.exp(0.3 * torch.randn(rows, 1, generator=gen, device=dev))


def _held(codes):
    """Codes in rows of a 16-byte pitch, as the products take them."""
    buf = torch.zeros(*codes.shape[:-1], _pitch(codes.shape[-1]), dtype=codes.dtype, device=codes.device)
    buf.view(torch.uint8)[..., : codes.shape[-1]] = codes.view(torch.uint8)
    return buf


def prepare(case, seed):
    c, op = case, case["op"]
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    s = dict(case=dict(c))
    if "groups" in c:
        lens = _lens(c["rows"], c["groups"], c["empty"], host)
        s["offsets"] = torch.nn.functional.pad(torch.cumsum(lens, 0), (1, 0)).to(torch.int32).to(dev)
        s["cap"] = max(1, int(lens.max()))
        s["padded"] = _padded(c["rows"], c["groups"])
    if op in ("quantize_rows", "quantize_cols"):
        s["x"] = _activations(c["source"] or c["rows"], c["cols"], gen).to(TYPE[c["x"]])
        s["index"] = None
        if c["source"]:
            index = torch.randint(0, c["source"], (c["rows"],), generator=gen, device=dev)
            s["index"] = torch.where(torch.rand(c["rows"], generator=gen, device=dev) < 0.01, -1, index).to(torch.int32)
        if op == "quantize_rows":
            s["q"] = torch.empty(c["rows"], c["cols"], dtype=CODE[c["q"]], device=dev)
            s["scales"] = torch.empty(_blocks(c["cols"]), c["rows"], device=dev)
        else:
            s["q"] = torch.empty(c["cols"], s["padded"], dtype=CODE[c["q"]], device=dev)
            s["scales"] = torch.empty(s["padded"] // BLOCK, c["cols"], device=dev)
    elif op == "quantize_tiles":
        b, r, n = c["batch"], c["rows"], c["cols"]
        s["x"] = (0.02 * torch.randn(b, r, n, generator=gen, device=dev)).to(TYPE[c["x"]])
        s["q"] = torch.empty(b, r, n, dtype=CODE[c["q"]], device=dev)
        s["qt"] = torch.empty(b, n, r, dtype=CODE[c["q"]], device=dev)
        s["scales"] = torch.empty(b, _blocks(r), _blocks(n), device=dev)
    elif op == "gemm":
        m, n, k = c["M"], c["N"], c["K"]
        a, s["sa"] = _rows_quantized(_activations(m, k, gen), c["q"], False)
        if c["per_row"]:
            b, s["sb"] = _rows_quantized(_activations(n, k, gen), c["q"], False)
        else:
            b, s["sb"] = _tiles_quantized(0.02 * torch.randn(1, n, k, generator=gen, device=dev), c["q"], False)
        s["a"], s["b"] = _held(a), _held(b.view(n, k))
        s["sb"] = s["sb"] if c["per_row"] else s["sb"][0]
        s["bias"] = (0.1 * torch.randn(n, generator=gen, device=dev)).to(torch.bfloat16) if c["bias"] else None
        s["c"] = torch.randn(m, n, generator=gen, device=dev).to(TYPE[c["d"]]) if c["beta"] else None
        s["d"] = torch.empty(m, n, dtype=TYPE[c["d"]], device=dev)
    elif op == "grouped":
        a, s["sa"] = _rows_quantized(_activations(c["rows"], c["K"], gen), c["q"], False)
        b, s["sb"] = _tiles_quantized(0.02 * torch.randn(c["groups"], c["N"], c["K"], generator=gen, device=dev), c["q"], False)
        s["a"], s["b"] = _held(a), _held(b)
        s["d"] = torch.empty(c["rows"], c["N"], dtype=TYPE[c["d"]], device=dev)
    elif op == "grouped_k":
        index = _padded_index(s["offsets"].long(), s["padded"])
        for name, scales, n in (("a", "sa", c["M"]), ("b", "sb", c["N"])):
            x = _gathered(_activations(c["rows"], n, gen), index)
            codes, s[scales] = _rows_quantized(x.t().contiguous(), c["q"], False)
            s[name] = _held(codes)
        s["c"] = torch.randn(c["groups"], c["M"], c["N"], generator=gen, device=dev).to(TYPE[c["d"]]) if c["beta"] else None
        s["d"] = torch.empty(c["groups"], c["M"], c["N"], dtype=TYPE[c["d"]], device=dev)
    else:
        t, e = c["tokens"], c["experts"]
        skew = torch.randn(e, generator=gen, device=dev)
        s["logits"] = (torch.randn(t, e, generator=gen, device=dev) + skew).to(TYPE[c["x"]])
        topk = torch.topk(s["logits"].float(), c["k"], dim=-1).indices
        s["topk"] = torch.where(torch.rand(t, c["k"], generator=gen, device=dev) < 0.02, -1, topk).to(torch.int32)
        s["mask"] = (torch.rand(t, generator=gen, device=dev) >= c["masked"]).to(torch.uint8)
        s["mask"][0] = 1
        s["coef"] = 0.01
        s["grad"] = 0.5 + torch.rand(1, generator=gen, device=dev)
        s["counts"] = torch.empty(e, dtype=torch.int32, device=dev)
        s["starts"] = torch.empty(e + 1, dtype=torch.int32, device=dev)
        s["valid"] = torch.empty(1, dtype=torch.int32, device=dev)
        s["loss"] = torch.empty(1, device=dev)
        s["dlogits"] = torch.empty_like(s["logits"])
    s["workspace"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------- runs


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "quantize_rows":
        q, scales = _rows_quantized(_gathered(s["x"].to(torch.float32), s["index"]), c["q"], c["pow2"])
        return dict(q=q, scales=scales)
    if op == "quantize_cols":
        x = _gathered(s["x"].to(torch.float32), s["index"])
        x = _gathered(x, _padded_index(s["offsets"].long(), s["padded"]))
        q, scales = _rows_quantized(x.t().contiguous(), c["q"], c["pow2"])
        return dict(q=q, scales=scales)
    if op == "quantize_tiles":
        q, scales = _tiles_quantized(s["x"].to(torch.float32), c["q"], c["pow2"])
        return dict(q=q, qt=q.view(torch.uint8).transpose(1, 2).contiguous().view(q.dtype), scales=scales)
    if op == "gemm":
        a = _wide(s["a"][:, : c["K"]], s["sa"], True)
        b = _wide(s["b"][:, : c["K"]], s["sb"], c["per_row"])
        y = a @ b.t()
        if c["beta"]:
            y = y + c["beta"] * s["c"].to(torch.float32)
        if c["bias"]:
            y = y + s["bias"].to(torch.float32)
        return _activated(y, c["act"]).to(TYPE[c["d"]])
    if op == "grouped":
        a = _wide(s["a"][:, : c["K"]], s["sa"], True)
        b = _wide(s["b"][..., : c["K"]], s["sb"], False)
        rows, real = _group_rows(s["offsets"].long(), s["cap"])
        y = torch.bmm(a[rows.clamp(max=c["rows"] - 1)], b.transpose(1, 2))
        at = torch.nonzero(real.view(-1)).view(-1)
        return y.view(-1, c["N"])[at].to(TYPE[c["d"]])
    if op == "grouped_k":
        a = _wide(s["a"], s["sa"], True).t()
        b = _wide(s["b"], s["sb"], True).t()
        lens = s["offsets"][1:] - s["offsets"][:-1]
        starts = torch.nn.functional.pad(torch.cumsum((lens + BLOCK - 1) // BLOCK * BLOCK, 0), (1, 0))
        rows, real = _group_rows(starts, _blocks(s["cap"]) * BLOCK)
        rows = rows.clamp(max=s["padded"] - 1)
        y = torch.bmm(torch.where(real[..., None], a[rows], 0.0).transpose(1, 2), b[rows])
        return (y + c["beta"] * s["c"].to(torch.float32) if c["beta"] else y).to(TYPE[c["d"]])
    p, f, loss, counts, starts, n = _router(s, torch.float32)
    out = dict(loss=loss.view(1), counts=counts.to(torch.int32), offsets=starts.to(torch.int32))
    if c["train"]:
        out["dlogits"] = _router_grad(s, p, f, n, torch.float32).to(TYPE[c["x"]])
    return out


def _run_own(s):
    import tiled_tensor_core_persistent_gb300 as tcg
    c, op = s["case"], s["case"]["op"]
    stream = torch.cuda.current_stream()
    if op == "quantize_rows":
        tcg.quantize_rows128(c["rows"], c["cols"], s["x"], c["cols"], c["x"], s["q"], c["cols"], c["q"], s["scales"], c["rows"],
                             row_index=s["index"], source_rows=c["source"], pow2=c["pow2"], stream=stream)
        return dict(q=s["q"], scales=s["scales"])
    if op == "quantize_cols":
        tcg.quantize_cols128(c["rows"], c["cols"], s["x"], c["cols"], c["x"], s["q"], s["padded"], c["q"], s["scales"], c["cols"],
                             padded_rows=s["padded"], num_groups=c["groups"], offsets=s["offsets"], row_index=s["index"],
                             source_rows=c["source"], pow2=c["pow2"], stream=stream)
        return dict(q=s["q"], scales=s["scales"])
    if op == "quantize_tiles":
        tcg.quantize_tiles128(c["batch"], c["rows"], c["cols"], s["x"], c["cols"], c["x"], s["q"], c["cols"], s["qt"], c["rows"], c["q"],
                              s["scales"], pow2=c["pow2"], stream=stream)
        return dict(q=s["q"], qt=s["qt"], scales=s["scales"])
    if op == "gemm":
        a = tcg.block_operand(s["a"], _pitch(c["K"]), s["sa"], 1, 1, c["M"])
        if c["per_row"]:
            b = tcg.block_operand(s["b"], _pitch(c["K"]), s["sb"], 1, 1, c["N"])
        else:
            b = tcg.block_operand(s["b"], _pitch(c["K"]), s["sb"], BLOCK, _blocks(c["K"]), 1)
        tcg.gemm_block128(c["M"], c["N"], c["K"], a, b, c["beta"], s["c"], c["N"], c["d"], s["d"], c["N"], c["d"], ab_dtype=c["q"],
                          bias=s["bias"], act=c["act"], workspace=s["workspace"], workspace_bytes=WORKSPACE_BYTES, stream=stream)
        return s["d"]
    if op == "grouped":
        kb = _blocks(c["K"])
        a = tcg.block_operand(s["a"], _pitch(c["K"]), s["sa"], 1, 1, c["rows"])
        b = tcg.block_operand(s["b"], _pitch(c["K"]), s["sb"], BLOCK, kb, 1, _blocks(c["N"]) * kb)
        tcg.gemm_block128_grouped(c["groups"], s["offsets"], c["rows"], c["N"], c["K"], a, b, s["d"], c["N"], c["d"], ab_dtype=c["q"],
                                  workspace=s["workspace"], workspace_bytes=WORKSPACE_BYTES, stream=stream)
        return s["d"]
    if op == "grouped_k":
        a = tcg.block_operand(s["a"], s["padded"], s["sa"], 1, 1, c["M"])
        b = tcg.block_operand(s["b"], s["padded"], s["sb"], 1, 1, c["N"])
        tcg.gemm_block128_grouped_k(c["groups"], s["offsets"], c["M"], c["N"], s["padded"], a, b, c["beta"], s["c"], c["N"], c["d"], s["d"],
                                    c["N"], c["d"], ab_dtype=c["q"], workspace=s["workspace"], workspace_bytes=WORKSPACE_BYTES,
                                    stream=stream)
        return s["d"]
    tcg.moe_balance(c["tokens"], c["experts"], c["k"], s["logits"], c["experts"], c["x"], s["topk"], c["k"], s["mask"], s["coef"],
                    s["counts"], s["starts"], s["valid"], s["loss"], workspace=s["workspace"], workspace_bytes=WORKSPACE_BYTES, stream=stream)
    out = dict(loss=s["loss"], counts=s["counts"], offsets=s["starts"])
    if c["train"]:
        tcg.moe_balance_backward(c["tokens"], c["experts"], c["k"], s["logits"], c["experts"], c["x"], s["mask"], s["coef"], s["counts"],
                                 s["valid"], s["grad"], s["dlogits"], c["experts"], c["x"], stream=stream)
        out["dlogits"] = s["dlogits"]
    return out


# ------------------------------------------------------------------- work


def work(case):
    c, op = case, case["op"]
    if op == "quantize_rows":
        read = min(c["rows"], c["source"]) if c["source"] else c["rows"]
        cells = c["rows"] * c["cols"]
        return dict(bytes=read * c["cols"] * SIZE[c["x"]] + cells + 4 * c["rows"] * _blocks(c["cols"]) + (4 * c["rows"] if c["source"] else 0),
                    flops=3 * cells)
    if op == "quantize_cols":
        padded = _padded(c["rows"], c["groups"])
        return dict(bytes=c["rows"] * c["cols"] * SIZE[c["x"]] + padded * c["cols"] + 4 * (padded // BLOCK) * c["cols"],
                    flops=3 * c["rows"] * c["cols"])
    if op == "quantize_tiles":
        cells = c["batch"] * c["rows"] * c["cols"]
        return dict(bytes=cells * (SIZE[c["x"]] + 2) + 4 * c["batch"] * _blocks(c["rows"]) * _blocks(c["cols"]), flops=3 * cells)
    if op == "gemm":
        m, n, k = c["M"], c["N"], c["K"]
        scales = 4 * _blocks(k) * (m + (n if c["per_row"] else _blocks(n)))
        return dict(bytes=(m + n) * k + scales + m * n * SIZE[c["d"]] * (2 if c["beta"] else 1) + (2 * n if c["bias"] else 0), flops=2 * m * n * k)
    if op == "grouped":
        m, n, k = c["rows"], c["N"], c["K"]
        used = min(c["groups"] - c["empty"], m)
        return dict(bytes=m * k + used * n * k + 4 * _blocks(k) * (m + used * _blocks(n)) + m * n * SIZE[c["d"]], flops=2 * m * n * k)
    if op == "grouped_k":
        m, n, t = c["M"], c["N"], c["rows"]
        return dict(bytes=(m + n) * (t + 4 * _blocks(t)) + c["groups"] * m * n * SIZE[c["d"]] * (2 if c["beta"] else 1), flops=2 * m * n * t)
    cells = c["tokens"] * c["experts"]
    once = cells * SIZE[c["x"]] + c["tokens"] * (4 * c["k"] + 1) + 8 * c["experts"] + 12
    return dict(bytes=once + (cells * SIZE[c["x"]] if c["train"] else 0), flops=(12 if c["train"] else 6) * cells)


# ------------------------------------------------------- values in 64 bits


def _rounded64(v, q):
    """v to the nearest value of the 8-bit format, ties to even, as a 64-bit number."""
    bits, lowest = (3, -6) if q == "e4m3" else (2, -14)
    e = torch.frexp(v.abs().clamp(min=2.0 ** -60))[1].to(torch.float64) - 1.0
    step = torch.exp2(e.clamp(min=lowest) - bits)
    return (torch.round(v / step) * step).clamp(-TOP[q], TOP[q])


def _scale64(amax, q, pow2):
    s = amax.clamp(min=TINY) / TOP[q]
    return torch.exp2(torch.ceil(torch.log2(s.float().double()))) if pow2 else s


def _blocked64(x, q, pow2):
    """The codes' values and scales (blocks x rows) of 1 x 128 blocks in 64 bits, a slab of rows at a time."""
    r, c = x.shape
    kb = _blocks(c)
    codes = torch.empty(r, c, dtype=torch.float32, device=x.device)
    scales = torch.empty(kb, r, dtype=torch.float64, device=x.device)
    for a in range(0, r, 4096):
        part = torch.zeros(min(4096, r - a), kb * BLOCK, dtype=torch.float64, device=x.device)
        part[:, :c] = x[a : a + 4096].double()
        part = part.reshape(-1, kb, BLOCK)
        sc = _scale64(part.abs().amax(2), q, pow2)
        scales[:, a : a + 4096] = sc.t()
        held = sc.float().double().unsqueeze(2)
        codes[a : a + 4096] = _rounded64(part / held, q).reshape(part.shape[0], -1)[:, :c].float()
    return codes, scales


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op in ("quantize_rows", "quantize_cols"):
        x = s["x"]
        if s["index"] is not None:
            x = x[s["index"].clamp(min=0).long()] * (s["index"] >= 0).to(x.dtype)[:, None]
        if op == "quantize_cols":
            lens = (s["offsets"][1:] - s["offsets"][:-1]).tolist()
            wide = torch.zeros(c["cols"], s["padded"], dtype=x.dtype, device=x.device)
            row = place = 0
            for n in lens:
                wide[:, place : place + n] = x[row : row + n].t()
                row, place = row + n, place + _blocks(n) * BLOCK
            x = wide
        codes, scales = _blocked64(x, c["q"], c["pow2"])
        return dict(q=codes, scales=scales)
    if op == "quantize_tiles":
        b, r, n = c["batch"], c["rows"], c["cols"]
        q = torch.empty(b, r, n, dtype=torch.float32, device="cuda")
        scales = torch.empty(b, _blocks(r), _blocks(n), dtype=torch.float64, device="cuda")
        for i in range(b):
            x = torch.zeros(_blocks(r) * BLOCK, _blocks(n) * BLOCK, dtype=torch.float64, device="cuda")
            x[:r, :n] = s["x"][i].double()
            amax = x.abs().reshape(_blocks(r), BLOCK, _blocks(n), BLOCK).amax(3).amax(1)
            scales[i] = _scale64(amax, c["q"], c["pow2"])
            held = scales[i].float().double()
            q[i] = _rounded64(x / torch.kron(held, torch.ones(BLOCK, BLOCK, dtype=torch.float64, device="cuda")), c["q"])[:r, :n].float()
        return dict(q=q, qt=q.permute(0, 2, 1).contiguous(), scales=scales)

    def values(codes, scales, tiles):
        """An operand's values in 64 bits: codes R x K."""
        r, k = codes.shape
        v = codes.float().double()
        for j in range(_blocks(k)):
            col = scales[:, j].double().repeat_interleave(BLOCK)[:r] if tiles else scales[j].double()
            v[:, j * BLOCK : (j + 1) * BLOCK] *= col[:, None]
        return v

    if op == "gemm":
        y = values(s["a"][:, : c["K"]], s["sa"], False) @ values(s["b"][:, : c["K"]], s["sb"], not c["per_row"]).t()
        if c["beta"]:
            y += c["beta"] * s["c"].double()
        if c["bias"]:
            y += s["bias"].double()[None, :]
        if c["act"] == "relu":
            y = torch.maximum(y, torch.zeros_like(y))
        elif c["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        return y
    if op == "grouped":
        a = values(s["a"][:, : c["K"]], s["sa"], False)
        at = s["offsets"].tolist()
        y = torch.empty(c["rows"], c["N"], dtype=torch.float64, device="cuda")
        for g in range(c["groups"]):
            if at[g + 1] > at[g]:
                y[at[g] : at[g + 1]] = a[at[g] : at[g + 1]] @ values(s["b"][g][:, : c["K"]], s["sb"][g], True).t()
        return y
    if op == "grouped_k":
        a, b = values(s["a"], s["sa"], False), values(s["b"], s["sb"], False)
        at = s["offsets"].tolist()
        y = torch.zeros(c["groups"], c["M"], c["N"], dtype=torch.float64, device="cuda")
        place = 0
        for g in range(c["groups"]):
            n = _blocks(at[g + 1] - at[g]) * BLOCK
            y[g] = a[:, place : place + n] @ b[:, place : place + n].t()
            place += n
        return y + c["beta"] * s["c"].double() if c["beta"] else y
    real = torch.nonzero(s["mask"]).view(-1)
    e, n = c["experts"], max(1, real.numel())
    p = torch.softmax(s["logits"][real].double(), 1)
    picked = s["topk"][real].reshape(-1).long()
    counts = torch.bincount(picked[picked >= 0], minlength=e)
    f = counts.double() * e / (c["k"] * n)
    out = dict(loss=(s["coef"] * (f * p.sum(0)).sum() / n).reshape(1), counts=counts,
               offsets=torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), torch.cumsum(counts, 0)]))
    if c["train"]:
        d = torch.zeros(c["tokens"], e, dtype=torch.float64, device="cuda")
        d[real] = p * (f[None, :] - p @ f[:, None]) * (float(s["grad"]) * s["coef"] / n)
        out["dlogits"] = d
    return out
