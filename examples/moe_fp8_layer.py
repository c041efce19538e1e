"""A mixture-of-experts layer in 8 bits with one fp32 scale per 128 elements:
forward, backward and the router's balance loss, on the library's operators.

    python examples/moe_fp8_layer.py [tokens hidden inner experts k]

The layer is y_t = sum over t's k experts e of w_te W2_e relu(W1_e x_t)^2, with
the router's softmax weights w.  Every product runs in 8 bits:

    router     tcg.moe_route chooses the experts and their weights,
               tcg.moe_sort puts the assignments in expert order
    dispatch   tcg.quantize_rows128 gathers the tokens into expert order
    experts    tcg.gemm_block128_grouped, twice (weights by 128 x 128 tiles)
    dx         the same products with the weights' transposed codes
    dW         tcg.quantize_cols128 and tcg.gemm_block128_grouped_k, into fp32
    combine    tcg.moe_combine sums a token's experts with their weights (and the
               tokens' gradients over their rows); tcg.moe_combine_backward
               makes the gradients of the experts' outputs and of the weights
    balance    tcg.moe_balance and tcg.moe_balance_backward: the balance loss and
               its gradient; tcg.moe_route_backward: the weights' part of the
               logits' gradient

The host never waits for the routing.  The activation and its gradient are
torch operations here.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tiled_tensor_core_persistent_gb300 as tcg  # noqa: E402


def blocks(n):
    return -(-n // 128)


class Fp8MoeLayer:
    """Holds the weights' codes and the buffers that every step reuses.  hidden
    and inner are multiples of 16 (rows of 8-bit operands start on 16 bytes)."""

    def __init__(self, w1, w2, k, coef=0.01):
        self.E, self.I, self.H = w1.shape     # w1: E x inner x hidden, w2: E x hidden x inner
        self.k, self.coef, dev = k, coef, w1.device
        self.codes = [self.quantize_weight(w) for w in (w1, w2)]
        self.ws = None

    def quantize_weight(self, w):
        """Codes, transposed codes and tile scales of E stacked matrices (after an optimizer step)."""
        e, n, k = w.shape
        q = torch.empty(e, n, k, dtype=torch.uint8, device=w.device)
        qt = torch.empty(e, k, n, dtype=torch.uint8, device=w.device)
        s = torch.empty(e, blocks(n), blocks(k), device=w.device)
        tcg.quantize_tiles128(e, n, k, w, k, "bf16", q, k, qt, n, "e4m3", s, stream=torch.cuda.current_stream())
        return q, qt, s

    def workspace(self, need):
        """The one workspace of all calls, which run one after the other."""
        if self.ws is None or self.ws.numel() < need:
            self.ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        return dict(workspace=self.ws, workspace_bytes=self.ws.numel(), stream=torch.cuda.current_stream())

    def rows(self, x, index=None, source=0):
        """x's rows (gathered) as an operand: codes, scales."""
        r = x.shape[0] if index is None else index.numel()
        c = x.shape[1]
        q = torch.empty(r, c, dtype=torch.uint8, device=x.device)
        s = torch.empty(blocks(c), r, device=x.device)
        tcg.quantize_rows128(r, c, x, c, "bf16", q, c, "e4m3", s, r, row_index=index, source_rows=source,
                             stream=torch.cuda.current_stream())
        return tcg.block_operand(q, c, s, 1, 1, r), (q, s)

    def cols(self, x, index=None, source=0):
        """x's columns over each expert's rows, transposed, as an operand of a weight gradient."""
        r = x.shape[0] if index is None else index.numel()
        c, places = x.shape[1], (r // 128 + self.E) * 128
        q = torch.empty(c, places, dtype=torch.uint8, device=x.device)
        s = torch.empty(places // 128, c, device=x.device)
        tcg.quantize_cols128(r, c, x, c, "bf16", q, places, "e4m3", s, c, padded_rows=places, num_groups=self.E, offsets=self.offsets,
                             row_index=index, source_rows=source, stream=torch.cuda.current_stream())
        return tcg.block_operand(q, places, s, 1, 1, c), (q, s), places

    def product(self, a, which, transposed, rows):
        """Each expert's rows times its weight (or its transpose: the scales' strides change places)."""
        q, qt, s = self.codes[which]
        n, k = q.shape[1:]
        nb, kb = s.shape[1:]
        if transposed:
            n, k = k, n
            b = tcg.block_operand(qt, k, s, 128, 1, kb, nb * kb)
        else:
            b = tcg.block_operand(q, k, s, 128, kb, 1, nb * kb)
        y = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
        tcg.gemm_block128_grouped(self.E, self.offsets, rows, n, k, a, b, y, n, "bf16", **self.workspace(tcg.block128_workspace_size(self.E, rows, n, k)))
        return y

    def weight_grad(self, da, xb, places, m, n):
        g = torch.empty(self.E, m, n, device="cuda")
        tcg.gemm_block128_grouped_k(self.E, self.offsets, m, n, places, da, xb, 0.0, None, n, "f32", g, n, "f32",
                                    **self.workspace(256))
        return g

    def forward(self, x, logits, mask=None):
        t, k, stream = x.shape[0], self.k, torch.cuda.current_stream()
        n = t * k
        ints = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.x, self.logits, self.mask = x, logits, mask
        self.expert, self.weight = ints(t, k), torch.empty(t, k, device="cuda")
        tcg.moe_route(t, self.E, k, logits, self.E, "bf16", mask, False, self.expert, k, self.weight, k, stream=stream)
        self.counts, self.valid, self.loss = ints(self.E), ints(1), torch.empty(1, device="cuda")
        tcg.moe_balance(t, self.E, k, logits, self.E, "bf16", self.expert, k, mask, self.coef, self.counts, None, self.valid, self.loss,
                        **self.workspace(tcg.moe_balance_workspace_size()))
        self.offsets, self.token, self.row_of = ints(self.E + 1), ints(n), ints(t, k)
        tcg.moe_sort(t, self.E, k, self.expert, k, mask, self.offsets, self.token, self.row_of, k,
                     **self.workspace(tcg.moe_sort_workspace_size(t, self.E, k)))
        # (rows past the last assignment belong to no expert: the products leave them as they are)
        self.live = (self.token >= 0)[:, None]
        a, keep = self.rows(x, self.token, t)
        self.h = self.product(a, 0, False, n)
        r = torch.relu(self.h.float())
        self.act = torch.where(self.live, r * r, 0.0).to(torch.bfloat16)
        a, keep = self.rows(self.act)
        self.out = self.product(a, 1, False, n)
        y = torch.empty(t, self.H, dtype=torch.bfloat16, device="cuda")
        tcg.moe_combine(t, k, self.H, n, self.out, self.H, "bf16", self.row_of, k, self.weight, k, y, self.H, "bf16", stream=stream)
        return y, self.loss

    def backward(self, dy, dloss):
        """Gradients of x, W1, W2 and the logits: of the balance loss, and of y through the weights."""
        t, k, n, stream = self.x.shape[0], self.k, self.token.numel(), torch.cuda.current_stream()
        do = torch.zeros(n, self.H, dtype=torch.bfloat16, device="cuda")
        dweight = torch.empty(t, k, device="cuda")
        tcg.moe_combine_backward(t, k, self.H, n, self.out, self.H, "bf16", self.row_of, k, self.weight, k, dy, self.H, "bf16", do, self.H,
                                 dweight, k, stream=stream)
        a, keep = self.rows(do)
        dact = self.product(a, 1, True, n)
        da, ka, places = self.cols(do)
        xb, kb, _ = self.cols(self.act)
        dw2 = self.weight_grad(da, xb, places, self.H, self.I)
        dh = torch.where(self.live, dact.float() * 2.0 * torch.relu(self.h.float()), 0.0).to(torch.bfloat16)
        a, keep = self.rows(dh)
        dxr = self.product(a, 0, True, n)
        da, ka, places = self.cols(dh)
        xb, kb, _ = self.cols(self.x, self.token, t)
        dw1 = self.weight_grad(da, xb, places, self.I, self.H)
        dx = torch.empty(t, self.H, device="cuda")
        tcg.moe_combine(t, k, self.H, n, dxr, self.H, "bf16", self.row_of, k, None, k, dx, self.H, "f32", stream=stream)
        dlogits, drouter = (torch.empty(self.logits.shape, device="cuda") for _ in range(2))
        tcg.moe_balance_backward(t, self.E, k, self.logits, self.E, "bf16", self.mask, self.coef, self.counts, self.valid, dloss, dlogits,
                                 self.E, "f32", stream=stream)
        # (kept apart to compare them; accumulate = True adds the second to the first)
        tcg.moe_route_backward(t, self.E, k, self.logits, self.E, "bf16", self.expert, k, False, dweight, k, False, drouter, self.E, "f32",
                               stream=stream)
        return dx, dw1, dw2, dlogits, drouter


def reference(x, w1, w2, logits, k, coef, dy, dloss, mask):
    """The same layer in fp32 torch with autograd."""
    x, w1, w2 = (v.float().requires_grad_() for v in (x, w1, w2))
    z, zr = logits.float().requires_grad_(), logits.float().requires_grad_()
    e = logits.shape[1]
    valid = torch.ones(x.shape[0], dtype=torch.bool, device=x.device) if mask is None else mask != 0
    p = torch.softmax(z, -1)
    weight, expert = torch.topk(torch.softmax(zr, -1), k, -1)
    y = torch.zeros_like(x)
    for i in range(e):
        t, j = torch.nonzero((expert == i) & valid[:, None], as_tuple=True)
        out = torch.relu(x[t] @ w1[i].t()).square() @ w2[i].t()
        y = y.index_add(0, t, out * weight[t, j, None])
    n = int(valid.sum())
    f = torch.bincount(expert[valid].reshape(-1), minlength=e).float() * e / (k * n)
    loss = coef * (f * p[valid].sum(0)).sum() / n
    ((y * dy.float()).sum() + loss * dloss[0]).backward()
    return y, loss, x.grad, w1.grad, w2.grad, z.grad, zr.grad


def run(tokens=2048, hidden=1024, inner=512, experts=16, k=2, seed=0, masked=True):
    """Relative differences (2-norm) of the 8-bit layer from fp32 torch."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rand(tokens, hidden).to(torch.bfloat16)
    w1 = (rand(experts, inner, hidden) / hidden ** 0.5).to(torch.bfloat16)
    w2 = (rand(experts, hidden, inner) / inner ** 0.5).to(torch.bfloat16)
    logits = rand(tokens, experts).to(torch.bfloat16)
    mask = (torch.rand(tokens, generator=g, device="cuda") < 0.9).to(torch.uint8) if masked else None
    dy, dloss = rand(tokens, hidden).to(torch.bfloat16), torch.ones(1, device="cuda")
    layer = Fp8MoeLayer(w1, w2, k)
    y, loss = layer.forward(x, logits, mask)
    got = (y, loss[0], *layer.backward(dy, dloss))
    want = reference(x, w1, w2, logits, k, layer.coef, dy, dloss, mask)
    names = ("y", "loss", "dx", "dW1", "dW2", "dlogits", "drouter")
    return {n: float((a.float() - b.detach()).norm() / b.detach().norm()) for n, a, b in zip(names, got, want)}


if __name__ == "__main__":
    print("relative difference from fp32:", {n: float("%.3g" % v) for n, v in run(*map(int, sys.argv[1:])).items()})
