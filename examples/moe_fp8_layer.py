"""A mixture-of-experts layer in 8 bits with one fp32 scale per 128 elements:
forward, backward and the router's balance loss, on the library's operators.

    python examples/moe_fp8_layer.py [tokens hidden inner experts k]

The layer is y_t = sum over t's k experts e of w_te W2_e relu(W1_e x_t)^2, with
the router's softmax weights w.  Every product runs in 8 bits:

    dispatch   tcg.quantize_rows128 gathers the tokens into expert order
    experts    tcg.gemm_block128_grouped, twice (weights by 128 x 128 tiles)
    dx         the same products with the weights' transposed codes
    dW         tcg.quantize_cols128 and tcg.gemm_block128_grouped_k, into fp32
    router     tcg.moe_balance writes the experts' offsets that the products
               read (the host never waits for the routing), the balance loss
               and, with tcg.moe_balance_backward, its gradient

Elementwise steps, the choice of experts and the sum over a token's experts
are torch operations here.
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
        self.balance_ws = torch.zeros(tcg.moe_balance_workspace_size(), dtype=torch.uint8, device=dev)
        self.ws = None

    def quantize_weight(self, w):
        """Codes, transposed codes and tile scales of E stacked matrices (after an optimizer step)."""
        e, n, k = w.shape
        q = torch.empty(e, n, k, dtype=torch.uint8, device=w.device)
        qt = torch.empty(e, k, n, dtype=torch.uint8, device=w.device)
        s = torch.empty(e, blocks(n), blocks(k), device=w.device)
        tcg.quantize_tiles128(e, n, k, w, k, "bf16", q, k, qt, n, "e4m3", s, stream=torch.cuda.current_stream())
        return q, qt, s

    def workspace(self, rows, n, k):
        need = tcg.block128_workspace_size(self.E, rows, n, k)
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
        tcg.gemm_block128_grouped(self.E, self.offsets, rows, n, k, a, b, y, n, "bf16", **self.workspace(rows, n, k))
        return y

    def weight_grad(self, da, xb, places, m, n):
        g = torch.empty(self.E, m, n, device="cuda")
        tcg.gemm_block128_grouped_k(self.E, self.offsets, m, n, places, da, xb, 0.0, None, n, "f32", g, n, "f32",
                                    **self.workspace(1, 1, 1))
        return g

    def forward(self, x, logits, mask=None):
        t = x.shape[0]
        p = torch.softmax(logits.float(), -1)
        weight, expert = torch.topk(p, self.k, -1)
        expert = expert.to(torch.int32)
        if mask is not None:
            expert = torch.where(mask[:, None] != 0, expert, self.E)   # padding goes to nobody
        self.counts = torch.empty(self.E, dtype=torch.int32, device="cuda")
        self.offsets = torch.empty(self.E + 1, dtype=torch.int32, device="cuda")
        self.valid = torch.empty(1, dtype=torch.int32, device="cuda")
        self.loss = torch.empty(1, device="cuda")
        tcg.moe_balance(t, self.E, self.k, logits, self.E, "bf16", expert, self.k, mask, self.coef, self.counts, self.offsets, self.valid,
                        self.loss, workspace=self.balance_ws, workspace_bytes=self.balance_ws.numel(),
                        stream=torch.cuda.current_stream())
        order = torch.argsort(expert.view(-1), stable=True)            # assignments in expert order, padding last
        self.token = (order // self.k).to(torch.int32)
        self.weight = weight.view(-1)[order]
        # (a masked token's weight is 0, so what its rows hold does not matter: they are gathered as zeros)
        gather = self.token
        if mask is not None:
            real = expert.view(-1)[order] < self.E
            self.weight = torch.where(real, self.weight, 0.0)
            gather = torch.where(real, gather, -1)
        self.gather, self.x, self.logits, self.mask, n = gather, x, logits, mask, order.numel()
        a, keep = self.rows(x, gather, t)
        self.h = self.product(a, 0, False, n)
        r = torch.relu(self.h.float())
        self.act = torch.where(self.weight[:, None] != 0, r * r, 0.0).to(torch.bfloat16)
        a, keep = self.rows(self.act)
        out = self.product(a, 1, False, n)
        y = torch.zeros(t, self.H, device="cuda")
        y.index_add_(0, self.token.long(), torch.where(self.weight[:, None] != 0, out.float() * self.weight[:, None], 0.0))
        return y.to(torch.bfloat16), self.loss

    def backward(self, dy, dloss):
        """Gradients of x, W1, W2 and, of the balance loss, of the logits."""
        n = self.token.numel()
        do = (dy.float()[self.token.long()] * self.weight[:, None]).to(torch.bfloat16)
        a, keep = self.rows(do)
        dact = self.product(a, 1, True, n)
        da, ka, places = self.cols(do)
        xb, kb, _ = self.cols(self.act)
        dw2 = self.weight_grad(da, xb, places, self.H, self.I)
        live = self.weight[:, None] != 0
        dh = torch.where(live, dact.float() * 2.0 * torch.relu(self.h.float()), 0.0).to(torch.bfloat16)
        a, keep = self.rows(dh)
        dxr = self.product(a, 0, True, n)
        da, ka, places = self.cols(dh)
        xb, kb, _ = self.cols(self.x, self.gather, self.x.shape[0])
        dw1 = self.weight_grad(da, xb, places, self.I, self.H)
        dx = torch.zeros(self.x.shape, device="cuda").index_add_(0, self.token.long(), torch.where(live, dxr.float(), 0.0))
        dlogits = torch.empty(self.logits.shape, device="cuda")
        tcg.moe_balance_backward(self.x.shape[0], self.E, self.k, self.logits, self.E, "bf16", self.mask, self.coef, self.counts, self.valid,
                                 dloss, dlogits, self.E, "f32", stream=torch.cuda.current_stream())
        return dx, dw1, dw2, dlogits


def reference(x, w1, w2, logits, k, coef, dy, dloss, mask):
    """The same layer in fp32 torch with autograd."""
    x, w1, w2 = (v.float().requires_grad_() for v in (x, w1, w2))
    z = logits.float().requires_grad_()
    e = logits.shape[1]
    valid = torch.ones(x.shape[0], dtype=torch.bool, device=x.device) if mask is None else mask != 0
    p = torch.softmax(z, -1)
    weight, expert = torch.topk(p.detach(), k, -1)
    y = torch.zeros_like(x)
    for i in range(e):
        t, j = torch.nonzero((expert == i) & valid[:, None], as_tuple=True)
        out = torch.relu(x[t] @ w1[i].t()).square() @ w2[i].t()
        y = y.index_add(0, t, out * weight[t, j, None])
    n = int(valid.sum())
    f = torch.bincount(expert[valid].reshape(-1), minlength=e).float() * e / (k * n)
    loss = coef * (f * p[valid].sum(0)).sum() / n
    ((y * dy.float()).sum() + loss * dloss[0]).backward()
    return y, loss, x.grad, w1.grad, w2.grad, z.grad


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
    names = ("y", "loss", "dx", "dW1", "dW2", "dlogits")
    return {n: float((a.float() - b.detach()).norm() / b.detach().norm()) for n, a, b in zip(names, got, want)}


if __name__ == "__main__":
    print("relative difference from fp32:", {n: float("%.3g" % v) for n, v in run(*map(int, sys.argv[1:])).items()})
