"""What is measured of the router's choice, the way of tokens to their experts and
back, and the loss over a large vocabulary.

What a mixture-of-experts model runs around the experts' products, and the loss
it is trained on:

  route     p = softmax of a token's logits; the k largest logits' experts in
            falling order (ties: the lower expert), and their weights p, or p
            over the k chosen only.  An expert whose logit is -inf is switched
            off: it is never chosen, -1 stands in its place with weight 0, as in
            every place of a masked token.  Training: the logits' gradient too.
  sort      the assignments in the order of their experts, and inside an expert
            in that of the tokens: where each expert's rows start, the token of
            every row (-1 past the last), and the row of every assignment (-1
            for those that were dropped or masked).
  dispatch  the row of x of every token goes to the rows of its assignments in
            the experts' input; rows of no assignment stay as they are.
            Training: with the gradient of x, each token's sum over its rows.
  combine   y_t = sum over j of w_tj x[row_of[t, j]].  Training: the gradients
            of the rows and of the weights.
  xent      lse_t = log sum_v exp(x_t . W_v), loss_t = lse_t - x_t . W_target,
            0 where the target names no word, and the mean over the others; the
            logits, tokens x vocabulary, are never kept.  Training: the
            gradients of x and W.
"""
import math

import torch

own = False

TYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
# columns of the vocabulary that the plain form holds at a time
PIECE = 8192


def listed():
    return [
        # the router of a small decode batch: latency
        dict(name="route 64x16", op="route", tokens=64, experts=16, k=2, x="f32", renormalize=True, masked=0.0, off=0.0, train=False),
        # the router of a training batch with padding: choice, weights, gradient of the logits
        dict(name="route 32768x256 train", op="route", tokens=32768, experts=256, k=8, x="bf16", renormalize=True, masked=0.1, off=0.0, train=True),
        # the same decode batch into expert order
        dict(name="sort 64x16", op="sort", tokens=64, experts=16, k=2, masked=0.0),
        # the training batch's 262144 assignments
        dict(name="sort 32768x256", op="sort", tokens=32768, experts=256, k=8, masked=0.1),
        # the decode batch's hidden states to the experts
        dict(name="dispatch 64x4096", op="dispatch", tokens=64, experts=16, k=2, cols=4096, x="bf16", masked=0.0, train=False),
        # a training batch's, with the gradient that comes back from the experts' inputs
        dict(name="dispatch 16384x4096 train", op="dispatch", tokens=16384, experts=16, k=2, cols=4096, x="bf16", masked=0.0, train=True),
        # the experts' outputs of a decode batch back to its tokens
        dict(name="combine 64x4096", op="combine", tokens=64, experts=16, k=2, cols=4096, x="bf16", masked=0.0, train=False),
        # of a training batch, with both gradients
        dict(name="combine 16384x4096 train", op="combine", tokens=16384, experts=16, k=2, cols=4096, x="bf16", masked=0.0, train=True),
        # the loss of a short prompt: the weights' bytes
        dict(name="xent 64x32768x4096", op="xent", tokens=64, vocab=32768, hidden=4096, x="bf16", ignored=0.0, train=False),
        # the loss of held-out text
        dict(name="xent 4096x131072x2048", op="xent", tokens=4096, vocab=131072, hidden=2048, x="bf16", ignored=0.0, train=False),
        # a fine-tuning step of odd sizes, the prompts' tokens not counted
        dict(name="xent 1000x50021x1280 train", op="xent", tokens=1000, vocab=50021, hidden=1280, x="bf16", ignored=0.3, train=True),
        # a training step
        dict(name="xent 4096x65536x4096 train", op="xent", tokens=4096, vocab=65536, hidden=4096, x="bf16", ignored=0.0, train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "sort", "dispatch", "combine", "xent", "xent"])
    x = rng.choice(["bf16", "bf16", "f16", "f32"])
    masked = rng.choice([0.0, 0.1, 0.5])
    train = rng.random() < 0.6
    if op == "xent":
        while True:
            c = dict(op=op, tokens=_log(rng, 1, 8192), vocab=_log(rng, 100, 131072), hidden=_log(rng, 64, 4096), x=rng.choice(["bf16", "bf16", "f16"]),
                     ignored=rng.choice([0.0, 0.1, 0.5]), train=train)
            if rng.random() < 0.7:
                c["hidden"] = -(-c["hidden"] // 64) * 64
            if _products(c) <= 8 * 4096 * 65536 * 4096:
                return c
    if op in ("route", "sort"):
        experts = _log(rng, 2, 512)
        c = dict(op=op, tokens=_log(rng, 1, 32768), experts=experts, k=rng.randrange(1, min(8, experts) + 1), masked=masked)
        if op == "route":
            c.update(x=x, renormalize=rng.random() < 0.5, off=rng.choice([0.0, 0.0, 0.3]), train=train)
        return c
    while True:
        experts = _log(rng, 2, 256)
        c = dict(op=op, tokens=_log(rng, 1, 32768), experts=experts, k=rng.randrange(1, min(8, experts) + 1), cols=_log(rng, 64, 8192), x=x,
                 masked=masked, train=train)
        if work(c)["bytes"] <= work(dict(c, tokens=16384, k=2, cols=4096, x="bf16", train=True))["bytes"]:
            return c


def _products(c):
    return (8 if c["train"] else 2) * c["tokens"] * c["vocab"] * c["hidden"]


# ------------------------------------------------------------- plain form


def _route_plain(x, mask, k, renormalize):
    """(experts, their weights, p) in the type of x."""
    x = torch.where(mask[:, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    z = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = z.sum(-1, keepdim=True)
    p = torch.where(total > 0, z / total, 0.0)
    value, index = torch.sort(x, dim=-1, descending=True, stable=True)
    index = torch.where(value[:, :k] == -math.inf, -1, index[:, :k])
    w = torch.where(index >= 0, p.gather(1, index.clamp(min=0)), 0.0)
    if renormalize:
        # (over the chosen logits, the largest of which is the token's largest)
        z = torch.where(index >= 0, z.gather(1, index.clamp(min=0)), 0.0)
        total = z.sum(-1, keepdim=True)
        w = torch.where(total > 0, z / total, 0.0)
    return index, w, p


def _route_grad_plain(index, w, p, g, renormalize):
    live = index >= 0
    g = torch.where(live, g, 0.0)
    if renormalize:
        part = w * (g - (w * g).sum(-1, keepdim=True))
        return torch.zeros_like(p).scatter_add(1, index.clamp(min=0), torch.where(live, part, 0.0))
    direct = torch.zeros_like(p).scatter_add(1, index.clamp(min=0), g)
    return p * (direct - (w * g).sum(-1, keepdim=True))


def _sorted_plain(topk, mask, experts):
    t, k = topk.shape
    key = torch.where(mask[:, None] & (topk >= 0) & (topk < experts), topk, experts).reshape(-1)
    order = torch.argsort(key, stable=True)
    real = key[order] < experts
    counts = (key[:, None] == torch.arange(experts, device=key.device)).sum(0) if key.numel() * experts <= 1 << 27 else torch.stack(
        [(key == e).sum() for e in range(experts)])
    offsets = torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0))
    row_token = torch.where(real, torch.div(order, k, rounding_mode="floor"), -1)
    row_of = torch.full_like(key, -1)
    row_of[order] = torch.where(real, torch.arange(key.numel(), device=key.device), -1)
    return dict(offsets=offsets.to(torch.int32), row_token=row_token.to(torch.int32), row_of=row_of.view(t, k).to(torch.int32))


def _gathered(x, index):
    """Rows of x in the order of index, zeros where it holds -1."""
    return torch.where((index >= 0)[:, None], x[index.clamp(min=0).long()], 0.0)


def _combined(x, row_of, w):
    y = torch.zeros(row_of.shape[0], x.shape[1], device=x.device)
    for j in range(row_of.shape[1]):
        y += _gathered(x, row_of[:, j]) * (1.0 if w is None else w[:, j, None])
    return y


def _xent_plain(s):
    c = s["case"]
    x = s["x"].to(torch.float32)
    target, v = s["target"].long(), c["vocab"]
    live = (target >= 0) & (target < v)
    top = torch.full((c["tokens"],), -math.inf, device=x.device)
    total = torch.zeros_like(top)
    picked = torch.zeros_like(top)
    for a in range(0, v, PIECE):
        z = x @ s["w"][a : a + PIECE].to(torch.float32).t()
        m = torch.maximum(top, z.amax(1))
        total = total * torch.exp(top - m) + torch.exp(z - m[:, None]).sum(1)
        top = m
        at = target - a
        inside = live & (at >= 0) & (at < z.shape[1])
        picked = torch.where(inside, z.gather(1, at.clamp(0, z.shape[1] - 1)[:, None])[:, 0], picked)
    lse = top + torch.log(total)
    loss = torch.where(live, lse - picked, 0.0)
    n = live.sum()
    out = dict(lse=lse, loss=loss, mean=(loss.sum() / n.clamp(min=1)).view(1), valid=n.view(1).to(torch.int32))
    if c["train"]:
        g = torch.where(live, s["grad"] / n.clamp(min=1), 0.0)
        dx = torch.zeros_like(x)
        dw = torch.empty_like(s["w"])
        rows = torch.arange(c["tokens"], device=x.device)
        for a in range(0, v, PIECE):
            w = s["w"][a : a + PIECE].to(torch.float32)
            d = torch.exp(x @ w.t() - lse[:, None])
            at = target - a
            inside = live & (at >= 0) & (at < d.shape[1])
            d[rows, at.clamp(0, d.shape[1] - 1)] -= inside.to(torch.float32)
            d *= g[:, None]
            dx += d @ w
            dw[a : a + PIECE] = (d.t() @ x).to(dw.dtype)
        out.update(dx=dx.to(s["x"].dtype), dw=dw)
    return out


# ----------------------------------------------------------------- states


def _held(x, dtype):
    """A matrix in rows of a 16-byte pitch, as the products take them."""
    pitch = -(-x.shape[1] // 8) * 8
    buf = torch.zeros(x.shape[0], pitch, dtype=dtype, device=x.device)
    buf[:, : x.shape[1]] = x.to(dtype)
    return buf[:, : x.shape[1]]


def _choice(t, e, k, gen):
    """Each token's k experts, some of them much liked, a few dropped."""
    liking = torch.randn(e, generator=gen, device=gen.device)
    topk = torch.topk(torch.randn(t, e, generator=gen, device=gen.device) + liking, k, dim=-1).indices
    return torch.where(torch.rand(t, k, generator=gen, device=gen.device) < 0.02, -1, topk).to(torch.int32)


def prepare(case, seed):
    c, op, t = case, case["op"], case["tokens"]
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    s = dict(case=dict(c))
    if op == "xent":
        v, h = c["vocab"], c["hidden"]
        w = randn(v, h) * (2.0 / math.sqrt(h))
        s["w"] = _held(w, TYPE[c["x"]])
        target = torch.randint(0, v, (t,), generator=gen, device=dev)
        # hidden states that lean towards the right word, more or less
        s["x"] = _held(randn(t, h) + 2.0 * rand(t, 1) * w[target], TYPE[c["x"]])
        del w
        target = torch.where(rand(t) < c["ignored"], -100, target)
        target[0] = target[0].clamp(min=0)
        s["target"] = target.to(torch.int32)
        s["lse"], s["loss"] = torch.empty(t, device=dev), torch.empty(t, device=dev)
        s["mean"], s["valid"] = torch.empty(1, device=dev), torch.empty(1, dtype=torch.int32, device=dev)
        s["grad"] = 0.5 + rand(1)
        if c["train"]:
            s["dx"], s["dw"] = torch.zeros_like(_whole(s["x"]))[:, :h], torch.zeros_like(_whole(s["w"]))[:, :h]
        if own:
            import tiled_tensor_core_persistent_gb300 as tcg
            s["ws_bytes"] = tcg.linear_xent_workspace_size(t, v, h, c["train"])
            s["workspace"] = torch.zeros(s["ws_bytes"], dtype=torch.uint8, device=dev)
        return s
    e, k = c["experts"], c["k"]
    s["mask"] = (rand(t) >= c["masked"]).to(torch.uint8)
    s["mask"][0] = 1
    if op == "route":
        x = randn(t, e) + randn(e)
        off = rand(e) < c["off"]
        off[0] = False
        s["logits"] = torch.where(off, -math.inf, x).to(TYPE[c["x"]])
        s["topk"] = torch.empty(t, k, dtype=torch.int32, device=dev)
        s["weights"] = torch.empty(t, k, device=dev)
        s["dweights"] = 0.1 * randn(t, k)
        s["dlogits"] = torch.empty_like(s["logits"])
        return s
    topk = _choice(t, e, k, gen)
    if op == "sort":
        s["topk"] = topk
        s["offsets"] = torch.empty(e + 1, dtype=torch.int32, device=dev)
        s["row_token"] = torch.empty(t * k, dtype=torch.int32, device=dev)
        s["row_of"] = torch.empty(t, k, dtype=torch.int32, device=dev)
        if own:
            import tiled_tensor_core_persistent_gb300 as tcg
            s["ws_bytes"] = tcg.moe_sort_workspace_size(t, e, k)
            s["workspace"] = torch.zeros(s["ws_bytes"], dtype=torch.uint8, device=dev)
        return s
    s.update(_sorted_plain(topk.long(), s["mask"].bool(), e))
    n, cols, dt = t * k, c["cols"], TYPE[c["x"]]
    if op == "dispatch":
        s["x"] = randn(t, cols).to(dt)
        s["out"] = torch.zeros(n, cols, dtype=dt, device=dev)    # (rows of no token stay as they are)
        if c["train"]:
            s["dout"] = (0.1 * randn(n, cols)).to(dt)
            s["dx"] = torch.empty(t, cols, dtype=dt, device=dev)
        return s
    s["x"] = randn(n, cols).to(dt)
    w = torch.exp(randn(t, k))
    s["weights"] = w / w.sum(1, keepdim=True)
    s["y"] = torch.empty(t, cols, dtype=dt, device=dev)
    if c["train"]:
        s["dy"] = (0.1 * randn(t, cols)).to(dt)
        s["dx"] = torch.zeros(n, cols, dtype=dt, device=dev)
        s["dweights"] = torch.empty(t, k, device=dev)
    return s


def _whole(held):
    """The padded matrix that a held one is the front of."""
    return held if held.is_contiguous() else held.as_strided((held.shape[0], held.stride(0)), (held.stride(0), 1))


# ------------------------------------------------------------------- runs


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "xent":
        return _xent_plain(s)
    if op == "route":
        index, w, p = _route_plain(s["logits"].to(torch.float32), s["mask"].bool(), c["k"], c["renormalize"])
        out = dict(topk=index.to(torch.int32), weights=w)
        if c["train"]:
            out["dlogits"] = _route_grad_plain(index, w, p, s["dweights"], c["renormalize"]).to(TYPE[c["x"]])
        return out
    if op == "sort":
        return _sorted_plain(s["topk"].long(), s["mask"].bool(), c["experts"])
    x = s["x"].to(torch.float32)
    if op == "dispatch":
        out = dict(out=_gathered(x, s["row_token"]).to(TYPE[c["x"]]))
        if c["train"]:
            out["dx"] = _combined(s["dout"].to(torch.float32), s["row_of"], None).to(TYPE[c["x"]])
        return out
    out = dict(y=_combined(x, s["row_of"], s["weights"]).to(TYPE[c["x"]]))
    if c["train"]:
        dy = s["dy"].to(torch.float32)
        dx = torch.zeros_like(x)
        dw = torch.zeros_like(s["weights"])
        for j in range(c["k"]):
            at = s["row_of"][:, j]
            live = at >= 0
            dw[:, j] = (dy * _gathered(x, at)).sum(1)
            dx[at[live].long()] = (dy * s["weights"][:, j, None])[live]
        out.update(dx=dx.to(TYPE[c["x"]]), dweights=dw)
    return out


def _run_own(s):
    import tiled_tensor_core_persistent_gb300 as tcg
    c, op, t = s["case"], s["case"]["op"], s["case"]["tokens"]
    stream = torch.cuda.current_stream()
    if op == "xent":
        v, h, ld = c["vocab"], c["hidden"], s["x"].stride(0)
        ws = dict(workspace=s["workspace"], workspace_bytes=s["ws_bytes"], stream=stream)
        tcg.linear_xent(t, v, h, c["x"], s["x"], ld, s["w"], s["w"].stride(0), s["target"], s["lse"], s["loss"], s["mean"], s["valid"], **ws)
        out = dict(lse=s["lse"], loss=s["loss"], mean=s["mean"], valid=s["valid"])
        if c["train"]:
            tcg.linear_xent_backward(t, v, h, c["x"], s["x"], ld, s["w"], s["w"].stride(0), s["target"], s["lse"], s["valid"], s["grad"], None,
                                     s["dx"], s["dx"].stride(0), c["x"], 0.0, s["dw"], s["dw"].stride(0), c["x"], **ws)
            out.update(dx=s["dx"], dw=s["dw"])
        return out
    e, k = c["experts"], c["k"]
    if op == "route":
        tcg.moe_route(t, e, k, s["logits"], e, c["x"], s["mask"], c["renormalize"], s["topk"], k, s["weights"], k, stream=stream)
        out = dict(topk=s["topk"], weights=s["weights"])
        if c["train"]:
            tcg.moe_route_backward(t, e, k, s["logits"], e, c["x"], s["topk"], k, c["renormalize"], s["dweights"], k, False, s["dlogits"], e,
                                   c["x"], stream=stream)
            out["dlogits"] = s["dlogits"]
        return out
    if op == "sort":
        tcg.moe_sort(t, e, k, s["topk"], k, s["mask"], s["offsets"], s["row_token"], s["row_of"], k, workspace=s["workspace"],
                     workspace_bytes=s["ws_bytes"], stream=stream)
        return dict(offsets=s["offsets"], row_token=s["row_token"], row_of=s["row_of"])
    n, cols, x = t * k, c["cols"], c["x"]
    if op == "dispatch":
        tcg.moe_dispatch(t, k, cols, n, s["x"], cols, x, s["row_of"], k, s["out"], cols, x, stream=stream)
        out = dict(out=s["out"])
        if c["train"]:
            tcg.moe_combine(t, k, cols, n, s["dout"], cols, x, s["row_of"], k, None, k, s["dx"], cols, x, stream=stream)
            out["dx"] = s["dx"]
        return out
    tcg.moe_combine(t, k, cols, n, s["x"], cols, x, s["row_of"], k, s["weights"], k, s["y"], cols, x, stream=stream)
    out = dict(y=s["y"])
    if c["train"]:
        tcg.moe_combine_backward(t, k, cols, n, s["x"], cols, x, s["row_of"], k, s["weights"], k, s["dy"], cols, x, s["dx"], cols,
                                 s["dweights"], k, stream=stream)
        out.update(dx=s["dx"], dweights=s["dweights"])
    return out


# ------------------------------------------------------------------- work


def work(case):
    c, op, t = case, case["op"], case["tokens"]
    if op == "xent":
        v, h = c["vocab"], c["hidden"]
        once = (t + v) * h * 2 + 12 * t + 8
        # (the gradient needs the logits' product, and one more for each of x and W)
        return dict(bytes=once + ((t + v) * h * 2 if c["train"] else 0), flops=(6 if c["train"] else 2) * t * v * h)
    e, k = c["experts"], c["k"]
    if op == "route":
        cells, size = t * e, SIZE[c["x"]]
        once = cells * size + t * (1 + 8 * k)
        return dict(bytes=once + (cells * size + 4 * t * k if c["train"] else 0), flops=(10 if c["train"] else 5) * cells)
    if op == "sort":
        return dict(bytes=t * (12 * k + 1) + 4 * (e + 1), flops=t * k)
    row, live = c["cols"] * SIZE[c["x"]], int(0.98 * (1.0 - c["masked"]) * t * k)
    if op == "dispatch":
        once = (t + live) * row + 4 * t * k
        return dict(bytes=once + ((live + t) * row + 4 * t * k if c["train"] else 0), flops=live * c["cols"] if c["train"] else 0)
    once = (live + t) * row + 8 * t * k
    if not c["train"]:
        return dict(bytes=once, flops=2 * live * c["cols"])
    # (the rows are needed once for y and both gradients)
    return dict(bytes=once + (t + live) * row + 4 * t * k, flops=5 * live * c["cols"])


# ------------------------------------------------------- values in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    c, op, t = case, case["op"], case["tokens"]
    f64 = torch.float64
    if op == "xent":
        if _products(c) > 10 ** 13:
            return None
        v, h = c["vocab"], c["hidden"]
        w = s["w"].to(f64)
        label = s["target"].long()
        counted = (label >= 0) & (label < v)
        n = max(1, int(counted.sum()))
        lse, loss = torch.empty(t, dtype=f64, device="cuda"), torch.zeros(t, dtype=f64, device="cuda")
        dx = torch.empty(t, h, dtype=f64, device="cuda") if c["train"] else None
        dw = torch.zeros(v, h, dtype=f64, device="cuda") if c["train"] else None
        step = max(1, (1 << 27) // v)
        for a in range(0, t, step):
            rows = slice(a, min(t, a + step))
            x = s["x"][rows].to(f64)
            z = torch.mm(x, w.t())
            lse[rows] = torch.logsumexp(z, 1)
            here = torch.nonzero(counted[rows]).view(-1)
            loss[rows][here] = lse[rows][here] - z[here, label[rows][here]]
            if c["train"]:
                z = torch.softmax(z, 1)
                z[here, label[rows][here]] -= 1.0
                z *= counted[rows].to(f64)[:, None] * (float(s["grad"]) / n)
                dx[rows] = torch.mm(z, w)
                dw.addmm_(z.t(), x)
        out = dict(lse=lse, loss=loss, mean=(loss.sum() / n).reshape(1), valid=counted.sum().reshape(1))
        if c["train"]:
            out.update(dx=dx, dw=dw)
        return out
    e, k = c["experts"], c["k"]
    real = torch.nonzero(s["mask"]).view(-1)
    if op == "route":
        x = s["logits"][real].to(f64)
        left = x.clone()
        rows = torch.arange(real.numel(), device="cuda")
        chosen = torch.full((real.numel(), k), -1, dtype=torch.long, device="cuda")
        for j in range(k):
            best = left.max(1).values
            first = torch.where(left == best[:, None], torch.arange(e, device="cuda"), e).min(1).values
            ok = best > -math.inf
            chosen[ok, j] = first[ok]
            left[rows, first] = -math.inf
        ok = chosen >= 0
        if c["renormalize"]:
            w = torch.softmax(torch.where(ok, x.gather(1, chosen.clamp(min=0)), -math.inf), 1)
        else:
            w = torch.softmax(x, 1).gather(1, chosen.clamp(min=0))
        w = torch.where(ok, w, 0.0)
        topk = torch.full((t, k), -1, dtype=torch.long, device="cuda")
        weights = torch.zeros(t, k, dtype=f64, device="cuda")
        topk[real], weights[real] = chosen, w
        out = dict(topk=topk, weights=weights)
        if c["train"]:
            g = torch.where(ok, s["dweights"][real].to(f64), 0.0)
            back = w * g
            mean = back.sum(1, keepdim=True)
            d = torch.zeros(real.numel(), e, dtype=f64, device="cuda")
            for j in range(k):
                at = torch.nonzero(ok[:, j]).view(-1)
                d[at, chosen[at, j]] = back[at, j] - (w[at, j] * mean[at, 0] if c["renormalize"] else 0.0)
            if not c["renormalize"]:
                d -= torch.softmax(x, 1) * mean
            dlogits = torch.zeros(t, e, dtype=f64, device="cuda")
            dlogits[real] = d
            out["dlogits"] = dlogits
        return out
    if op == "sort":
        chosen = s["topk"].cpu()
        chosen[s["mask"].cpu() == 0] = -1
        flat = chosen.reshape(-1)
        lists = [torch.nonzero(flat == i).view(-1) for i in range(e)]
        at = torch.cat(lists)
        offsets = torch.zeros(e + 1, dtype=torch.long)
        offsets[1:] = torch.cumsum(torch.tensor([q.numel() for q in lists]), 0)
        row_token = torch.full((t * k,), -1, dtype=torch.long)
        row_token[: at.numel()] = at // k
        row_of = torch.full((t * k,), -1, dtype=torch.long)
        row_of[at] = torch.arange(at.numel())
        return dict(offsets=offsets.cuda(), row_token=row_token.cuda(), row_of=row_of.view(t, k).cuda())
    n, cols = t * k, c["cols"]
    live = int(s["offsets"][-1])
    token = s["row_token"][:live].long()
    if op == "dispatch":
        out = torch.zeros(n, cols, dtype=f64, device="cuda")
        out[:live] = s["x"].to(f64)[token]
        if not c["train"]:
            return dict(out=out)
        return dict(out=out, dx=torch.zeros(t, cols, dtype=f64, device="cuda").index_add_(0, token, s["dout"][:live].to(f64)))
    slot = torch.zeros(n, dtype=torch.long, device="cuda")
    at = torch.nonzero(s["row_of"].reshape(-1) >= 0).view(-1)
    slot[s["row_of"].reshape(-1)[at].long()] = at
    slot = slot[:live]
    w = s["weights"].reshape(-1)[slot].to(f64)
    x = s["x"][:live].to(f64)
    out = dict(y=torch.zeros(t, cols, dtype=f64, device="cuda").index_add_(0, token, x * w[:, None]))
    if c["train"]:
        dy = s["dy"].to(f64)[token]
        dx = torch.zeros(n, cols, dtype=f64, device="cuda")
        dx[:live] = dy * w[:, None]
        dw = torch.zeros(n, dtype=f64, device="cuda")
        dw[slot] = (dy * x).sum(1)
        out.update(dx=dx, dweights=dw.view(t, k))
    return out
