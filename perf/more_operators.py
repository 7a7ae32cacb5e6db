"""Cases of the library's products of rows grouped by expert, its LM-head loss
and its embedding lookup, each with its gradient.

``run`` computes a case in plain torch operations (``own`` false) or through
the library (``own`` true); ``exact`` computes it in 64 bits.  The sizes are
the GLM-scale layer's (hidden 6144, 256 routed experts of 2048, 8 picks a
token), the 1-bit GEMV's model (hidden 2560, 151936 tokens of vocabulary), the
tiny layer's, or generic ones.
"""
import math

import torch

own = False


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # a decode batch of 16 requests through the gate and up matrices of the
        # GLM-scale layer's experts: one or two rows an expert, the weights' bytes
        dict(name="product-16", op="product", tokens=16, top_k=8, experts=256, local=256, n=4096,
             k=6144, dtype="bf16"),
        # a ragged prefill chunk on one of four ranks that share the experts, odd
        # matrix sizes, fp32 outputs for an fp32 combination
        dict(name="product-1021-share", op="product", tokens=1021, top_k=6, experts=64, local=16,
             n=1000, k=1416, dtype="f32"),
        # a large chunk of few experts: 1024 rows each, the matrix cores' case
        dict(name="product-8192", op="product", tokens=8192, top_k=8, experts=64, local=64, n=4096,
             k=6144, dtype="bf16"),
        # gradients of an odd micro-batch of small experts, fp32 weight gradients
        dict(name="product-grads-301", op="product_backward", tokens=301, top_k=4, experts=32,
             local=32, n=504, k=1000, dtype="f32"),
        # gradients of a training micro-batch
        dict(name="product-grads-4096", op="product_backward", tokens=4096, top_k=8, experts=64,
             local=64, n=4096, k=6144, dtype="bf16"),
        # log-probabilities of 8 rows, a verify step's: the head's bytes
        dict(name="loss-8", op="loss", rows=8, vocab=151936, hidden=2560),
        # the loss of a training micro-batch
        dict(name="loss-4096", op="loss", rows=4096, vocab=151936, hidden=2560),
        # gradients of an odd batch over a small odd vocabulary
        dict(name="loss-grads-333", op="loss_backward", rows=333, vocab=32003, hidden=1000,
             dtype="bf16"),
        # gradients of a training micro-batch
        dict(name="loss-grads-4096", op="loss_backward", rows=4096, vocab=151936, hidden=2560,
             dtype="bf16"),
        # the first rows of a prefill chunk
        dict(name="embed-8192", op="embed", rows=8192, vocab=151936, hidden=2560, dtype="bf16"),
        # gradient of a small model's table, odd rows in fp32: latency
        dict(name="embed-grad-61", op="embed_backward", rows=61, vocab=1000, hidden=257, dtype="f32",
             out="f32"),
        # gradient of a training micro-batch of text: few tokens make up most rows
        dict(name="embed-grad-8192", op="embed_backward", rows=8192, vocab=151936, hidden=2560,
             dtype="bf16", out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("product", "product_backward", "loss", "loss_backward", "embed", "embed_backward"))
    if op in ("product", "product_backward"):
        n, k = 8 * _log(rng, 16, 768), 8 * _log(rng, 16, 768)
        experts = _log(rng, 4, 256)
        if op == "product_backward":
            experts = min(experts, max(4, 64 * 4096 * 6144 // (n * k)))
        top_k = min(experts, rng.choice((1, 2, 4, 6, 8)))
        # operations of the largest listed case
        rows = int(min(65536, (65536 if op == "product" else 32768) * 4096 * 6144 / (n * k)))
        c = dict(op=op, tokens=_log(rng, 1, max(2, rows // top_k)), top_k=top_k, experts=experts,
                 n=n, k=k, dtype=rng.choice(("bf16", "f32")))
        c["local"] = rng.choice((experts, max(1, experts // 4)))
        return c
    if op in ("loss", "loss_backward"):
        vocab, hidden = _log(rng, 500, 151936), 8 * _log(rng, 16, 768)
        rows = int(min(8192, 4096 * 151936 * 2560 / (vocab * hidden)))
        c = dict(op=op, rows=_log(rng, 1, max(2, rows)), vocab=vocab, hidden=hidden)
        if op == "loss_backward":
            c["dtype"] = "bf16"
        return c
    vocab, hidden = _log(rng, 100, 151936), rng.choice((_log(rng, 64, 4096), 8 * _log(rng, 8, 512)))
    rows = int(min(32768, 8192 * 2 * 2560 / hidden))
    c = dict(op=op, rows=_log(rng, 1, rows), vocab=vocab, hidden=hidden,
             dtype=rng.choice(("bf16", "f32")))
    if op == "embed_backward":
        c["out"] = rng.choice((c["dtype"], "f32"))
    return c


# ---------------------------------------------------------------------- inputs
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EMBED_SCALE = 1.7


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    """Normal numbers, drawn in parts: a large matrix's 32-bit form is not kept."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for part in flat.split(1 << 28):
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda").mul_(std))
    return out


def _offsets(case, g):
    """The experts' first rows, of a router whose experts differ in popularity."""
    z = torch.randn(case["tokens"], case["experts"], generator=g, device="cuda")
    z += 0.5 * torch.randn(case["experts"], generator=g, device="cuda")
    ids = z.topk(case["top_k"], dim=1).indices.reshape(-1)
    # picks of experts past the local ones belong to another rank
    count = torch.bincount(ids, minlength=case["experts"])[:case["local"]]
    return torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)


def _tokens(rows, vocab, g):
    """Token ids with a text's frequencies (the i-th most frequent one's goes as
    1/(i + 3)), in an order of their own; one in twenty is none (-1, padding)."""
    u = torch.rand(rows, generator=g, device="cuda", dtype=torch.float64)
    rank = (3.0 * (((vocab + 3.0) / 3.0) ** u - 1.0)).long().clamp(0, vocab - 1)
    ids = torch.randperm(vocab, generator=g, device="cuda")[rank]
    none = torch.rand(rows, generator=g, device="cuda") < 0.05
    return torch.where(none, torch.full_like(ids, -1), ids).to(torch.int32)


def _inputs(case, seed):
    """The case's inputs, the same for every side."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    if op in ("product", "product_backward"):
        rows, e, n, k = case["tokens"] * case["top_k"], case["local"], case["n"], case["k"]
        s = dict(offsets=_offsets(case, g), x=_normal(g, rows, k),
                 w=_normal(g, e, n, k, std=k ** -0.5))
        if op == "product_backward":
            s["dy"] = _normal(g, rows, n)
        return s
    if op in ("loss", "loss_backward"):
        r, v, h = case["rows"], case["vocab"], case["hidden"]
        s = dict(h=_normal(g, r, h), w=_normal(g, v, h, std=2.0 * h ** -0.5),
                 targets=_tokens(r, v, g))
        if op == "loss_backward":
            # the mean over the rows with a target, and what a forward pass gave
            s["dloss"] = torch.full((r,), 1.0, device="cuda") / (s["targets"] >= 0).sum().clamp(min=1)
            s["lse"] = torch.empty(r, device="cuda")
            for i in range(0, r, 1024):
                z = s["h"][i:i + 1024].float() @ s["w"].float().T
                s["lse"][i:i + 1024] = torch.logsumexp(z, 1)
        return s
    r, v, h, dt = case["rows"], case["vocab"], case["hidden"], TYPES[case["dtype"]]
    s = dict(ids=_tokens(r, v, g))
    if op == "embed":
        s["table"] = _normal(g, v, h, dtype=dt)
    else:
        s["dout"] = _normal(g, r, h, dtype=dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        _prepare_own(case, s)
    return s


def _prepare_own(case, s):
    """What a program keeps beside its inputs: outputs and workspaces.  Rows
    behind the last expert's are left as they were: 0."""
    from bit_moe_decode_amd import binding as B
    op = case["op"]
    space = lambda n: torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")  # noqa: E731
    if op in ("product", "product_backward"):
        rows, e, n, k, dt = s["x"].shape[0], case["local"], case["n"], case["k"], TYPES[case["dtype"]]
        if op == "product":
            s["y"] = torch.zeros(rows, n, dtype=dt, device="cuda")
            s["ws"] = space(B.moe_product_workspace_size(rows, e, n, k))
        else:
            s["dx"] = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
            s["dw"] = torch.empty(e, n, k, dtype=dt, device="cuda")
            s["ws"] = space(B.moe_product_backward_workspace_size(rows, e, n, k))
    elif op in ("loss", "loss_backward"):
        r, v, h = case["rows"], case["vocab"], case["hidden"]
        if op == "loss":
            s["loss"], s["lse"] = torch.empty(r, device="cuda"), torch.empty(r, device="cuda")
            s["ws"] = space(B.lm_head_loss_workspace_size(r, v, h))
        else:
            s["dh"] = torch.empty(r, h, dtype=torch.bfloat16, device="cuda")
            s["dw"] = torch.empty(v, h, dtype=TYPES[case["dtype"]], device="cuda")
            s["ws"] = space(B.lm_head_loss_backward_workspace_size(r, v, h))
    elif op == "embed":
        s["out"] = torch.empty(case["rows"], case["hidden"], dtype=TYPES[case["dtype"]], device="cuda")
    else:
        s["dtable"] = torch.empty(case["vocab"], case["hidden"], dtype=TYPES[case["out"]], device="cuda")
        s["ws"] = space(B.embed_backward_workspace_size(case["rows"], case["vocab"], case["hidden"]))


# ------------------------------------------------------------------------- run
def run(state):
    return (_run_own if own else _run_plain)(state["case"], state)


def _run_own(case, s):
    from bit_moe_decode_amd import binding as B
    op = case["op"]
    if op == "product":
        B.moe_product(s["x"], s["w"], s["offsets"], s["y"], s["ws"])
        return s["y"]
    if op == "product_backward":
        B.moe_product_backward(s["dy"], s["x"], s["w"], s["offsets"], s["dx"], s["dw"], s["ws"])
        return dict(dx=s["dx"], dw=s["dw"])
    if op == "loss":
        B.lm_head_loss(s["h"], s["w"], s["targets"], s["loss"], s["lse"], s["ws"])
        return dict(loss=s["loss"], lse=s["lse"])
    if op == "loss_backward":
        B.lm_head_loss_backward(s["h"], s["w"], s["targets"], s["lse"], s["dloss"], s["dh"], s["dw"],
                                s["ws"])
        return dict(dh=s["dh"], dw=s["dw"])
    if op == "embed":
        B.embed(s["ids"], s["table"], s["out"], EMBED_SCALE)
        return s["out"]
    B.embed_backward(s["ids"], s["dout"], s["dtable"], s["ws"], EMBED_SCALE)
    return s["dtable"]


def _run_plain(case, s):
    op = case["op"]
    if op in ("product", "product_backward"):
        dt = TYPES[case["dtype"]]
        at = s["offsets"].tolist()
        if op == "product":
            y = torch.zeros(s["x"].shape[0], case["n"], dtype=dt, device="cuda")
            for e, (i, j) in enumerate(zip(at, at[1:])):
                if i < j:
                    y[i:j] = (s["x"][i:j].float() @ s["w"][e].float().T).to(dt)
            return y
        dx = torch.zeros_like(s["x"])
        dw = torch.zeros(s["w"].shape, dtype=dt, device="cuda")
        for e, (i, j) in enumerate(zip(at, at[1:])):
            if i < j:
                dy = s["dy"][i:j].float()
                dx[i:j] = (dy @ s["w"][e].float()).to(dx.dtype)
                dw[e] = (dy.T @ s["x"][i:j].float()).to(dt)
        return dict(dx=dx, dw=dw)
    if op in ("loss", "loss_backward"):
        h, w, t = s["h"].float(), s["w"].float(), s["targets"].long()
        live, at = t >= 0, t.clamp(min=0)[:, None]
        z = h @ w.T
        if op == "loss":
            m = z.amax(1, keepdim=True)
            lse = m[:, 0] + torch.log(torch.exp(z - m).sum(1))
            loss = torch.where(live, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
            return dict(loss=loss, lse=lse)
        d = torch.exp(z - s["lse"][:, None])
        d.scatter_add_(1, at, torch.full_like(s["lse"], -1.0)[:, None])
        d *= torch.where(live, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
        return dict(dh=(d @ w).to(torch.bfloat16), dw=(d.T @ h).to(TYPES[case["dtype"]]))
    live, at = s["ids"] >= 0, s["ids"].clamp(min=0).long()
    if op == "embed":
        out = s["table"][at].float() * EMBED_SCALE
        return torch.where(live[:, None], out, torch.zeros_like(out)).to(s["table"].dtype)
    d = torch.where(live[:, None], s["dout"].float() * EMBED_SCALE, torch.zeros_like(s["dout"], dtype=torch.float32))
    out = torch.zeros(case["vocab"], case["hidden"], device="cuda").index_add_(0, at, d)
    return out.to(TYPES[case["out"]])


# ----------------------------------------------------------------------- exact
def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("product", "product_backward"):
        at = s["offsets"].tolist()
        x = s["x"].double()
        if op == "product":
            y = torch.zeros(x.shape[0], case["n"], dtype=torch.float64, device="cuda")
            for e in range(case["local"]):
                part = slice(at[e], at[e + 1])
                y[part] = x[part] @ s["w"][e].double().t()
            return y
        dy = s["dy"].double()
        dx, dw = torch.zeros_like(x), torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
        for e in range(case["local"]):
            part = slice(at[e], at[e + 1])
            dx[part] = dy[part] @ s["w"][e].double()
            dw[e] = dy[part].t() @ x[part]
        return dict(dx=dx, dw=dw)
    if op == "loss":
        h, t = s["h"].double(), s["targets"].long()
        lse = torch.full((h.shape[0],), -math.inf, dtype=torch.float64, device="cuda")
        for i in range(0, case["vocab"], 16384):
            z = h @ s["w"][i:i + 16384].double().t()
            lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
        own_logit = (h * s["w"][t.clamp(min=0)].double()).sum(1)
        return dict(loss=torch.where(t >= 0, lse - own_logit, torch.zeros_like(lse)), lse=lse)
    if op == "loss_backward":
        h, t = s["h"].double(), s["targets"].long()
        scale = torch.where(t >= 0, s["dloss"].double(), torch.zeros_like(h[:, 0]))[:, None]
        dh = torch.zeros_like(h)
        dw = torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
        for i in range(0, case["vocab"], 16384):
            w = s["w"][i:i + 16384].double()
            hit = torch.arange(i, i + w.shape[0], device="cuda")[None] == t[:, None]
            d = (torch.exp(h @ w.t() - s["lse"].double()[:, None]) - hit.double()) * scale
            dh += d @ w
            dw[i:i + 16384] = d.t() @ h
        return dict(dh=dh, dw=dw)
    ids = s["ids"].long()
    if op == "embed":
        out = torch.zeros(case["rows"], case["hidden"], dtype=torch.float64, device="cuda")
        kept = (ids >= 0).nonzero()[:, 0]
        out[kept] = s["table"][ids[kept]].double() * EMBED_SCALE
        return out
    out = torch.zeros(case["vocab"], case["hidden"], dtype=torch.float64, device="cuda")
    kept = (ids >= 0).nonzero()[:, 0]
    return out.index_add_(0, ids[kept], s["dout"][kept].double() * EMBED_SCALE)


# ------------------------------------------------------------------------ work
def _different(rows, vocab):
    """About how many tokens occur among the rows."""
    ln = math.log((vocab + 3.0) / 3.0)
    edge = rows / ln - 3.0  # up to this rank a token is expected once
    if edge <= 0:
        return min(rows, vocab)
    return min(vocab, rows, edge + rows / ln * math.log((vocab + 3.0) / (edge + 3.0)) if edge < vocab else vocab)


def work(case):
    op = case["op"]
    if op in ("product", "product_backward"):
        e, n, k = case["local"], case["n"], case["k"]
        rows = case["tokens"] * case["top_k"] * e / case["experts"]
        used = e * (1 - (1 - case["top_k"] / case["experts"]) ** case["tokens"])
        size = 2 if case["dtype"] == "bf16" else 4
        if op == "product":
            return dict(bytes=2 * rows * k + size * rows * n + 2 * used * n * k, flops=2 * rows * n * k)
        # dy, x, the weights, dx, dw
        return dict(bytes=2 * rows * (n + 2 * k) + 2 * used * n * k + size * e * n * k,
                    flops=4 * rows * n * k)
    if op in ("loss", "loss_backward"):
        r, v, h = case["rows"], case["vocab"], case["hidden"]
        if op == "loss":
            return dict(bytes=2 * h * (r + v) + 12 * r, flops=2 * r * v * h)
        # the logits again, which nobody kept, and the two gradients
        return dict(bytes=4 * h * (r + v) + 12 * r, flops=6 * r * v * h)
    r, v, h = case["rows"], case["vocab"], case["hidden"]
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "embed":
        return dict(bytes=(0.95 * r + _different(r, v)) * h * size + 4 * r, flops=r * h)
    return dict(bytes=r * h * size + v * h * (2 if case["out"] == "bf16" else 4) + 4 * r, flops=2 * r * h)
