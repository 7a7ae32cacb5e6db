"""Cases of the library's operators on rows grouped by an expert or an adapter:
the sort of tokens by expert with the gather of their rows, the weighted
combination back, the gradients of both, the experts' step for any number of
tokens, and low-rank adapters of many requests beside a projection.

``run`` computes a case in plain torch operations (``own`` false) or through
the library (``own`` true); ``exact`` computes it in 64 bits.  The sizes are
the GLM-scale layer's (hidden 6144, 256 routed experts of 2048, 8 picks a
token, one shared expert) and the 1-bit GEMV's MLP shapes, or generic ones.
"""
import math

import torch

own = False

FP8_MAX = 448.0
EPS = 1e-6


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # a decode batch of 16 requests: latency of the sort and the gather
        dict(name="dispatch-16", op="dispatch", tokens=16, top_k=8, experts=256, local=256,
             hidden=6144, dtype="bf16"),
        # a prefill chunk of 8192 tokens: the rows' traffic
        dict(name="dispatch-8192", op="dispatch", tokens=8192, top_k=8, experts=256, local=256,
             hidden=6144, dtype="bf16"),
        # the same decode batch on the way back
        dict(name="combine-32", op="combine", tokens=32, top_k=8, experts=256, local=256,
             hidden=6144, dtype="bf16", add=True),
        # a ragged prefill chunk on one of four ranks that share the experts:
        # three quarters of the picks are another rank's, fp32 rows
        dict(name="combine-8191-share", op="combine", tokens=8191, top_k=8, experts=256, local=64,
             hidden=6144, dtype="f32", add=False),
        # backward of both movements, an odd micro-batch with odd row sizes
        dict(name="backward-1021", op="backward", tokens=1021, top_k=6, experts=64, local=64,
             hidden=1001, dtype="f32"),
        # backward of a training micro-batch
        dict(name="backward-4096", op="backward", tokens=4096, top_k=8, experts=256, local=256,
             hidden=6144, dtype="bf16"),
        # 16 requests decoding together: twice the rows of the widest decode step
        dict(name="wide-16", op="wide", tokens=16, hidden=6144, inter=2048, experts=256,
             shared=True),
        # a small prefill chunk: every expert is read for a few rows each
        dict(name="wide-300", op="wide", tokens=300, hidden=6144, inter=2048, experts=256,
             shared=True),
        # a large prefill chunk: bound by the products
        dict(name="wide-4096", op="wide", tokens=4096, hidden=6144, inter=2048, experts=256,
             shared=True),
        # one request on the 1-bit MLP up projection, its adapter beside it
        dict(name="lora-gemv-1", op="lora_gemv", rows=1, n=9728, k=2560, rank=16, adapters=32,
             fmt="q1", ragged=False),
        # 64 requests decoding, nearly every one with an adapter of its own
        dict(name="lora-64", op="lora", rows=64, n=6144, k=6144, rank=16, adapters=128,
             segment=1, ragged=True),
        # prefill: 6001 rows of requests of some 200 rows each
        dict(name="lora-6001", op="lora", rows=6001, n=6144, k=6144, rank=64, adapters=24,
             segment=200, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("dispatch", "combine", "backward", "wide", "lora", "lora_gemv"))
    if op in ("dispatch", "combine", "backward"):
        dtype = rng.choice(("bf16", "f32"))
        hidden = rng.choice((_log(rng, 100, 8192), 8 * _log(rng, 16, 1024), 6144))
        top_k = rng.choice((1, 2, 4, 6, 8, 8))
        experts = 16 * _log(rng, 1, 32)
        most = 8192 if op != "backward" else 4096
        most = min(most, int(most * 8 * 6144 / (top_k * hidden)) // (1 if dtype == "bf16" else 2))
        c = dict(op=op, tokens=_log(rng, 1, max(2, min(most, 32768))), top_k=top_k,
                 experts=max(experts, top_k), hidden=hidden, dtype=dtype)
        c["local"] = rng.choice((c["experts"], max(1, c["experts"] // 4)))
        if op == "combine":
            c["add"] = rng.choice((True, False))
        return c
    if op == "wide":
        return dict(op=op, tokens=_log(rng, 9, 4000), hidden=128 * _log(rng, 4, 48),
                    inter=128 * _log(rng, 2, 16), experts=16 * _log(rng, 2, 16),
                    shared=rng.choice((True, False)))
    rank = rng.choice((8, 16, 16, 24, 32, 64, 128))
    if op == "lora":
        n, k = 8 * _log(rng, 64, 1024), 64 * _log(rng, 8, 128)
        most = int(min(6000, 6000 * 64 * 12288 / (rank * (n + k)), 6000 * 3 * 6144 / (k + 2 * n)))
        return dict(op=op, rows=_log(rng, 1, most), n=n, k=k, rank=rank, adapters=_log(rng, 1, 128),
                    segment=rng.choice((1, 1, 17, 200)), ragged=rng.choice((True, False)))
    return dict(op=op, rows=rng.randint(1, 8), n=128 * _log(rng, 4, 96), k=256 * _log(rng, 2, 32),
                rank=rank, adapters=_log(rng, 1, 64), fmt=rng.choice(("q1", "fp8", "bf16")),
                ragged=rng.choice((True, False)))


# ---------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _routing(tokens, top_k, experts, g):
    """The picks and gates of a router whose experts differ in popularity."""
    z = torch.randn(tokens, experts, generator=g, device="cuda")
    z += 0.5 * torch.randn(experts, generator=g, device="cuda")
    top = z.topk(top_k, dim=1)
    return top.indices.to(torch.int32).contiguous(), torch.softmax(top.values, 1).contiguous()


def _fp8_matrices(count, n, k, g):
    """FP8 E4M3 codes [count, n, k] of N(0, 1/k) weights with the fp32 scale
    amax/448 of each 128x128 block."""
    codes = torch.empty(count, n, k, dtype=torch.uint8, device="cuda")
    scales = torch.empty(count, n // 128, k // 128, device="cuda")
    step = max(1, (1 << 28) // (n * k))
    for i in range(0, count, step):
        c = min(step, count - i)
        w = torch.randn(c, n // 128, 128, k // 128, 128, generator=g, device="cuda")
        w *= k ** -0.5
        s = w.abs().amax(dim=(2, 4)) / FP8_MAX
        w /= s[:, :, None, :, None]
        codes[i:i + c] = w.to(torch.float8_e4m3fn).view(torch.uint8).view(c, n, k)
        scales[i:i + c] = s
    return codes, scales


def _adapters(case, g):
    a = case["adapters"]
    d = dict(
        a=(torch.randn(a, case["rank"], case["k"], generator=g, device="cuda") * case["k"] ** -0.5).to(torch.bfloat16),
        b=(torch.randn(a, case["n"], case["rank"], generator=g, device="cuda") * 0.25).to(torch.bfloat16),
        scale=torch.rand(a, generator=g, device="cuda") + 0.5,
        rank=None)
    if case["ragged"]:
        d["rank"] = (8 * torch.randint(1, case["rank"] // 8 + 1, (a,), generator=g, device="cuda")).to(torch.int32)
    return d


def _adapter_ids(rows, adapters, segment, g):
    """The adapter of each row: requests of up to 2 * segment rows, about one
    in nine of them with none (-1)."""
    ids = torch.randint(-1, adapters, (rows,), generator=g, device="cuda")
    none = torch.rand(rows, generator=g, device="cuda") < 0.1
    ids = torch.where(none, torch.full_like(ids, -1), ids)
    if segment > 1:
        cut = torch.rand(rows, generator=g, device="cuda") < 1.0 / segment
        ids = ids[torch.cumsum(cut, 0) % rows]
    return ids.to(torch.int32).contiguous()


def _projection(case, g):
    n, k = case["n"], case["k"]
    if case["fmt"] == "bf16":
        return dict(codes=(torch.randn(n, k, generator=g, device="cuda") * k ** -0.5).to(torch.bfloat16),
                    scales=None)
    if case["fmt"] == "fp8":
        c, s = _fp8_matrices(1, n, k, g)
        return dict(codes=c[0], scales=s[0])
    d = (torch.randn(n, k // 128, generator=g, device="cuda") * 0.02).abs().to(torch.float16)
    blocks = torch.empty(n, k // 128, 18, dtype=torch.uint8, device="cuda")
    blocks[..., :2] = d.view(torch.uint8).view(n, k // 128, 2)
    blocks[..., 2:] = torch.randint(0, 256, (n, k // 128, 16), generator=g, device="cuda",
                                    dtype=torch.uint8)
    return dict(codes=blocks, scales=None)


def _inputs(case, seed):
    """The case's inputs, the same for every side."""
    g = _generator(seed)
    op = case["op"]
    if op in ("dispatch", "combine", "backward"):
        t, k, h, dt = case["tokens"], case["top_k"], case["hidden"], _dtype(case)
        ids, gates = _routing(t, k, case["experts"], g)
        # picks of experts past the local ones belong to another rank
        ids = torch.where(ids < case["local"], ids, torch.full_like(ids, -1))
        s = dict(ids=ids, gates=gates)
        rows = lambda n: torch.randn(n, h, generator=g, device="cuda").to(dt)  # noqa: E731
        if op == "dispatch":
            s["x"] = rows(t)
            return s
        s["y"] = rows(t * k)
        if op == "combine":
            s["add"] = rows(t) if case["add"] else None
        else:
            s["dout"], s["dxs"] = rows(t), rows(t * k)
        _, _, s["pos"] = _plain_sort(s["ids"], case["local"])
        return s
    if op == "wide":
        t, h, i, e = case["tokens"], case["hidden"], case["inter"], case["experts"]
        ids, gates = _routing(t, 8, e, g)
        s = dict(ids=ids, gates=gates,
                 x=torch.randn(t, h, generator=g, device="cuda").to(torch.bfloat16),
                 gamma=(torch.rand(h, generator=g, device="cuda") * 0.4 + 0.8).to(torch.bfloat16),
                 routed=[_fp8_matrices(e, i, h, g), _fp8_matrices(e, i, h, g), _fp8_matrices(e, h, i, g)],
                 shared=None)
        if case["shared"]:
            s["shared"] = [_fp8_matrices(1, i, h, g), _fp8_matrices(1, i, h, g), _fp8_matrices(1, h, i, g)]
        return s
    s = _adapters(case, g)
    r = case["rows"]
    s["x"] = torch.randn(r, case["k"], generator=g, device="cuda").to(torch.bfloat16)
    s["ids"] = _adapter_ids(r, case["adapters"], case.get("segment", 1), g)
    if op == "lora":
        s["base"] = torch.randn(r, case["n"], generator=g, device="cuda").to(torch.bfloat16)
    else:
        s["w"] = _projection(case, g)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        _prepare_own(case, s)
    return s


def _prepare_own(case, s):
    """What a program keeps beside its inputs: outputs, workspaces, structs."""
    from bit_moe_decode_amd import binding as B
    op = case["op"]
    space = lambda n: torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")  # noqa: E731
    if op in ("dispatch", "combine", "backward"):
        t, k, h, e = case["tokens"], case["top_k"], case["hidden"], case["local"]
        if op == "dispatch":
            s["offsets"] = torch.empty(e + 1, dtype=torch.int32, device="cuda")
            s["order"] = torch.empty(t * k, dtype=torch.int32, device="cuda")
            s["pos"] = torch.empty(t, k, dtype=torch.int32, device="cuda")
            s["xs"] = torch.empty(t * k, h, dtype=_dtype(case), device="cuda")
            s["ws"] = space(B.moe_sort_workspace_size(t, k, e))
        elif op == "combine":
            s["out"] = torch.empty(t, h, dtype=_dtype(case), device="cuda")
        else:
            s["dy"] = torch.empty(t * k, h, dtype=_dtype(case), device="cuda")
            s["dgates"] = torch.empty(t, k, device="cuda")
            s["dx"] = torch.empty(t, h, dtype=_dtype(case), device="cuda")
    elif op == "wide":
        s["cfg"] = B.Config(case["hidden"], case["inter"], case["experts"], 8,
                            case["inter"] if case["shared"] else 0, 8, EPS, B.FMT_FP8, B.FMT_FP8,
                            0, B.ACT_FP8)
        sh = None
        if case["shared"]:
            sh = [(c[0], sc[0]) for c, sc in s["shared"]]
        s["weights"] = B.make_weights(s["gamma"], None, s["routed"], sh)
        s["out"] = torch.empty_like(s["x"])
        s["ws"] = space(B.moe_wide_workspace_size(s["cfg"], case["tokens"]))
    else:
        s["lora"] = B.make_lora(s["a"], s["b"], s["scale"], s["rank"])
        s["ws"] = space(B.lora_workspace_size(s["lora"], case["rows"]))
        s["y"] = torch.empty(case["rows"], case["n"], dtype=torch.bfloat16, device="cuda")
        if op == "lora_gemv":
            fmt = {"q1": B.FMT_Q1, "fp8": B.FMT_FP8, "bf16": B.FMT_BF16}[case["fmt"]]
            s["matrix"] = B.make_matrix(fmt, case["n"], case["k"], s["w"]["codes"], s["w"]["scales"])


# ------------------------------------------------------------------------- run
def run(state):
    return (_run_own if own else _run_plain)(state["case"], state)


def _run_own(case, s):
    from bit_moe_decode_amd import binding as B
    op = case["op"]
    # rows that no pick has are left as they were: where there are such, the pass
    # clears the buffers
    some = case.get("local", 0) < case.get("experts", 0)
    if op == "dispatch":
        if some:
            s["order"].fill_(-1)
            s["xs"].zero_()
        B.moe_sort(s["ids"], case["local"], s["offsets"], s["order"], s["pos"], s["ws"])
        B.moe_gather(s["x"], s["pos"], s["xs"])
        return {n: s[n] for n in ("offsets", "order", "pos", "xs")}
    if op == "combine":
        B.moe_combine(s["y"], s["pos"], s["gates"], s["out"], s["add"])
        return s["out"]
    if op == "backward":
        if some:
            s["dy"].zero_()
        B.moe_combine_backward(s["dout"], s["y"], s["pos"], s["gates"], s["dy"], s["dgates"])
        B.moe_gather_backward(s["dxs"], s["pos"], s["dx"])
        return {n: s[n] for n in ("dy", "dgates", "dx")}
    if op == "wide":
        B.moe_wide_step(s["cfg"], s["x"], s["ids"], s["gates"], s["weights"], s["out"], s["ws"])
        return s["out"]
    if op == "lora":
        B.lora_apply(s["lora"], s["x"], s["ids"], s["base"], s["y"], s["ws"])
        return s["y"]
    B.lowbit_gemv_lora(s["matrix"], s["lora"], s["x"], s["ids"], s["y"], s["ws"])
    return s["y"]


def _plain_sort(ids, experts):
    flat = ids.reshape(-1).long()
    kept = (flat >= 0) & (flat < experts)
    key = torch.where(kept, flat, torch.full_like(flat, experts))
    rank, by = torch.sort(key, stable=True)
    offsets = torch.searchsorted(rank, torch.arange(experts + 1, device=ids.device))
    order = torch.where(rank < experts, by, torch.full_like(by, -1))
    pos = torch.empty_like(flat)
    pos[by] = torch.arange(flat.numel(), device=ids.device)
    pos = torch.where(kept, pos, torch.full_like(pos, -1))
    return offsets.int(), order.int(), pos.int().view(ids.shape)


def _plain_blocks(v):
    """FP8 E4M3 values and fp32 scales of the 1x128 blocks of v, multiplied
    out again.  The quotients of bf16 inputs often lie on a border between two
    codes: they are formed in 64 bits and rounded to fp32."""
    b = v.view(v.shape[0], -1, 128)
    s = (b.abs().amax(dim=2, keepdim=True).double() / FP8_MAX).float()
    q = (b.double() / torch.where(s > 0, s, torch.ones_like(s))).float().to(torch.float8_e4m3fn)
    return (q.float() * s).view(v.shape)


def _plain_matrix(codes, scales):
    n, k = codes.shape
    w = codes.view(torch.float8_e4m3fn).float().view(n // 128, 128, k // 128, 128)
    return (w * scales[:, None, :, None]).view(n, k)


def _plain_expert(m, rows, e, rstd):
    g = (rows @ _plain_matrix(m[0][0][e], m[0][1][e]).T) * rstd
    u = (rows @ _plain_matrix(m[1][0][e], m[1][1][e]).T) * rstd
    mid = g / (1 + torch.exp(-g)) * u
    return _plain_blocks(mid) @ _plain_matrix(m[2][0][e], m[2][1][e]).T


def _plain_lora(s, x):
    """scale * B (A x) of every row's adapter; 0 for rows without one."""
    ids, a, b = s["ids"].long(), s["a"], s["b"]
    keep = torch.ones(a.shape[0], a.shape[1], device=x.device)
    if s["rank"] is not None:
        keep = (torch.arange(a.shape[1], device=x.device) < s["rank"][:, None]).float()
    out = torch.zeros(x.shape[0], b.shape[1], device=x.device)
    if x.shape[0] <= a.shape[0]:
        at = ids.clamp(min=0)
        v = torch.bmm(a[at].float(), x[:, :, None]) * keep[at][:, :, None]
        d = torch.bmm(b[at].float(), v)[:, :, 0] * s["scale"][at][:, None]
        return torch.where((ids >= 0)[:, None], d, out)
    for i in range(a.shape[0]):
        v = (x @ a[i].float().T) * keep[i]
        d = (v @ b[i].float().T) * s["scale"][i]
        out = torch.where((ids == i)[:, None], d, out)
    return out


def _plain_projection(case, s, x):
    w = s["w"]
    if case["fmt"] == "bf16":
        return x @ w["codes"].float().T
    if case["fmt"] == "fp8":
        return x @ _plain_matrix(w["codes"], w["scales"]).T
    blk = w["codes"]
    d = blk[..., :2].contiguous().view(torch.float16).float()
    bit = (blk[..., 2:, None] >> torch.arange(8, device=x.device, dtype=torch.uint8)) & 1
    sign = (1.0 - 2.0 * bit.float()).view(blk.shape[0], blk.shape[1], 128)
    return x @ (sign * d).view(blk.shape[0], -1).T


def _run_plain(case, s):
    op = case["op"]
    if op == "dispatch":
        offsets, order, pos = _plain_sort(s["ids"], case["local"])
        xs = s["x"][order.clamp(min=0).long() // case["top_k"]]
        xs = torch.where((order >= 0)[:, None], xs, torch.zeros_like(xs))
        return dict(offsets=offsets, order=order, pos=pos, xs=xs)
    if op == "combine":
        kept = s["pos"] >= 0
        g = torch.where(kept, s["gates"], torch.zeros_like(s["gates"]))
        out = torch.zeros(case["tokens"], case["hidden"], device="cuda")
        for j in range(case["top_k"]):
            out += g[:, j, None] * s["y"][s["pos"][:, j].clamp(min=0).long()].float()
        if s["add"] is not None:
            out += s["add"].float()
        return out.to(s["y"].dtype)
    if op == "backward":
        kept = s["pos"] >= 0
        g = torch.where(kept, s["gates"], torch.zeros_like(s["gates"]))
        dout = s["dout"].float()
        dy = torch.zeros_like(s["y"])
        dg = torch.zeros_like(g)
        dx = torch.zeros_like(dout)
        at = torch.where(kept, s["pos"], torch.full_like(s["pos"], dy.shape[0])).long()
        spare = torch.cat([dy, dy[:1]])  # a row for the dropped picks' writes
        for j in range(case["top_k"]):
            rows = s["pos"][:, j].clamp(min=0).long()
            spare[at[:, j]] = (g[:, j, None] * dout).to(dy.dtype)
            dg[:, j] = torch.where(kept[:, j], (dout * s["y"][rows].float()).sum(1), dg[:, j])
            dx += torch.where(kept[:, j, None], s["dxs"][rows].float(), torch.zeros_like(dx))
        return dict(dy=spare[:-1], dgates=dg, dx=dx.to(s["dxs"].dtype))
    x = s["x"].float()
    if op == "wide":
        rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
        act = _plain_blocks((x * s["gamma"].float()).to(torch.bfloat16).float())
        offsets, order, _ = _plain_sort(s["ids"], case["experts"])
        out = torch.zeros_like(x)
        if s["shared"] is not None:
            out += _plain_expert(s["shared"], act, 0, rstd)
        at = offsets.tolist()
        y = torch.empty(order.numel(), x.shape[1], device="cuda")
        for e in range(case["experts"]):
            if at[e + 1] > at[e]:
                t = order[at[e]:at[e + 1]].long() // 8
                y[order[at[e]:at[e + 1]].long()] = _plain_expert(s["routed"], act[t], e, rstd[t])
        out += (y.view(x.shape[0], 8, -1) * s["gates"][:, :, None]).sum(1)
        return out.to(torch.bfloat16)
    if op == "lora":
        return (s["base"].float() + _plain_lora(s, x)).to(torch.bfloat16)
    return (_plain_projection(case, s, x) + _plain_lora(s, x)).to(torch.bfloat16)


# ----------------------------------------------------------------------- exact
def _e4m3(v):
    """The E4M3 value nearest to v (|v| at most 448 after rounding), ties to
    the even mantissa."""
    _, e = torch.frexp(v.abs())
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-FP8_MAX, FP8_MAX)


def _exact_blocks(v):
    """FP8 blocks by their definition: s = fp32(amax/448), q = E4M3(fp32(v/s))."""
    out = torch.empty_like(v)
    v = v.float().double()
    for b in range(0, v.shape[1], 128):
        c = v[:, b:b + 128]
        s = (c.abs().amax(1) / FP8_MAX).float().double()[:, None]
        q = _e4m3((c / s.clamp(min=1e-300)).float().double())
        out[:, b:b + 128] = q * s
    return out


def _exact_matrix(codes, scales):
    c = codes.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, torch.ldexp(1 + m / 8, e - 7), torch.ldexp(m / 8, torch.full_like(e, -6)))
    v = torch.where(c >= 128, -v, v)
    return v * scales.double().repeat_interleave(128, 0).repeat_interleave(128, 1)


def _exact_expert(m, e, act, rstd):
    g = act @ _exact_matrix(m[0][0][e], m[0][1][e]).t() * rstd
    u = act @ _exact_matrix(m[1][0][e], m[1][1][e]).t() * rstd
    return _exact_blocks(g * torch.sigmoid(g) * u) @ _exact_matrix(m[2][0][e], m[2][1][e]).t()


def _exact_adapters(s, x, out):
    for r, i in enumerate(s["ids"].tolist()) if x.shape[0] <= 64 else ():
        if i >= 0:
            n = s["a"].shape[1] if s["rank"] is None else int(s["rank"][i])
            v = s["a"][i, :n].double() @ x[r]
            out[r] += s["scale"][i].double() * (s["b"][i, :, :n].double() @ v)
    for i in range(s["a"].shape[0]) if x.shape[0] > 64 else ():
        n = s["a"].shape[1] if s["rank"] is None else int(s["rank"][i])
        at = (s["ids"] == i).nonzero()[:, 0]
        v = x[at] @ s["a"][i, :n].double().t()
        out[at] += s["scale"][i].double() * (v @ s["b"][i, :, :n].double().t())
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "dispatch":
        ids = s["ids"].cpu().reshape(-1).tolist()
        by = sorted((i for i, e in enumerate(ids) if 0 <= e < case["local"]), key=lambda i: (ids[i], i))
        xs = torch.zeros(len(ids), case["hidden"], dtype=torch.float64, device="cuda")
        at = torch.tensor(by, device="cuda", dtype=torch.long)
        xs[:len(by)] = s["x"].double()[at // case["top_k"]]
        return dict(offsets=None, order=None, pos=None, xs=xs)
    if op in ("combine", "backward"):
        t, k = torch.nonzero(s["pos"] >= 0, as_tuple=True)
        at = s["pos"][t, k].long()
        gates = s["gates"].double()[t, k]
        if op == "combine":
            out = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
            for c in range(0, at.numel(), 8192):  # in parts, for memory
                part = slice(c, c + 8192)
                out.index_add_(0, t[part], s["y"][at[part]].double() * gates[part, None])
            return out if s["add"] is None else out + s["add"].double()
        dy = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        dg = torch.zeros(s["gates"].shape, dtype=torch.float64, device="cuda")
        dx = torch.zeros(s["dout"].shape, dtype=torch.float64, device="cuda")
        for c in range(0, at.numel(), 8192):
            part = slice(c, c + 8192)
            d = s["dout"][t[part]].double()
            dy[at[part]] = d * gates[part, None]
            dg[t[part], k[part]] = (d * s["y"][at[part]].double()).sum(1)
            dx.index_add_(0, t[part], s["dxs"][at[part]].double())
        return dict(dy=dy, dgates=dg, dx=dx)
    x = s["x"].double()
    if op == "wide":
        rstd = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
        act = _exact_blocks((x * s["gamma"].double()).to(torch.bfloat16).double())
        out = torch.zeros_like(x)
        if s["shared"] is not None:
            out += _exact_expert(s["shared"], 0, act, rstd)
        for e in range(case["experts"]):
            t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
            if t.numel():
                y = _exact_expert(s["routed"], e, act[t], rstd[t])
                out.index_add_(0, t, y * s["gates"].double()[t, j, None])
        return out
    if op == "lora":
        return _exact_adapters(s, x, s["base"].double())
    w = s["w"]
    if case["fmt"] == "bf16":
        m = w["codes"].double()
    elif case["fmt"] == "fp8":
        m = _exact_matrix(w["codes"], w["scales"])
    else:
        d = w["codes"][..., :2].contiguous().view(torch.float16).double()
        bits = w["codes"][..., 2:].long()
        sign = torch.stack([1 - 2 * ((bits >> i) & 1) for i in range(8)], -1).double()
        m = (sign.view(case["n"], -1, 128) * d).view(case["n"], case["k"])
    return _exact_adapters(s, x, x @ m.t())


# ------------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op in ("dispatch", "combine", "backward"):
        t, s, h = case["tokens"], case["tokens"] * case["top_k"], case["hidden"]
        size = 2 if case["dtype"] == "bf16" else 4
        kept = s * case["local"] / case["experts"]
        if op == "dispatch":
            return dict(bytes=(t + kept) * h * size + 12 * s + 4 * case["local"], flops=0)
        if op == "combine":
            return dict(bytes=(kept + t * (2 if case["add"] else 1)) * h * size + 8 * s,
                        flops=2 * kept * h)
        # dout, y, dy and dxs, dx; the gates, their gradient, the positions
        return dict(bytes=(2 * t + 3 * kept) * h * size + 12 * s, flops=4 * kept * h)
    if op == "wide":
        t, h, i, e = case["tokens"], case["hidden"], case["inter"], case["experts"]
        used = e * (1 - (1 - 8 / e) ** t) + (1 if case["shared"] else 0)
        return dict(bytes=used * 3 * h * i + 4 * t * h + 64 * t,
                    flops=6 * h * i * t * (9 if case["shared"] else 8))
    r, n, k = case["rows"], case["n"], case["k"]
    rank = (case["rank"] + 8) / 2 if case["ragged"] else case["rank"]
    live = 0.9 * r
    a = case["adapters"]
    used = min(a, live) if case.get("segment", 1) > 1 else a * (1 - (1 - 1 / a) ** live)
    if op == "lora":
        # x and y of the rows, y written; the adapters that are used
        return dict(bytes=2 * r * (k + 2 * n) + 2 * used * rank * (k + n) + 4 * r,
                    flops=2 * live * rank * (k + n))
    w = {"q1": n * k * 18 / 128, "fp8": n * k, "bf16": 2 * n * k}[case["fmt"]]
    return dict(bytes=w + 2 * r * (k + n) + 2 * used * rank * (k + n) + 4 * r,
                flops=2 * r * n * k + 2 * live * rank * (k + n))
