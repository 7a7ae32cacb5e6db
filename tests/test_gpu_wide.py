"""The experts' step for any number of token rows (moe_wide_step) against its
definition in float64, and against the decode step and its oracle.

Tolerance, element by element.  Gate and up are sums of K / 128 scaled FP8
MFMAs, bounded by the model in tests/parity.py (MFMA8_GROUP per group of 8
products, MFMA8_SUMS and (K/128 + 7) fp32 roundings of the terms, the row's
rstd folded into the scale being one more); mid_tau carries them through
SiLU * up.  mid within tau of its exact value gives a block scale within
tau / 448 of the exact one and a code between the roundings of the window's
ends, so mid's dequantised value is off by at most D = the larger distance of
the two ends' values from the exact one's; down adds |W| D and its own MFMA
bound; the gate-weighted sum adds 10 fp32 roundings; the result is rounded to
bf16 once (2^-8).
"""
import numpy as np
import pytest
import torch

from bit_moe_decode_amd import binding as B
from bit_moe_decode_amd import synth as S
from tests import parity as P

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


def _say(*a):
    print(*a, flush=True)


def _e4m3(v):
    """Nearest E4M3 value, ties to the even mantissa, saturating at 448."""
    _, e = torch.frexp(v.abs())
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _scales(v):
    return (v.float().double().view(v.shape[0], -1, 128).abs().amax(2) / 448.0).float().double()


def _blocks(v):
    s = _scales(v).repeat_interleave(128, 1)
    q = _e4m3((v.float().double() / s.clamp(min=1e-300)).float().double())
    return torch.where(s > 0, q * s, torch.zeros_like(q))


def _matrix(m, e):
    w = m[0][e].view(torch.float8_e4m3fn).double()
    return w * m[1][e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)


def _product(h, w, nkb):
    """(h w^T, bound of its FP8 MFMA sums): h [n, K], w [N, K], float64."""
    ref, terms = h @ w.t(), h.abs() @ w.abs().t()
    gmax = torch.zeros_like(ref)
    wg = w.abs().view(w.shape[0], -1, 8)
    for i in range(h.shape[0]):
        gmax[i] = (wg * h[i].abs().view(1, -1, 8)).amax(2).sum(1)
    return ref, P.MFMA8_GROUP * gmax + (P.MFMA8_SUMS + (nkb + 7) * U32) * terms


def _expert(m, e, h, rstd):
    """(y, its bound) of expert e on rows h (dequantised activations)."""
    nkb = h.shape[1] // 128
    g, dg = _product(h, _matrix(m.gate, e), nkb)
    u, du = _product(h, _matrix(m.up, e), nkb)
    g, dg, u, du = g * rstd, dg * rstd, u * rstd, du * rstd
    sig = torch.sigmoid(g)
    mid = g * sig * u
    # |d mid| <= |d/dg| dg + |d/du| du + dg du, and eight roundings of the evaluation
    tau = ((sig * (1 + g * (1 - sig)) * u).abs() * dg + (g * sig).abs() * du + 2 * dg * du
           + (8 + g.abs()) * U32 * mid.abs())
    s = _scales(mid)
    ds = tau.view(tau.shape[0], -1, 128).amax(2) / 448.0 + 2 * U32 * s
    s, ds = s.repeat_interleave(128, 1), ds.repeat_interleave(128, 1)
    exact = _blocks(mid)
    low = (s - ds).clamp(min=1e-300)
    off = torch.zeros_like(mid)
    for a in (mid - tau, mid + tau):
        for b in (low, s + ds):
            q = _e4m3(a / b)  # the code the window's corner rounds to, at either scale
            for c in (s - ds, s + ds):
                off = torch.maximum(off, (q * c - exact).abs())
    w = _matrix(m.down, e)
    y, dy = _product(exact, w, mid.shape[1] // 128)
    return y, dy + off @ w.abs().t() * (1 + 2.0 ** -9)


def _reference(layer, x, ids, gates):
    x = x.cuda().double()
    rstd = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + float(np.float32(layer.rms_eps)))
    u = (x * layer.gamma.double()).to(torch.bfloat16).double()
    act = _blocks(u)
    out, tol = torch.zeros_like(x), torch.zeros_like(x)
    size = torch.zeros_like(x)
    for e in range(layer.n_experts):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not t.numel():
            continue
        y, dy = _expert(layer.routed, e, act[t], rstd[t])
        w = gates.double()[t, j, None]
        out.index_add_(0, t, w * y)
        tol.index_add_(0, t, w.abs() * dy)
        size.index_add_(0, t, (w * y).abs())
    if layer.shared is not None:
        y, dy = _expert(layer.shared, 0, act, rstd)
        out, tol, size = out + y, tol + dy, size + y.abs()
    return out, tol + 10 * U32 * size


def _layer(hidden, inter, experts, shared, seed):
    return S.make_layer(dict(hidden=hidden, inter=inter, n_experts=experts,
                             shared_inter=inter if shared else 0, router_std=0.02),
                        seed=seed, device="cuda")


def _cfg(layer):
    return B.Config(layer.hidden, layer.inter, layer.n_experts, 8, layer.shared_inter, 8,
                    float(layer.rms_eps), B.FMT_FP8, B.FMT_FP8, 0, B.ACT_FP8)


def _run(layer, x, ids, gates, ws=None, stream=None):
    cfg = _cfg(layer)
    if ws is None:
        ws = torch.empty(max(1, B.moe_wide_workspace_size(cfg, x.shape[0])), dtype=torch.uint8,
                         device="cuda")
        ws.fill_(0xFF)  # NaN everywhere: what is not written is not read
    w = B.LayerRunner.weights_for(layer)
    w.router_w = None
    out = torch.full_like(x, float("nan"))
    B.moe_wide_step(cfg, x, ids, gates, w, out, ws, stream)
    return out


def _routing(t, e, mode, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    gates = torch.softmax(torch.randn(t, 8, generator=g, device="cuda"), 1)
    if mode == "one":      # every pick the same expert, the same index eight times a token
        ids = torch.full((t, 8), e - 1, device="cuda")
    elif mode == "none":
        ids = torch.full((t, 8), -1, device="cuda")
    else:
        ids = torch.randn(t, e, generator=g, device="cuda").topk(8, 1).indices
        if mode == "dropped":
            drop = torch.rand(t, 8, generator=g, device="cuda") < 0.5
            ids = torch.where(drop, torch.full_like(ids, e + 3), ids)
            ids[0] = -1
            gates = torch.where(ids < e, gates, torch.full_like(gates, float("nan")))
    return ids.to(torch.int32).contiguous(), gates.contiguous()


# rows per expert from none to hundreds: every tile size, ends inside a tile
@pytest.mark.parametrize("t,hidden,inter,experts,shared,mode", [
    (1, 256, 128, 16, True, "top"), (1, 128, 128, 16, False, "top"), (9, 384, 256, 32, True, "top"),
    (31, 640, 128, 16, False, "dropped"), (40, 256, 384, 16, True, "one"),
    (100, 256, 128, 16, True, "top"), (130, 512, 256, 16, False, "top"),
    (300, 256, 128, 16, True, "dropped"), (515, 384, 128, 16, True, "top"),
    (70, 256, 128, 16, False, "one"), (17, 256, 128, 32, True, "none"),
    (1100, 128, 128, 32, False, "top")])
def test_against_the_definition(t, hidden, inter, experts, shared, mode):
    _say("wide", t, hidden, inter, experts, shared, mode)
    layer = _layer(hidden, inter, experts, shared, seed=t + hidden)
    x = S.make_x(t, hidden, seed=t).cuda()
    ids, gates = _routing(t, experts, mode, t + 1)
    out = _run(layer, x, ids, gates)
    torch.cuda.synchronize()
    safe = torch.where((ids >= 0) & (ids < experts), gates, torch.zeros_like(gates))
    ref, tol = _reference(layer, x, ids, safe)
    bound = tol + 2.0 ** -8 * (ref.abs() + tol)
    err = (out.double() - ref).abs()
    assert bool((err <= bound).all()), (int((err > bound).sum()), float((err - bound).max()))
    # the bound is for the worst case of every rounding; in the mean the
    # outputs are as near as the decode step's tolerance asks of each
    assert float(err.norm()) <= P.OUT_TOL * float(ref.norm())
    assert torch.equal(_run(layer, x, ids, gates), out)  # the same bits again


def _check_definition(layer, x, ids, gates):
    out = _run(layer, x, ids, gates)
    torch.cuda.synchronize()
    ref, tol = _reference(layer, x, ids, gates)
    bound = tol + 2.0 ** -8 * (ref.abs() + tol)
    err = (out.double() - ref).abs()
    assert bool((err <= bound).all()), (int((err > bound).sum()), float((err - bound).max()))
    assert float(err.norm()) <= P.OUT_TOL * float(ref.norm())


# rows of an expert: every number of row tiles of 16, full, one short and one over
COUNTS = [1, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 79, 80, 81, 95, 96, 97, 111, 112, 113,
          126, 127, 128, 129, 144, 191, 192, 193, 255, 257]


@pytest.mark.parametrize("hidden,inter,shared", [(128, 128, False), (256, 256, True), (384, 640, False),
                                                 (640, 384, True)])
def test_every_number_of_rows_an_expert(hidden, inter, shared):
    _say("wide rows", hidden, inter, shared)
    experts = len(COUNTS)
    flat = torch.repeat_interleave(torch.arange(experts), torch.tensor(COUNTS))
    flat = torch.cat([flat, torch.full((-flat.numel() % 8,), -1)])
    flat = flat[torch.randperm(flat.numel(), generator=torch.Generator().manual_seed(hidden))]
    ids = flat.view(-1, 8).to(torch.int32).cuda()
    layer = _layer(hidden, inter, experts, shared, seed=inter)
    x = S.make_x(ids.shape[0], hidden, seed=inter + 1).cuda()
    gates = torch.softmax(torch.randn(ids.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(3)), 1)
    _check_definition(layer, x, ids, torch.where(ids >= 0, gates, torch.zeros_like(gates)))


@pytest.mark.parametrize("t,hidden,inter", [(20, 16384, 128), (20, 128, 16384), (160, 16384, 128),
                                            (160, 128, 16384)])
def test_the_longest_rows(t, hidden, inter):
    _say("wide long", t, hidden, inter)
    layer = _layer(hidden, inter, 16, True, seed=t)
    x = S.make_x(t, hidden, seed=t + 1).cuda()
    ids, gates = _routing(t, 16, "top", t + 2)
    _check_definition(layer, x, ids, gates)


@pytest.mark.parametrize("mode", ["top", "one"])
def test_a_token_does_not_touch_the_others(mode):
    """NaN and infinities of some tokens stay in their outputs."""
    t, experts = 90, 16
    layer = _layer(256, 256, experts, True, 31)
    x = S.make_x(t, 256, seed=32).cuda()
    ids, gates = _routing(t, experts, mode, 33)
    out = _run(layer, x, ids, gates)
    bad = x.clone()
    bad[::7] = float("nan")
    bad[1::7, 5] = float("inf")
    got = _run(layer, bad, ids, gates)
    torch.cuda.synchronize()
    clean = torch.ones(t, dtype=torch.bool, device="cuda")
    clean[::7] = clean[1::7] = False
    assert torch.equal(got[clean], out[clean])
    assert bool(torch.isnan(got[~clean]).all())


def test_no_picks_and_no_shared_expert():
    layer = _layer(256, 128, 16, False, 3)
    x = S.make_x(33, 256, seed=4).cuda()
    ids, gates = _routing(33, 16, "none", 5)
    out = _run(layer, x, ids, gates)
    torch.cuda.synchronize()
    assert bool((out == 0).all())
    empty = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    _run(layer, empty, ids[:0], gates[:0])


@pytest.mark.parametrize("rows", [1, 4, 8])
def test_the_decode_steps_rows(rows):
    """The decode step's own rows, picks and gates: within the decode step's
    output tolerance of the oracle, as the decode step is."""
    layer = _layer(512, 256, 32, True, 1234)
    x = S.make_x(rows, 512, seed=9 + rows, mode="corr")
    runner = B.LayerRunner(layer, rows)
    decode = runner.run(x.cuda())
    torch.cuda.synchronize()
    dbg = runner.debug(rows)
    _, ref = P.oracle_for(layer, x, dbg["logits"])
    ids = torch.from_numpy(dbg["ids"].copy()).cuda()
    gates = torch.from_numpy(dbg["gates"].copy()).cuda()
    out = _run(layer, x.cuda(), ids, gates)
    torch.cuda.synchronize()
    scale = np.abs(ref["out_f64"]).max()
    for o in (out, decode):
        err = np.abs(o.double().cpu().numpy() - ref["out_f64"]).max()
        assert err <= P.OUT_TOL * scale, float(err / scale)


def test_the_set_together():
    """The wide step, and the same step put together from the operators: sort,
    gather, a wide step of each expert's rows alone, combine; then adapters on
    its output beside a projection."""
    t, hidden, inter, experts = 150, 256, 128, 16
    layer = _layer(hidden, inter, experts, False, 77)
    x = S.make_x(t, hidden, seed=78).cuda()
    ids, gates = _routing(t, experts, "top", 79)
    out = _run(layer, x, ids, gates)
    offsets = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
    order = torch.empty(t * 8, dtype=torch.int32, device="cuda")
    pos = torch.empty(t, 8, dtype=torch.int32, device="cuda")
    B.moe_sort(ids, experts, offsets, order, pos)
    xs = torch.empty(t * 8, hidden, dtype=torch.bfloat16, device="cuda")
    B.moe_gather(x, pos, xs)
    y = torch.empty_like(xs)
    at = offsets.tolist()
    for e in range(experts):
        n = at[e + 1] - at[e]
        one = torch.full((n, 8), -1, dtype=torch.int32, device="cuda")
        one[:, 0] = e
        y[at[e]:at[e + 1]] = _run(layer, xs[at[e]:at[e + 1]].contiguous(), one,
                                  torch.ones(n, 8, device="cuda"))
    out2 = torch.empty_like(out)
    B.moe_combine(y, pos, gates, out2)
    torch.cuda.synchronize()
    ref, tol = _reference(layer, x, ids, gates)
    # each expert's output was rounded to bf16 once more
    size = torch.zeros_like(ref)
    for j in range(8):
        size += (gates[:, j, None].double() * y[pos[:, j].long()].double()).abs()
    for o, more in ((out, 0.0), (out2, 2.0 ** -8 * (size + tol))):
        bound = tol + more + 2.0 ** -8 * (ref.abs() + tol + more)
        assert bool(((o.double() - ref).abs() <= bound).all())
    # adapters beside the projection that follows
    n, mr = 128, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(80)
    a = (torch.randn(3, mr, hidden, generator=g, device="cuda") / 16).to(torch.bfloat16)
    b = torch.randn(3, n, mr, generator=g, device="cuda").to(torch.bfloat16)
    scale = torch.rand(3, generator=g, device="cuda")
    who = torch.randint(-1, 3, (t,), generator=g, device="cuda").to(torch.int32)
    w = (torch.randn(n, hidden, generator=g, device="cuda") / 16).to(torch.bfloat16)
    base = (out.double() @ w.double().t()).to(torch.bfloat16)
    lora = B.make_lora(a, b, scale)
    z = torch.empty_like(base)
    ws = torch.empty(B.lora_workspace_size(lora, t), dtype=torch.uint8, device="cuda")
    B.lora_apply(lora, out, who, base, z, ws)
    torch.cuda.synchronize()
    ref, tol = base.double(), torch.zeros(t, n, dtype=torch.float64, device="cuda")
    for i in range(3):
        r = who == i
        v, va = out[r].double() @ a[i].double().t(), out[r].double().abs() @ a[i].double().abs().t()
        ref[r] += scale[i].double() * v @ b[i].double().t()
        tol[r] += scale[i].double() * ((va * (hidden + 8) * 2.0 ** -23 + v.abs() * 2.0 ** -15) @ b[i].double().abs().t())
    assert bool(((z.double() - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol)).all())


def test_streams_graph_and_two_workspaces():
    """Two wide steps of other inputs on two streams at once, each with its own
    workspace, then both captured into one graph: every replay on new inputs
    gives the eager bits."""
    t, hidden, inter, experts = 90, 256, 128, 32
    layer = _layer(hidden, inter, experts, True, 91)
    inputs = [(S.make_x(t, hidden, seed=92 + i).cuda(), *_routing(t, experts, "top", 95 + i))
              for i in range(3)]
    want = []
    for i in inputs:
        want.append(_run(layer, *i))
        torch.cuda.synchronize()
    cfg, w = _cfg(layer), B.LayerRunner.weights_for(layer)
    n = B.moe_wide_workspace_size(cfg, t)
    spaces = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty(t, hidden, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            B.moe_wide_step(cfg, *inputs[i], w, outs[i], spaces[i], streams[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    cur = [[v.clone() for v in inputs[i]] for i in range(2)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(2):
            B.moe_wide_step(cfg, *cur[i], w, outs[i], spaces[i], torch.cuda.current_stream())
    for rep in range(3):
        for i in range(2):
            for d, v in zip(cur[i], inputs[(rep + i) % 3]):
                d.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[(rep + i) % 3]), (rep, i)
        _run(layer, *inputs[rep])
        torch.cuda.synchronize()
    del g
