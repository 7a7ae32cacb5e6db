"""How the experts' step of many rows (moe_wide_step) adds: in fp32 up to 16
picks an expert, and for the shared expert's gate and up in every batch; by the
FP8 MFMA for the rest of wider batches.

The measure is rms(out - bf16(definition)) / rms(definition).  Rounding the
definition as the kernel rounds its result takes that rounding out of it, and
what is left are values that lie on the other side of a border between two
codes: a relative error d of a sum moves the share 2 d / step of the quotients
across one, by `step` of their value each, an rms of sqrt(2 d step), step <=
2^-3 for E4M3 and <= 2^-7 for bf16.

Limit of fp32 sums: d = 2^-21, eight fp32 roundings of 2^-24 (the sums' own, the
scales, the row's rstd, SiLU): sqrt(2 * 2^-21 * 2^-3) = 3.5e-4 from mid and
sqrt(2 * 2^-21 * 2^-7) = 0.9e-4 from the output; 7e-4 allows each twice.
Limit of the FP8 MFMA: it drops 1.33e-5 of a sum (rms, measured on N(0, 1)
blocks), gate and up together 1.9e-5: sqrt(2 * 1.9e-5 * 2^-3) = 2.2e-3; 2.5e-3
with the output's sqrt(2 * 1.9e-5 * 2^-7) = 0.6e-3 in quadrature, and no factor.

The bounds of single elements are tests/test_gpu_wide.py's, with the fp32 sums'
own model in place of the FP8 MFMA's: 128 products in fp32 with truncation,
128 * 2^-23 of their size.
"""
import pytest
import torch

from tests import test_gpu_wide as W

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
FP32_LIMIT, FP8_LIMIT = 7e-4, 2.5e-3


def _power(e):
    """2^e exactly, from the bits of a double."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(v):
    """Nearest E4M3 value, ties to the even mantissa (float64)."""
    _, e = torch.frexp(v.abs())
    step = _power((e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _fp32_product(h, w, nkb):
    ref, terms = h @ w.t(), h.abs() @ w.abs().t()
    return ref, (128 * 2.0 ** -23 + (nkb + 7) * U32) * terms


@pytest.fixture
def exact_codes(monkeypatch):
    monkeypatch.setattr(W, "_e4m3", _e4m3)


def _case(t, hidden, inter, experts, shared, mode, seed):
    layer = W._layer(hidden, inter, experts, shared, seed)
    x = W.S.make_x(t, hidden, seed=seed + 1).cuda()
    ids, gates = W._routing(t, experts, "top" if mode == "skewed" else mode, seed + 2)
    if mode == "skewed":  # most tokens pick expert 0, whose rows pass a half tile
        ids[: (4 * t) // 5, 0] = 0
    return layer, x, ids, gates


def _apart(out, ref):
    return float((out.double() - ref.to(torch.bfloat16).double()).norm() / ref.norm())


@pytest.mark.parametrize("t,hidden,inter,experts,shared,mode", [
    (16, 2048, 1024, 32, True, "top"), (96, 2048, 1024, 64, True, "skewed"),
    (96, 1024, 512, 64, False, "skewed"), (32, 512, 256, 16, True, "dropped")])
def test_few_picks_an_expert(exact_codes, monkeypatch, t, hidden, inter, experts, shared, mode):
    print("wide sums", t, hidden, inter, experts, shared, mode, flush=True)
    assert t * 8 <= 16 * experts
    monkeypatch.setattr(W, "_product", _fp32_product)
    layer, x, ids, gates = _case(t, hidden, inter, experts, shared, mode, t + hidden)
    out = W._run(layer, x, ids, gates)
    torch.cuda.synchronize()
    safe = torch.where((ids >= 0) & (ids < experts), gates, torch.zeros_like(gates))
    ref, tol = W._reference(layer, x, ids, safe)
    bound = tol + 2.0 ** -8 * (ref.abs() + tol)
    err = (out.double() - ref).abs()
    assert bool((err <= bound).all()), (int((err > bound).sum()), float((err - bound).max()))
    apart = _apart(out, ref)
    print("apart", apart, flush=True)
    assert apart <= FP32_LIMIT


@pytest.mark.parametrize("t", [33, 80, 81, 130, 160, 161, 300])
def test_the_shared_expert_of_any_batch(exact_codes, t):
    """No pick is in a group: the outputs are the shared expert's, whose gate
    and up are summed in fp32 in batches of more than 16 picks an expert too.
    Its down is the FP8 MFMA's, 1.33e-5 off: sqrt(2 * 1.33e-5 * 2^-7) = 4.6e-4
    from the output's rounding instead of 0.9e-4, twice that in quadrature with
    twice 3.5e-4."""
    assert t * 8 > 16 * 16
    layer, x, ids, gates = _case(t, 2048, 1024, 16, True, "none", t)
    out = W._run(layer, x, ids, gates)
    torch.cuda.synchronize()
    ref, _ = W._reference(layer, x, ids, gates)
    apart = _apart(out, ref)
    print("apart", apart, flush=True)
    assert apart <= 1.16e-3


@pytest.mark.parametrize("t,shared", [(200, False), (300, True)])
def test_many_picks_an_expert(exact_codes, t, shared):
    layer, x, ids, gates = _case(t, 1024, 512, 16, shared, "top", t)
    out = W._run(layer, x, ids, gates)
    torch.cuda.synchronize()
    ref, _ = W._reference(layer, x, ids, gates)
    apart = _apart(out, ref)
    print("apart", apart, flush=True)
    assert apart <= FP8_LIMIT


@pytest.mark.parametrize("t,more,experts", [(20, 37, 32), (150, 333, 16), (31, 97, 64)])
def test_a_tokens_bits_in_two_batches(t, more, experts):
    """Batches on the same side of 16 picks an expert: the first tokens' results
    are the same bits alone and among others, at other places in the sorted
    order and in tiles of other sizes."""
    layer, x, ids, gates = _case(t + more, 512, 384, experts, True, "top", 7 * t)
    both = W._run(layer, x, ids, gates)
    alone = W._run(layer, x[:t].contiguous(), ids[:t].contiguous(), gates[:t].contiguous())
    at = torch.randperm(t + more, generator=torch.Generator().manual_seed(t)).cuda()
    moved = W._run(layer, x[at].contiguous(), ids[at].contiguous(), gates[at].contiguous())
    torch.cuda.synchronize()
    as_bits = lambda v: v.view(torch.int16)  # noqa: E731
    assert torch.equal(as_bits(both[:t]), as_bits(alone))
    assert torch.equal(as_bits(both[at]), as_bits(moved))


@pytest.mark.parametrize("hidden,inter,shared", [(128, 128, False), (256, 128, True), (384, 256, True),
                                                 (640, 384, False)])
def test_every_number_of_rows_an_expert_in_fp32(exact_codes, monkeypatch, hidden, inter, shared):
    """Experts of 0 to 257 rows, every number of row tiles of 16 of a tile of 80,
    full, one short and one over, in a batch of few picks an expert."""
    print("wide fp32 rows", hidden, inter, shared, flush=True)
    monkeypatch.setattr(W, "_product", _fp32_product)
    counts = W.COUNTS + [159, 160, 161]
    experts = -(-sum(counts) // 256) * 16
    flat = torch.repeat_interleave(torch.arange(len(counts)) * 5 % experts, torch.tensor(counts))
    flat = torch.cat([flat, torch.full((-flat.numel() % 8,), -1)])
    flat = flat[torch.randperm(flat.numel(), generator=torch.Generator().manual_seed(hidden))]
    ids = flat.view(-1, 8).to(torch.int32).cuda()
    assert ids.numel() <= 16 * experts
    assert torch.bincount(flat[flat >= 0]).max() == max(counts)
    layer = W._layer(hidden, inter, experts, shared, inter)
    x = W.S.make_x(ids.shape[0], hidden, seed=inter + 1).cuda()
    gates = torch.softmax(torch.randn(ids.shape, device="cuda",
                                      generator=torch.Generator("cuda").manual_seed(3)), 1)
    gates = torch.where(ids >= 0, gates, torch.zeros_like(gates))
    out = W._run(layer, x, ids, gates)
    torch.cuda.synchronize()
    ref, tol = W._reference(layer, x, ids, gates)
    bound = tol + 2.0 ** -8 * (ref.abs() + tol)
    err = (out.double() - ref).abs()
    assert bool((err <= bound).all()), (int((err > bound).sum()), float((err - bound).max()))
    apart = _apart(out, ref)
    print("apart", apart, flush=True)
    assert apart <= FP32_LIMIT


@pytest.mark.parametrize("t,experts", [(40, 32), (70, 16)])
def test_tokens_of_tiny_values(t, experts):
    """Values whose products lie where a block's scale, a 448th of its largest
    mid, is a rounded subnormal: finite outputs, of the products' size.  With x up
    to 2^(e + 2), weights up to 2^3 and rstd 2^10 (1 / sqrt(eps)), sums of 256
    N(0, 1) products give gate and up below 2^(e + 21), mid below 2^(2 e + 41),
    sums of 128 of them and of 9 experts below 2^(2 e + 52)."""
    layer = W._layer(256, 128, experts, True, t)
    x0 = W.S.make_x(t, 256, seed=t + 1).cuda().float()
    ids, gates = W._routing(t, experts, "top", t + 2)
    for e in range(-92, -78):
        out = W._run(layer, (x0 * 2.0 ** e).to(torch.bfloat16), ids, gates)
        torch.cuda.synchronize()
        assert bool(torch.isfinite(out).all()), e
        assert float(out.float().abs().max()) <= 2.0 ** (2 * e + 52), e


def test_two_batches_in_a_graph():
    """A batch of few picks an expert and one of many, each with its workspace,
    captured into one graph: every replay on other inputs gives the eager bits."""
    few, many = W._layer(256, 384, 32, True, 5), W._layer(384, 256, 16, True, 6)
    sizes = ((few, 60), (many, 200))
    sets = [[(W.S.make_x(t, l.hidden, seed=9 * s + i).cuda(), *W._routing(t, l.n_experts, "top", 20 * s + i))
             for i, (l, t) in enumerate(sizes)] for s in range(3)]
    want = [[W._run(l, *x) for (l, _), x in zip(sizes, one)] for one in sets]
    torch.cuda.synchronize()
    cur = [[v.clone() for v in x] for x in sets[0]]
    outs = [torch.empty_like(x[0]) for x in cur]
    cfgs = [W._cfg(l) for l, _ in sizes]
    weights = [W.B.LayerRunner.weights_for(l) for l, _ in sizes]
    spaces = [torch.empty(W.B.moe_wide_workspace_size(c, t), dtype=torch.uint8, device="cuda")
              for c, (_, t) in zip(cfgs, sizes)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(2):
            W.B.moe_wide_step(cfgs[i], *cur[i], weights[i], outs[i], spaces[i], torch.cuda.current_stream())
    for rep in range(6):
        for c, x in zip(cur, sets[rep % 3]):
            for d, v in zip(c, x):
                d.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[rep % 3][i]), (rep, i)
        W._run(few, *sets[rep % 3][0])
        torch.cuda.synchronize()
    del g
