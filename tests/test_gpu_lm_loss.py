"""The LM head's loss and its gradients (lm_head_loss, lm_head_loss_backward)
against the definition in float64, through the C ABI.

Logits: products of two bf16 are exact in fp32 and an addition is off by 2^-23 of
a partial sum at most: |err z| <= hidden 2^-23 sum|terms| =: e.  exp(z - big) is
off by e, the rounding of the difference and of its exponent (2^-22 (1 + |z -
big|) of it together), and below 2^-126 may be 0; so the sum of vocab of them,
added in fp32, and with it lse, is off by e + 2^-22 (1 + spread) + vocab 2^-23 at
most, plus 2^-22 of lse.  The additions' term is for one chain; they run in
chains of at most 64 and then over the tiles: (64 + vocab / 64) 2^-23.

d is (p - hit) dloss, p off by (e + 2^-22 (2 + |z - lse|)) of it, rounded to bf16
once: 2^-8 of it (or below 2^-126 maybe 0); at the target it is the sum of two
bf16, 2^-16.  dh and dw add d times w (h) in fp32.
"""
import math

import pytest
import torch

from bit_moe_decode_amd import binding as B

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -23
BF16 = 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


def _say(*a):
    print(*a, flush=True)


def _inputs(rows, vocab, hidden, seed, size=2.0, none=0.2):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.randn(rows, hidden, generator=g, device="cuda").to(BF)
    w = (torch.randn(vocab, hidden, generator=g, device="cuda") * size * hidden ** -0.5).to(BF)
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    t = torch.where(torch.rand(rows, generator=g, device="cuda") < none, torch.full_like(t, -100), t)
    dloss = torch.rand(rows, generator=g, device="cuda") - 0.25
    return h, w, t.to(torch.int32), dloss


def _loss(h, w, t, stream=None):
    rows = h.shape[0]
    loss, lse = torch.full((rows,), -7.0, device="cuda"), torch.full((rows,), -7.0, device="cuda")
    ws = torch.empty(max(1, B.lm_head_loss_workspace_size(rows, *w.shape)), dtype=torch.uint8, device="cuda")
    B.lm_head_loss(h, w, t, loss, lse, ws, stream)
    return loss, lse


def _grads(h, w, t, lse, dloss, dtype=F32, add=None, which="both"):
    dh = torch.full(h.shape, -7.0, dtype=BF, device="cuda") if which != "dw" else None
    dw = (torch.full(w.shape, float("nan"), dtype=dtype, device="cuda") if add is None else add.clone()) \
        if which != "dh" else None
    ws = torch.empty(max(1, B.lm_head_loss_backward_workspace_size(h.shape[0], *w.shape)), dtype=torch.uint8,
                     device="cuda")
    B.lm_head_loss_backward(h, w, t, lse, dloss, dh, dw, ws, add is not None)
    return dh, dw


def _logits(h, w):
    hd, wd = h.double(), w.double()
    return hd @ wd.t(), h.shape[1] * U32 * (hd.abs() @ wd.abs().t())


def _check_loss(loss, lse, h, w, t):
    z, e = _logits(h, w)
    ref = torch.logsumexp(z, 1)
    worst = e.amax(1)
    vocab = w.shape[0]
    tol = worst + U32 * (2 + 2 * (z.amax(1) - z.amin(1)) + 64 + vocab / 64) + 2 * U32 * ref.abs()
    assert bool(((lse.double() - ref).abs() <= tol).all()), float(((lse.double() - ref).abs() - tol).max())
    live = (t >= 0) & (t < vocab)
    at = z.gather(1, t.long().clamp(0, vocab - 1)[:, None])[:, 0]
    want = torch.where(live, ref - at, torch.zeros_like(ref))
    err = (loss.double() - want).abs()
    assert bool((err <= torch.where(live, 2 * tol + 2 * U32 * at.abs(), torch.zeros_like(tol))).all()), float(err.max())


def _check_grads(dh, dw, h, w, t, lse, dloss, add=None):
    z, e = _logits(h, w)
    vocab = w.shape[0]
    live = ((t >= 0) & (t < vocab))[:, None]
    x = z - lse.double()[:, None]
    p = torch.exp(x)
    hit = torch.arange(vocab, device="cuda")[None] == t[:, None]
    dl = dloss.double()[:, None]
    zero = torch.zeros_like(p)
    d = torch.where(live, (p - hit.double()) * dl, zero)
    off = torch.where(live, p * (e + 2 * U32 * (2 + x.abs())) * dl.abs() + 2 * U32 * d.abs() + 2.0 ** -125, zero)
    off = off + torch.where(hit, 2.0 ** -16, BF16) * (d.abs() + off)
    hd, wd = torch.where(live, h.double(), torch.zeros((), device="cuda", dtype=torch.float64)), w.double()
    for got, ref, terms, part, c in (
            (dh, d @ wd, d.abs() @ wd.abs(), off @ wd.abs(), vocab + 40),
            (dw, d.t() @ hd, d.abs().t() @ hd.abs(), off.t() @ hd.abs(), h.shape[0] + 1)):
        if got is None:
            continue
        if got is dw and add is not None:
            ref, terms = ref + add.double(), terms + add.double().abs()
        tol = part + c * U32 * (terms + part)
        if got.dtype is BF:
            tol = tol + BF16 * (ref.abs() + tol)
        err = (got.double() - ref).abs()
        assert bool(torch.isfinite(got).all())
        assert bool((err <= tol).all()), (got is dw, float((err - tol).max()), float(err.max()))


SHAPES = [(1, 1, 8), (1, 1000, 64), (3, 7, 16), (5, 130, 40), (8, 4099, 256), (33, 256, 72), (64, 513, 128),
          (65, 511, 136), (130, 1003, 264), (257, 2050, 96), (600, 5003, 200)]


@pytest.mark.parametrize("rows,vocab,hidden", SHAPES)
def test_loss(rows, vocab, hidden):
    _say("loss", rows, vocab, hidden)
    h, w, t, _ = _inputs(rows, vocab, hidden, rows + vocab)
    loss, lse = _loss(h, w, t)
    torch.cuda.synchronize()
    _check_loss(loss, lse, h, w, t)


@pytest.mark.parametrize("dtype,add", [(F32, False), (F32, True), (BF, False), (BF, True)])
@pytest.mark.parametrize("rows,vocab,hidden", SHAPES)
def test_gradients(rows, vocab, hidden, dtype, add):
    _say("loss gradients", rows, vocab, hidden, dtype, add)
    h, w, t, dloss = _inputs(rows, vocab, hidden, rows + vocab)
    base = torch.randn(vocab, hidden, device="cuda").to(dtype) if add else None
    lse = torch.logsumexp(_logits(h, w)[0], 1).float()
    dh, dw = _grads(h, w, t, lse, dloss, dtype, base)
    torch.cuda.synchronize()
    _check_grads(dh, dw, h, w, t, lse, dloss, base)


def test_several_pieces_of_the_vocabulary():
    """Rows enough that the vocabulary is taken in pieces: 40000 rows of 3 pieces."""
    rows, vocab, hidden = 40000, 4500, 16
    _say("pieces", rows, vocab, hidden)
    h, w, t, dloss = _inputs(rows, vocab, hidden, 3)
    loss, lse = _loss(h, w, t)
    dh, dw = _grads(h, w, t, lse, dloss)
    torch.cuda.synchronize()
    _check_loss(loss, lse, h, w, t)
    _check_grads(dh, dw, h, w, t, lse, dloss)


def test_every_row_has_a_target_and_none_has():
    h, w, t, dloss = _inputs(70, 300, 64, 5)
    for targets in (torch.full_like(t, 299), torch.zeros_like(t), torch.full_like(t, -1), torch.full_like(t, 300),
                    torch.full_like(t, 2 ** 31 - 1), torch.full_like(t, -2 ** 31)):
        _say("targets", int(targets[0]))
        loss, lse = _loss(h, w, targets)
        dh, dw = _grads(h, w, targets, lse, dloss)
        torch.cuda.synchronize()
        _check_loss(loss, lse, h, w, targets)
        _check_grads(dh, dw, h, w, targets, lse, dloss)
        if not 0 <= int(targets[0]) < 300:
            assert bool((loss == 0).all()) and bool((dh == 0).all()) and bool((dw == 0).all())


@pytest.mark.parametrize("size", [30.0, 200.0])
def test_large_logits(size):
    """Probabilities of 0 and 1: exponentials that would overflow without the
    largest, and ones that vanish."""
    h, w, t, dloss = _inputs(90, 700, 64, 6, size)
    t[:40] = _logits(h, w)[0].argmax(1)[:40].to(torch.int32)
    loss, lse = _loss(h, w, t)
    dh, dw = _grads(h, w, t, lse, dloss)
    torch.cuda.synchronize()
    assert float(lse.max()) > 2 * size
    _check_loss(loss, lse, h, w, t)
    _check_grads(dh, dw, h, w, t, lse, dloss)


@pytest.mark.parametrize("rows", [20, 100])
def test_infinite_logits(rows):
    """Weights of infinity: a row with a logit of +inf has an lse of +inf, one
    whose other logits are -inf keeps the rest, one of -inf alone has -inf."""
    _say("infinite logits", rows)
    h = torch.zeros(rows, 8, dtype=BF, device="cuda")
    w = torch.zeros(300, 8, dtype=BF, device="cuda")
    h[:, 0] = 1.0
    t = torch.zeros(rows, dtype=torch.int32, device="cuda")
    big = 3e38  # bf16's largest is 3.39e38: its square is infinite
    h[1, 1], h[2, 1] = big, -big
    h[3, :2] = torch.tensor([-big, 0.0])
    w[5:9, 1] = big
    w[:, 0] = 0.0
    loss, lse = _loss(h, w, t)
    w2 = torch.zeros_like(w)
    w2[:, 0] = big
    _, lse2 = _loss(h, w2, t)
    torch.cuda.synchronize()
    assert float(lse[1]) == math.inf and float(loss[1]) == math.inf
    assert abs(float(lse[2]) - math.log(296)) < 1e-5
    assert abs(float(lse[0]) - math.log(300)) < 1e-5
    assert float(lse2[3]) == -math.inf


def test_rows_without_a_target_take_no_part():
    """Whatever h, lse and dloss they hold: the same bits in all else."""
    h, w, t, dloss = _inputs(150, 700, 72, 8)
    loss, lse = _loss(h, w, t)
    dh, dw = _grads(h, w, t, lse, dloss)
    none = t < 0
    h2, lse2, dl2 = h.clone(), lse.clone(), dloss.clone()
    h2[none], lse2[none], dl2[none] = float("nan"), float("nan"), float("inf")
    loss2, _ = _loss(h2, w, t)
    dh2, dw2 = _grads(h2, w, t, lse2, dl2)
    torch.cuda.synchronize()
    assert bool(none.any()) and torch.equal(dh, dh2) and torch.equal(dw, dw2) and torch.equal(loss, loss2)
    assert bool((dh[none] == 0).all())


def test_nan_stays_in_its_row():
    h, w, t, dloss = _inputs(100, 400, 64, 9, none=0.0)
    loss, lse = _loss(h, w, t)
    h2 = h.clone()
    h2[37] = float("nan")
    loss2, lse2 = _loss(h2, w, t)
    torch.cuda.synchronize()
    keep = [i for i in range(100) if i != 37]
    assert torch.equal(loss[keep], loss2[keep]) and torch.equal(lse[keep], lse2[keep])
    assert math.isnan(float(loss2[37])) and math.isnan(float(lse2[37]))
    dh, _ = _grads(h2, w, t, lse2, dloss)
    dh1, _ = _grads(h, w, t, lse, dloss)
    assert torch.equal(dh[keep], dh1[keep]) and bool(torch.isnan(dh[37]).all())


def test_one_gradient_alone_and_the_same_bits_again():
    h, w, t, dloss = _inputs(300, 1500, 136, 10)
    _, lse = _loss(h, w, t)
    dh, dw = _grads(h, w, t, lse, dloss)
    only_dh, _ = _grads(h, w, t, lse, dloss, which="dh")
    _, only_dw = _grads(h, w, t, lse, dloss, which="dw")
    torch.cuda.synchronize()
    assert torch.equal(dh, only_dh) and torch.equal(dw, only_dw)


def test_no_rows():
    w = torch.randn(50, 16, device="cuda").to(BF)
    h, e = torch.empty(0, 16, dtype=BF, device="cuda"), torch.empty(0, device="cuda")
    t = torch.empty(0, dtype=torch.int32, device="cuda")
    B.lm_head_loss(h, w, t, e, e, None)
    for dtype in (BF, F32):
        dw = torch.full((50, 16), float("nan"), dtype=dtype, device="cuda")
        B.lm_head_loss_backward(h, w, t, e, e, h, dw)
        kept = torch.ones(50, 16, dtype=dtype, device="cuda")
        B.lm_head_loss_backward(h, w, t, e, e, h, kept, add=True)
        torch.cuda.synchronize()
        assert bool((dw == 0).all()) and bool((kept == 1).all())


def test_gradients_are_the_differences():
    """sum(dloss loss(h, w)) moves by dh and dw: differences in float64 of the
    definition against the library's gradients (bf16 2^-8, d's and dh's own)."""
    h, w, t, dloss = _inputs(4, 30, 8, 11, none=0.0)
    _, lse = _loss(h, w, t)
    dh, dw = _grads(h, w, t, lse, dloss)

    def value(hd, wd):
        z = hd @ wd.t()
        return float((dloss.double() * (torch.logsumexp(z, 1) - z.gather(1, t.long()[:, None])[:, 0])).sum())

    step = 2.0 ** -12
    for which, got in (("h", dh), ("w", dw)):
        for i, j in ((0, 0), (3, 7), (2, 5)):
            p, m = (h.double(), h.double()) if which == "h" else (w.double(), w.double())
            p = p.clone()
            p[i, j] += step
            m = m.clone()
            m[i, j] -= step
            d = (value(p, w.double()) - value(m, w.double())) if which == "h" else \
                (value(h.double(), p) - value(h.double(), m))
            terms = float((dloss.abs().double()[:, None] * 2).sum()) * 2
            assert abs(d / (2 * step) - float(got[i, j])) <= 2 * BF16 * terms


def test_on_another_stream_and_in_a_graph():
    h, w, t, dloss = _inputs(90, 700, 136, 12)
    loss, lse = torch.zeros(90, device="cuda"), torch.zeros(90, device="cuda")
    dh, dw = torch.zeros_like(h), torch.zeros(w.shape, device="cuda")
    ws = torch.empty(max(B.lm_head_loss_workspace_size(90, 700, 136),
                         B.lm_head_loss_backward_workspace_size(90, 700, 136)), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.lm_head_loss(h, w, t, loss, lse, ws, stream=side)
    side.synchronize()
    _check_loss(loss, lse, h, w, t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = torch.cuda.current_stream()
        B.lm_head_loss(h, w, t, loss, lse, ws, stream=s)
        B.lm_head_loss_backward(h, w, t, lse, dloss, dh, dw, ws, stream=s)
    for i in range(3):
        h2, _, t2, _ = _inputs(90, 700, 136, 20 + i)
        h.copy_(h2)
        t.copy_(t2)
        graph.replay()
        torch.cuda.synchronize()
        rl, re = _loss(h, w, t)
        rh, rw = _grads(h, w, t, re, dloss)
        torch.cuda.synchronize()
        assert torch.equal(loss, rl) and torch.equal(lse, re) and torch.equal(dh, rh) and torch.equal(dw, rw)


@pytest.mark.parametrize("rows", [16384 + 40, 16384 + 300])
def test_several_launches_of_rows(rows):
    """More rows than a launch takes; the last launch's in small tiles."""
    vocab, hidden = 4000, 8
    _say("launches", rows)
    h, w, t, _ = _inputs(rows, vocab, hidden, rows)
    loss, lse = _loss(h, w, t)
    torch.cuda.synchronize()
    for i in (0, 16384):
        part = slice(i, min(rows, i + 3000))
        _check_loss(loss[part], lse[part], h[part], w, t[part])


@pytest.mark.parametrize("rows,vocab,hidden", [(5000, 300, 24), (70, 9000, 16), (400, 70000, 264), (4200, 1003, 520)])
def test_shapes_between_the_tiles(rows, vocab, hidden):
    """Tiles of either size, rows placed by counting and by a sort, dh split."""
    _say("between", rows, vocab, hidden)
    h, w, t, dloss = _inputs(rows, vocab, hidden, rows + vocab)
    loss, lse = _loss(h, w, t)
    dh, dw = _grads(h, w, t, lse, dloss)
    torch.cuda.synchronize()
    _check_loss(loss, lse, h, w, t)
    _check_grads(dh, dw, h, w, t, lse, dloss)
