"""Tokens sorted by expert and back (moe_sort, moe_gather, moe_combine and
the gradients) against plain numpy / float64 forms, through the C ABI.

Sort, gather and dy of fp32 rows are compared bitwise.  Sums: the kernels add
the k terms of an element in fp32 in pick order (k products, k + 1 additions),
so |err| <= (k + 3) * 2^-24 * sum|terms|, and a result rounded to bf16 is off
by half a step more, 2^-8 of its value.  dgates adds H products in fp32:
(H + 8) * 2^-24 * sum|terms|.
"""
import numpy as np
import pytest
import torch

from bit_moe_decode_amd import binding as B

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
BF16 = 2.0 ** -8
I32 = torch.int32


def _say(*a):
    print(*a, flush=True)


def _ids(t, k, e, mode, seed):
    g = np.random.default_rng(seed)
    if mode == "same":
        return np.full((t, k), e - 1, np.int32)
    if mode == "none":
        return np.full((t, k), -1, np.int32)
    ids = g.integers(0, e, (t, k)).astype(np.int32)
    if mode == "outside":
        ids = np.where(g.random((t, k)) < 0.4,
                       g.choice(np.array([-1, -2 ** 31, e, 2 ** 31 - 1, e + 77], np.int64), (t, k)),
                       ids).astype(np.int32)
    return ids


def _sort_ref(ids, e):
    flat = ids.reshape(-1)
    kept = np.nonzero((flat >= 0) & (flat < e))[0]
    by = kept[np.argsort(flat[kept], kind="stable")]
    pos = np.full(flat.size, -1, np.int32)
    pos[by] = np.arange(by.size)
    offsets = np.searchsorted(np.sort(flat[kept]), np.arange(e + 1)).astype(np.int32)
    return offsets, by.astype(np.int32), pos.reshape(ids.shape)


def _sort(ids, e, stream=None, ws=None):
    t, k = ids.shape
    offsets = torch.full((e + 1,), -7, dtype=I32, device="cuda")
    order = torch.full((t * k,), -7, dtype=I32, device="cuda")
    pos = torch.full((t, k), -7, dtype=I32, device="cuda")
    n = B.moe_sort_workspace_size(t, k, e)
    if ws is None and n:
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    B.moe_sort(ids, e, offsets, order, pos, ws, stream)
    return offsets, order, pos


@pytest.mark.parametrize("t,k,e", [(1, 1, 1), (1, 8, 256), (3, 6, 16), (16, 8, 256), (61, 16, 1000),
                                   (512, 8, 256), (1024, 8, 256), (1025, 8, 256), (8193, 1, 1024), (5000, 7, 33),
                                   (40001, 8, 256)])
@pytest.mark.parametrize("mode", ["random", "outside", "same", "none"])
def test_sort(t, k, e, mode):
    _say("sort", t, k, e, mode)
    ids = _ids(t, k, e, mode, seed=t + k + e)
    offsets, order, pos = _sort(torch.from_numpy(ids).cuda(), e)
    torch.cuda.synchronize()
    ro, rb, rp = _sort_ref(ids, e)
    assert np.array_equal(offsets.cpu().numpy(), ro)
    assert np.array_equal(pos.cpu().numpy(), rp)
    order = order.cpu().numpy()
    assert np.array_equal(order[:rb.size], rb)
    assert (order[rb.size:] == -7).all()  # rows behind the last group: left as they were


def test_sort_of_no_tokens():
    offsets, _, _ = _sort(torch.empty(0, 8, dtype=I32, device="cuda"), 64)
    torch.cuda.synchronize()
    assert bool((offsets == 0).all())


def _rows(n, h, dtype, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(n, h, generator=g).to(dtype)


def _case(t, k, e, h, dtype, seed, share=1):
    """(ids' pos on the device and host, sorted rows, gates); with share > 1
    only the experts below e // share are in a group, and the sorted buffers
    hold just their picks."""
    ids = _ids(t, k, e, "random", seed)
    _, by, pos = _sort_ref(ids, max(1, e // share))
    rows = max(by.size, 1) if share > 1 else t * k
    gates = torch.rand(t, k, generator=torch.Generator().manual_seed(seed + 1))
    gates[torch.from_numpy(pos) < 0] = float("nan")  # not read
    return torch.from_numpy(pos), rows, gates


SHAPES = [(1, 1, 4, 1, 1), (1, 8, 256, 6144, 1), (5, 8, 16, 7, 1), (33, 6, 64, 1001, 4),
          (7, 16, 40, 2050, 1), (130, 8, 256, 640, 4), (3, 3, 8, 8200, 2)]
DTYPES = [torch.bfloat16, torch.float32]


def _nan_rows(rows, h, dtype):
    return torch.full((rows, h), float("nan"), dtype=dtype, device="cuda")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,k,e,h,share", SHAPES)
def test_gather(t, k, e, h, share, dtype):
    _say("gather", t, k, e, h, share, dtype)
    pos, rows, _ = _case(t, k, e, h, dtype, 11, share)
    x = _rows(t, h, dtype, 12)
    x[0, 0] = float("inf")
    xs = torch.full((rows, h), 3.0, dtype=dtype, device="cuda")
    B.moe_gather(x.cuda(), pos.cuda(), xs)
    torch.cuda.synchronize()
    ref = torch.full((rows, h), 3.0, dtype=dtype)
    for a in range(t):
        for j in range(k):
            if pos[a, j] >= 0:
                ref[pos[a, j]] = x[a]
    assert torch.equal(xs.cpu(), ref)


def _terms(y, pos, w):
    """[T, H, k] float64 terms w y[pos], 0 for picks without a row."""
    at = pos.clamp(min=0).long()
    f = y.double()[at.reshape(-1)].view(*pos.shape, -1)
    keep = (pos >= 0)[..., None]
    f = torch.where(keep, f, torch.zeros_like(f))
    w = torch.where(pos >= 0, w.double(), torch.zeros(()).double())
    return (f * w[..., None]).permute(0, 2, 1)


def _assert_sum(out, terms, k):
    ref = terms.sum(-1)
    err = (out.double().cpu() - ref).abs()
    bound = (k + 3) * U32 * terms.abs().sum(-1)
    if out.dtype == torch.bfloat16:
        bound = bound + BF16 * (ref.abs() + bound)
    assert bool((err <= bound).all()), float((err - bound).max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,k,e,h,share", SHAPES)
def test_combine(t, k, e, h, share, dtype):
    _say("combine", t, k, e, h, share, dtype)
    pos, rows, gates = _case(t, k, e, h, dtype, 21, share)
    y = _rows(rows, h, dtype, 22)
    used = torch.zeros(rows, dtype=torch.bool)
    used[pos[pos >= 0].long()] = True
    y[~used] = float("nan")  # rows of no pick are not read
    add = _rows(t, h, dtype, 23)
    for extra in (None, add):
        out = _nan_rows(t, h, dtype)
        B.moe_combine(y.cuda(), pos.cuda(), gates.cuda(), out, None if extra is None else extra.cuda())
        torch.cuda.synchronize()
        terms = _terms(torch.where(used[:, None], y, torch.zeros_like(y)), pos, gates)
        if extra is not None:
            terms = torch.cat([terms, extra.double()[..., None]], -1)
        _assert_sum(out, terms, k)
    # out may be add itself
    out2 = add.cuda()
    B.moe_combine(y.cuda(), pos.cuda(), gates.cuda(), out2, out2)
    torch.cuda.synchronize()
    assert torch.equal(out2, out)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,k,e,h,share", SHAPES)
def test_gather_backward(t, k, e, h, share, dtype):
    _say("gather backward", t, k, e, h, share, dtype)
    pos, rows, _ = _case(t, k, e, h, dtype, 31, share)
    dxs = _rows(rows, h, dtype, 32)
    dx = _nan_rows(t, h, dtype)
    B.moe_gather_backward(dxs.cuda(), pos.cuda(), dx)
    torch.cuda.synchronize()
    _assert_sum(dx, _terms(dxs, pos, torch.ones(t, k)), k)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,k,e,h,share", SHAPES)
def test_combine_backward(t, k, e, h, share, dtype):
    _say("combine backward", t, k, e, h, share, dtype)
    pos, rows, gates = _case(t, k, e, h, dtype, 41, share)
    y, dout = _rows(rows, h, dtype, 42), _rows(t, h, dtype, 43)
    used = torch.zeros(rows, dtype=torch.bool)
    used[pos[pos >= 0].long()] = True
    y[~used] = float("inf")
    dy = torch.full((rows, h), 3.0, dtype=dtype, device="cuda")
    dg = torch.full((t, k), float("nan"), device="cuda")
    B.moe_combine_backward(dout.cuda(), y.cuda(), pos.cuda(), gates.cuda(), dy, dg)
    torch.cuda.synchronize()
    dy, dg = dy.cpu(), dg.cpu()
    assert bool((dy[~used] == 3.0).all())
    for a in range(t):
        for j in range(k):
            p = int(pos[a, j])
            if p < 0:
                assert float(dg[a, j]) == 0.0
                continue
            # one fp32 product, rounded once more for bf16: the same bits
            assert torch.equal(dy[p], (gates[a, j] * dout[a].float()).to(dtype))
            terms = dout[a].double() * y[p].double()
            assert abs(float(dg[a, j]) - float(terms.sum())) <= (h + 8) * U32 * float(terms.abs().sum())


def test_gradients_against_differences():
    """combine is linear in y and in the gates: its difference over a whole
    step is the gradient's product with that step.  The two sides differ by
    their roundings, (k + 3) and (H + 8) of 2^-24 of the terms."""
    t, k, e, h = 9, 4, 8, 96
    pos, rows, gates = _case(t, k, e, h, torch.float32, 51)
    y, dy_step = _rows(rows, h, torch.float32, 52), _rows(rows, h, torch.float32, 53)
    gate_step = torch.randn(t, k, generator=torch.Generator().manual_seed(54))
    dout = _rows(t, h, torch.float32, 55)

    def loss(yy, gg):
        out = torch.empty(t, h, device="cuda")
        B.moe_combine(yy.cuda(), pos.cuda(), gg.cuda(), out)
        return float((out.double().cpu() * dout.double()).sum())

    dy = torch.zeros(rows, h, device="cuda")
    dg = torch.empty(t, k, device="cuda")
    B.moe_combine_backward(dout.cuda(), y.cuda(), pos.cuda(), gates.cuda(), dy, dg)
    dx = torch.empty(t, h, device="cuda")
    B.moe_gather_backward(y.cuda(), pos.cuda(), dx)
    torch.cuda.synchronize()

    def size(yy, gg):  # sum of the loss' terms
        return float((_terms(yy.abs(), pos, gg.abs()) * dout.double().abs()[..., None]).sum())

    eps = (k + h + 16) * U32
    tol = eps * (size(y + dy_step, gates) + size(y, gates) + size(dy_step, gates))
    d = loss(y + dy_step, gates) - loss(y, gates)
    assert abs(d - float((dy.double().cpu() * dy_step.double()).sum())) <= tol + 2 * U32 * size(y + dy_step, gates)
    tol = eps * (size(y, gates + gate_step) + size(y, gates) + size(y, gate_step))
    d = loss(y, gates + gate_step) - loss(y, gates)
    assert abs(d - float((dg.double().cpu() * gate_step.double()).sum())) <= tol + 2 * U32 * size(y, gates + gate_step)
    # gather: <gather(x), s> = <x, gather_backward(s)>
    x = _rows(t, h, torch.float32, 56)
    xs = torch.zeros(rows, h, device="cuda")
    B.moe_gather(x.cuda(), pos.cuda(), xs)
    a = float((xs.double().cpu() * y.double()).sum())
    b = float((x.double() * dx.double().cpu()).sum())
    assert abs(a - b) <= eps * float((xs.double().cpu().abs() * y.double().abs()).sum())


def test_every_pick_dropped():
    t, k, h = 6, 8, 72
    pos = torch.full((t, k), -1, dtype=I32, device="cuda")
    bad = torch.full((t * k, h), float("nan"), device="cuda")
    gates = torch.full((t, k), float("inf"), device="cuda")
    out = _nan_rows(t, h, torch.float32)
    B.moe_combine(bad, pos, gates, out)
    dx = _nan_rows(t, h, torch.float32)
    B.moe_gather_backward(bad, pos, dx)
    dg = torch.full((t, k), float("nan"), device="cuda")
    dy = torch.full((t * k, h), 2.0, device="cuda")
    B.moe_combine_backward(torch.ones(t, h, device="cuda"), bad, pos, gates, dy, dg)
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool((dx == 0).all()) and bool((dg == 0).all())
    assert bool((dy == 2.0).all())


def test_a_position_behind_the_buffer_is_a_pick_without_a_row():
    t, k, h = 4, 2, 64
    pos = torch.tensor([[0, 5], [2 ** 31 - 1, 1], [-3, 2], [3, 4]], dtype=I32, device="cuda")
    x = _rows(t, h, torch.float32, 61).cuda()
    xs = torch.zeros(4, h, device="cuda")
    B.moe_gather(x, pos, xs)
    out = _nan_rows(t, h, torch.float32)
    B.moe_combine(xs, pos, torch.ones(t, k, device="cuda"), out)
    torch.cuda.synchronize()
    assert torch.equal(xs.cpu(), torch.stack([x[0], x[1], x[2], x[3]]).cpu())
    assert torch.equal(out, x)


def test_on_another_stream_and_in_a_graph():
    """The four movements on a stream of their own, and captured: every replay
    on new inputs gives the eager bits, with eager work between replays."""
    t, k, e, h = 300, 8, 64, 520
    dt = torch.bfloat16
    picks = [torch.from_numpy(_ids(t, k, e, "outside", s)).cuda() for s in (71, 72, 73)]
    xs_in = [_rows(t, h, dt, 74 + i).cuda() for i in range(3)]
    gates = torch.rand(t, k, device="cuda")
    ids, x = picks[0].clone(), xs_in[0].clone()
    mk = lambda: dict(offsets=torch.zeros(e + 1, dtype=I32, device="cuda"),  # noqa: E731
                      order=torch.zeros(t * k, dtype=I32, device="cuda"),
                      pos=torch.zeros(t, k, dtype=I32, device="cuda"),
                      xs=torch.zeros(t * k, h, dtype=dt, device="cuda"),
                      out=torch.zeros(t, h, dtype=dt, device="cuda"),
                      dy=torch.zeros(t * k, h, dtype=dt, device="cuda"),
                      dg=torch.zeros(t, k, device="cuda"), dx=torch.zeros(t, h, dtype=dt, device="cuda"),
                      ws=torch.empty(max(1, B.moe_sort_workspace_size(t, k, e)), dtype=torch.uint8,
                                     device="cuda"))

    def run(b, ids, x, stream):
        B.moe_sort(ids, e, b["offsets"], b["order"], b["pos"], b["ws"], stream)
        B.moe_gather(x, b["pos"], b["xs"], stream)
        B.moe_combine(b["xs"], b["pos"], gates, b["out"], x, stream)
        B.moe_combine_backward(x, b["xs"], b["pos"], gates, b["dy"], b["dg"], stream)
        B.moe_gather_backward(b["xs"], b["pos"], b["dx"], stream)

    names = ("offsets", "pos", "out", "dg", "dx")
    side = torch.cuda.Stream()
    want = []
    for p, xi in zip(picks, xs_in):
        b = mk()
        torch.cuda.synchronize()
        run(b, p, xi, side)
        torch.cuda.synchronize()
        want.append({n: b[n].clone() for n in names})
    b = mk()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(b, ids, x, torch.cuda.current_stream())
    for rep in range(2):
        for p, xi, w in zip(picks, xs_in, want):
            ids.copy_(p)
            x.copy_(xi)
            g.replay()
            torch.cuda.synchronize()
            for n in names:
                assert torch.equal(b[n], w[n]), (rep, n)
            run(mk(), p, xi, torch.cuda.current_stream())
            torch.cuda.synchronize()
    del g
