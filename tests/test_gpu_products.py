"""Products of rows grouped by expert and their gradients (moe_product,
moe_product_backward) against the definition in float64, through the C ABI.

A product of two bf16 is exact in fp32, and the c products of a sum are added in
fp32 in some order.  An addition is off by one step at most, 2^-23 of a partial
sum, and no partial sum is above sum|terms|: |err| <= c 2^-23 sum|terms|, plus
half a step of a bf16 result, 2^-8 of it.
"""
import numpy as np
import pytest
import torch

from bit_moe_decode_amd import binding as B

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -23
BF16 = 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


def _say(*a):
    print(*a, flush=True)


def _normal(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(BF)


def _offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), device="cuda")


def _near(got, ref, terms, c):
    """got against ref, whose sum|terms| is `terms`, of c products a sum."""
    tol = c * U32 * terms
    if got.dtype is BF:
        tol = tol + BF16 * (ref.abs() + tol)
    err = (got.double() - ref).abs()
    assert bool(torch.isfinite(got).all())
    assert bool((err <= tol).all()), (float((err - tol).max()), float(err.max()))


def _space(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


def _product(x, w, offsets, dtype, rows=None):
    y = torch.full((x.shape[0], w.shape[1]), -7.0, dtype=dtype, device="cuda")
    B.moe_product(x, w, offsets, y, _space(B.moe_product_workspace_size(x.shape[0], *w.shape)))
    return y


def _backward(dy, x, w, offsets, dtype, add=None):
    dx = torch.full(x.shape, -7.0, dtype=BF, device="cuda")
    dw = torch.full(w.shape, float("nan"), dtype=dtype, device="cuda") if add is None else add.clone()
    B.moe_product_backward(dy, x, w, offsets, dx, dw,
                           _space(B.moe_product_backward_workspace_size(x.shape[0], *w.shape)),
                           add is not None)
    return dx, dw


def _check_product(y, x, w, counts):
    at = 0
    for e, m in enumerate(counts):
        xe, we = x[at:at + m].double(), w[e].double()
        _near(y[at:at + m], xe @ we.t(), xe.abs() @ we.abs().t(), x.shape[1])
        at += m
    assert bool((y[at:] == -7).all())  # rows behind the last expert's: left as they were


def _check_backward(dx, dw, dy, x, w, counts, add=None):
    at = 0
    for e, m in enumerate(counts):
        d, xe, we = dy[at:at + m].double(), x[at:at + m].double(), w[e].double()
        _near(dx[at:at + m], d @ we, d.abs() @ we.abs(), w.shape[1])
        base = torch.zeros_like(we) if add is None else add[e].double()
        if m == 0:
            assert torch.equal(dw[e].double(), base)
        else:
            _near(dw[e], d.t() @ xe + base, d.abs().t() @ xe.abs() + base.abs(), m + 1)
        at += m
    assert bool((dx[at:] == -7).all())


# counts of rows an expert, rows behind the last, n, k
CASES = [
    ([1], 0, 8, 8),
    ([0, 1, 0], 2, 24, 40),
    ([3, 0, 17, 1], 5, 200, 136),
    ([33, 64, 65, 0, 31, 129], 0, 264, 1000),
    ([5] * 40, 3, 128, 72),
    ([0, 0], 4, 64, 64),
    ([260, 100, 0, 511], 1, 504, 248),
    ([1] * 300, 0, 72, 104),
    ([0] * 1000 + [3] + [0] * 23, 0, 16, 48),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_product(i, dtype):
    counts, more, n, k = CASES[i]
    _say("product", i, n, k, dtype)
    rows = sum(counts) + more
    x, w = _normal(i, rows, k), _normal(100 + i, len(counts), n, k)
    y = _product(x, w, _offsets(counts), dtype)
    torch.cuda.synchronize()
    _check_product(y, x, w, counts)


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_product_backward(i, dtype, add):
    counts, more, n, k = CASES[i]
    _say("product backward", i, n, k, dtype, add)
    rows = sum(counts) + more
    x, w, dy = _normal(i, rows, k), _normal(100 + i, len(counts), n, k), _normal(200 + i, rows, n)
    base = _normal(300 + i, len(counts), n, k).to(dtype) if add else None
    dx, dw = _backward(dy, x, w, _offsets(counts), dtype, base)
    torch.cuda.synchronize()
    _check_backward(dx, dw, dy, x, w, counts, base)


# large tiles: rows enough for tiles of 256, one of which ends after each number
# of rows of interest
LARGE = [
    ([256 + r for r in (0, 1, 31, 32, 33, 64, 65, 100, 128, 129, 200, 255)] + [700, 0, 1], 4, 1096, 2056),
    ([2049, 300, 0, 513], 0, 4104, 520),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", range(len(LARGE)))
def test_product_of_many_rows(i, dtype):
    counts, more, n, k = LARGE[i]
    _say("product", counts, n, k, dtype)
    rows = sum(counts) + more
    x, w, dy = _normal(i, rows, k), _normal(100 + i, len(counts), n, k), _normal(200 + i, rows, n)
    y = _product(x, w, _offsets(counts), dtype)
    dx, dw = _backward(dy, x, w, _offsets(counts), dtype)
    torch.cuda.synchronize()
    _check_product(y, x, w, counts)
    _check_backward(dx, dw, dy, x, w, counts)


@pytest.mark.parametrize("k", [8, 24, 32, 40, 64, 96, 128, 136, 160, 168, 200])
def test_product_of_every_number_of_steps(k):
    _say("product, k", k)
    counts, n = [70, 0, 3], 48
    x, w, dy = _normal(k, 73, k), _normal(k + 1, 3, n, k), _normal(k + 2, 73, n)
    y = _product(x, w, _offsets(counts), F32)
    dx, dw = _backward(_normal(k + 3, 73, k), _normal(k + 4, 73, n), w.transpose(1, 2).contiguous().transpose(1, 2)
                       .reshape(3, n, k).transpose(1, 2).contiguous(), _offsets(counts), F32)
    torch.cuda.synchronize()
    _check_product(y, x, w, counts)
    _check_backward(dx, dw, _normal(k + 3, 73, k), _normal(k + 4, 73, n), w.transpose(1, 2).contiguous(), counts)
    del dy


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("counts,more,n,k", [([3, 0, 5], 4, 72, 8200), ([40], 0, 8, 32768), ([1], 0, 200, 4104)])
def test_product_of_long_sums(counts, more, n, k, dtype):
    """A few tiles, whose sums are split."""
    _say("long sums", counts, n, k, dtype)
    rows = sum(counts) + more
    assert B.moe_product_workspace_size(rows, len(counts), n, k) > 0
    x, w = _normal(1, rows, k), _normal(2, len(counts), n, k)
    y = _product(x, w, _offsets(counts), dtype)
    torch.cuda.synchronize()
    _check_product(y, x, w, counts)


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("counts,n,k", [([2500, 0, 3, 1601], 72, 136), ([5000], 264, 8), ([1, 8000], 40, 296)])
def test_gradients_of_many_rows_of_small_experts(counts, n, k, dtype, add):
    _say("many rows", counts, n, k, dtype, add)
    rows = sum(counts)
    assert B.moe_product_backward_workspace_size(rows, len(counts), n, k) > 0
    x, w, dy = _normal(1, rows, k), _normal(2, len(counts), n, k), _normal(3, rows, n)
    base = _normal(4, len(counts), n, k).to(dtype) if add else None
    dx, dw = _backward(dy, x, w, _offsets(counts), dtype, base)
    torch.cuda.synchronize()
    _check_backward(dx, dw, dy, x, w, counts, base)


def test_product_of_no_rows():
    w = _normal(1, 3, 16, 24)
    offsets = _offsets([0, 0, 0])
    x, y = torch.empty(0, 24, dtype=BF, device="cuda"), torch.empty(0, 16, dtype=BF, device="cuda")
    B.moe_product(x, w, offsets, y)
    dw = torch.full(w.shape, float("nan"), dtype=F32, device="cuda")
    B.moe_product_backward(y, x, w, offsets, x, dw)
    torch.cuda.synchronize()
    assert bool((dw == 0).all())


def test_one_gradient_alone_and_the_same_bits_again():
    counts, n, k = [40, 0, 300], 136, 200
    x, w, dy = _normal(1, 340, k), _normal(2, 3, n, k), _normal(3, 340, n)
    off = _offsets(counts)
    dx, dw = _backward(dy, x, w, off, F32)
    only_dx, only_dw = torch.full_like(dx, -7.0), torch.zeros_like(dw)
    B.moe_product_backward(dy, None, w, off, dx=only_dx)
    B.moe_product_backward(dy, x, None, off, dw=only_dw)
    B.moe_product_backward(dy, x, w, off)  # neither: nothing
    torch.cuda.synchronize()
    assert torch.equal(dx, only_dx) and torch.equal(dw, only_dw)


def test_rows_do_not_depend_on_others():
    """A row's results are the same bits whatever the other rows and experts hold,
    NaN and infinities among them."""
    counts, n, k = [70, 200, 90], 264, 328
    x, w, dy = _normal(1, 360, k), _normal(2, 3, n, k), _normal(3, 360, n)
    off = _offsets(counts)
    y, (dx, dw) = _product(x, w, off, F32), _backward(dy, x, w, off, F32)
    for t in (x, dy):
        t[70:270] = float("nan")
        t[300] = float("inf")
    w[1] = float("nan")
    y2, (dx2, dw2) = _product(x, w, off, F32), _backward(dy, x, w, off, F32)
    torch.cuda.synchronize()
    keep = [*range(70), *range(270, 300), *range(301, 360)]
    assert torch.equal(y[keep], y2[keep]) and torch.equal(dx[keep], dx2[keep])
    assert torch.equal(dw[0], dw2[0])
    assert bool(torch.isnan(y2[70:270]).all()) and bool(torch.isnan(dw2[1]).all())
    assert not bool(torch.isfinite(y2[300]).any())


@pytest.mark.parametrize("offsets", [[0, 10, 5, 40], [-3, 20, 60, 2 ** 31 - 1], [7, 7, 7, 30], [40, 30, 20, 10],
                                     [-2 ** 31, 2 ** 31 - 1, -5, 12]])
def test_offsets_that_are_not_ascending_stay_inside(offsets):
    """No access leaves the buffers: what lies around them is kept."""
    _say("offsets", offsets)
    n, k, rows = 40, 72, 40
    whole = torch.full((rows + 64, n), 5.0, dtype=BF, device="cuda")
    whole_dx = torch.full((rows + 64, k), 5.0, dtype=BF, device="cuda")
    x, w, dy = _normal(1, rows, k), _normal(2, 3, n, k), _normal(3, rows, n)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    B.moe_product(x, w, off, whole[32:32 + rows])
    dw = torch.empty(3, n, k, device="cuda")
    B.moe_product_backward(dy, x, w, off, whole_dx[32:32 + rows], dw)
    torch.cuda.synchronize()
    for t in (whole, whole_dx):
        assert bool((t[:32] == 5).all()) and bool((t[32 + rows:] == 5).all())


def test_product_gradients_are_the_differences():
    """sum(dy y(x, w)) moves by dx and dw: differences in float64 around bf16
    inputs, by the definition, against the library's gradients (bf16 2^-8 and
    sums of at most 4 terms of size 1: 2^-5)."""
    counts, n, k = [2, 3], 8, 8
    x, w, dy = _normal(1, 5, k), _normal(2, 2, n, k), _normal(3, 5, n)
    dx, dw = _backward(dy, x, w, _offsets(counts), F32)

    def value(xd, wd):
        y = torch.cat([xd[:2] @ wd[0].t(), xd[2:] @ wd[1].t()])
        return float((dy.double() * y).sum())

    h = 2.0 ** -10
    for r, c in ((0, 0), (1, 7), (4, 3)):
        p, m = x.double(), x.double()
        p[r, c] += h
        m[r, c] -= h
        d = (value(p, w.double()) - value(m, w.double())) / (2 * h)
        assert abs(d - float(dx[r, c])) <= BF16 * abs(d) + 1e-6
    for e, i, c in ((0, 0, 0), (1, 7, 2)):
        p, m = w.double(), w.double()
        p[e, i, c] += h
        m[e, i, c] -= h
        d = (value(x.double(), p) - value(x.double(), m)) / (2 * h)
        assert abs(d - float(dw[e, i, c])) <= 1e-5 * (1 + abs(d))


def test_product_on_another_stream_and_in_a_graph():
    counts, n, k = [40, 0, 90], 136, 264
    x, w, dy = _normal(1, 130, k), _normal(2, 3, n, k), _normal(3, 130, n)
    off = _offsets(counts)
    y = torch.zeros(130, n, dtype=BF, device="cuda")
    dx, dw = torch.zeros(130, k, dtype=BF, device="cuda"), torch.zeros(3, n, k, device="cuda")
    ws = _space(max(B.moe_product_workspace_size(130, 3, n, k), B.moe_product_backward_workspace_size(130, 3, n, k)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.moe_product(x, w, off, y, ws, stream=side)
    side.synchronize()
    _check_product(y, x, w, counts)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = torch.cuda.current_stream()
        B.moe_product(x, w, off, y, ws, stream=s)
        B.moe_product_backward(y, x, w, off, dx, dw, ws, stream=s)
    for i in range(3):
        x.copy_(_normal(10 + i, 130, k))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        _check_product(y, x, w, counts)
        rx, rw = _backward(y, x, w, off, F32)
        assert torch.equal(dx, rx) and torch.equal(dw, rw)
