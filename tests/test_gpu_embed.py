"""The embedding lookup and its gradient (embed, embed_backward) against the
definition in float64, through the C ABI.

Lookup: one product in fp32 (2^-24 of it), rounded to the table's type.
Gradient: a token's m rows are added in fp32 (an addition off by 2^-24 of a
partial sum), times scale, plus what dtable held: (m + 2) 2^-24 sum|terms|, and
half a step of a bf16 result, 2^-8 of it.
"""
import pytest
import torch

from bit_moe_decode_amd import binding as B

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
BF16 = 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32
TYPES = [BF, F32]


def _say(*a):
    print(*a, flush=True)


def _ids(rows, vocab, mode, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if mode == "same":
        return torch.full((rows,), vocab - 1, dtype=torch.int32, device="cuda")
    if mode == "none":
        return torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    if mode == "few":  # a few tokens make up all rows, in runs of every length
        ids = torch.randint(0, min(vocab, 5), (rows,), generator=g, device="cuda")
    else:
        ids = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    if mode == "outside":
        bad = torch.tensor([-1, -2 ** 31, vocab, 2 ** 31 - 1], device="cuda")
        pick = torch.randint(0, 4, (rows,), generator=g, device="cuda")
        ids = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.4, bad[pick], ids)
    return ids.to(torch.int32)


def _rows(n, h, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(n, h, generator=g, device="cuda").to(dtype)


def _space(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


SIZES = [(1, 1, 1), (1, 5, 8), (7, 3, 9), (61, 1000, 257), (64, 1024, 512), (65, 1025, 513), (130, 40, 2050),
         (1024, 300, 40), (1025, 5000, 24), (3000, 151936, 17), (8192, 700, 72), (8193, 40000, 33),
         (20000, 1 << 20, 8)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab,hidden", SIZES)
def test_embed(rows, vocab, hidden, dtype):
    _say("embed", rows, vocab, hidden, dtype)
    ids, table = _ids(rows, vocab, "outside", rows), _rows(vocab, hidden, dtype, 1)
    out = torch.full((rows, hidden), float("nan"), dtype=dtype, device="cuda")
    B.embed(ids, table, out, 1.7)
    plain = torch.empty_like(out)
    B.embed(ids, table, plain)
    torch.cuda.synchronize()
    live = (ids >= 0) & (ids < vocab)
    ref = torch.where(live[:, None], table[ids.long().clamp(0, vocab - 1)], torch.zeros((), dtype=dtype, device="cuda"))
    assert torch.equal(plain, ref)
    want = ref.double() * float(torch.tensor(1.7))
    assert bool(((out.double() - want).abs() <= (BF16 if dtype is BF else 0) * want.abs() * 1.01 + U32 * want.abs()).all())


def _check(dtable, ids, dout, scale, base=None):
    vocab = dtable.shape[0]
    live = (ids >= 0) & (ids < vocab)
    at = ids.long()[live]
    d = dout.double()[live] * scale
    ref = torch.zeros(dtable.shape, dtype=torch.float64, device="cuda").index_add_(0, at, d)
    terms = torch.zeros(dtable.shape, dtype=torch.float64, device="cuda").index_add_(0, at, d.abs())
    m = torch.bincount(at, minlength=vocab)[:, None]
    if base is not None:
        ref, terms = ref + base.double(), terms + base.double().abs()
        assert torch.equal(dtable[m[:, 0] == 0], base[m[:, 0] == 0])
    else:
        assert bool((dtable[m[:, 0] == 0] == 0).all())
    tol = (m + 2) * U32 * terms
    if dtable.dtype is BF:
        tol = tol + BF16 * (ref.abs() + tol)
    err = (dtable.double() - ref).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float(err.max()))


def _grad(ids, dout, vocab, dtype, scale=1.0, base=None, ws=None):
    rows, hidden = dout.shape
    dtable = torch.full((vocab, hidden), float("nan"), dtype=dtype, device="cuda") if base is None else base.clone()
    if ws is None:
        ws = _space(B.embed_backward_workspace_size(rows, vocab, hidden))
    B.embed_backward(ids, dout, dtable, ws, scale, base is not None)
    return dtable


@pytest.mark.parametrize("mode,dtype,table_dtype", [("outside", a, b) for a in TYPES for b in TYPES] + [
    ("random", BF, BF), ("few", BF, BF), ("few", F32, F32), ("same", BF, F32), ("none", F32, BF)])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("rows,vocab,hidden", SIZES)
def test_embed_backward(rows, vocab, hidden, dtype, table_dtype, add, mode):
    if vocab * hidden > 1 << 21 and mode in ("few", "none"):
        vocab = 70000
    _say("embed backward", rows, vocab, hidden, dtype, table_dtype, add, mode)
    ids, dout = _ids(rows, vocab, mode, rows), _rows(rows, hidden, dtype, 2)
    base = _rows(vocab, hidden, table_dtype, 3) if add else None
    dtable = _grad(ids, dout, vocab, table_dtype, 0.5, base)
    torch.cuda.synchronize()
    _check(dtable, ids, dout, 0.5, base)


@pytest.mark.parametrize("rows", [40000, 300000])
def test_embed_backward_of_many_rows(rows):
    """Chunks longer than 16 rows, sorts of several blocks, one token in half of
    the rows."""
    vocab, hidden = 30000, 24
    _say("embed backward", rows)
    ids, dout = _ids(rows, vocab, "outside", 5), _rows(rows, hidden, F32, 6)
    ids[torch.arange(0, rows, 2, device="cuda")] = 17
    for dtype in TYPES:
        dtable = _grad(ids, dout, vocab, dtype)
        torch.cuda.synchronize()
        _check(dtable, ids, dout, 1.0)


@pytest.mark.parametrize("rows", [200, 5000])
def test_rows_without_a_token_are_not_read_into_others(rows):
    ids, dout = _ids(rows, 900, "outside", 7), _rows(rows, 40, F32, 8)
    ids[3] = 5
    want = _grad(ids, dout, 900, F32)
    live = (ids >= 0) & (ids < 900)
    dout[~live] = float("nan")
    got = _grad(ids, dout, 900, F32)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    dout[3] = float("inf")
    got = _grad(ids, dout, 900, F32)
    torch.cuda.synchronize()
    keep = torch.arange(900, device="cuda") != 5
    assert torch.equal(got[keep], want[keep]) and bool((got[5] == float("inf")).all())


@pytest.mark.parametrize("rows", [30, 2000])
def test_a_scale_that_is_not_finite(rows):
    """Tokens without rows have a gradient of 0 all the same, rows without a token
    an embedding of 0."""
    ids, dout = _ids(rows, 5000, "outside", 12), _rows(rows, 16, F32, 13)
    dtable = _grad(ids, dout, 5000, F32, float("inf"))
    out = torch.empty(rows, 16, dtype=BF, device="cuda")
    B.embed(ids, _rows(5000, 16, BF, 14), out, float("nan"))
    torch.cuda.synchronize()
    live = (ids >= 0) & (ids < 5000)
    used = torch.zeros(5000, dtype=torch.bool, device="cuda")
    used[ids[live].long()] = True
    assert bool((dtable[~used] == 0).all()) and not bool(torch.isfinite(dtable[used]).any())
    assert bool((out[~live] == 0).all()) and bool(torch.isnan(out[live]).all())


def test_no_rows():
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    table, dout = _rows(50, 7, BF, 1), torch.empty(0, 7, dtype=BF, device="cuda")
    B.embed(ids, table, dout)
    dtable = torch.full((50, 7), float("nan"), dtype=BF, device="cuda")
    B.embed_backward(ids, dout, dtable)
    kept = table.clone()
    B.embed_backward(ids, dout, kept, add=True)
    torch.cuda.synchronize()
    assert bool((dtable == 0).all()) and torch.equal(kept, table)


def test_gradient_is_the_difference():
    """sum(dout embed(table)) moves by dtable: differences in float64."""
    ids, dout = _ids(20, 6, "outside", 9), _rows(20, 4, F32, 10)
    table, dtable = _rows(6, 4, F32, 11), _grad(ids, dout, 6, F32, 1.5)
    live = (ids >= 0) & (ids < 6)

    def value(t):
        return float((dout.double()[live] * 1.5 * t[ids.long()[live]]).sum())

    for i, j in ((0, 0), (3, 2), (5, 3)):
        p, m = table.double(), table.double()
        p[i, j] += 0.5
        m[i, j] -= 0.5
        assert abs(value(p) - value(m) - float(dtable[i, j])) < 1e-5 * (1 + abs(float(dtable[i, j])))


@pytest.mark.parametrize("rows,vocab", [(40, 300), (3000, 2000), (9000, 2000)])
def test_on_another_stream_and_in_a_graph(rows, vocab):
    _say("graph", rows, vocab)
    ids, dout = _ids(rows, vocab, "outside", 1), _rows(rows, 72, BF, 2)
    table, out = _rows(vocab, 72, BF, 3), torch.zeros(rows, 72, dtype=BF, device="cuda")
    dtable = torch.zeros(vocab, 72, device="cuda")
    ws = _space(B.embed_backward_workspace_size(rows, vocab, 72))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.embed_backward(ids, dout, dtable, ws, stream=side)
    side.synchronize()
    _check(dtable, ids, dout, 1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = torch.cuda.current_stream()
        B.embed(ids, table, out, 2.0, stream=s)
        B.embed_backward(ids, out, dtable, ws, 0.5, stream=s)
    for i in range(3):
        ids.copy_(_ids(rows, vocab, "outside", 20 + i))
        dtable.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(out)
        B.embed(ids, table, want, 2.0)
        assert torch.equal(out, want)
        assert torch.equal(dtable, _grad(ids, out, vocab, F32, 0.5))
        _check(dtable, ids, out, 0.5)
