"""The operators on grouped rows where an element's place passes 2^31, at the
largest batches they take, and at more tokens than one launch holds.

Movements of one pick a token are copies or one fp32 product rounded once:
compared bitwise.  The others use the tolerances of their own small tests
(tests/test_gpu_lora.py, tests/test_gpu_wide.py) on some of the rows.
"""
import pytest
import torch

from bit_moe_decode_amd import binding as B
from tests import test_gpu_lora as L
from tests import test_gpu_wide as W

pytestmark = pytest.mark.gpu

I32 = torch.int32


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def test_refusal_of_a_workspace_in_host_memory():
    """Refused before anything is enqueued; so is a part of a strided one."""
    ids = torch.zeros(4000, 8, dtype=I32, device="cuda")
    offsets = torch.zeros(17, dtype=I32, device="cuda")
    order, pos = torch.zeros(32000, dtype=I32, device="cuda"), torch.zeros_like(ids)
    n = B.moe_sort_workspace_size(4000, 8, 16)
    for ws in (torch.zeros(n, dtype=torch.uint8),
               torch.zeros(n, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(B.MoeError):
            B.moe_sort(ids, 16, offsets, order, pos, ws)
    a, b, scale, rank = L._adapters(2, 8, 64, 64, 1, False)
    lora = B.make_lora(a, b, scale, rank)
    x = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    some = torch.zeros(3, dtype=I32, device="cuda")
    with pytest.raises(B.MoeError):
        B.lora_apply(lora, x, some, x, torch.empty_like(x), torch.zeros(1 << 16, dtype=torch.uint8))
    matrix = B.make_matrix(B.FMT_BF16, 128, 64, torch.zeros(128, 64, dtype=torch.bfloat16))
    a, b, scale, rank = L._adapters(2, 8, 128, 64, 2, False)
    with pytest.raises(B.MoeError):  # the matrix in host memory
        B.lowbit_gemv_lora(matrix, B.make_lora(a, b, scale, rank), x, some,
                           torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda"),
                           torch.zeros(1 << 16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("tokens,h,dtype", [
    (2 ** 23 + 5, 2, torch.bfloat16),    # more blocks than one launch
    (2 ** 23 + 5, 3, torch.float32),
    (350000, 6144, torch.bfloat16)])     # 2^31 elements and more
def test_movements_of_many_rows(tokens, h, dtype):
    print("movements", tokens, h, dtype, flush=True)
    g = _gen(tokens + h)
    x = torch.randn(tokens, h, generator=g, device="cuda").to(dtype) if h < 8 else \
        torch.randint(2 ** 13, 2 ** 14, (tokens, h), generator=g, device="cuda",
                      dtype=torch.int16).view(dtype)  # 2^-63 .. 2
    order = torch.randperm(tokens, generator=g, device="cuda")
    pos = order.to(I32).view(-1, 1)
    pos[tokens // 2] = -1
    gates = torch.randn(tokens, 1, generator=g, device="cuda")
    xs = torch.zeros_like(x)
    B.moe_gather(x, pos, xs)
    torch.cuda.synchronize()
    some = torch.cat([torch.arange(0, tokens, max(1, tokens // 999), device="cuda"),
                      torch.arange(tokens - 300, tokens, device="cuda")])
    some = some[some != tokens // 2]
    assert torch.equal(xs[order[some]], x[some])
    assert bool((xs[order[tokens // 2]] == 0).all())

    out = torch.full_like(x, float("nan"))
    B.moe_combine(xs, pos, gates, out)
    dx = torch.full_like(x, float("nan"))
    B.moe_gather_backward(xs, pos, dx)
    torch.cuda.synchronize()
    assert torch.equal(out[some], (gates[some] * x[some].float()).to(dtype))
    assert torch.equal(dx[some], x[some])
    assert bool((out[tokens // 2] == 0).all()) and bool((dx[tokens // 2] == 0).all())

    del dx
    dy = torch.zeros_like(x)
    dg = torch.full((tokens, 1), float("nan"), device="cuda")
    B.moe_combine_backward(x, xs, pos, gates, dy, dg)
    torch.cuda.synchronize()
    assert torch.equal(dy[order[some]], (gates[some] * x[some].float()).to(dtype))
    v = x[some].double()
    dot, terms = (v * v).sum(1), (v * v).sum(1)
    assert bool(((dg[some, 0].double() - dot).abs() <= (h + 8) * 2.0 ** -24 * terms).all())
    assert float(dg[tokens // 2]) == 0.0


@pytest.mark.parametrize("rows,n,k", [(66000, 64, 32768), (66000, 32768, 64)])
def test_adapters_of_many_wide_rows(rows, n, k):
    print("lora", rows, n, k, flush=True)
    a, b, scale, rank = L._adapters(3, 16, n, k, rows + n, False)
    g = _gen(n)
    ids = torch.randint(-1, 3, (rows,), generator=g, device="cuda").to(I32)
    x = torch.randn(rows, k, generator=g, device="cuda", dtype=torch.bfloat16)
    base = torch.randn(rows, n, generator=g, device="cuda", dtype=torch.bfloat16)
    lora = B.make_lora(a, b, scale, rank)
    y = torch.full_like(base, float("nan"))
    B.lora_apply(lora, x, ids, base, y, L._space(lora, rows))
    torch.cuda.synchronize()
    for at in (slice(0, 100), slice(rows - 200, rows)):
        d, tol = L._delta(a, b, scale, rank, x[at], ids[at])
        L._assert_close(y[at], base[at].double() + d, tol)


def test_the_most_adapters_rows():
    rows, n, k = 2 ** 20, 8, 64
    a, b, scale, rank = L._adapters(1023, 8, n, k, 5, True)
    g = _gen(6)
    ids = torch.randint(-1, 1024, (rows,), generator=g, device="cuda").to(I32)
    x = torch.randn(rows, k, generator=g, device="cuda", dtype=torch.bfloat16)
    base = torch.randn(rows, n, generator=g, device="cuda", dtype=torch.bfloat16)
    lora = B.make_lora(a, b, scale, rank)
    y = torch.full_like(base, float("nan"))
    B.lora_apply(lora, x, ids, base, y, L._space(lora, rows))
    torch.cuda.synchronize()
    for at in (slice(0, 500), slice(rows - 500, rows)):
        d, tol = L._delta(a, b, scale, rank, x[at], ids[at])
        L._assert_close(y[at], base[at].double() + d, tol)


def test_the_wide_steps_most_tokens():
    """65536 tokens of 6144: 3.6e9 elements of the experts' fp32 outputs."""
    t, hidden, inter, experts = 65536, 6144, 128, 16
    layer = W._layer(hidden, inter, experts, True, 21)
    g = _gen(22)
    x = torch.randn(t, hidden, generator=g, device="cuda", dtype=torch.bfloat16)
    ids, gates = W._routing(t, experts, "top", 23)
    out = W._run(layer, x, ids, gates)
    torch.cuda.synchronize()
    some = torch.cat([torch.arange(0, 4, device="cuda"), torch.arange(t - 12, t, device="cuda")])
    ref, tol = W._reference(layer, x[some], ids[some], gates[some])
    bound = tol + 2.0 ** -8 * (ref.abs() + tol)
    # and in a batch of their own (whose tiles, and with them the sums, differ)
    few = W._run(layer, x[some].contiguous(), ids[some].contiguous(), gates[some].contiguous())
    torch.cuda.synchronize()
    for got in (out[some], few):
        err = (got.double() - ref).abs()
        assert bool((err <= bound).all()), (int((err > bound).sum()), float((err - bound).max()))
