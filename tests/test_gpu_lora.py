"""Low-rank adapters of many requests (lora_apply, lowbit_gemv_lora) against a
float64 form, through the C ABI.

Tolerance.  A x is a sum of K products in fp32 and B v one of `rank` products;
they may be formed by bf16 matrix instructions, whose sums truncate: (K + 8)
and (rank + 8) of 2^-23 of the sums' terms.  A v that such an instruction
takes is split into two bf16 parts, which keeps 16 bits: 2^-16 of B v's terms.
The projection adds (K + 8) * 2^-24 of its terms (the bound of lowbit_gemv's
own tests), and the result is rounded to bf16 once: 2^-8 of its value.
"""
import numpy as np
import pytest
import torch

from bit_moe_decode_amd import binding as B
from bit_moe_decode_amd import synth as S

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, flush=True)


def _adapters(adapters, max_rank, n, k, seed, ragged):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    a = (torch.randn(adapters, max_rank, k, generator=g, device="cuda") * k ** -0.5).to(torch.bfloat16)
    b = torch.randn(adapters, n, max_rank, generator=g, device="cuda").to(torch.bfloat16)
    scale = torch.rand(adapters, generator=g, device="cuda") + 0.5
    rank = None
    if ragged:  # any rank, 0 and max_rank among them; what lies past it is not used
        rank = torch.randint(0, max_rank + 1, (adapters,), generator=g, device="cuda").to(torch.int32)
        rank[0] = 0
        rank[-1] = max_rank
        for i, r in enumerate(rank.tolist()):
            a[i, r:] = float("nan")
            b[i, :, r:] = float("inf")
    return a, b, scale, rank


def _ids(rows, adapters, seed, segment=1):
    g = torch.Generator()
    g.manual_seed(seed)
    ids = torch.randint(-1, adapters + 1, (rows,), generator=g)  # -1 and `adapters`: none
    if segment > 1:
        ids = ids[torch.arange(rows) // segment]
    return ids.to(torch.int32).cuda()


def _delta(a, b, scale, rank, x, ids):
    """(scale B (A x), the error its sums may have), float64 [rows, n]."""
    rows, k = x.shape
    n, mr = b.shape[1:]
    out = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    xd = x.double()
    for i in range(a.shape[0]):
        at = (ids == i).nonzero()[:, 0]
        r = mr if rank is None else int(rank[i])
        if at.numel() == 0 or r == 0:
            continue
        ad, bd, s = a[i, :r].double(), b[i, :, :r].double(), scale[i].double()
        v = xd[at] @ ad.t()
        va = xd[at].abs() @ ad.abs().t()
        out[at] = s * (v @ bd.t())
        tol[at] = s * ((va * (k + 8) * 2.0 ** -23) @ bd.abs().t()
                       + (v.abs() @ bd.abs().t()) * ((r + 8) * 2.0 ** -23 + 2.0 ** -16))
    return out, tol


def _assert_close(y, ref, tol):
    bound = tol + 2.0 ** -8 * (ref.abs() + tol)
    err = (y.double() - ref).abs()
    assert bool((err <= bound).all()), (int((err > bound).sum()), float((err / bound.clamp(min=1e-300)).max()))


def _space(lora, rows):
    return torch.empty(max(1, B.lora_workspace_size(lora, rows)), dtype=torch.uint8, device="cuda")


# (rows, n, k, max_rank, adapters, segment)
SHAPES = [(1, 8, 64, 8, 1, 1), (1, 6144, 6144, 16, 3, 1), (3, 264, 192, 24, 2, 1),
          (8, 1000, 1088, 8, 9, 1), (17, 520, 4160, 64, 40, 1), (64, 2048, 2560, 16, 128, 1),
          (65, 136, 640, 128, 5, 7), (200, 1024, 1024, 32, 3, 90), (777, 392, 704, 40, 11, 50),
          (1025, 2056, 512, 128, 1000, 1), (2500, 512, 2048, 64, 6, 400), (130, 64, 32768, 16, 4, 1), (150, 128, 256, 16, 3, 1),
          (70, 264, 64, 8, 3, 1), (300, 64, 576, 16, 2, 40)]


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("rows,n,k,mr,adapters,segment", SHAPES)
def test_lora_apply(rows, n, k, mr, adapters, segment, ragged):
    _say("lora", rows, n, k, mr, adapters, segment, ragged)
    a, b, scale, rank = _adapters(adapters, mr, n, k, rows + n, ragged)
    ids = _ids(rows, adapters, rows + k, segment)
    x = S.make_x(rows, k, seed=rows).cuda()
    base = S.make_x(rows, n, seed=rows + 1).cuda()
    lora = B.make_lora(a, b, scale, rank)
    y = torch.full_like(base, float("nan"))
    B.lora_apply(lora, x, ids, base, y, _space(lora, rows))
    torch.cuda.synchronize()
    d, tol = _delta(a, b, scale, rank, x, ids)
    _assert_close(y, base.double() + d, tol)
    none = (ids < 0) | (ids >= adapters)
    assert torch.equal(y[none], base[none])
    # in place, and the same bits again
    y2 = base.clone()
    B.lora_apply(lora, x, ids, y2, y2, _space(lora, rows))
    torch.cuda.synchronize()
    assert torch.equal(y2, y)


def _projection(fmt, n, k, seed):
    if fmt == B.FMT_Q1:
        return S.make_q1(n, k, seed, device="cuda"), None
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = torch.randn(n, k, generator=g, device="cuda") * 0.05
    return (w.to(torch.bfloat16), None) if fmt == B.FMT_BF16 else S.encode_fp8_blocks(w)


def _project(fmt, codes, scales, x):
    """float64 (W x, sum of its terms' sizes)."""
    c = codes.cpu()
    if fmt == B.FMT_BF16:
        w = c.double()
    elif fmt == B.FMT_FP8:
        w = c.view(torch.float8_e4m3fn).double()
        w = w * torch.from_numpy(np.kron(scales.cpu().double().numpy(), np.ones((128, 128))))
    else:
        d = c[..., :2].contiguous().view(torch.float16).double()
        bits = torch.from_numpy(np.unpackbits(c[..., 2:].numpy(), axis=-1, bitorder="little"))
        w = ((1 - 2 * bits.double()) * d).reshape(c.shape[0], -1)
    w = w.cuda()
    return x.double() @ w.t(), x.double().abs() @ w.abs().t()


# every form of the GEMVs: 1-bit tables, generic, MFMA and wide MFMA; FP8; bf16
GEMVS = [(B.FMT_Q1, 1, 9728, 2560), (B.FMT_Q1, 1, 40, 384), (B.FMT_Q1, 5, 1032, 512),
         (B.FMT_Q1, 8, 2560, 9728), (B.FMT_Q1, 3, 32776, 1024), (B.FMT_FP8, 1, 6144, 6144),
         (B.FMT_FP8, 8, 256, 384), (B.FMT_BF16, 1, 512, 192), (B.FMT_BF16, 7, 2048, 2560)]


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("fmt,rows,n,k", GEMVS)
def test_lowbit_gemv_lora(fmt, rows, n, k, ragged):
    _say("gemv + lora", fmt, rows, n, k, ragged)
    codes, scales = _projection(fmt, n, k, n + k)
    for mr, adapters in ((16, 5), (128, 2)):
        a, b, scale, rank = _adapters(adapters, mr, n, k, rows + n, ragged)
        ids = _ids(rows, adapters, rows + n + mr)
        if rows == 1:
            ids[0] = adapters - 1
        x = S.make_x(rows, k, seed=rows + 3).cuda()
        lora = B.make_lora(a, b, scale, rank)
        m = B.make_matrix(fmt, n, k, codes, scales)
        y = torch.full((rows, n), float("nan"), dtype=torch.bfloat16, device="cuda")
        B.lowbit_gemv_lora(m, lora, x, ids, y, _space(lora, rows))
        plain = torch.empty_like(y)
        assert B.lib().lowbit_gemv(m, x.data_ptr(), rows, plain.data_ptr(), None) == B.MOE_OK
        torch.cuda.synchronize()
        d, tol = _delta(a, b, scale, rank, x, ids)
        ref, terms = _project(fmt, codes, scales, x)
        _assert_close(y, ref + d, tol + (k + 8) * 2.0 ** -24 * terms)
        none = (ids < 0) | (ids >= adapters)
        assert torch.equal(y[none], plain[none])  # a row without an adapter: lowbit_gemv's bits


def test_no_adapters_and_no_rows():
    n, k = 128, 128
    empty = torch.empty(0, 8, k, dtype=torch.bfloat16, device="cuda")
    lora = B.make_lora(empty, torch.empty(0, n, 8, dtype=torch.bfloat16, device="cuda"),
                       torch.empty(0, device="cuda"))
    for rows in (1, 70):
        base = S.make_x(rows, n, seed=1).cuda()
        x = S.make_x(rows, k, seed=2).cuda()
        y = torch.zeros_like(base)
        B.lora_apply(lora, x, torch.zeros(rows, dtype=torch.int32, device="cuda"), base, y, _space(lora, rows))
        torch.cuda.synchronize()
        assert torch.equal(y, base)
    none = torch.empty(0, k, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(0, n, dtype=torch.bfloat16, device="cuda")
    B.lora_apply(lora, none, torch.empty(0, dtype=torch.int32, device="cuda"), out, out, _space(lora, 1))


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("rows,mr", [(256, 8), (257, 8), (128, 16), (129, 16), (32, 64), (33, 64),
                                     (16, 128), (17, 128)])
def test_few_and_many_rows(rows, mr, ragged):
    """Either side of the row count from which rows are grouped."""
    n, k, adapters = 520, 704, 5
    _say("lora", rows, mr, ragged)
    a, b, scale, rank = _adapters(adapters, mr, n, k, rows + mr, ragged)
    ids = _ids(rows, adapters, rows)
    x = S.make_x(rows, k, seed=rows).cuda()
    base = S.make_x(rows, n, seed=rows + 1).cuda()
    lora = B.make_lora(a, b, scale, rank)
    y = torch.full_like(base, float("nan"))
    B.lora_apply(lora, x, ids, base, y, _space(lora, rows))
    torch.cuda.synchronize()
    d, tol = _delta(a, b, scale, rank, x, ids)
    _assert_close(y, base.double() + d, tol)


def test_no_adapters_and_grouped_rows():
    n, k, rows = 128, 128, 300
    lora = B.make_lora(torch.empty(0, 8, k, dtype=torch.bfloat16, device="cuda"),
                       torch.empty(0, n, 8, dtype=torch.bfloat16, device="cuda"),
                       torch.empty(0, device="cuda"))
    base = S.make_x(rows, n, seed=1).cuda()
    y = torch.zeros_like(base)
    B.lora_apply(lora, S.make_x(rows, k, seed=2).cuda(), torch.zeros(rows, dtype=torch.int32, device="cuda"),
                 base, y, _space(lora, rows))
    torch.cuda.synchronize()
    assert torch.equal(y, base)


def test_a_row_does_not_depend_on_the_batch_around_it():
    """NaN and infinities in other rows stay there."""
    rows, n, k, mr, adapters = 300, 256, 256, 16, 4
    a, b, scale, rank = _adapters(adapters, mr, n, k, 5, False)
    ids = torch.arange(rows, device="cuda").remainder(adapters).to(torch.int32)
    x = S.make_x(rows, k, seed=6).cuda()
    base = S.make_x(rows, n, seed=7).cuda()
    lora = B.make_lora(a, b, scale, rank)
    y = torch.empty_like(base)
    B.lora_apply(lora, x, ids, base, y, _space(lora, rows))
    bad = x.clone()
    bad[::3] = float("nan")
    bad[1::3, 0] = float("inf")
    y2 = torch.empty_like(base)
    B.lora_apply(lora, bad, ids, base, y2, _space(lora, rows))
    torch.cuda.synchronize()
    assert torch.equal(y2[2::3], y[2::3])
    assert bool(torch.isnan(y2[::3]).all())


def test_streams_and_graph():
    n, k, mr, adapters = 512, 512, 16, 6
    a, b, scale, rank = _adapters(adapters, mr, n, k, 8, True)
    lora = B.make_lora(a, b, scale, rank)
    codes, scales = _projection(B.FMT_FP8, n, k, 9)
    m = B.make_matrix(B.FMT_FP8, n, k, codes, scales)
    sizes = (4, 40, 500)
    sets = [[(S.make_x(r, k, seed=10 * s + r).cuda(), _ids(r, adapters, 10 * s + r, 1 + r // 100),
              S.make_x(r, n, seed=10 * s + r + 1).cuda()) for r in sizes] for s in range(3)]

    def run(inputs, ys, wss, stream):
        for (x, ids, base), y, ws in zip(inputs, ys, wss):
            B.lora_apply(lora, x, ids, base, y, ws, stream)
        x, ids, _ = inputs[0]
        B.lowbit_gemv_lora(m, lora, x, ids, ys[3], wss[3], stream)

    def buffers():
        return ([torch.zeros(r, n, dtype=torch.bfloat16, device="cuda") for r in sizes + (4,)],
                [_space(lora, r) for r in sizes + (4,)])

    side = torch.cuda.Stream()
    want = []
    for s in sets:
        ys, wss = buffers()
        torch.cuda.synchronize()
        run(s, ys, wss, side)
        torch.cuda.synchronize()
        want.append(ys)
    cur = [tuple(t.clone() for t in c) for c in sets[0]]
    ys, wss = buffers()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(cur, ys, wss, torch.cuda.current_stream())
    for rep in range(2):
        for s, w in zip(sets, want):
            for c, i in zip(cur, s):
                for d, t in zip(c, i):
                    d.copy_(t)
            g.replay()
            torch.cuda.synchronize()
            for i, (p, q) in enumerate(zip(ys, w)):
                assert torch.equal(p, q), (rep, i)
            run(s, *buffers(), torch.cuda.current_stream())
            torch.cuda.synchronize()
    del g
