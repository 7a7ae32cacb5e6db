"""The products by expert, the LM head's loss, the embedding and their gradients at
the largest and smallest sizes that they take, and two calls under way at once.

Where a sum is long its terms are small whole numbers, whose sums below 2^24 are
exact in fp32 in any order: the results are equal to the definition's.
"""
import pytest
import torch

from bit_moe_decode_amd import binding as B
from tests.test_gpu_lm_loss import _check_grads, _check_loss, _inputs

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _say(*a):
    print(*a, flush=True)


def _whole(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=g, device="cuda", dtype=torch.int8).to(BF)


def _space(n):
    return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("counts,more,n,k", [([2 ** 24 - 1005, 0, 1000], 5, 8, 8), ([3], 0, 32768, 8), ([0, 70], 1, 8, 32768),
                                             ([1] * 1024, 0, 8, 8)])
def test_products_at_their_limits(counts, more, n, k):
    _say("product", counts[:3], n, k)
    rows, e = sum(counts) + more, len(counts)
    offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).to(I32)
    x, w, dy = _whole(1, rows, k), _whole(2, e, n, k), _whole(3, rows, n)
    y = torch.full((rows, n), -7.0, device="cuda")
    dx = torch.full((rows, k), -7.0, dtype=BF, device="cuda")
    dw = torch.full((e, n, k), float("nan"), device="cuda")
    B.moe_product(x, w, offsets, y, _space(B.moe_product_workspace_size(rows, e, n, k)))
    B.moe_product_backward(dy, x, w, offsets, dx, dw, _space(B.moe_product_backward_workspace_size(rows, e, n, k)))
    torch.cuda.synchronize()
    at = 0
    for i, m in enumerate(counts):
        for j in range(at, at + m, 1 << 21):
            part = slice(j, min(at + m, j + (1 << 21)))
            assert torch.equal(y[part].double(), x[part].double() @ w[i].double().t())
            assert torch.equal(dx[part], (dy[part].double() @ w[i].double()).to(BF))
        ref = torch.zeros(n, k, dtype=torch.float64, device="cuda")
        for j in range(at, at + m, 1 << 21):
            part = slice(j, min(at + m, j + (1 << 21)))
            ref += dy[part].double().t() @ x[part].double()
        assert torch.equal(dw[i].double(), ref)
        at += m
    assert bool((y[at:] == -7).all()) and bool((dx[at:] == -7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,vocab,hidden", [(1 << 20, 1, 8), (1 << 20, 3, 8), (3, 1 << 20, 8), (3, 70, 32768), (1, 1, 8)])
def test_loss_at_its_limits(rows, vocab, hidden, dtype):
    _say("loss", rows, vocab, hidden, dtype)
    h, w, t, dloss = _inputs(rows, vocab, hidden, 7)
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dh = torch.full_like(h, -7.0)
    dw = torch.full((vocab, hidden), float("nan"), dtype=dtype, device="cuda")
    ws = _space(max(B.lm_head_loss_workspace_size(rows, vocab, hidden),
                    B.lm_head_loss_backward_workspace_size(rows, vocab, hidden)))
    B.lm_head_loss(h, w, t, loss, lse, ws)
    B.lm_head_loss_backward(h, w, t, lse, dloss, dh, dw, ws)
    torch.cuda.synchronize()
    _check_loss(loss, lse, h, w, t)
    _check_grads(dh, dw, h, w, t, lse, dloss)


@pytest.mark.parametrize("rows,vocab,hidden", [(1 << 24, 1, 1), (1 << 24, 1 << 20, 2), (3, 1 << 20, 1), (1025, 1 << 20, 3)])
def test_embedding_at_its_limits(rows, vocab, hidden):
    _say("embedding", rows, vocab, hidden)
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    ids = torch.randint(-1 if vocab > 1 else 0, vocab, (rows,), generator=g, device="cuda").to(I32)
    table = torch.randn(vocab, hidden, generator=g, device="cuda")
    out = torch.full((rows, hidden), float("nan"), device="cuda")
    B.embed(ids, table, out)
    live = ids >= 0
    ref = torch.where(live[:, None], table[ids.long().clamp(min=0)], 0.0)
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    dout = _whole(5, rows, hidden).float()
    dtable = torch.full((vocab, hidden), float("nan"), device="cuda")
    ws = _space(B.embed_backward_workspace_size(rows, vocab, hidden))
    B.embed_backward(ids, dout, dtable, ws)
    torch.cuda.synchronize()
    ref = torch.zeros(vocab, hidden, dtype=torch.float64, device="cuda")
    ref.index_add_(0, ids[live].long(), dout[live].double())
    assert torch.equal(dtable.double(), ref)
    B.embed_backward(ids, dout, dtable, ws, 1.0, True)
    torch.cuda.synchronize()
    assert torch.equal(dtable.double(), 2 * ref)


def test_calls_under_way_at_once():
    """Two streams, each with outputs and a workspace of its own."""
    shapes = [(300, 1500, 136), (900, 25000, 264)]
    streams = [torch.cuda.Stream() for _ in shapes]
    calls, alone = [], []
    for rows, vocab, hidden in shapes:
        h, w, t, dloss = _inputs(rows, vocab, hidden, rows)
        offsets = torch.tensor([0, rows // 3, rows], dtype=I32, device="cuda")
        w2 = _whole(4, 2, 264, hidden)
        loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        dh, dw = torch.empty_like(h), torch.empty(vocab, hidden, device="cuda")
        y = torch.empty(rows, 264, dtype=BF, device="cuda")
        ws = [_space(n) for n in (B.lm_head_loss_workspace_size(rows, vocab, hidden),
                                  B.lm_head_loss_backward_workspace_size(rows, vocab, hidden),
                                  B.moe_product_workspace_size(rows, 2, 264, hidden),
                                  B.embed_backward_workspace_size(rows, vocab, hidden))]

        def call(stream, h=h, w=w, t=t, dloss=dloss, offsets=offsets, w2=w2, loss=loss, lse=lse, dh=dh, dw=dw, y=y, ws=ws):
            B.lm_head_loss(h, w, t, loss, lse, ws[0], stream)
            B.lm_head_loss_backward(h, w, t, lse, dloss, dh, dw, ws[1], stream=stream)
            B.moe_product(dh, w2, offsets, y, ws[2], stream)
            B.embed_backward(t, dh, dw, ws[3], 2.0, True, stream)
            return loss, lse, dh, dw, y

        calls.append(call)
        alone.append([v.clone() for v in call(None)])
    torch.cuda.synchronize()
    for i in range(5):
        _say("at once", i)
        got = [call(s) for call, s in zip(calls, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
