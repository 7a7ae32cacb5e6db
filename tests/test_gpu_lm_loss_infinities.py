"""Gradients of lm_head_loss where weights or rows hold infinities: wherever the
definition, term by term in float64, gives an infinity, a NaN or a number, so does
the library.

A number is off by a bf16 d's 2^-8 of each term at most (and 2^-16 for the rest of
what makes d: logits of 8 products, their exponential), by the result's own
rounding, 2^-8, and by less than 2^-12 of the terms for their fp32 sums of up to
25000.
"""
import math

import pytest
import torch

from bit_moe_decode_amd import binding as B

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _sum(a, b):
    """sum_i a[i, m] b[i, n] term by term, so that 0 times an infinity is NaN."""
    return torch.stack([(a * b[:, c, None]).sum(0) for c in range(b.shape[1])], 1)


def _same(got, ref, terms):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), (int(torch.isnan(got).sum()), int(torch.isnan(ref).sum()))
    big = torch.isinf(ref)
    assert torch.equal(got[big], ref[big])
    fine = torch.isfinite(ref)
    err = (got - ref).abs()[fine]
    tol = (2.0 ** -8 + 2.0 ** -16 + 2.0 ** -12) * terms[fine] + 2.0 ** -8 * ref[fine].abs() * (1 + 2.0 ** -7)
    assert bool((err <= tol).all()), float((err - tol).max())


def _check(h, w, t, dloss, dtype):
    """Both gradients against the definition; returns the references."""
    rows, vocab = h.shape[0], w.shape[0]
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ws = torch.empty(max(B.lm_head_loss_workspace_size(rows, vocab, 8),
                         B.lm_head_loss_backward_workspace_size(rows, vocab, 8)), dtype=torch.uint8, device="cuda")
    B.lm_head_loss(h, w, t, loss, lse, ws)
    dh = torch.zeros_like(h)
    dw = torch.zeros(vocab, 8, dtype=dtype, device="cuda")
    B.lm_head_loss_backward(h, w, t, lse, dloss, dh, dw, ws)
    torch.cuda.synchronize()
    hd, wd, live = h.double(), w.double(), t >= 0
    z = _sum(hd.t(), wd.t())
    d = torch.exp(z - lse.double()[:, None])
    d[live, t[live].long()] -= 1.0
    d = torch.where(live[:, None], d * dloss.double()[:, None], 0.0)
    keep = live.nonzero()[:, 0]
    ref_h, terms_h = _sum(d.t(), wd.double()), _sum(d.t().abs(), wd.abs())
    ref_h[~live], terms_h[~live] = 0.0, 0.0
    ref_w, terms_w = _sum(d[keep], hd[keep]), _sum(d[keep].abs(), hd[keep].abs())
    _same(dh, ref_h, terms_h)
    _same(dw, ref_w, terms_w)
    return loss, ref_h, ref_w


def _inputs(rows, vocab, scale):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    h = torch.randn(rows, 8, generator=g, device="cuda").to(BF)
    w = torch.randn(vocab, 8, generator=g, device="cuda").to(BF)
    t = torch.randint(20, vocab, (rows,), generator=g, device="cuda").to(torch.int32)
    t[rows - 1] = -1
    dloss = torch.full((rows,), scale, device="cuda")
    dloss[::2] = -scale
    sign = torch.where(torch.rand(vocab, generator=g, device="cuda") < 0.5, 1.0, -1.0).to(BF)
    return h, w, t, dloss, sign


# a dloss that bf16 holds, and ones that it rounds up and down
CASES = [(r, v, s, d) for r, v in ((20, 300), (100, 300), (600, 25000)) for s in (0.5, 0.3, 0.7) for d in (BF, F32)]


@pytest.mark.parametrize("rows,vocab,scale,dtype", CASES)
def test_infinite_weight_of_a_target(rows, vocab, scale, dtype):
    """Token 7's logit is -inf in all rows; rows 3 and 4 have it as their target."""
    print("infinite weight", rows, vocab, scale, dtype, flush=True)
    h, w, t, dloss, _ = _inputs(rows, vocab, scale)
    h[:, 1], w[:, 1] = -1.0, 0.25
    w[7, 1] = math.inf
    t[3:5] = 7
    loss, dh, dw = _check(h, w, t, dloss, dtype)
    assert bool((loss[3:5] == math.inf).all())
    assert dh[3:5, 1].tolist() == [-float(d) * math.inf for d in dloss[3:5]] and bool(torch.isfinite(dw).all())


@pytest.mark.parametrize("rows,vocab,scale,dtype", CASES)
def test_infinite_rows(rows, vocab, scale, dtype):
    """Row 5's logits are infinite, that of its target, token 11, -inf."""
    print("infinite rows", rows, vocab, scale, dtype, flush=True)
    h, w, t, dloss, sign = _inputs(rows, vocab, scale)
    h[5, 2], t[5] = math.inf, 11
    w[:, 2] = sign
    w[11, 2] = -1.0
    loss, dh, dw = _check(h, w, t, dloss, dtype)
    assert float(loss[5]) == math.inf and bool(torch.isnan(dh[5]).all())
    assert float(dw[11, 2]) == -float(dloss[5]) * math.inf and bool(torch.isfinite(dw[11, 3:]).all())
