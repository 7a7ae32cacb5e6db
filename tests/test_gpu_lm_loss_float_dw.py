"""The fp32 dw of lm_head_loss_backward against the definition in float64, through
the C ABI: it enters its sums as two bf16, so that it is an fp32 result and not a
bf16 one's size of error in fp32.

h holds one number a row, in column r % hidden: a logit is one product, exact in
fp32, and column c's sums of dw are those of rows / hidden rows, the other terms
being 0, which an addition leaves exact.  So with n such rows

  p is off by 2^-22 (2 + |z - lse|) of it (the difference's rounding, that of its
  product with log2 e and the exponential's), d by that and 2^-22 of it;
  the two bf16 of d leave 2^-8 of 2^-8 of it, 2^-16, or what is below 2^-126;
  a sum of 2 n terms (and dw's old value) is off by 2^-23 of sum|terms| an addition.

A bf16 d would be off by up to 2^-8: at n = 1 the bound is below a hundredth of that.
"""
import pytest
import torch

from bit_moe_decode_amd import binding as B

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

# the small tiles of 16, 32 and 64 rows, of more; large ones of d with dw's of 128
# and of 256, rows placed by counting and by a sort, one piece and two
SHAPES = [(1, 1000, 64), (20, 4099, 72), (50, 513, 128), (130, 1003, 136), (600, 25000, 200), (5000, 9000, 264),
          (2300, 33000, 264), (30000, 2500, 512)]


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("rows,vocab,hidden", SHAPES)
def test_float_dw_is_of_float_accuracy(rows, vocab, hidden, add):
    print("float dw", rows, vocab, hidden, add, flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + vocab)
    at = torch.arange(rows, device="cuda") % hidden
    h = torch.zeros(rows, hidden, device="cuda")
    h[torch.arange(rows, device="cuda"), at] = torch.randn(rows, generator=g, device="cuda") * 2
    h = h.to(BF)
    w = torch.randn(vocab, hidden, generator=g, device="cuda").to(BF)
    t = torch.randint(-1, vocab, (rows,), generator=g, device="cuda").to(torch.int32)
    dloss = torch.rand(rows, generator=g, device="cuda") - 0.25
    z = h[torch.arange(rows, device="cuda"), at].double()[:, None] * w.double()[:, at].t()
    lse = torch.logsumexp(z, 1).float()
    base = torch.randn(vocab, hidden, generator=g, device="cuda") if add else None
    dw = base.clone() if add else torch.full((vocab, hidden), float("nan"), device="cuda")
    ws = torch.empty(B.lm_head_loss_backward_workspace_size(rows, vocab, hidden), dtype=torch.uint8, device="cuda")
    B.lm_head_loss_backward(h, w, t, lse, dloss, None, dw, ws, add)
    torch.cuda.synchronize()
    x = z - lse.double()[:, None]
    del z
    p = torch.exp(x)
    d = p.clone()
    live = t >= 0
    d[live, t[live].long()] -= 1.0
    scale = torch.where(live, dloss.double(), 0.0)[:, None]
    d *= scale
    off = p * 2.0 ** -22 * (2 + x.abs()) * scale.abs() + (2.0 ** -22 + 2.0 ** -16) * d.abs() + 2.0 ** -124 * live[:, None]
    del p, x
    hd = h.double()
    ref, terms, part = d.t() @ hd, d.abs().t() @ hd.abs(), off.t() @ hd.abs()
    if add:
        ref, terms = ref + base.double(), terms + base.double().abs()
    c = 2 * -(-rows // hidden) + 1
    err, tol = (dw.double() - ref).abs(), part + c * 2.0 ** -23 * (terms + part)
    assert bool(torch.isfinite(dw).all())
    assert bool((err <= tol).all()), (float((err - tol).max()), float(err.norm() / ref.norm()))


def test_dh_is_the_same_beside_either_dw():
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    h, w = (torch.randn(*s, generator=g, device="cuda").to(BF) for s in ((700, 200), (21000, 200)))
    t = torch.randint(-1, 21000, (700,), generator=g, device="cuda").to(torch.int32)
    lse = torch.logsumexp(h.double() @ w.double().t(), 1).float()
    dloss = torch.rand(700, generator=g, device="cuda")
    ws = torch.empty(B.lm_head_loss_backward_workspace_size(700, 21000, 200), dtype=torch.uint8, device="cuda")
    got = []
    for dtype in (BF, F32, None):
        dh = torch.full_like(h, -7.0)
        dw = None if dtype is None else torch.zeros(21000, 200, dtype=dtype, device="cuda")
        B.lm_head_loss_backward(h, w, t, lse, dloss, dh, dw, ws)
        got.append(dh)
    torch.cuda.synchronize()
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
