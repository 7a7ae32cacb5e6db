"""Adapters (lora_apply) whose B holds infinities, and whose A x is near
fp32's largest number: the definition's infinities and NaN, at the places where
it has them, whether rows are taken one by one or grouped.

A x is made of whole numbers below 2^24, so it is exact in fp32; where it is
also a bf16 number its low bf16 part is 0.  Finite outputs are within
(rank + 8) * 2^-23 + 2^-16 of the terms and one bf16 rounding, as in
tests/test_gpu_lora.py.
"""
import pytest
import torch

from bit_moe_decode_amd import binding as B
from tests import test_gpu_lora as L

pytestmark = pytest.mark.gpu


def _terms(b, v, scale):
    """scale B v of every row as its terms, float64 [rows, n, rank]."""
    return scale * b.double()[None] * v.double()[:, None, :]


@pytest.mark.parametrize("rows,mr,ragged", [(8, 16, False), (16, 128, True), (70, 64, False),
                                            (300, 16, False), (300, 24, True), (65, 128, True)])
def test_infinities_in_b(rows, mr, ragged):
    print("lora, infinite B", rows, mr, ragged, flush=True)
    n, k = 264, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + mr)
    x = torch.randint(1, 3, (rows, k), generator=g, device="cuda").to(torch.bfloat16)
    x[3::7] = 0                                     # v is 0: an infinity times 0
    x[5::7, 1:] = 0                                 # v is a bf16 number
    sign = torch.randint(0, 2, (1, mr, 1), generator=g, device="cuda") * 2 - 1
    a = (sign * torch.ones(1, mr, k, device="cuda", dtype=torch.int64)).to(torch.bfloat16)
    b = torch.randn(1, n, mr, generator=g, device="cuda").to(torch.bfloat16)
    used = mr - 5 if ragged else mr
    b[0, 1, 0], b[0, 2, used - 1], b[0, 130, 7] = float("inf"), -float("inf"), float("inf")
    b[0, 131, 3] = b[0, 131, 4] = float("inf")      # of v's two signs, or of one
    b[0, n - 1, 2], b[0, n - 1, 1] = -float("inf"), float("nan")
    if ragged:
        a[:, used:], b[..., used:] = float("nan"), float("inf")
    rank = torch.tensor([used], dtype=torch.int32, device="cuda") if ragged else None
    scale = torch.full((1,), 0.5, device="cuda")
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    ids[::9] = -1
    base = torch.randn(rows, n, generator=g, device="cuda").to(torch.bfloat16)
    lora = B.make_lora(a, b, scale, rank)
    y = torch.empty_like(base)
    B.lora_apply(lora, x, ids, base, y, L._space(lora, rows))
    torch.cuda.synchronize()

    v = (a[0, :used].double()[None] * x.double()[:, None, :]).sum(2)
    t = _terms(b[0, :, :used], v, 0.5)
    t[::9] = 0
    ref = base.double() + t.sum(2)
    got = y.double()
    assert bool(torch.isinf(ref).any()) and bool(torch.isnan(ref).any())
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    fin = torch.isfinite(ref)
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf])
    size = t.abs().sum(2)
    tol = ((used + 8) * 2.0 ** -23 + 2.0 ** -16) * size
    bound = tol + 2.0 ** -8 * (ref.abs() + tol)
    assert bool(((got - ref).abs() <= bound)[fin].all())


@pytest.mark.parametrize("rows", [4, 300])
def test_the_largest_products(rows):
    """A x above bf16's largest number, 3.39e38, and below fp32's."""
    n, k, mr = 64, 64, 16
    x = torch.zeros(rows, k, device="cuda")
    x[:, 0], x[:, 1] = 3.38e38, 2e36
    x = x.to(torch.bfloat16)
    a = torch.zeros(1, mr, k, device="cuda")
    a[0, 0, :2], a[0, 1, :2] = 1.0, -1.0
    b = torch.zeros(1, n, mr, device="cuda")
    b[0, :, 0], b[0, 5:, 1] = 2.0 ** -10, 2.0 ** -12
    a, b = a.to(torch.bfloat16), b.to(torch.bfloat16)
    v = x.double() @ a[0].double().t()
    assert 3.3961776e38 < float(v[0, 0]) < 3.4028e38
    lora = B.make_lora(a, b, torch.ones(1, device="cuda"))
    base = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(base)
    B.lora_apply(lora, x, torch.zeros(rows, dtype=torch.int32, device="cuda"), base, y,
                 L._space(lora, rows))
    torch.cuda.synchronize()
    ref = v @ b[0].double().t()
    size = v.abs() @ b[0].double().abs().t()
    tol = ((mr + 8) * 2.0 ** -23 + 2.0 ** -16) * size
    assert bool(((y.double() - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol)).all())
