"""Rows without an adapter keep their projection's bits, the sign of a zero and
a NaN's own bits among them, in every form: taken one by one, grouped, in
place, and in the GEMVs' epilogue."""
import pytest
import torch

from bit_moe_decode_amd import binding as B
from bit_moe_decode_amd import synth as S
from tests import test_gpu_lora as L

pytestmark = pytest.mark.gpu


def _bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("rows,adapters", [(5, 3), (300, 3), (4, 0), (300, 0)])
def test_bits_of_the_base(rows, adapters):
    print("lora, rows without an adapter", rows, adapters, flush=True)
    n, k, mr = 264, 128, 16
    a, b, scale, _ = L._adapters(max(adapters, 1), mr, n, k, rows, False)
    lora = B.make_lora(a[:adapters].contiguous(), b[:adapters].contiguous(), scale[:adapters].contiguous())
    base = S.make_x(rows, n, seed=rows).cuda()
    base[:, ::3] = -0.0
    _bits(base)[:, 1::9] = 0x7FA5  # a NaN whose payload an addition would change
    ids = torch.arange(rows, device="cuda", dtype=torch.int32) % (adapters + 1) - 1  # -1: none
    ids[1::5] = adapters
    none = (ids < 0) | (ids >= adapters)
    assert bool(none.any())
    x = S.make_x(rows, k, seed=1).cuda()
    y = torch.zeros_like(base)
    B.lora_apply(lora, x, ids, base, y, L._space(lora, rows))
    same = base.clone()
    B.lora_apply(lora, x, ids, same, same, L._space(lora, rows))
    torch.cuda.synchronize()
    assert torch.equal(_bits(y[none]), _bits(base[none]))
    assert torch.equal(_bits(same[none]), _bits(base[none]))
    assert torch.equal(_bits(same), _bits(y))


@pytest.mark.parametrize("fmt,rows,n,k", L.GEMVS)
def test_bits_of_the_gemv(fmt, rows, n, k):
    """x of zeros of either sign: sums that are zeros of either sign, too."""
    print("gemv, rows without an adapter", fmt, rows, n, k, flush=True)
    codes, scales = L._projection(fmt, n, k, n + k)
    a, b, scale, _ = L._adapters(2, 16, n, k, rows, False)
    lora = B.make_lora(a, b, scale)
    m = B.make_matrix(fmt, n, k, codes, scales)
    x = S.make_x(rows, k, seed=rows + 3).cuda()
    x[rows // 2:] = -0.0
    ids = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    y = torch.full((rows, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    B.lowbit_gemv_lora(m, lora, x, ids, y, L._space(lora, rows))
    plain = torch.empty_like(y)
    assert B.lib().lowbit_gemv(m, x.data_ptr(), rows, plain.data_ptr(), None) == B.MOE_OK
    torch.cuda.synchronize()
    assert torch.equal(_bits(y), _bits(plain))
