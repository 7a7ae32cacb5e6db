"""The binding's structs of weights refuse tensors that the kernels would read
past or misread: make_matrix.  No kernel runs."""
import pytest
import torch

from bit_moe_decode_amd import binding as B

U8, F32, BF, F8 = torch.uint8, torch.float32, torch.bfloat16, torch.float8_e4m3fn


def z(dtype, *shape):
    return torch.zeros(shape, dtype=U8 if dtype is F8 else dtype).view(dtype)


@pytest.mark.parametrize("fmt,codes,scales", [
    (B.FMT_Q1, z(U8, 256, 3, 18), None), (B.FMT_FP8, z(U8, 256, 384), z(F32, 2, 3)),
    (B.FMT_FP8, z(F8, 256, 384), z(F32, 2, 3)), (B.FMT_BF16, z(BF, 256, 384), None)])
def test_matrices(fmt, codes, scales):
    m = B.make_matrix(fmt, 256, 384, codes, scales)
    assert (m.fmt, m.n, m.k, m.codes) == (fmt, 256, 384, codes.data_ptr())
    assert m.scales == (None if scales is None else scales.data_ptr())
    assert m.tensors == (codes, scales)


@pytest.mark.parametrize("fmt,codes,scales", [
    (B.FMT_FP8, z(U8, 256, 384), None),                       # no scales
    (B.FMT_FP8, z(U8, 384, 256), z(F32, 2, 3)),               # transposed
    (B.FMT_FP8, z(U8, 384, 256).t(), z(F32, 2, 3)),           # a transposed view
    (B.FMT_FP8, z(U8, 256, 400)[:, :384], z(F32, 2, 3)),      # a part of wider rows
    (B.FMT_FP8, z(U8, 255, 384), z(F32, 2, 3)),               # too short
    (B.FMT_FP8, z(U8, 256, 384), z(F32, 2, 2)), (B.FMT_FP8, z(U8, 256, 384), z(F32, 3, 2).t()),
    (B.FMT_FP8, z(U8, 256, 384), z(BF, 2, 3)), (B.FMT_FP8, z(BF, 256, 384), z(F32, 2, 3)),
    (B.FMT_Q1, z(U8, 256, 3, 16), None), (B.FMT_Q1, z(U8, 256, 2, 18), None),
    (B.FMT_Q1, z(U8, 128, 3, 18), None), (B.FMT_Q1, z(U8, 256, 54), None),
    (B.FMT_Q1, z(F32, 256, 3, 18), None), (B.FMT_Q1, z(U8, 256, 6, 18)[:, ::2], None),
    (B.FMT_BF16, z(torch.float16, 256, 384), None), (B.FMT_BF16, z(BF, 384, 256).t(), None),
    (B.FMT_BF16, z(BF, 256, 383), None)])
def test_matrices_that_are_refused(fmt, codes, scales):
    with pytest.raises(B.MoeError) as e:
        B.make_matrix(fmt, 256, 384, codes, scales)
    assert e.value.status == B.MOE_ERR_INVALID_ARG
