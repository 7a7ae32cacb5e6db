"""The binding's structs of weights refuse tensors that the kernels would read
past or misread: make_matrix, and moe_wide_step for make_weights'.  No kernel
runs."""
import gc
import os
import subprocess
import sys
import weakref

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


H, I, E, SHARED = 256, 384, 16, 384


def weights(shared=True, **kw):
    """make_weights of a small layer; kw replaces tensors: gamma, gate_c, sh_down_s, .."""
    def mats(pre, lead):
        out = []
        for name, n, k in (("gate", I, H), ("up", I, H), ("down", H, I)):
            out.append((kw.get(f"{pre}{name}_c", z(U8, *lead, n, k)),
                        kw.get(f"{pre}{name}_s", z(F32, *lead, n // 128, k // 128))))
        return out
    return B.make_weights(kw.get("gamma", z(BF, H)), None, mats("", (E,)), mats("sh_", (1,)) if shared else None)


def wide(w, shared=SHARED, **kw):
    """The error of a call on the CPU, where every call is refused."""
    c = dict(hidden=H, inter=I, n_experts=E, top_k=8, shared_inter=shared, max_rows=8, rms_eps=1e-6,
             routed_fmt=B.FMT_FP8, shared_fmt=B.FMT_FP8, flags=0, act_fmt=B.ACT_FP8)
    c.update(kw)
    x = z(BF, 20, c["hidden"])
    with pytest.raises(B.MoeError) as e:
        B.moe_wide_step(B.Config(*c.values()), x, z(torch.int32, 20, 8), z(F32, 20, 8), w, z(BF, 20, c["hidden"]), None)
    assert e.value.status == B.MOE_ERR_INVALID_ARG
    return str(e.value)


ONLY_DEVICE = "not on the current device"  # all that is wrong with a call on the CPU


def test_wide_weights():
    assert ONLY_DEVICE in wide(weights())
    assert ONLY_DEVICE in wide(weights(shared=False), shared=0)
    assert ONLY_DEVICE in wide(weights(gate_c=z(F8, E, I, H)))
    one = dict(sh_gate_c=z(U8, I, H), sh_up_c=z(U8, I, H), sh_down_c=z(U8, H, I), sh_gate_s=z(F32, 3, 2),
               sh_up_s=z(F32, 3, 2), sh_down_s=z(F32, 2, 3))
    assert ONLY_DEVICE in wide(weights(**one))
    assert ONLY_DEVICE in wide(B.Weights())  # addresses alone: the caller's word


@pytest.mark.parametrize("name,t", [
    ("gamma", z(BF, H - 8)), ("gamma", z(F32, H)), ("gate_c", z(U8, E, H, I)), ("gate_c", z(U8, E - 1, I, H)),
    ("gate_c", z(U8, E * I, H)), ("up_c", z(U8, E, H, I).transpose(1, 2)), ("up_c", z(BF, E, I, H)),
    ("down_c", z(U8, E, H, I + 128)[..., :I]), ("gate_s", None), ("up_s", z(F32, E, 2, 3)),
    ("down_s", z(torch.float64, E, 2, 3)), ("sh_gate_c", z(U8, 1, H, I)), ("sh_up_s", None),
    ("sh_down_c", z(U8, H, I - 128)), ("sh_down_s", z(F32, 2, 2))])
def test_wide_weights_that_are_refused(name, t):
    e = wide(weights(**{name: t})) if t is not None or "sh_" not in name else None
    if e is None:  # make_weights itself takes no shared matrix without scales
        with pytest.raises(AttributeError):
            weights(**{name: t})
    else:
        assert ONLY_DEVICE not in e and "is not a contiguous" in e


def test_wide_weights_of_two_configurations():
    w = weights()
    for _ in range(2):  # a call that found them right does not speak for another configuration's
        assert ONLY_DEVICE in wide(w)
        assert ONLY_DEVICE not in wide(w, n_experts=32)
        assert ONLY_DEVICE in wide(w, shared=0)


def test_wide_weights_of_another_layer():
    assert ONLY_DEVICE not in wide(weights(), n_experts=32)
    assert ONLY_DEVICE not in wide(weights(), hidden=512)
    assert ONLY_DEVICE not in wide(weights(), inter=256, shared=256)
    assert "no shared expert" in wide(weights(shared=False))


def test_structs_keep_their_tensors():
    codes = z(U8, E, I, H)
    gone = weakref.ref(codes)
    w = weights(gate_c=codes)
    del codes
    gc.collect()
    assert gone() is not None and w.gate.codes == gone().data_ptr()
    del w
    gc.collect()
    assert gone() is None


def test_the_binding_loads_without_torch():
    """As far as it takes no tensors: the library, its sizes, its statuses."""
    code = ("import sys; sys.modules['torch'] = None\n"
            "from bit_moe_decode_amd import binding as B\n"
            "c = B.Config(256, 128, 32, 8, 0, 8, 1e-6, B.FMT_FP8, B.FMT_FP8, 0, B.ACT_FP8)\n"
            "assert B.workspace_size(c) > 0 and B.moe_wide_workspace_size(c, 20) > 0\n"
            "assert 'ok' in B.status_string(B.MOE_OK)\n"
            "assert 'moe_sort' in B.declared_functions()\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-500:]
