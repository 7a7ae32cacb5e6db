"""Host-side refusals of the operators on grouped rows and of the adapters (no
kernel is launched by any call here: every call is refused, or has nothing to
do)."""
import ctypes

import pytest

from bit_moe_decode_amd import binding as B

P = 1 << 24  # an aligned address; nothing reads it


def ptr(i):
    return P * (i + 1)


def sort(tokens=4, top_k=8, n=16, ids=ptr(0), offsets=ptr(1), order=ptr(2), pos=ptr(3), ws=None, nb=0):
    return B.lib().moe_sort(ids, tokens, top_k, n, offsets, order, pos, ws, nb, None)


@pytest.mark.parametrize("kw,st", [
    (dict(tokens=-1), B.MOE_ERR_INVALID_ARG), (dict(top_k=0), B.MOE_ERR_INVALID_ARG),
    (dict(n=0), B.MOE_ERR_INVALID_ARG), (dict(top_k=17), B.MOE_ERR_UNSUPPORTED),
    (dict(n=1025), B.MOE_ERR_UNSUPPORTED), (dict(tokens=(1 << 21) + 1), B.MOE_ERR_UNSUPPORTED),
    (dict(ids=None), B.MOE_ERR_INVALID_ARG), (dict(offsets=None), B.MOE_ERR_INVALID_ARG),
    (dict(order=None), B.MOE_ERR_INVALID_ARG), (dict(pos=None), B.MOE_ERR_INVALID_ARG),
    (dict(ids=ptr(0) + 2), B.MOE_ERR_INVALID_ARG), (dict(pos=ptr(2) + 64), B.MOE_ERR_INVALID_ARG),
    (dict(offsets=ptr(0) + 4), B.MOE_ERR_INVALID_ARG),
    (dict(tokens=40960), B.MOE_ERR_WORKSPACE),
    (dict(tokens=40960, ws=ptr(4), nb=16), B.MOE_ERR_WORKSPACE),
    (dict(tokens=40960, ws=ptr(2) + 64, nb=1 << 20), B.MOE_ERR_INVALID_ARG)])
def test_sort_refusals(kw, st):
    assert sort(**kw) == st


def test_sort_workspace_size():
    assert B.moe_sort_workspace_size(16, 8, 256) == 0
    assert B.moe_sort_workspace_size(40960, 8, 256) > 0
    assert B.moe_sort_workspace_size(4096, 17, 256) == 0
    assert B.moe_sort_workspace_size(-1, 8, 256) == 0


SHAPE = dict(dtype=0, tokens=4, top_k=8, hidden=64, rows=32)


def shape(**kw):
    return B.RowShape(*dict(SHAPE, **kw).values())


def gather(sh, x=ptr(0), pos=ptr(1), xs=ptr(2)):
    return B.lib().moe_gather(sh, x, pos, xs, None)


def gather_backward(sh, dxs=ptr(0), pos=ptr(1), dx=ptr(2)):
    return B.lib().moe_gather_backward(sh, dxs, pos, dx, None)


def combine(sh, y=ptr(0), pos=ptr(1), gates=ptr(2), add=ptr(3), out=ptr(4)):
    return B.lib().moe_combine(sh, y, pos, gates, add, out, None)


def combine_backward(sh, dout=ptr(0), y=ptr(1), pos=ptr(2), gates=ptr(3), dy=ptr(4), dg=ptr(5)):
    return B.lib().moe_combine_backward(sh, dout, y, pos, gates, dy, dg, None)


@pytest.mark.parametrize("f", [gather, gather_backward, combine, combine_backward])
@pytest.mark.parametrize("kw,st", [
    (dict(dtype=2), B.MOE_ERR_UNSUPPORTED), (dict(dtype=-1), B.MOE_ERR_UNSUPPORTED),
    (dict(tokens=-1), B.MOE_ERR_INVALID_ARG), (dict(top_k=0), B.MOE_ERR_INVALID_ARG),
    (dict(hidden=0), B.MOE_ERR_INVALID_ARG), (dict(rows=-1), B.MOE_ERR_INVALID_ARG),
    (dict(top_k=17), B.MOE_ERR_UNSUPPORTED), (dict(tokens=1 << 22), B.MOE_ERR_UNSUPPORTED),
    (dict(hidden=(1 << 20) + 1), B.MOE_ERR_UNSUPPORTED), (dict(tokens=0), B.MOE_OK)])
def test_row_shape_refusals(f, kw, st):
    assert f(ctypes.byref(shape(**kw))) == st


@pytest.mark.parametrize("f,names", [
    (gather, ("x", "pos", "xs")), (gather_backward, ("dxs", "pos", "dx")),
    (combine, ("y", "pos", "gates", "out")), (combine_backward, ("dout", "y", "pos", "gates", "dy", "dg"))])
def test_row_pointer_refusals(f, names):
    sh = ctypes.byref(shape())
    assert f(None) == B.MOE_ERR_INVALID_ARG
    for n in names:
        assert f(sh, **{n: None}) == B.MOE_ERR_INVALID_ARG, n
        assert f(sh, **{n: ptr(9) + 2}) == B.MOE_ERR_INVALID_ARG, n  # misaligned


def test_row_overlaps():
    sh = ctypes.byref(shape())
    bad = B.MOE_ERR_INVALID_ARG
    assert gather(sh, xs=ptr(0) + 256) == bad
    assert gather(sh, xs=ptr(1)) == bad
    assert gather_backward(sh, dx=ptr(0) + 16) == bad
    assert gather_backward(sh, dx=ptr(1)) == bad
    assert combine(sh, out=ptr(0)) == bad
    assert combine(sh, out=ptr(1)) == bad
    assert combine(sh, out=ptr(2)) == bad
    assert combine(sh, out=ptr(3) + 16) == bad  # add itself is allowed, a shifted one is not
    assert combine(sh, add=ptr(3) + 8) == bad
    for a in range(4):
        assert combine_backward(sh, dy=ptr(a)) == bad
        assert combine_backward(sh, dg=ptr(a)) == bad
    assert combine_backward(sh, dg=ptr(4) + 16) == bad


def cfg(**kw):
    base = dict(hidden=512, inter=256, n_experts=32, top_k=8, shared_inter=256, max_rows=8,
                rms_eps=1e-6, routed_fmt=B.FMT_FP8, shared_fmt=B.FMT_FP8, flags=0, act_fmt=B.ACT_FP8)
    base.update(kw)
    return B.Config(*base.values())


def weights(**kw):
    w = B.Weights()
    w.rms_gamma = ptr(10)
    for i, n in enumerate(("gate", "up", "down", "sh_gate", "sh_up", "sh_down")):
        setattr(w, n, B.Tensor(ptr(20 + i), ptr(30 + i)))
    for n, v in kw.items():
        setattr(w, n, v)
    return w


def wide(c=None, x=ptr(0), tokens=20, ids=ptr(1), gates=ptr(2), w=None, out=ptr(3), ws=ptr(4), nb=None):
    c = c or cfg()
    nb = B.moe_wide_workspace_size(c, tokens) if nb is None else nb
    return B.lib().moe_wide_step(ctypes.byref(c), x, tokens, ids, gates,
                                 ctypes.byref(w or weights()), out, ws, nb, None)


@pytest.mark.parametrize("kw", [dict(routed_fmt=B.FMT_MXFP4), dict(routed_fmt=B.FMT_Q1),
                                dict(act_fmt=B.ACT_BF16), dict(hidden=500), dict(top_k=4),
                                dict(n_experts=24), dict(shared_inter=128)])
def test_wide_unsupported_configs(kw):
    assert B.moe_wide_workspace_size(cfg(**kw), 16) == 0
    assert wide(cfg(**kw), nb=1 << 30) == B.MOE_ERR_UNSUPPORTED


def test_wide_refusals():
    bad = B.MOE_ERR_INVALID_ARG
    assert B.moe_wide_workspace_size(cfg(), 65537) == 0
    assert wide(tokens=65537, nb=1 << 40) == B.MOE_ERR_UNSUPPORTED
    assert wide(tokens=-1, nb=1 << 30) == bad
    assert wide(tokens=0) == B.MOE_OK
    for n in ("x", "ids", "gates", "out"):
        assert wide(**{n: None}) == bad, n
        assert wide(**{n: ptr(8) + 2}) == bad, n
    assert wide(w=weights(rms_gamma=None)) == bad
    assert wide(w=weights(down=B.Tensor(ptr(22), None))) == bad
    assert wide(w=weights(sh_up=B.Tensor(ptr(24) + 8, ptr(34)))) == bad
    assert wide(ws=None) == B.MOE_ERR_WORKSPACE
    assert wide(ws=ptr(4) + 16) == B.MOE_ERR_WORKSPACE
    assert wide(nb=B.moe_wide_workspace_size(cfg(), 20) - 1) == B.MOE_ERR_WORKSPACE
    assert wide(out=ptr(0) + 1024) == bad   # overlaps x
    assert wide(out=ptr(1)) == bad          # the picks
    assert wide(out=ptr(2)) == bad          # the gates
    assert wide(x=ptr(4) + 256) == bad      # in the workspace


def lora_set(**kw):
    base = dict(n_adapters=4, max_rank=16, n=256, k=512, a=ptr(10), b=ptr(11), rank=None, scale=ptr(12))
    base.update(kw)
    return B.LoraSet(*base.values())


def apply(l=None, x=ptr(0), ids=ptr(1), rows=5, base=ptr(2), y=ptr(3), ws=ptr(4), nb=1 << 22):
    return B.lib().lora_apply(ctypes.byref(l or lora_set()), x, ids, rows, base, y, ws, nb, None)


@pytest.mark.parametrize("kw,st", [
    (dict(n_adapters=-1), B.MOE_ERR_INVALID_ARG), (dict(n_adapters=1025), B.MOE_ERR_UNSUPPORTED),
    (dict(max_rank=0), B.MOE_ERR_UNSUPPORTED), (dict(max_rank=12), B.MOE_ERR_UNSUPPORTED),
    (dict(max_rank=136), B.MOE_ERR_UNSUPPORTED), (dict(n=-8), B.MOE_ERR_INVALID_ARG),
    (dict(n=100), B.MOE_ERR_UNSUPPORTED), (dict(k=0), B.MOE_ERR_INVALID_ARG),
    (dict(k=96), B.MOE_ERR_UNSUPPORTED), (dict(k=32832), B.MOE_ERR_UNSUPPORTED),
    (dict(a=None), B.MOE_ERR_INVALID_ARG), (dict(b=ptr(11) + 8), B.MOE_ERR_INVALID_ARG),
    (dict(scale=None), B.MOE_ERR_INVALID_ARG), (dict(rank=ptr(13) + 1), B.MOE_ERR_INVALID_ARG)])
def test_lora_set_refusals(kw, st):
    assert apply(lora_set(**kw)) == st
    if st == B.MOE_ERR_UNSUPPORTED:
        assert B.lora_workspace_size(lora_set(**kw), 5) == 0


def test_lora_refusals():
    bad = B.MOE_ERR_INVALID_ARG
    assert B.lib().lora_apply(None, ptr(0), ptr(1), 1, ptr(2), ptr(3), ptr(4), 1 << 20, None) == bad
    for n in ("x", "ids", "base", "y"):
        assert apply(**{n: None}) == bad, n
        assert apply(**{n: ptr(8) + 2}) == bad, n
    assert apply(rows=-1) == bad
    assert apply(rows=(1 << 20) + 1) == B.MOE_ERR_UNSUPPORTED
    assert apply(rows=0) == B.MOE_OK
    assert apply(lora_set(n=0)) == B.MOE_OK
    assert apply(ws=None) == B.MOE_ERR_WORKSPACE
    assert apply(ws=ptr(4) + 8) == B.MOE_ERR_WORKSPACE
    assert apply(nb=B.lora_workspace_size(lora_set(), 5) - 1) == B.MOE_ERR_WORKSPACE
    assert apply(y=ptr(0) + 64) == bad
    assert apply(y=ptr(1)) == bad
    assert apply(y=ptr(2) + 64) == bad  # base itself is allowed, a shifted one is not
    assert apply(ws=ptr(0) + 64) == bad
    assert apply(ws=ptr(3) + 64) == bad
    assert apply(ws=ptr(2) + 64) == bad


def test_gemv_lora_refusals():
    def call(l=None, fmt=B.FMT_FP8, n=256, k=512, rows=3, x=ptr(0), ids=ptr(1), y=ptr(3), ws=ptr(4),
             nb=1 << 22):
        m = B.LowbitMatrix(fmt, n, k, ptr(5), ptr(6))
        return B.lib().lowbit_gemv_lora(ctypes.byref(m), ctypes.byref(l or lora_set()), x, ids, rows,
                                        y, ws, nb, None)

    bad = B.MOE_ERR_INVALID_ARG
    assert call(rows=9) == B.MOE_ERR_UNSUPPORTED
    assert call(rows=0) == B.MOE_OK
    assert call(fmt=B.FMT_MXFP4) == B.MOE_ERR_UNSUPPORTED
    assert call(lora_set(n=128)) == bad     # not the projection's
    assert call(lora_set(k=256)) == bad
    assert call(lora_set(max_rank=4)) == B.MOE_ERR_UNSUPPORTED
    assert call(x=None) == bad
    assert call(ids=None) == bad
    assert call(y=ptr(0) + 64) == bad
    assert call(ws=None) == B.MOE_ERR_WORKSPACE
    assert call(nb=15) == B.MOE_ERR_WORKSPACE


def test_lora_refuses_wide_outputs_and_a_workspace_on_the_ids():
    assert apply(lora_set(n=(1 << 20) + 8)) == B.MOE_ERR_UNSUPPORTED
    assert B.lora_workspace_size(lora_set(n=1 << 20), 5) > 0
    assert apply(ids=ptr(4) + 16) == B.MOE_ERR_INVALID_ARG


def test_binding_refuses_host_tensors():
    import torch
    ids = torch.zeros(4, 8, dtype=torch.int32)
    with pytest.raises(B.MoeError):
        B.moe_sort(ids, 16, torch.zeros(17, dtype=torch.int32), ids.view(-1).clone(), ids.clone())
    with pytest.raises(B.MoeError):
        B.make_lora(torch.zeros(1, 8, 64, dtype=torch.bfloat16), torch.zeros(1, 8, 8, dtype=torch.bfloat16),
                    torch.zeros(1))
