"""Host-side refusals of the products of rows grouped by expert, the LM head's
loss and the embedding lookup, with their gradients (no kernel is launched by any
call here: every call is refused, or has nothing to do)."""
import ctypes

import pytest

from bit_moe_decode_amd import binding as B

P = 1 << 32  # an aligned address; nothing reads it
BAD, NOT, WS, OK = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE, B.MOE_OK


def ptr(i):
    return P * (i + 1)


def product_shape(**kw):
    return B.ProductShape(*dict(dict(dtype=0, n_experts=16, rows=4096, n=1024, k=512), **kw).values())


def product(sh, x=ptr(0), w=ptr(1), offsets=ptr(2), y=ptr(3), ws=None, nb=0):
    return B.lib().moe_product(ctypes.byref(sh) if sh else None, x, w, offsets, y, ws, nb, None)


def product_backward(sh, dy=ptr(0), x=ptr(1), w=ptr(2), offsets=ptr(3), dx=ptr(4), dw=ptr(5), ws=None, nb=0):
    return B.lib().moe_product_backward(ctypes.byref(sh) if sh else None, dy, x, w, offsets, dx, dw, 0, ws, nb, None)


def head_shape(**kw):
    return B.HeadShape(*dict(dict(dtype=0, rows=64, vocab=1000, hidden=128), **kw).values())


def loss(sh, h=ptr(0), w=ptr(1), targets=ptr(2), loss=ptr(3), lse=ptr(4), ws=ptr(5), nb=1 << 31):
    return B.lib().lm_head_loss(ctypes.byref(sh) if sh else None, h, w, targets, loss, lse, ws, nb, None)


def loss_backward(sh, h=ptr(0), w=ptr(1), targets=ptr(2), lse=ptr(3), dloss=ptr(4), dh=ptr(5), dw=ptr(6), ws=ptr(7),
                  nb=1 << 31):
    return B.lib().lm_head_loss_backward(ctypes.byref(sh) if sh else None, h, w, targets, lse, dloss, dh, dw, 0, ws,
                                         nb, None)


def embed_shape(**kw):
    return B.EmbedShape(*dict(dict(dtype=0, rows=4000, vocab=1000, hidden=128), **kw).values())


def embed(sh, ids=ptr(0), table=ptr(1), out=ptr(2)):
    return B.lib().embed(ctypes.byref(sh) if sh else None, ids, table, 1.0, out, None)


def embed_backward(sh, ids=ptr(0), dout=ptr(1), dtable=ptr(2), ws=ptr(3), nb=1 << 31, table_dtype=0, add=0):
    return B.lib().embed_backward(ctypes.byref(sh) if sh else None, ids, dout, 1.0, table_dtype, dtable, add, ws, nb,
                                  None)


@pytest.mark.parametrize("f", [product, product_backward])
@pytest.mark.parametrize("kw,st", [
    (dict(dtype=2), NOT), (dict(dtype=-1), NOT), (dict(n_experts=0), BAD), (dict(n_experts=1025), NOT),
    (dict(rows=-1), BAD), (dict(rows=(1 << 24) + 1), NOT), (dict(n=0), BAD), (dict(n=12), NOT), (dict(n=32776), NOT),
    (dict(k=-8), BAD), (dict(k=4), NOT), (dict(k=32776), NOT)])
def test_product_shape_refusals(f, kw, st):
    assert f(product_shape(**kw)) == st
    assert B.moe_product_workspace_size(*[dict(dict(rows=4096, n_experts=16, n=1024, k=512), **kw)[i]
                                          for i in ("rows", "n_experts", "n", "k")]) == 0


@pytest.mark.parametrize("f,names", [(product, ("x", "w", "offsets", "y")),
                                     (product_backward, ("dy", "x", "w", "offsets"))])
def test_product_pointer_refusals(f, names):
    assert f(None) == BAD
    for n in names:
        assert f(product_shape(), **{n: None}) == BAD, n
        assert f(product_shape(), **{n: ptr(9) + 2}) == BAD, n
    for n in names:  # 16 bytes, offsets 4
        if n != "offsets":
            assert f(product_shape(), **{n: ptr(9) + 8}) == BAD, n


def test_product_overlaps_and_nothing_to_do():
    sh = product_shape()
    for i in range(3):
        assert product(sh, y=ptr(i) + 16) == BAD
    for i in range(4):
        assert product_backward(sh, dx=ptr(i) + 16) == BAD
        assert product_backward(sh, dw=ptr(i) + 16) == BAD
    assert product_backward(sh, dx=ptr(4), dw=ptr(4) + 1024) == BAD
    assert product_backward(sh, dx=ptr(4) + 8) == BAD and product_backward(sh, dw=ptr(5) + 8) == BAD
    assert product(product_shape(rows=0), None, None, None, None) == OK
    assert product_backward(sh, None, None, None, None, None, None) == OK
    assert product_backward(product_shape(rows=0), None, None, None, ptr(3), ptr(4), None) == OK  # dx of no rows


def test_product_workspaces():
    few, many = product_shape(n_experts=2, rows=8, n=64, k=8192), product_shape(n_experts=2, rows=9000, n=64, k=64)
    need = B.moe_product_workspace_size(8, 2, 64, 8192)
    assert need > 0 and need % 4 == 0
    assert product(few) == WS and product(few, ws=ptr(5), nb=need - 1) == WS and product(few, ws=ptr(5) + 8, nb=need) == WS
    assert product(few, ws=ptr(3), nb=need) == BAD and product(few, ws=ptr(0) + 64, nb=need) == BAD
    need = B.moe_product_backward_workspace_size(9000, 2, 64, 64)
    assert need > 0
    assert product_backward(many) == WS and product_backward(many, ws=ptr(6), nb=need - 1) == WS
    assert product_backward(many, ws=ptr(5), nb=need) == BAD


@pytest.mark.parametrize("f", [loss, loss_backward])
@pytest.mark.parametrize("kw,st", [
    (dict(dtype=2), NOT), (dict(rows=-1), BAD), (dict(rows=(1 << 20) + 1), NOT), (dict(vocab=0), BAD),
    (dict(vocab=(1 << 20) + 1), NOT), (dict(hidden=0), BAD), (dict(hidden=12), NOT), (dict(hidden=32776), NOT)])
def test_loss_shape_refusals(f, kw, st):
    assert f(head_shape(**kw)) == st
    if "dtype" not in kw:
        at = [dict(dict(rows=64, vocab=1000, hidden=128), **kw)[i] for i in ("rows", "vocab", "hidden")]
        assert B.lm_head_loss_workspace_size(*at) == 0 and B.lm_head_loss_backward_workspace_size(*at) == 0


@pytest.mark.parametrize("f,wide,words", [(loss, ("h", "w"), ("targets", "loss", "lse")),
                                          (loss_backward, ("h", "w"), ("targets", "lse", "dloss"))])
def test_loss_pointer_refusals(f, wide, words):
    sh = head_shape()
    assert f(None) == BAD
    for n in wide + words:
        assert f(sh, **{n: None}) == BAD, n
        assert f(sh, **{n: ptr(9) + 2}) == BAD, n
    for n in wide:
        assert f(sh, **{n: ptr(9) + 4}) == BAD, n
    assert f(sh, ws=None) == WS and f(sh, nb=16) == WS and f(sh, ws=ptr(9) + 8) == WS


def test_loss_overlaps_and_nothing_to_do():
    sh = head_shape()
    for i in range(3):
        assert loss(sh, loss=ptr(i) + 16) == BAD and loss(sh, lse=ptr(i) + 16) == BAD and loss(sh, ws=ptr(i) + 16) == BAD
    assert loss(sh, lse=ptr(3) + 16) == BAD
    for i in range(5):
        assert loss_backward(sh, dh=ptr(i) + 16) == BAD and loss_backward(sh, dw=ptr(i) + 16) == BAD
        assert loss_backward(sh, ws=ptr(i) + 16) == BAD
    assert loss_backward(sh, dw=ptr(5) + 16) == BAD and loss_backward(sh, dh=ptr(5) + 8) == BAD
    none = head_shape(rows=0)
    assert loss(none, None, None, None, None, None, None, 0) == OK
    assert loss_backward(sh, dh=None, dw=None) == OK
    assert loss_backward(none, None, None, None, None, None, ptr(5), None, None, 0) == OK
    assert B.lm_head_loss_workspace_size(0, 1000, 128) == 0


@pytest.mark.parametrize("f", [embed, embed_backward])
@pytest.mark.parametrize("kw,st", [
    (dict(dtype=2), NOT), (dict(rows=-1), BAD), (dict(rows=(1 << 24) + 1), NOT), (dict(vocab=0), BAD),
    (dict(vocab=(1 << 20) + 1), NOT), (dict(hidden=0), BAD), (dict(hidden=(1 << 20) + 1), NOT)])
def test_embed_shape_refusals(f, kw, st):
    assert f(embed_shape(**kw)) == st


def test_embed_refusals():
    sh = embed_shape()
    for n in ("ids", "table", "out"):
        assert embed(sh, **{n: None}) == BAD and embed(sh, **{n: ptr(9) + 2}) == BAD, n
    for n in ("ids", "dout", "dtable"):
        assert embed_backward(sh, **{n: None}) == BAD and embed_backward(sh, **{n: ptr(9) + 2}) == BAD, n
    assert embed(None) == BAD and embed_backward(None) == BAD
    assert embed(sh, out=ptr(0) + 16) == BAD and embed(sh, out=ptr(1) + 16) == BAD
    for i in range(2):
        assert embed_backward(sh, dtable=ptr(i) + 16) == BAD and embed_backward(sh, ws=ptr(i) + 16) == BAD
    assert embed_backward(sh, ws=ptr(2) + 16) == BAD
    assert embed_backward(sh, table_dtype=2) == NOT
    assert embed_backward(sh, ws=None) == WS and embed_backward(sh, nb=16) == WS
    assert embed(embed_shape(rows=0), None, None, None) == OK
    assert embed_backward(embed_shape(rows=0), None, None, None, None, 0, add=1) == OK
    assert B.embed_backward_workspace_size(1024, 1000, 128) == 0 and B.embed_backward_workspace_size(1025, 1000, 128) > 0


def _big(*shape, dtype="bfloat16"):
    import torch
    return torch.empty(shape, dtype=getattr(torch, dtype), device="meta")


@pytest.mark.parametrize("call", [
    lambda n: B.moe_product_workspace_size(n, 16, 64, 64),
    lambda n: B.moe_product_backward_workspace_size(n, 16, 64, 64),
    lambda n: B.lm_head_loss_workspace_size(n, 500, 64),
    lambda n: B.lm_head_loss_backward_workspace_size(n, 500, 64),
    lambda n: B.embed_backward_workspace_size(n, 500, 64),
    lambda n: B.moe_product(_big(n, 8), _big(4, 8, 8), _big(5, dtype="int32"), _big(n, 8)),
    lambda n: B.moe_product_backward(_big(n, 8), None, _big(4, 8, 8), _big(5, dtype="int32"), dx=_big(n, 8)),
    lambda n: B.lm_head_loss(_big(n, 8), _big(40, 8), _big(n, dtype="int32"), _big(n, dtype="float32"),
                             _big(n, dtype="float32"), None),
    lambda n: B.lm_head_loss_backward(_big(n, 8), _big(40, 8), _big(n, dtype="int32"), _big(n, dtype="float32"),
                                      _big(n, dtype="float32"), dh=_big(n, 8)),
    lambda n: B.embed(_big(n, dtype="int32"), _big(40, 1), _big(n, 1)),
    lambda n: B.embed_backward(_big(n, dtype="int32"), _big(n, 1), _big(40, 1)),
])
def test_sizes_past_32_bits_are_not_cut(call):
    """2^32 + 16 rows are not the 16 of their low bits."""
    with pytest.raises(B.MoeError, match="sizes of"):
        call((1 << 32) + 16)
