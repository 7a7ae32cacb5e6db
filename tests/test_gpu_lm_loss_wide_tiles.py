"""The loss and its gradients in the largest tiles: 256 x 256 for the loss, for d and
for both gradients, the vocabulary in two pieces, and a last tile of rows of each
height (of 1..32, 33..64, 65..128 and more rows), whatever form dw has.  Bounds as
in test_gpu_lm_loss.py.
"""
import pytest
import torch

from bit_moe_decode_amd import binding as B
from tests.test_gpu_lm_loss import _check_grads, _check_loss, _inputs

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
VOCAB, HIDDEN = 33000, 264


@pytest.mark.parametrize("rows,live", [(2048 + 30, 2048 + 17), (2048 + 62, 2048 + 40), (2048 + 126, 2048 + 100),
                                       (2048 + 250, 2048 + 200)])
def test_loss_and_gradients_in_wide_tiles(rows, live):
    h, w, t, dloss = _inputs(rows, VOCAB, HIDDEN, rows, none=0.0)
    order = torch.randperm(rows, device="cuda", generator=torch.Generator(device="cuda").manual_seed(rows))
    t[order[live:]] = -1
    ws = torch.empty(max(B.lm_head_loss_workspace_size(rows, VOCAB, HIDDEN),
                         B.lm_head_loss_backward_workspace_size(rows, VOCAB, HIDDEN)), dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    print("wide tiles", rows, live, flush=True)
    B.lm_head_loss(h, w, t, loss, lse, ws)
    torch.cuda.synchronize()
    _check_loss(loss, lse, h, w, t)
    for dtype in (BF, F32):
        for add in (False, True):
            print("wide tiles", rows, live, dtype, add, flush=True)
            base = torch.randn(VOCAB, HIDDEN, device="cuda").to(dtype) if add else None
            dh = torch.full_like(h, -7.0)
            dw = base.clone() if add else torch.full((VOCAB, HIDDEN), float("nan"), dtype=dtype, device="cuda")
            B.lm_head_loss_backward(h, w, t, lse, dloss, dh, dw, ws, add)
            torch.cuda.synchronize()
            _check_grads(dh, dw, h, w, t, lse, dloss, base)
