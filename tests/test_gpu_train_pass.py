"""One pass of a small MoE language model through the operators together, as a
training step calls them: embed, sort, gather, the experts' two products, combine,
the LM head's loss over the tied table, and every gradient back to the table and
the experts' matrices.  And what the binding refuses.

The reference computes each stage in float64 from the stage before it and rounds
where the library rounds (to bf16).  A stage's fp32 sums may put a value on the
other side of a border between two bf16, one step, 2^-7 of it, away; 12 roundings
follow each other at most (embed, up, activation, down, combine; d, dh, dy, the
activation's, dxs, dx, dtable).  So each result is within 12 2^-7 of the
reference's size, in the 2-norm, if every value moved at every stage.
"""
import pytest
import torch

from bit_moe_decode_amd import binding as B

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
STEP = 12 * 2.0 ** -7


def _space(n):
    return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")


def _bf(v):
    return v.to(BF).double()


def _act(up):
    """mid = silu(gate) up of [rows, 2 inter], in float64, rounded."""
    g, u = up.double().chunk(2, 1)
    return (g * torch.sigmoid(g) * u).to(BF)


def _act_backward(up, dmid):
    g, u = up.double().chunk(2, 1)
    s, d = torch.sigmoid(g), dmid.double()
    return torch.cat([d * u * s * (1 + g * (1 - s)), d * g * s], 1).to(BF)


class Model:
    def __init__(self, tokens, vocab, hidden, inter, experts, top_k, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        normal = lambda std, *s: (torch.randn(s, generator=g, device="cuda") * std).to(BF)  # noqa: E731
        self.table = normal(hidden ** -0.5 * 3, vocab, hidden)
        self.up, self.down = normal(hidden ** -0.5, experts, 2 * inter, hidden), normal(inter ** -0.5, experts, hidden, inter)
        self.ids = torch.randint(-1, vocab, (tokens,), generator=g, device="cuda").to(I32)
        self.targets = torch.randint(-1, vocab, (tokens,), generator=g, device="cuda").to(I32)
        z = torch.randn(tokens, experts, generator=g, device="cuda")
        top = z.topk(top_k, 1)
        self.picks, self.gates = top.indices.to(I32).contiguous(), torch.softmax(top.values, 1)
        self.scale = hidden ** 0.5

    def library(self):
        (v, h), e, inter, t = self.table.shape, self.up.shape[0], self.down.shape[2], self.ids.numel()
        k = self.picks.shape[1]
        new = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        x, xs, up, y, out = new(t, h), new(t * k, h), new(t * k, 2 * inter), new(t * k, h), new(t, h)
        offsets, order, pos = new(e + 1, dtype=I32), new(t * k, dtype=I32), new(t, k, dtype=I32)
        loss, lse = new(t, dtype=F32), new(t, dtype=F32)
        B.embed(self.ids, self.table, x, self.scale)
        B.moe_sort(self.picks, e, offsets, order, pos, _space(B.moe_sort_workspace_size(t, k, e)))
        B.moe_gather(x, pos, xs)
        B.moe_product(xs, self.up, offsets, up, _space(B.moe_product_workspace_size(t * k, e, 2 * inter, h)))
        mid = _act(up)
        B.moe_product(mid, self.down, offsets, y, _space(B.moe_product_workspace_size(t * k, e, h, inter)))
        B.moe_combine(y, pos, self.gates, out, x)
        B.lm_head_loss(out, self.table, self.targets, loss, lse, _space(B.lm_head_loss_workspace_size(t, v, h)))
        live = int((self.targets >= 0).sum())
        dloss = torch.full((t,), 1.0 / live, device="cuda")
        dout, dtable, dy, dgates = new(t, h), new(v, h, dtype=F32), new(t * k, h), new(t, k, dtype=F32)
        dmid, dup_w, ddown_w = new(t * k, inter), new(*self.up.shape, dtype=F32), new(*self.down.shape, dtype=F32)
        dxs, dx = new(t * k, h), new(t, h)
        B.lm_head_loss_backward(out, self.table, self.targets, lse, dloss, dout, dtable,
                                _space(B.lm_head_loss_backward_workspace_size(t, v, h)))
        B.moe_combine_backward(dout, y, pos, self.gates, dy, dgates)
        B.moe_product_backward(dy, mid, self.down, offsets, dmid, ddown_w,
                               _space(B.moe_product_backward_workspace_size(t * k, e, h, inter)))
        dup = _act_backward(up, dmid)
        B.moe_product_backward(dup, xs, self.up, offsets, dxs, dup_w,
                               _space(B.moe_product_backward_workspace_size(t * k, e, 2 * inter, h)))
        B.moe_gather_backward(dxs, pos, dx)
        dx += dout  # the residual
        B.embed_backward(self.ids, dx, dtable, _space(B.embed_backward_workspace_size(t, v, h)), self.scale, add=True)
        torch.cuda.synchronize()
        return dict(loss=loss, dgates=dgates, up=dup_w, down=ddown_w, table=dtable)

    def reference(self):
        table, t, e = self.table.double(), self.ids.numel(), self.up.shape[0]
        known, live = self.ids >= 0, self.targets >= 0
        x = _bf(torch.where(known[:, None], table[self.ids.long().clamp(min=0)], 0.0) * self.scale)
        up_w, down_w, gates = self.up.double(), self.down.double(), self.gates.double()
        rows = []  # (token, pick, up, mid, y) of every expert
        out = x.clone()
        for i in range(e):
            tok, pick = torch.nonzero(self.picks == i, as_tuple=True)
            up = _bf(x[tok] @ up_w[i].t())
            mid = _act(up).double()
            y = _bf(mid @ down_w[i].t())
            out.index_add_(0, tok, y * gates[tok, pick, None])
            rows.append((tok, pick, up, mid, y))
        out = _bf(out)
        z = out @ table.t()
        lse = torch.logsumexp(z, 1)
        at = self.targets.long().clamp(min=0)[:, None]
        loss = torch.where(live, lse - z.gather(1, at)[:, 0], 0.0)
        d = torch.exp(z - lse[:, None])
        d.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
        d = torch.where(live[:, None], d / live.sum(), 0.0)
        dout, dtable = _bf(d @ table), d.t() @ out
        dx, dup_w, ddown_w = torch.zeros_like(x), torch.zeros_like(up_w), torch.zeros_like(down_w)
        dgates = torch.zeros_like(gates)
        for i, (tok, pick, up, mid, y) in enumerate(rows):
            dgates[tok, pick] = (dout[tok] * y).sum(1)
            dy = _bf(dout[tok] * gates[tok, pick, None])
            ddown_w[i] = dy.t() @ mid
            dup = _act_backward(up, _bf(dy @ down_w[i])).double()
            dup_w[i] = dup.t() @ x[tok]
            dx.index_add_(0, tok, _bf(dup @ up_w[i]))
        dx = _bf(_bf(dx) + dout)
        dtable.index_add_(0, self.ids.long()[known], dx[known] * self.scale)
        return dict(loss=loss, dgates=dgates, up=dup_w, down=ddown_w, table=dtable)


@pytest.mark.parametrize("shape", [(61, 300, 72, 40, 6, 2), (600, 1003, 256, 128, 16, 4), (1, 50, 64, 64, 4, 2)])
def test_training_pass(shape):
    print("pass", shape, flush=True)
    model = Model(*shape, seed=sum(shape))
    if shape[0] == 1:
        model.ids[:], model.targets[:] = 7, 3
    got, ref = model.library(), model.reference()
    for name, want in ref.items():
        err, size = float((got[name].double() - want).norm()), float(want.norm())
        print(name, err / size, flush=True)
        assert bool(torch.isfinite(got[name]).all()) and err <= STEP * size, name


def _t(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def test_binding_refuses_tensors_that_do_not_fit():
    off = _t(4, dtype=I32)
    x, w, y, dy = _t(8, 16), _t(3, 24, 16), _t(8, 24), _t(8, 24)
    ids, table, rows = _t(8, dtype=I32), _t(50, 16), _t(8, 16)
    f = _t(8, dtype=F32)
    ws = _t(1 << 22, dtype=torch.uint8)
    for call in (
            lambda: B.moe_product(x.float(), w, off, y), lambda: B.moe_product(x, w[:, :, :8], off, y),
            lambda: B.moe_product(x, w, off[:3], y), lambda: B.moe_product(x, w, off.long(), y),
            lambda: B.moe_product(x, w, off, y[:4]), lambda: B.moe_product(x, w, off, y.half()),
            lambda: B.moe_product(x, w.cpu(), off, y), lambda: B.moe_product(x, w.transpose(0, 1), off, y),
            lambda: B.moe_product(x, w, off, y, ws.cpu()),
            lambda: B.moe_product_backward(dy, None, w, off, dw=w), lambda: B.moe_product_backward(dy, x, None, off, dx=x),
            lambda: B.moe_product_backward(dy, x, w, off, dx=x.float()),
            lambda: B.moe_product_backward(dy, x, w, off, dw=w.half()),
            lambda: B.moe_product_backward(dy[:4], x, w, off, dx=_t(8, 16)),
            lambda: B.lm_head_loss(rows, table.float(), ids, f, f.clone(), ws),
            lambda: B.lm_head_loss(rows, table, ids.long(), f, f.clone(), ws),
            lambda: B.lm_head_loss(rows, table, ids, f[:4], f.clone(), ws),
            lambda: B.lm_head_loss(rows, _t(50, 24), ids, f, f.clone(), ws),
            lambda: B.lm_head_loss_backward(rows, table, ids, f, f[:4], _t(8, 16), None, ws),
            lambda: B.lm_head_loss_backward(rows, table, ids, f, f.clone(), _t(8, 16, dtype=F32), None, ws),
            lambda: B.lm_head_loss_backward(rows, table, ids, f, f.clone(), None, _t(50, 8), ws),
            lambda: B.embed(ids.long(), table, rows), lambda: B.embed(ids, table, rows.float()),
            lambda: B.embed(ids, table, _t(8, 24)), lambda: B.embed(ids, table.half(), rows.half()),
            lambda: B.embed_backward(ids, _t(8, 24), table), lambda: B.embed_backward(ids[:4], rows, table),
            lambda: B.embed_backward(ids, rows.half(), table), lambda: B.embed_backward(ids, rows.cpu(), table)):
        with pytest.raises(B.MoeError):
            call()
