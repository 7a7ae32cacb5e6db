"""moe_sort at the most picks it takes, bitwise against torch's stable sort."""
import pytest
import torch

from bit_moe_decode_amd import binding as B

pytestmark = pytest.mark.gpu

I32 = torch.int32


@pytest.mark.parametrize("tokens,k,experts,mode", [
    (1 << 21, 8, 256, "outside"), (1 << 20, 16, 1024, "all"), (1 << 24, 1, 1, "all"),
    ((1 << 21) - 3, 8, 1000, "last")])
def test_the_most_picks(tokens, k, experts, mode):
    print("sort", tokens, k, experts, mode, flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(experts)
    ids = torch.randint(0, experts, (tokens, k), generator=g, device="cuda", dtype=I32)
    if mode == "outside":  # some in no group
        ids[torch.rand(tokens, k, generator=g, device="cuda") < 0.3] = experts
        ids[::5, 0] = -1
    if mode == "last":     # nearly all picks in one group
        ids[torch.rand(tokens, k, generator=g, device="cuda") < 0.99] = experts - 1
    offsets = torch.full((experts + 1,), -7, dtype=I32, device="cuda")
    order = torch.full((tokens * k,), -7, dtype=I32, device="cuda")
    pos = torch.full((tokens, k), -7, dtype=I32, device="cuda")
    ws = torch.empty(B.moe_sort_workspace_size(tokens, k, experts), dtype=torch.uint8, device="cuda")
    B.moe_sort(ids, experts, offsets, order, pos, ws)
    torch.cuda.synchronize()
    flat = ids.view(-1).long()
    flat = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    key, by = torch.sort(flat, stable=True)
    n = int((key < experts).sum())
    assert torch.equal(offsets.long(), torch.searchsorted(key, torch.arange(experts + 1, device="cuda")))
    assert torch.equal(order[:n].long(), by[:n])
    assert bool((order[n:] == -7).all())
    want = torch.full_like(flat, -1)
    want[by[:n]] = torch.arange(n, device="cuda")
    assert torch.equal(pos.view(-1).long(), want)
