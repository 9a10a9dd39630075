"""The gate's gradient at masked experts, whose logit is -inf: their weight is 0, so their entries
count as none whatever dw holds.  Where the softmax runs over nothing else (every chosen logit with
renormalize, every logit without) the token's gradient is 0, and no other token sees it."""
import pytest
import torch

import combine_moe_route_count_amd as moe
from _gpu_util import DEV, note

pytestmark = pytest.mark.gpu


# every group width and list length of the kernel: 16 lanes up to 64 logits, 64 lanes past that, and
# 16 again for many tokens
@pytest.mark.parametrize("T,E", [(9, 4), (9, 20), (9, 50), (9, 100), (9, 200), (9, 400), (9, 1000), (4099, 128),
                                 (4099, 256)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
def test_masked_token_with_entries_in_range(T, E, dt, renorm):
    note(f"masked token {T} {E} {dt} {renorm}")
    g = torch.Generator().manual_seed(E)
    K = 4
    logits = torch.randn((T, E), generator=g).to(dt).to(DEV)
    idx = torch.argsort(torch.rand((T, E), generator=g), 1)[:, :K].int().to(DEV)
    dw = torch.randn((T, K), generator=g).to(DEV)
    want = moe.gate_backward(logits, idx, dw, renormalize=renorm)
    dead = [1, 4, T - 1]
    for bad in (float("nan"), float("inf"), float("-inf"), 1.0):
        l, d = logits.clone(), dw.clone()
        l[dead] = -torch.inf
        d[dead] = 0.0
        d[dead, 2] = bad
        got = moe.gate_backward(l, idx, d, renormalize=renorm)
        assert (got[dead] == 0).all(), (bad, got[dead])
        live = torch.ones(T, dtype=torch.bool, device=DEV)
        live[dead] = False
        assert torch.equal(got[live], want[live])


@pytest.mark.parametrize("E", [16, 64, 128, 300])
def test_chosen_experts_masked_among_others(E):
    """renormalize: the softmax runs over the chosen alone, so -inf there is nothing at all."""
    note(f"masked choice {E}")
    logits = torch.zeros((3, E), device=DEV)
    idx = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32, device=DEV)
    logits[1, 2:4] = -torch.inf
    dw = torch.tensor([[1.0, 3.0], [torch.nan, torch.inf], [2.0, -2.0]], device=DEV)
    got = moe.gate_backward(logits, idx, dw)
    assert (got[1] == 0).all()
    # two equal logits: p = 1/2 each, so the gradient is +-(dw_0 - dw_1) / 4, exact in f32
    assert got[0, :2].tolist() == [-0.5, 0.5] and got[2, 4:6].tolist() == [1.0, -1.0]
    assert (got[0, 2:] == 0).all() and (got[2, :4] == 0).all()


@pytest.mark.parametrize("E", [16, 64, 128, 300])
@pytest.mark.parametrize("renorm", [True, False])
def test_masked_entry_of_a_live_token(E, renorm):
    """An entry that names a masked expert counts as none, as gate itself would have left it."""
    note(f"masked entry {E} {renorm}")
    g = torch.Generator().manual_seed(E)
    T, K = 21, 5
    logits = torch.randn((T, E), generator=g).to(DEV)
    idx = torch.argsort(torch.rand((T, E), generator=g), 1)[:, :K].int().to(DEV)
    logits[torch.arange(T, device=DEV), idx[:, 2].long()] = -torch.inf
    dw = torch.randn((T, K), generator=g).to(DEV)
    none = idx.clone()
    none[:, 2] = -1
    want = moe.gate_backward(logits, none, dw, renormalize=renorm)
    assert torch.isfinite(want).all()
    for bad in (float("nan"), float("inf"), 2.0):
        dw[:, 2] = bad
        assert torch.equal(moe.gate_backward(logits, idx, dw, renormalize=renorm), want), bad
