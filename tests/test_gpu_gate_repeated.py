"""The gate's gradient for ids that name an expert more than once: the softmax over the chosen runs
over the entries, and the expert gets the gradients of all of them.

Tolerance.  u = 2^-24.  Logits lie within d of each other.  A weight is off by (2.25 d + 2 n + 8) u
relative, n the number of terms of its softmax: 2.2 d for the rounded argument of exp, which weighs
terms p_j and so adds at most 0.81 n for the sum, n for its additions, 6 for the power, the division
and the product.  The gradient p (dw - sum p dw) takes two of them and K + 6 more roundings, each of
them against the sum of the magnitudes."""
import pytest
import torch

import combine_moe_route_count_amd as moe
from _gpu_util import DEV, note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _by_autograd(logits, idx, dw, renorm, scale):
    """64 bits, from the definition of the weights: entry k has exp(l[idx_k]) over the sum of the
    entries' own exps, or of all experts'."""
    z = logits.double().cpu().requires_grad_()
    at = idx.long().cpu()
    w = torch.softmax(z.gather(1, at), 1) if renorm else torch.softmax(z, 1).gather(1, at)
    (w * scale * dw.double().cpu()).sum().backward()
    return z.grad.to(logits.device)


# one case for each list length of the two group widths, and one past the switch for many tokens
@pytest.mark.parametrize("T,E", [(12, 3), (12, 16), (12, 30), (12, 64), (12, 120), (12, 256), (12, 500), (12, 1024),
                                 (4100, 128), (4100, 256)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
def test_repeated_experts(T, E, dt, renorm):
    note(f"repeated experts {T} {E} {dt} {renorm}")
    g = torch.Generator().manual_seed(7 * E + T)
    K, scale = min(E, 6), 2.5
    logits = torch.randn((T, E), generator=g).clamp(-4, 4).to(dt).to(DEV)
    idx = torch.randint(0, E, (T, K), generator=g).int().to(DEV)
    idx[0] = E - 1                        # one expert, K times
    idx[1, K // 2:] = idx[1, 0]
    idx[2, -1] = idx[2, 0]                # the first and the last entry
    dw = torch.randn((T, K), generator=g).to(DEV)
    got = moe.gate_backward(logits, idx, dw, renormalize=renorm, scale=scale).double()
    ref = _by_autograd(logits, idx, dw, renorm, scale)
    n = K if renorm else E
    z = logits.double()
    e = torch.zeros_like(z).scatter_add_(1, idx.long(), torch.ones_like(dw, dtype=torch.float64))
    p = torch.exp(z) * e
    p = p / p.sum(1, keepdim=True) if renorm else torch.softmax(z, 1)
    most = dw.double().abs().sum(1, keepdim=True)            # of K entries, repeated ones together
    mag = scale * p * (most + (torch.softmax(z, 1).gather(1, idx.long()) if not renorm else
                               torch.softmax(z.gather(1, idx.long()), 1)).mul(dw.double().abs()).sum(1, keepdim=True))
    lim = mag * (2 * (2.25 * 8 + 2 * n + 8) + K + 6) * U * (1 + 2.0 ** -7)
    lim = lim + ref.abs() * (torch.finfo(dt).eps / 2) * (1 + 2.0 ** -7) + 1e-37
    worst = ((got - ref).abs() / lim).max().item()
    assert worst <= 1, worst
    if renorm:                            # the whole softmax on one expert: no gradient but rounding
        assert (got[0, :E - 1] == 0).all()
    again = moe.gate_backward(logits, idx, dw, renormalize=renorm, scale=scale).double()
    assert torch.equal(got, again)
