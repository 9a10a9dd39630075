"""GPU tests of silu inside the products: silu(g) * u of f32 results keeps its digits at every g,
as moe_swiglu's does.

Inputs are small whole multiples of a power of two, so that both sums are exact and what is left
is the activation.  Tolerances, u = 2^-24: t = exp(-|g|) is off by at most 6u (its argument is held in
two parts, 1u each; exp2 2u, the correction 2u), 1 + t by u more than half of that, its reciprocal by
2u more: 6u, t times it 13u, and the two products 1u each: 15u.  exp2 has no subnormal results: t below
2^-126 is 0, which moves s by at most 2^-126, an absolute error of 2^-126 |g u|.  experts_decode adds
its three parts of h in f32 (2u each, twice) and holds 24 bits of it (u / 2 and less): 20u."""
import pytest
import torch

import combine_moe_route_count_amd as moe
from _gpu_util import DEV, note
from test_gpu_experts_decode import _values

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def _silu_product(g, u):
    """silu(g) * u in 64 bits, without a cancellation."""
    t = torch.exp(-g.abs())
    return g * u * torch.where(g < 0, t / (1 + t), 1 / (1 + t))


def _check(got, g, u, steps, what):
    want = _silu_product(g, u)
    lim = want.abs() * steps * U + (g * u).abs() * 2.0 ** -126
    over = (got.cpu().double() - want).abs() > lim
    assert (g < -20).any() and (g < -80).any() and (g > 20).any()
    assert not over.any(), (what, int(over.sum()), over.numel(),
                            (((got.cpu().double() - want).abs() - lim / 15) / want.abs() / U)[over].max())


@pytest.mark.parametrize("rows,N", [(40, 512), (64, 9472), (200, 20480), (512, 20480)])
def test_product(rows, N):
    """One expert, in tiles of 32, 64, 128 and 256 rows."""
    note(f"silu of the product rows={rows} N={N}")
    gen = torch.Generator()
    gen.manual_seed(rows)
    H = 32
    a = torch.randint(0, 256, (rows, H // 2), generator=gen, dtype=torch.uint8)
    sa = torch.full((rows, 1), 127, dtype=torch.uint8)
    w = torch.randint(0, 256, (1, N, H // 2), generator=gen, dtype=torch.uint8)
    sw = torch.randint(125, 128, (1, N, 1), generator=gen, dtype=torch.uint8)
    cnt, off = torch.tensor([rows], dtype=torch.int32), torch.tensor([0, rows], dtype=torch.int32)
    y = moe.expert_product_mxfp4(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), cnt.to(DEV), off.to(DEV),
                                 swiglu=True, out_dtype=F32)
    torch.cuda.synchronize()
    z = _values(a, sa) @ _values(w, sw)[0].t()
    _check(y, *z.chunk(2, 1), 15, "product")


@pytest.mark.parametrize("T,I", [(4, 64), (40, 1664)])
@pytest.mark.parametrize("mx", [False, True])
def test_decode(mx, T, I):
    """The second product's weights pick single h's out."""
    note(f"silu of experts_decode mx={mx} T={T} I={I}")
    gen = torch.Generator()
    gen.manual_seed(T)
    H = 64
    x = torch.randint(-7, 8, (T, H), generator=gen).to(BF16)
    if mx:
        w13 = torch.randint(0, 256, (1, 2 * I, H // 2), generator=gen, dtype=torch.uint8)
        s13 = torch.full((1, 2 * I, H // 32), 126, dtype=torch.uint8)
        v13 = _values(w13, s13)[0]
        w2, s2 = torch.zeros((1, H, I // 2), dtype=torch.uint8), torch.full((1, H, I // 32), 127, dtype=torch.uint8)
        for r in range(H):
            w2[0, r, r // 2] = 2 << 4 * (r % 2)
    else:
        w13 = (torch.randint(-6, 7, (1, 2 * I, H), generator=gen) * 0.5).to(BF16)
        v13, s13, s2 = w13[0].double(), None, None
        w2 = torch.eye(H, I, dtype=BF16).unsqueeze(0)
    on = lambda t: None if t is None else t.to(DEV)
    y = moe.experts_decode(on(x), torch.zeros((T, 1), dtype=torch.int32, device=DEV),
                           torch.ones((T, 1), device=DEV), on(w13), on(w2), on(s13), on(s2), out_dtype=F32)
    torch.cuda.synchronize()
    z = x.double() @ v13.t()
    g, u = z.chunk(2, 1)
    _check(y, g[:, :H], u[:, :H], 20, "decode")
