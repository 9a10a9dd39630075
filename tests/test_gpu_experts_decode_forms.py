"""GPU tests of experts_decode in each of its kernels, at sizes that the rules give to them
(_experts_forms.py), against the definition in 64 bits: evenly spread entries with some that
name no expert, and crowds that take an expert's weights more than one pass.

Tolerances are those of test_gpu_experts_decode.py, from the same sums of magnitudes.  Sums are
computed on the GPU in 64 bits, by torch, one expert at a time."""
import pytest
import torch

import combine_moe_route_count_amd as moe
from _experts_forms import BF16 as BF16_FORMS
from _experts_forms import MXFP4 as MXFP4_FORMS
from _gpu_util import DEV, note
from test_gpu_expert_product_tiles import _values

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def _weights(g, E, rows, cols, mx):
    if mx:
        return (torch.randint(0, 256, (E, rows, cols // 2), generator=g, dtype=torch.uint8, device=DEV),
                torch.randint(119, 125, (E, rows, cols // 32), generator=g, dtype=torch.uint8, device=DEV))
    return (torch.randn((E, rows, cols), generator=g, device=DEV) * cols ** -0.5).to(BF16), None


def _of(w, e):
    return w[0][e].double() if w[1] is None else _values(w[0][e], w[1][e])


def _inputs(T, H, I, E, K, mx, crowd, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn((T, H), generator=g, device=DEV).to(BF16)
    idx = torch.randint(0, E, (T, K), generator=g, device=DEV).int()
    if crowd:       # half of all entries on one expert
        idx[torch.rand((T, K), generator=g, device=DEV) < 0.5] = E // 2
    idx[torch.rand((T, K), generator=g, device=DEV) < 0.1] = -1
    w = torch.softmax(torch.randn((T, K), generator=g, device=DEV), -1)
    return x, idx, w, _weights(g, E, 2 * I, H, mx), _weights(g, E, H, I, mx)


def _check(got, x, idx, w, w13, w2, P):
    T, H = x.shape
    K = idx.shape[1]
    I = w13[0].shape[1] // 2
    out, tol = (torch.zeros((T, H), dtype=torch.float64, device=DEV) for _ in range(2))
    xd = x.double()
    for e in idx.unique().tolist():
        if e < 0:
            continue
        t, k = torch.nonzero(idx == e, as_tuple=True)
        v = _of(w13, e)
        z, d = xd[t] @ v.t(), (xd[t].abs() @ v.abs().t()) * (2 * H * U)
        (g, u), (dg, du) = z.chunk(2, 1), d.chunk(2, 1)
        act = g * torch.sigmoid(g)
        h = act * u
        dh = 1.1 * dg * u.abs() + act.abs() * du + dg * du + h.abs() * (20 + g.abs()) * U
        v = _of(w2, e)
        y = h @ v.t()
        dy = (dh + h.abs() * (2.0 ** (-9 * P) + 2 * P * I * U * (1 + 2.0 ** -8))) @ v.abs().t()
        c = w[t, k].double().unsqueeze(1)
        out.index_add_(0, t, c * y)
        tol.index_add_(0, t, c * dy + (c * y).abs() * (K + 10) * U)
    lim = (tol + out.abs() * (torch.finfo(got.dtype).eps / 2)) * (1 + 2.0 ** -7) + 1e-37
    over = ~((got.double() - out).abs() <= lim)
    assert not over.any(), (int(over.sum()), over.numel(), over.nonzero()[:4].tolist())


CASES = [(False, s) for s in BF16_FORMS] + [(True, s) for s in MXFP4_FORMS]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("crowd", [False, True])
@pytest.mark.parametrize("mx,size", CASES)
def test_forms(mx, size, crowd, out):
    T, H, I, E, K = size
    note(f"decode form mx={mx} {size} crowd={crowd} {out}")
    args = _inputs(T, H, I, E, K, mx, crowd, T + H)
    x, idx, w, w13, w2 = args
    y = torch.full((T, H), 7.0, dtype=out, device=DEV)
    moe.experts_decode(x, idx, w, w13[0], w2[0], w13[1], w2[1], out=y)
    torch.cuda.synchronize()
    _check(y, *args, 3 if out == F32 else 2)


@pytest.mark.parametrize("mx,size", CASES)
def test_bits_do_not_change(mx, size):
    """Also with weights that begin elsewhere: at 16 bytes into a cache line."""
    T, H, I, E, K = size
    note(f"decode repeat mx={mx} {size}")
    x, idx, w, w13, w2 = _inputs(T, H, I, E, K, mx, True, T + I)
    first = moe.experts_decode(x, idx, w, w13[0], w2[0], w13[1], w2[1], out_dtype=F32)

    def moved(t):
        n = 16 // t.element_size()
        flat = torch.empty(t.numel() + n, dtype=t.dtype, device=DEV)
        flat[n:] = t.flatten()
        return flat[n:].view(t.shape)
    a, b = moved(w13[0]), moved(w2[0])
    for _ in range(2):
        assert torch.equal(first, moe.experts_decode(x, idx, w, w13[0], w2[0], w13[1], w2[1], out_dtype=F32))
        assert torch.equal(first, moe.experts_decode(x, idx, w, a, b, w13[1], w2[1], out_dtype=F32))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,H,I,E,K", [(1, 1 << 20, 32, 2, 2), (1, 32, 1 << 20, 2, 2), (1024, 1 << 20, 32, 3, 1),
                                       (1024, 32, 1 << 20, 3, 1), (64, 1 << 20, 64, 40, 1)])
def test_largest_sizes(T, H, I, E, K, mx):
    """Rows of 2^20 elements, x and the parts of h of 2 GiB."""
    note(f"decode largest T={T} H={H} I={I} mx={mx}")
    args = _inputs(T, H, I, E, K, mx, False, T + H)
    x, idx, w, w13, w2 = args
    y = moe.experts_decode(x, idx, w, w13[0], w2[0], w13[1], w2[1], out_dtype=F32)
    torch.cuda.synchronize()
    _check(y, *args, 3)
    torch.cuda.empty_cache()
