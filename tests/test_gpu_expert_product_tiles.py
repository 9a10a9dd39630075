"""GPU tests of the grouped MXFP4 product in each of its tiles, at sizes that the rules give to them
(_experts_forms.py), against the definition in 64 bits: every scale and code random, K of one
block to several rounds of scale loads with every kind of rest, full, part-filled and half-full
tiles, scales that begin at any byte, padded segments.

Tolerances are those of test_gpu_expert_product.py: a sum of H products, each exact, is off by at
most 2*H*u of the sum of their magnitudes (u = 2^-24), and SwiGLU by 1.1*dg*|up| + |silu(g)|*du +
dg*du and 20 + |g| further roundings.  Sums and magnitudes are computed on the GPU in 64 bits, by
torch, one expert at a time."""
import numpy as np
import pytest
import torch

import combine_moe_route_count_amd as moe
from _experts_forms import PRODUCT
from _gpu_util import DEV, note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
TABLE = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                     dtype=torch.float64)


def _values(codes, scales):
    """MXFP4 values in 64 bits, on the GPU."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    s = torch.from_numpy(np.ldexp(1.0, np.arange(256) - 127)).to(DEV)[scales.long()]
    return (TABLE.to(DEV)[c].unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def _random(g, shape):
    H = shape[-1]
    c = torch.randint(0, 256, shape[:-1] + (H // 2,), generator=g, dtype=torch.uint8, device=DEV)
    s = torch.randint(120, 132, shape[:-1] + (H // 32,), generator=g, dtype=torch.uint8, device=DEV)
    return c, s


def _counts(rng, rows, E, height):
    """Uneven, some a row more or less than whole or half tiles, one expert in four without rows."""
    special = [height, height // 2, height + 1, height // 2 + 1, 1]
    cnt = [0 if E > 3 and e % 4 == 2 else special[int(rng.integers(5))] if e % 2 else int(rng.integers(1, 2 * height))
           for e in range(E)]
    while sum(cnt) > rows:
        e = int(np.argmax(cnt))
        cnt[e] -= min(cnt[e], sum(cnt) - rows)
    cnt[0] += rows - sum(cnt)
    return cnt


def _check(y, a, w, cnt, off, swiglu, what):
    rows, H = a[0].shape[0], 2 * a[0].shape[1]
    va = _values(*a)
    owned = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for e, (c, o) in enumerate(zip(cnt.tolist(), off.tolist())):
        if c == 0:
            continue
        owned[o:o + c] = True
        x, v = va[o:o + c], _values(w[0][e], w[1][e])
        z, d = x @ v.t(), (x.abs() @ v.abs().t()) * (2 * H * U)
        if swiglu:
            (g, u), (dg, du) = z.chunk(2, 1), d.chunk(2, 1)
            act = g * torch.sigmoid(g)
            d = 1.1 * dg * u.abs() + act.abs() * du + dg * du + (act * u).abs() * (20 + g.abs()) * U
            z = act * u
        lim = (d + z.abs() * (torch.finfo(y.dtype).eps / 2)) * (1 + 2.0 ** -7) + 1e-37
        over = ~((y[o:o + c].double() - z).abs() <= lim)
        assert not over.any(), (what, e, int(over.sum()), over.numel(), over.nonzero()[:4].tolist())
    assert (y[~owned] == 7).all(), (what, "rows that nobody owns were written")


def _shifted(t, by):
    flat = torch.full((t.numel() + 8,), 255, dtype=torch.uint8, device=DEV)    # NaN around it
    flat[by:by + t.numel()] = t.flatten()
    return flat[by:by + t.numel()].view(t.shape)


def _case(height, size, H, swiglu, out, at=(0, 0), padded=False):
    rows, E, N = size
    note(f"tiles height={height} rows={rows} E={E} N={N} H={H} swiglu={swiglu} {out} at={at} padded={padded}")
    rng = np.random.default_rng(rows + H)
    if padded:
        cap = rows // E
        cnt = torch.tensor([int(rng.integers(0, cap + 1)) for _ in range(E)], dtype=torch.int32)
        off = torch.arange(E + 1, dtype=torch.int32) * cap
    else:     # three rows in front of the first segment and two or more behind the last are nobody's
        cnt = torch.tensor(_counts(rng, rows - 5, E, height), dtype=torch.int32)
        off = torch.zeros(E + 1, dtype=torch.int32)
        off[1:] = torch.cumsum(cnt, 0)
        off += 3
    g = torch.Generator(device=DEV)
    g.manual_seed(rows * 31 + H)
    a, w = _random(g, (rows, H)), _random(g, (E, N, H))
    y = torch.full((rows, N // 2 if swiglu else N), 7.0, dtype=out, device=DEV)
    moe.expert_product_mxfp4(a[0], _shifted(a[1], at[0]), w[0], _shifted(w[1], at[1]), cnt.to(DEV), off.to(DEV),
                             swiglu=swiglu, y=y)
    torch.cuda.synchronize()
    _check(y, a, w, cnt, off, swiglu, "tiles")
    return a, w, cnt, off, y


SIZES = [(h, s) for h, sizes in PRODUCT.items() for s in sizes]

# K in blocks of 32: one; 23; one pair of rounds; a pair, whole rounds and a rest; two pairs and a rest
# that no word holds; more pairs than are loaded ahead with a rest, in whole words and not
DEPTHS = [32, 736, 1024, 1664, 2976, 5888, 5856]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("H", DEPTHS)
@pytest.mark.parametrize("height,size", SIZES)
def test_tiles(height, size, H, swiglu):
    _case(height, size, H, swiglu, F32 if (H // 32 + size[0]) % 2 else BF16)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("height", list(PRODUCT))
def test_both_results(height, out, swiglu):
    _case(height, PRODUCT[height][1], 800, swiglu, out)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("H", [1664, 5888, 2144])
@pytest.mark.parametrize("at", [(1, 0), (2, 3)])
@pytest.mark.parametrize("height", list(PRODUCT))
def test_scales_that_begin_anywhere(height, at, H, swiglu):
    _case(height, PRODUCT[height][-1], H, swiglu, F32, at=at)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("height", list(PRODUCT))
def test_padded_segments(height, swiglu):
    _case(height, PRODUCT[height][1], 1120, swiglu, BF16, padded=True)


@pytest.mark.parametrize("height", list(PRODUCT))
def test_bits_do_not_change(height):
    a, w, cnt, off, y = _case(height, PRODUCT[height][-1], 1056, True, F32)
    for _ in range(3):
        again = torch.full_like(y, 7.0)
        moe.expert_product_mxfp4(*a, *w, cnt.to(DEV), off.to(DEV), swiglu=True, y=again)
        assert torch.equal(y, again)


@pytest.mark.parametrize("height", list(PRODUCT))
def test_nan_scales(height):
    """A NaN scale reaches its row or column only, wherever in K it stands."""
    rows, E, N = PRODUCT[height][1]
    H = 1376
    note(f"tiles NaN height={height}")
    g = torch.Generator(device=DEV)
    g.manual_seed(height)
    a, w = _random(g, (rows, H)), _random(g, (E, N, H))
    cnt = torch.full((E,), rows // E, dtype=torch.int32)
    off = torch.arange(E + 1, dtype=torch.int32) * (rows // E)
    want = torch.zeros((rows, N), dtype=torch.bool, device=DEV)
    want_up = torch.zeros((rows, N // 2), dtype=torch.bool, device=DEV)
    for i, b in enumerate(range(0, H // 32, 7)):
        r, n, e = (i * 29 + 1) % (rows // E), (i * 37 + 5) % N, i % E
        a[1][e * (rows // E) + r, b] = 255
        w[1][e, n, b] = 255
        want[e * (rows // E) + r] = True
        want_up[e * (rows // E) + r] = True
        want[e * (rows // E):(e + 1) * (rows // E), n] = True
        want_up[e * (rows // E):(e + 1) * (rows // E), n % (N // 2)] = True
    y = moe.expert_product_mxfp4(*a, *w, cnt.to(DEV), off.to(DEV), out_dtype=F32)
    z = moe.expert_product_mxfp4(*a, *w, cnt.to(DEV), off.to(DEV), swiglu=True)
    torch.cuda.synchronize()
    mine = rows // E * E
    assert torch.equal(torch.isnan(y[:mine]), want[:mine])
    assert torch.equal(torch.isnan(z[:mine]), want_up[:mine])


@pytest.mark.parametrize("E", [256, 257, 300, 513, 1024])
@pytest.mark.parametrize("rows,N", [(700, 48), (1500, 1072)])
def test_many_experts(E, rows, N):
    """More experts than are looked at together, most of them without a row, the last with some."""
    note(f"many experts E={E} rows={rows} N={N}")
    rng = np.random.default_rng(E)
    cnt = np.zeros(E, dtype=np.int32)
    for e in [0, E - 1, 255] + rng.integers(0, E, 40).tolist():
        cnt[e] = min(int(rng.integers(1, 40)), rows - 5 - int(cnt.sum()) + int(cnt[e]))
    cnt = torch.from_numpy(cnt)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(cnt, 0)
    off += 3
    g = torch.Generator(device=DEV)
    g.manual_seed(E)
    a, w = _random(g, (rows, 160)), _random(g, (E, N, 160))
    for swiglu in (False, True):
        y = torch.full((rows, N // 2 if swiglu else N), 7.0, dtype=F32, device=DEV)
        moe.expert_product_mxfp4(*a, *w, cnt.to(DEV), off.to(DEV), swiglu=swiglu, y=y)
        torch.cuda.synchronize()
        _check(y, a, w, cnt, off, swiglu, "experts")


def test_longest_rows():
    """H = 2^24, with scales of 1: every sum is a multiple of 1/4 below 2^22, and exact."""
    rows, E, N, H = 5, 2, 16, 1 << 24
    note("longest rows of the product")
    g = torch.Generator(device=DEV)
    g.manual_seed(24)
    a, w = _random(g, (rows, H)), _random(g, (E, N, H))
    a[1].fill_(127)
    w[1].fill_(127)
    cnt, off = torch.tensor([2, 3], dtype=torch.int32), torch.tensor([0, 2, 5], dtype=torch.int32)
    y = moe.expert_product_mxfp4(*a, *w, cnt.to(DEV), off.to(DEV), out_dtype=F32)
    torch.cuda.synchronize()
    va = _values(*a)
    for e in range(E):
        z = va[off[e]:off[e + 1]] @ _values(w[0][e], w[1][e]).t()
        assert z.abs().max() < 2.0 ** 20          # and so are the sums on the way, of random signs
        assert torch.equal(y[off[e]:off[e + 1]].double(), z)
