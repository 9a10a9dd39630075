"""GPU tests of the grouped MXFP4 product against its definition in 64 bits.

Tolerances.  u = 2^-24.  Products of two e2m1 codes and two scales are exact in f32;
the sum of H of them, in any order, is off by at most H*u times the sum of their
magnitudes, the matrix instruction's own additions included (each rounds to f32, or is
cut there, which costs twice as much: 2*H*u is allowed).  Where all partial sums are
whole multiples of one unit below 2^24 nothing is lost, and results are compared bit
for bit.  SwiGLU of sums that are off by dg and du: silu' is at most 1.1 in magnitude,
so 1.1*dg*|u| + |silu(g)|*du + dg*du, and 20u for its own steps (exp2's argument is
rounded once: |g| u more)."""
import numpy as np
import pytest
import torch

import combine_moe_route_count_amd as moe
from _gpu_util import DEV, note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _codes(g, shape, lo=120, hi=132):
    """Random codes [..., H/2] and scales [..., H/32] of shape [..., H]."""
    H = shape[-1]
    c = torch.randint(0, 256, shape[:-1] + (H // 2,), generator=g, dtype=torch.uint8)
    s = torch.randint(lo, hi, shape[:-1] + (H // 32,), generator=g, dtype=torch.uint8)
    return c, s


def _values(codes, scales):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    v = torch.where(c >= 8, -E2M1[c & 7], E2M1[c & 7]).unflatten(-1, (-1, 32))
    s = torch.from_numpy(np.ldexp(1.0, scales.numpy().astype(np.int64) - 127))
    s = torch.where(scales == 255, torch.tensor(float("nan"), dtype=torch.float64), s)
    return (v * s.unsqueeze(-1)).flatten(-2)


def _ref(a, w, cnt, off, rows, swiglu):
    """(y, bound of its error before rounding, which rows are written)."""
    H = a.shape[1]
    N = w.shape[1]
    cols = N // 2 if swiglu else N
    y, tol = (torch.zeros((rows, cols), dtype=torch.float64) for _ in range(2))
    mine = torch.zeros(rows, dtype=torch.bool)
    for e, (c, o) in enumerate(zip(cnt.tolist(), off.tolist())):
        lo, hi = max(0, o), max(0, min(rows, o + c))
        if hi <= lo:
            continue
        mine[lo:hi] = True
        z = a[lo:hi] @ w[e].t()
        d = (a[lo:hi].abs() @ w[e].abs().t()) * (2 * H * U)
        if swiglu:
            g, u = z.chunk(2, 1)
            dg, du = d.chunk(2, 1)
            act = g * torch.sigmoid(g)
            y[lo:hi] = act * u
            tol[lo:hi] = 1.1 * dg * u.abs() + act.abs() * du + dg * du + (act * u).abs() * (20 + g.abs()) * U
        else:
            y[lo:hi], tol[lo:hi] = z, d
    return y, tol, mine


def _check(got, ref, what):
    y, tol, mine = ref
    g = got.cpu().double()
    lim = (tol + y.abs() * (torch.finfo(got.dtype).eps / 2)) * (1 + 2.0 ** -7) + 1e-37
    nan = torch.isnan(y)
    assert torch.equal(torch.isnan(g[mine]), nan[mine]), f"{what}: NaN in other places"
    over = ((g - y).abs() > lim)[mine] & ~nan[mine]
    assert not over.any(), f"{what}: {over.sum().item()} of {over.numel()} past the bound"
    assert (g[~mine] == 7).all(), f"{what}: rows that nobody owns were written"


def _compact(counts, tail=0, first=0):
    cnt = torch.tensor(counts, dtype=torch.int32)
    off = torch.zeros(len(counts) + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(cnt, 0)
    return cnt, off + first, first + int(cnt.sum()) + tail


def _padded(counts, cap):
    cnt = torch.tensor(counts, dtype=torch.int32)
    return cnt, torch.arange(len(counts) + 1, dtype=torch.int32) * cap, cap * len(counts)


def _run(cnt, off, rows, N, H, swiglu, out, seed, lo=120, hi=132):
    g = _gen(seed)
    E = cnt.numel()
    note(f"product rows={rows} E={E} N={N} H={H} swiglu={swiglu} {out}")
    a, sa = _codes(g, (rows, H), lo, hi)
    w, sw = _codes(g, (E, N, H), lo, hi)
    y = torch.full((rows, N // 2 if swiglu else N), 7.0, dtype=out, device=DEV)
    moe.expert_product_mxfp4(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), cnt.to(DEV),
                             off.to(DEV), swiglu=swiglu, y=y)
    torch.cuda.synchronize()
    return a, sa, w, sw, y


SEGS = {
    "one_row": _compact([1]),
    "few": _compact([2, 0, 1, 3, 0], tail=3),
    "late": _compact([5, 17], first=9, tail=2),
    "tiles": _compact([16, 17, 33, 0, 64, 65], tail=1),
    "padded": _padded([7, 0, 20, 12], 20),
    "long": _compact([300, 5, 131]),
    "many": _compact([1, 0, 2] * 40),
}


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("N,H", [(16, 32), (48, 96), (272, 256), (208, 1056), (528, 544)])
@pytest.mark.parametrize("segs", list(SEGS))
def test_matches_definition(segs, N, H, out, swiglu):
    cnt, off, rows = SEGS[segs]
    a, sa, w, sw, y = _run(cnt, off, rows, N, H, swiglu, out, N + H)
    _check(y, _ref(_values(a, sa), _values(w, sw), cnt, off, rows, swiglu), segs)


@pytest.mark.parametrize("mean", [4, 30, 60, 120, 260])
def test_every_tile_height(mean):
    """Rows per expert from a few to more than a tile, uneven."""
    g = _gen(mean)
    counts = torch.randint(0, 2 * mean + 1, (6,), generator=g).tolist()
    cnt, off, rows = _compact(counts)
    a, sa, w, sw, y = _run(cnt, off, rows, 344, 736, False, F32, mean)
    _check(y, _ref(_values(a, sa), _values(w, sw), cnt, off, rows, False), mean)


@pytest.mark.parametrize("H", [32, 64, 224, 256, 288, 480, 512, 544, 768, 1024])
def test_whole_numbers_are_exact(H):
    """Scales of 1: every partial sum is a multiple of 1/4 below 2^24."""
    cnt, off, rows = _compact([40, 3, 70])
    a, sa, w, sw, y = _run(cnt, off, rows, 264, H, False, F32, H, lo=127, hi=128)
    ref, _, mine = _ref(_values(a, sa), _values(w, sw), cnt, off, rows, False)
    assert torch.equal(y.cpu().double(), ref)


@pytest.mark.parametrize("mean", [3, 50, 150])
@pytest.mark.parametrize("H", [1024, 1056, 1120, 2144])
@pytest.mark.parametrize("at", [(1, 0), (0, 3), (2, 2), (3, 1)])
def test_scales_that_begin_anywhere(at, H, mean):
    """Views whose first byte is not the first of a word, rows of 32, 33, 35 and 67 scales."""
    g = _gen(mean + H)
    cnt, off, rows = _compact([mean, 0, 2 * mean + 1, 7])
    note(f"scales at {at} H={H} rows={rows}")
    E, N = 4, 304
    a, sa = _codes(g, (rows, H))
    w, sw = _codes(g, (E, N, H))

    def shifted(t, by):
        flat = torch.full((t.numel() + 8,), 255, dtype=torch.uint8, device=DEV)    # NaN around it
        flat[by:by + t.numel()] = t.to(DEV).flatten()
        return flat[by:by + t.numel()].view(t.shape)
    for swiglu in (False, True):
        y = torch.full((rows, N // 2 if swiglu else N), 7.0, dtype=F32, device=DEV)
        moe.expert_product_mxfp4(a.to(DEV), shifted(sa, at[0]), w.to(DEV), shifted(sw, at[1]), cnt.to(DEV),
                                 off.to(DEV), swiglu=swiglu, y=y)
        torch.cuda.synchronize()
        _check(y, _ref(_values(a, sa), _values(w, sw), cnt, off, rows, swiglu), "shifted")


def test_plain_product_of_odd_columns():
    """N a multiple of 8 but of no more."""
    cnt, off, rows = _compact([19, 40])
    a, sa, w, sw, y = _run(cnt, off, rows, 8 * 33, 320, False, BF16, 5)
    _check(y, _ref(_values(a, sa), _values(w, sw), cnt, off, rows, False), "odd")


def test_extreme_scales():
    """Scales from 2^-127 to 2^127, and NaN: a NaN block reaches its row or column only."""
    g = _gen(77)
    rows, E, N, H = 21, 2, 32, 160
    cnt, off, _ = _compact([13, 8])
    a, sa = _codes(g, (rows, H))
    w, sw = _codes(g, (E, N, H))
    sa[0], sw[0, 0] = 0, 254        # 2^-127 * 2^127
    sa[1], sw[0, 1] = 200, 54
    sa[2, 4] = 255
    sw[1, 5, 0] = 255
    y = torch.full((rows, N), 7.0, device=DEV)
    moe.expert_product_mxfp4(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), cnt.to(DEV),
                             off.to(DEV), y=y)
    torch.cuda.synchronize()
    ref = _ref(_values(a, sa), _values(w, sw), cnt, off, rows, False)
    nan = torch.isnan(ref[0])
    assert nan[2].all() and nan[13:, 5].all() and nan.sum() == N + 8
    big = ref[0].abs() > 3.4e38
    ref[0][big], ref[1][big] = 0, 0
    got = y.clone()
    got[big.to(DEV)] = 0
    _check(got, ref, "scales")


def test_bad_segments_do_not_fault():
    """Counts and offsets outside the buffer: only what lies inside is touched."""
    rows, E, N, H = 50, 6, 40, 64
    cnt = torch.tensor([5, -3, 1 << 30, 4, 2147483647, 7], dtype=torch.int32)
    off = torch.tensor([0, 5, 40, 60, 2147483647, -4, 0], dtype=torch.int32)
    a, sa, w, sw, y = _run(cnt, off, rows, N, H, False, F32, 3)
    want = torch.full((rows,), False)
    want[0:5] = want[40:50] = True
    # expert 5's segment is -4 .. 2: rows 0 to 2, which expert 0 has as well
    ref = _ref(_values(a, sa), _values(w, sw), cnt[:5], off[:6], rows, False)
    got = y.clone()
    got[:3] = 7
    ref[2][:3] = False
    assert torch.equal(ref[2], want & (torch.arange(rows) >= 3))
    _check(got, ref, "bad")


def test_dense_product():
    """One expert that owns every row is an ordinary product."""
    cnt, off, rows = _compact([77])
    a, sa, w, sw, y = _run(cnt, off, rows, 128, 512, False, BF16, 8)
    _check(y, _ref(_values(a, sa), _values(w, sw), cnt, off, rows, False), "dense")


def test_no_rows():
    g = _gen(1)
    w, sw = _codes(g, (3, 16, 64))
    a, sa = _codes(g, (0, 64))
    cnt, off, _ = _compact([0, 0, 0])
    y = moe.expert_product_mxfp4(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), cnt.to(DEV), off.to(DEV))
    assert y.shape == (0, 16)
    a, sa = _codes(g, (5, 64))
    y = torch.full((5, 16), 7.0, device=DEV)
    moe.expert_product_mxfp4(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), cnt.to(DEV), off.to(DEV), y=y)
    torch.cuda.synchronize()
    assert (y == 7).all()


def test_bits_do_not_change():
    cnt, off, rows = SEGS["long"]
    a, sa, w, sw, y = _run(cnt, off, rows, 272, 1056, True, F32, 2)
    for _ in range(3):
        again = torch.full_like(y, 7.0)
        moe.expert_product_mxfp4(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), cnt.to(DEV),
                                 off.to(DEV), swiglu=True, y=again)
        assert torch.equal(y, again)


def test_weights_past_32_bit_offsets():
    """The last expert of a weight array of more than 4 GiB, and rows behind 4 GiB of y."""
    E, N, H = 40, 32768, 7168
    note("product long")
    w = torch.zeros((E, N, H // 2), dtype=torch.uint8, device=DEV)
    sw = torch.full((E, N, H // 32), 127, dtype=torch.uint8, device=DEV)
    rows = 40000
    a = torch.zeros((rows, H // 2), dtype=torch.uint8, device=DEV)
    sa = torch.full((rows, H // 32), 127, dtype=torch.uint8, device=DEV)
    g = _gen(6)
    la, lsa = _codes(g, (3, H), 127, 128)
    lw, lsw = _codes(g, (64, H), 127, 128)
    a[-3:], sa[-3:] = la.to(DEV), lsa.to(DEV)
    w[-1, -64:], sw[-1, -64:] = lw.to(DEV), lsw.to(DEV)
    cnt = torch.zeros(E, dtype=torch.int32)
    cnt[0], cnt[-1] = rows - 3, 3
    off = torch.full((E + 1,), rows - 3, dtype=torch.int32)
    off[0], off[-1] = 0, rows
    y = moe.expert_product_mxfp4(a, sa, w, sw, cnt.to(DEV), off.to(DEV), out_dtype=F32)
    torch.cuda.synchronize()
    assert torch.equal(y[-3:, -64:].cpu().double(), _values(la, lsa) @ _values(lw, lsw).t())
    assert not y[-3:, :-64].any() and not y[:-3].any()
