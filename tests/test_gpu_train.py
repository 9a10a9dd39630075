"""GPU tests of the training-side operators against plain torch in 64 bits: the
top-k gate, the embedding lookup, and the gradients of gate, dispatch, combine
and lookup.

Tolerances.  u = 2^-24 is the most that one f32 rounding is off, relative to its
result; finfo(t).eps / 2 the same for a stored type t.  A sum of n terms in any
order is off by at most n*u times the sum of the terms' magnitudes (first order);
the bounds below use that with the number of additions a sum can take, plus one u
for every other rounding on the way, each stated where it is used."""
import numpy as np
import pytest
import torch

import combine_moe_route_count_amd as moe
from _gpu_util import DEV, note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
TINY = 1e-37                      # absolute: results near the subnormal range


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _randn(g, shape, dt=F32, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dt).to(DEV)


def _same(a, b, what):
    torch.cuda.synchronize()
    assert a.dtype == b.dtype and a.shape == b.shape, (what, a.dtype, b.dtype, a.shape, b.shape)
    x, y = a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)
    assert torch.equal(x, y), f"{what}: {(x != y).sum().item()} of {x.numel()} bytes differ"


def _near(got, want, tol, what):
    """|got - want| <= tol (f64 tensors), plus the rounding of got's own type."""
    torch.cuda.synchronize()
    bad_want = ~torch.isfinite(want)
    g = got.double()
    assert torch.equal(torch.isnan(g), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(g[bad_want & ~torch.isnan(want)], want[bad_want & ~torch.isnan(want)]), what
    err = (g - want).abs()
    lim = tol * (1 + 2.0 ** -7) + want.abs() * (torch.finfo(got.dtype).eps / 2) * (1 + 2.0 ** -7) + TINY
    over = (err > lim) & ~bad_want
    assert not over.any(), (f"{what}: {over.sum().item()} of {over.numel()} past the bound, worst "
                            f"{(err / lim)[~bad_want].max().item():.3g} times it")


# ---------------------------------------------------------------------------
# gate
# ---------------------------------------------------------------------------

def _choice(l, K):
    """Stable descending order of each row; -inf is never chosen."""
    v, i = torch.sort(l.float().cpu(), dim=1, descending=True, stable=True)
    return torch.where(torch.isneginf(v[:, :K]), -1, i[:, :K]).int().to(l.device)


def _gate_ref(l, idx, renorm, scale):
    """(w, p over all) in f64, and the magnitude D = max |l_j - top| that bounds exp's argument."""
    z = l.double()
    E = z.shape[1]
    at = idx.clamp(min=0).long()
    chosen = torch.zeros((z.shape[0], E + 1), dtype=torch.bool, device=z.device)
    chosen.scatter_(1, torch.where(idx < 0, E, idx).long(), True)
    live = z.masked_fill(~chosen[:, :E], -torch.inf) if renorm else z
    p = torch.softmax(live, 1)
    p = torch.where(torch.isneginf(live).all(1, keepdim=True), 0.0, p)
    w = torch.where(idx >= 0, p.gather(1, at) * scale, 0.0)
    return w, p


def _gate_rel(l, K):
    """Relative error of a weight, in units of u.  exp(x), x = l - top <= 0, as 2^(x*log2 e): x and
    the product are rounded once each and log2(e) is 0.2 u off, all of it in the exponent, so
    2.2 |x|; the power itself 2.  The sum: terms weigh p_j = e^x_j / S with S >= 1, so their own
    errors add sum p_j (2.2 |x_j| + 2) <= 2.2 E/e + 2 < 0.81 E + 2 (t e^-t <= 1/e), its additions at
    most E.  Then a division and a product: 2.2 d + 1.81 E + 6 in all.  Arguments past 104
    underflow f32 and only matter below TINY."""
    z = torch.where(torch.isfinite(l.double()), l.double(), 0.0)
    d = (z.amax(1, keepdim=True) - z.amin(1, keepdim=True)).clamp(max=104.0)
    return (2.25 * d + 2 * l.shape[1] + 8) * U


def _logits(g, T, E, dt, kind):
    l = _randn(g, (T, E), dt, 2.0)
    if kind == "ties":
        l = (l * 2).round() / 2
    elif kind == "masked" and T > 0:
        l[:, torch.randperm(E, generator=g)[: max(1, E // 3)].to(DEV)] = -torch.inf
        l[::3, E // 2:] = -torch.inf
        l[::5] = -torch.inf                      # nothing left
        l[1::7] = torch.finfo(dt).min            # the type's lowest value is a value
    elif kind == "wide":
        l = l * 40
    return l


GATE_SHAPES = [(1, 1, 1), (1, 8, 8), (3, 16, 16), (5, 63, 5), (7, 64, 6), (130, 65, 4), (33, 128, 8),
               (257, 200, 8), (64, 256, 8), (19, 257, 3), (9, 511, 16), (6, 512, 10), (5, 1000, 16),
               (31, 1024, 8), (4097, 100, 8), (4101, 256, 4), (4098, 192, 16)]


@pytest.mark.parametrize("kind", ["normal", "ties", "masked", "wide"])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,E,K", GATE_SHAPES)
def test_gate(T, E, K, dt, kind):
    note(f"gate {T} {E} {K} {dt} {kind}")
    l = _logits(_gen(T * 1000 + E + K), T, E, dt, kind)
    for renorm, scale in ((True, 1.0), (False, 2.5)):
        idx, w = moe.gate(l, K, renormalize=renorm, scale=scale)
        want = _choice(l, K)
        assert torch.equal(idx, want), (idx != want).nonzero()[:5]
        ref, _ = _gate_ref(l, want, renorm, scale)
        _near(w, ref, ref.abs() * _gate_rel(l, K), f"w renorm={renorm}")


def test_gate_nan_and_infinities():
    note("gate nan")
    l = torch.zeros((6, 40))
    l[0, 7] = torch.nan                         # the largest value
    l[1, 30] = torch.inf
    l[2] = torch.nan
    l[3, 3], l[3, 5] = -0.0, 0.0                # equal: ids 0, 1, 2, ... by order
    l[4] = -torch.inf
    l[4, 39] = -3e38
    l[5, 11], l[5, 2] = torch.nan, torch.inf
    l = l.to(DEV)
    for renorm in (True, False):
        idx, w = moe.gate(l, 4, renormalize=renorm)
        want = torch.tensor([[7, 0, 1, 2], [30, 0, 1, 2], [0, 1, 2, 3], [0, 1, 2, 3], [39, -1, -1, -1],
                             [11, 2, 0, 1]], dtype=torch.int32)
        assert torch.equal(idx.cpu(), want), idx
        w = w.cpu()
        assert torch.isnan(w[[0, 1, 2, 5]]).all(), w
        assert torch.equal(w[4], torch.tensor([1.0, 0, 0, 0])), w[4]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("E", [8, 60, 64, 128, 256, 512, 1024])
def test_gate_on_unaligned_logits(E, dt):
    """Rows whose vectors straddle 16 bytes give the same bits as aligned ones."""
    note(f"gate unaligned {E} {dt}")
    T, K = 37, 6
    g = _gen(E)
    l = _randn(g, (T, E), dt, 2.0)
    odd = torch.empty(T * E + 1, dtype=dt, device=DEV)[1:].view(T, E)
    odd.copy_(l)
    dw = _randn(g, (T, K))
    for renorm in (True, False):
        a, b = moe.gate(l, K, renormalize=renorm), moe.gate(odd, K, renormalize=renorm)
        _same(a[0], b[0], "idx")
        _same(a[1], b[1], "w")
        want = moe.gate_backward(l, a[0], dw, renormalize=renorm)
        got = torch.empty(T * E + 1, dtype=dt, device=DEV)[1:].view(T, E)
        _same(moe.gate_backward(odd, a[0], dw, renormalize=renorm, dlogits=got), want, "dlogits")
        _same(moe.gate_backward(odd, a[0], dw, renormalize=renorm), want, "dlogits, one side")


def test_nothing_to_do():
    """No tokens, no rows: empty outputs, and rows without entries are still zeroed."""
    note("empty")
    z = lambda *s, dt=F32: torch.zeros(s, dtype=dt, device=DEV)                     # noqa: E731
    idx, w = moe.gate(z(0, 8), 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    assert moe.gate_backward(z(0, 8), idx, w).shape == (0, 8)
    tm = z(0, 2, dt=torch.int64)
    assert moe.dispatch_backward(z(0, 16), tm).shape == (0, 16)
    dy, dw = moe.combine_backward(z(0, 16), z(5, 16), tm, w)
    assert dy.shape == (5, 16) and dw.shape == (0, 2)
    dy = torch.full((5, 16), 3.0, device=DEV)
    moe.combine_backward(z(0, 16), z(5, 16), tm, w, dy=dy, packed_cnt=z(2, dt=torch.int32),
                         packed_off=z(3, dt=torch.int32))
    assert (dy == 0).all()
    dy, dw = moe.combine_backward(torch.ones((3, 16), device=DEV), z(0, 16), torch.full((3, 2), -1, device=DEV),
                                  torch.ones((3, 2), device=DEV))
    assert dy.shape == (0, 16) and (dw == 0).all()
    assert (moe.dispatch_backward(z(0, 16), torch.full((3, 2), -1, device=DEV)) == 0).all()
    assert moe.embedding(z(0, dt=torch.int32), z(4, 8)).shape == (0, 8)
    assert (moe.embedding_backward(z(0, 8), z(0, dt=torch.int64), 4) == 0).all()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,E,K", GATE_SHAPES)
@pytest.mark.parametrize("kind", ["normal", "masked"])
def test_gate_backward(T, E, K, dt, kind):
    note(f"gate_backward {T} {E} {K} {dt} {kind}")
    g = _gen(T + 31 * E + K)
    l = _logits(g, T, E, dt, kind)
    dw = _randn(g, (T, K))
    idx = _choice(l, K)
    if T > 4 and K > 2:
        idx[4, 0] = -1                          # entries the caller took out
        idx[4, 1] = E
        dw[4, 0] = torch.nan                    # their dw is not looked at
        dw[4, 1] = torch.inf
    live = (idx >= 0) & (idx < E)
    for renorm, scale in ((True, 1.0), (False, 2.5)):
        got = moe.gate_backward(l, idx, dw, renormalize=renorm, scale=scale)
        assert got.dtype == dt
        used = torch.where(live, idx, -1)
        _, p = _gate_ref(l, used, renorm, 1.0)
        dp = torch.zeros_like(p)
        dwx = torch.where(live, dw.double(), 0.0) * scale
        dp.scatter_add_(1, used.clamp(min=0).long(), torch.where(live, dwx, 0.0))
        ref = p * (dp - (p * dp).sum(1, keepdim=True))
        # each p carries _gate_rel; the K-term sum, two products and the difference add K + 6 u
        mag = p * (dp.abs() + (p * dp.abs()).sum(1, keepdim=True))
        _near(got, ref, mag * (2 * _gate_rel(l, K) + (K + 6) * U), f"dlogits renorm={renorm}")
        if renorm and T > 0:
            out = torch.ones((T, E + 1), dtype=torch.bool, device=DEV)
            out.scatter_(1, torch.where(live, idx, E).long(), False)
            assert (got[out[:, :E]] == 0).all()


def test_gate_backward_repeated_expert():
    """An expert named twice by a token gets both entries' gradients."""
    note("gate_backward repeated")
    l = _randn(_gen(1), (4, 20))
    idx = torch.tensor([[3, 3], [19, 0], [7, 7], [0, 1]], dtype=torch.int32, device=DEV)
    dw = _randn(_gen(2), (4, 2))
    got = moe.gate_backward(l, idx, dw, renormalize=False)
    p = torch.softmax(l.double(), 1)
    dp = torch.zeros_like(p).scatter_add_(1, idx.long(), dw.double())
    ref = p * (dp - (p * dp).sum(1, keepdim=True))
    mag = p * (dp.abs() + (p * dp.abs()).sum(1, keepdim=True))
    _near(got, ref, mag * (2 * _gate_rel(l, 2) + 8 * U), "dlogits")


@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_against_differences(renorm):
    """Central differences of the gate's own weights.  With h = 2^-6 (exact in f32) a difference
    is off by h^2/6 times the third derivative (at most 1 for a softmax weight) and by twice a
    weight's error over 2h; logits are spaced so that no step changes the choice."""
    note(f"gate differences {renorm}")
    E, K, h = 24, 4, 2.0 ** -6
    g = _gen(77)
    base = (torch.randperm(E, generator=g).float() * 0.25 - 2.0)
    dw = torch.randn((1, K), generator=g).to(DEV)
    rows = base.repeat(2 * E, 1)
    for j in range(E):
        rows[2 * j, j] += h
        rows[2 * j + 1, j] -= h
    idx0, _ = moe.gate(base[None].to(DEV), K, renormalize=renorm)
    idx, w = moe.gate(rows.to(DEV), K, renormalize=renorm)
    assert torch.equal(idx, idx0.expand(2 * E, K))
    loss = (w.double() * dw.double()).sum(1)
    num = (loss[0::2] - loss[1::2]) / (2 * h)
    got = moe.gate_backward(base[None].to(DEV), idx0, dw, renormalize=renorm)[0].double()
    size = dw.abs().sum().item()
    tol = size * (h * h / 6 + 2 * (2 * 8 + E + 8) * U / (2 * h) + 100 * U)
    assert (got - num).abs().max().item() <= tol, ((got - num).abs().max().item(), tol)


# ---------------------------------------------------------------------------
# dispatch and combine
# ---------------------------------------------------------------------------

def _routing(g, T, E, K, cap, drop=0.05):
    """(idx, dispatch outputs) through the library's own dispatch of a narrow payload."""
    idx = torch.argsort(torch.rand((T, E), generator=g), 1)[:, :K].int()
    idx[torch.rand((T, K), generator=g) < drop] = -1
    if T > 3:
        idx[T // 2] = -1                         # a token without any expert
    idx = idx.to(DEV)
    rows = E * cap if cap else T * K
    d = moe.dispatch(torch.zeros((T, 8), dtype=F32, device=DEV), idx, E, cap=cap, packed_rows=rows)
    return idx, d, rows


E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def _expert_rows(g, rows, H, kind):
    """(y as given, scales, values in f64)."""
    if kind in ("bf16", "f32"):
        y = _randn(g, (rows, H), BF16 if kind == "bf16" else F32)
        return y, None, y.double()
    sc = (torch.rand((rows, H // 128), generator=g) * 2 + 0.25).to(DEV)
    rep = sc.double().repeat_interleave(128, 1)
    if kind == "fp8":
        y = _randn(g, (rows, H)).to(torch.float8_e4m3fn)
        return y.view(torch.uint8), sc, y.double() * rep
    y = torch.randint(0, 256, (rows, H // 2), generator=g, dtype=torch.uint8).to(DEV)
    code = torch.stack((y & 15, y >> 4), -1).view(rows, H).long()
    return y, sc, E2M1.to(DEV)[code] * rep


COMBINE = [(1, 8, 1, 1, 0), (1, 256, 8, 2, 3), (3, 1000, 5, 3, 0), (17, 136, 16, 8, 0), (64, 256, 8, 2, 0),
           (40, 4104, 12, 6, 25), (129, 1024, 64, 16, 0), (200, 520, 7, 4, 90), (33, 7168, 32, 8, 12),
           (9, 16392, 4, 2, 0), (1030, 64, 256, 8, 40)]


def _combine_check(T, H, E, K, cap, ykind, ddt, dydt, seed, dow):
    g = _gen(seed)
    idx, d, rows = _routing(g, T, E, K, cap)
    y, sc, yv = _expert_rows(g, rows, H, ykind)
    w = torch.rand((T, K), generator=g).to(DEV)
    dout = _randn(g, (T, H), ddt)
    dwt = _randn(g, (T,)) if dow else None
    dy, dw = moe.combine_backward(dout, y, d.tok_map, w, y_scales=sc, fp4=ykind == "fp4",
                                  dout_weights=dwt, packed_cnt=d.packed_cnt, packed_off=d.packed_off,
                                  dy_dtype=dydt)
    assert dy.dtype == dydt
    tm = d.tok_map
    want = torch.zeros((rows, H), dtype=F32, device=DEV)
    dref = torch.zeros((T, K), dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(dref)
    for k in range(K):
        t = (tm[:, k] >= 0).nonzero().flatten()
        r = tm[t, k]
        want[r] = w[t, k, None] * dout[t].float()        # one f32 product, then one rounding
        prod = dout[t].double() * yv[r]
        dref[t, k] = prod.sum(1) + (dwt.double()[t] if dow else 0.0)
        mag[t, k] = prod.abs().sum(1) + (dwt.double()[t].abs() if dow else 0.0)
    _same(dy, want.to(dydt), "dy")
    # at least 8 partial sums share a row's H products, so no product passes more than
    # H/8 + 16 additions; a code times its scale is rounded once more
    _near(dw, dref, mag * ((H / 8 + 17) * U), "dw")
    assert (dw[tm < 0] == 0).all()
    return dy, dw


@pytest.mark.parametrize("ddt", [F32, BF16])
@pytest.mark.parametrize("ykind", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E,K,cap", COMBINE)
def test_combine_backward(T, H, E, K, cap, ykind, ddt):
    note(f"combine_backward {T} {H} {E} {K} {cap} {ykind} {ddt}")
    _combine_check(T, H, E, K, cap, ykind, ddt, ddt, T + H, T % 2 == 0)


@pytest.mark.parametrize("ykind", ["fp8", "fp4"])
@pytest.mark.parametrize("T,H,E,K,cap", [(1, 128, 4, 1, 0), (5, 256, 8, 8, 0), (37, 384, 16, 5, 9),
                                         (64, 1280, 32, 16, 0), (21, 7168, 8, 4, 20)])
def test_combine_backward_quantized(T, H, E, K, cap, ykind):
    note(f"combine_backward {T} {H} {E} {K} {cap} {ykind}")
    _combine_check(T, H, E, K, cap, ykind, BF16, BF16, T + H, True)
    _combine_check(T, H, E, K, cap, ykind, F32, BF16, T + H + 1, False)


@pytest.mark.parametrize("ddt,dydt", [(F32, BF16), (BF16, F32)])
def test_combine_backward_mixed_types(ddt, dydt):
    note(f"combine_backward mixed {ddt} {dydt}")
    _combine_check(50, 328, 8, 3, 20, "bf16", ddt, dydt, 5, True)


def test_combine_backward_codes_without_scales():
    note("combine_backward direct cast")
    g = _gen(3)
    _, d, rows = _routing(g, 30, 8, 4, 0)
    y, _, _ = _expert_rows(g, rows, 256, "fp8")
    w, dout = torch.rand((30, 4), generator=g).to(DEV), _randn(g, (30, 256), BF16)
    a = moe.combine_backward(dout, y, d.tok_map, w, packed_cnt=d.packed_cnt, packed_off=d.packed_off)
    b = moe.combine_backward(dout, y.view(torch.float8_e4m3fn), d.tok_map, w, packed_cnt=d.packed_cnt,
                             packed_off=d.packed_off,
                             y_scales=torch.ones((rows, 2), dtype=F32, device=DEV))
    _same(a[0], b[0], "dy")
    _same(a[1], b[1], "dw")


def test_combine_backward_one_output_and_untouched_rows():
    """dy or dw alone equal the pair; without packed_cnt the rows of no entry keep their bytes."""
    note("combine_backward parts")
    T, H, E, K, cap = 45, 264, 8, 4, 40
    g = _gen(8)
    _, d, rows = _routing(g, T, E, K, cap)
    y = _randn(g, (rows, H), BF16)
    w, dout = torch.rand((T, K), generator=g).to(DEV), _randn(g, (T, H), BF16)
    dy, dw = moe.combine_backward(dout, y, d.tok_map, w, packed_cnt=d.packed_cnt, packed_off=d.packed_off)
    none, dw2 = moe.combine_backward(dout, y, d.tok_map, None, want_dy=False)
    assert none is None
    _same(dw2, dw, "dw alone")
    mine = torch.full((rows, H), 7.0, dtype=BF16, device=DEV)
    dy3, none = moe.combine_backward(dout, None, d.tok_map, w, dy=mine, want_dw=False)
    assert none is None and dy3 is mine
    owned = torch.zeros(rows, dtype=torch.bool, device=DEV)
    owned[d.tok_map[d.tok_map >= 0]] = True
    assert 0 < owned.sum().item() < rows
    _same(mine[owned], dy[owned], "owned rows")
    assert (mine[~owned] == 7.0).all() and (dy[~owned] == 0).all()


def test_combine_backward_bad_rows_and_nonfinite():
    """Rows outside [0, y_rows) are no rows; what is not finite stays where it belongs."""
    note("combine_backward bad rows")
    T, H, K = 6, 128, 2
    tm = torch.tensor([[0, 1], [2, 1 << 40], [-5, 3], [4, 12], [5, -1], [-1, -1]], device=DEV)
    g = _gen(4)
    y, dout = _randn(g, (12, H)), _randn(g, (T, H))
    w = torch.rand((T, K), generator=g).to(DEV)
    dout[5] = torch.nan                                   # a token without rows
    y[6:] = torch.nan                                     # rows without entry
    y[3, 7] = torch.inf
    dout[4, 0] = torch.inf
    dy = torch.full((12, H), 9.0, device=DEV)
    _, dw = moe.combine_backward(dout, y, tm, w, dy=dy)
    valid = torch.tensor([[1, 1], [1, 0], [0, 1], [1, 0], [1, 0], [0, 0]], dtype=torch.bool, device=DEV)
    assert (dw[~valid] == 0).all()
    assert torch.isinf(dw[2, 1]) and not torch.isfinite(dw[4, 0])
    assert torch.isfinite(dw[[0, 0, 1, 3], [0, 1, 0, 0]]).all()
    assert (dy[6:] == 9.0).all() and torch.isfinite(dy[:5]).all() and torch.isinf(dy[5, 0])


@pytest.mark.parametrize("ddt,odt", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("T,H,E,K,cap", COMBINE)
def test_dispatch_backward(T, H, E, K, cap, ddt, odt):
    note(f"dispatch_backward {T} {H} {E} {K} {cap} {ddt} {odt}")
    g = _gen(T * 7 + H)
    _, d, rows = _routing(g, T, E, K, cap)
    dp = _randn(g, (rows, H), ddt)
    res = _randn(g, (T, H), odt)
    valid = d.tok_map >= 0
    for r in (None, res):
        acc = torch.zeros((T, H), device=DEV) if r is None else r.float()
        for k in range(K):                                # the same f32 additions in the same order
            row = dp[d.tok_map[:, k].clamp(min=0)].float()
            acc = torch.where(valid[:, k, None], acc + row, acc)
        got = moe.dispatch_backward(dp, d.tok_map, residual=r, dx_dtype=odt)
        _same(got, acc.to(odt), f"dx residual={r is not None}")
    mine = res.clone()
    assert moe.dispatch_backward(dp, d.tok_map, residual=mine, dx=mine) is mine
    _same(mine, acc.to(odt), "dx in place")


def test_dispatch_backward_ignores_unowned_rows():
    note("dispatch_backward unowned")
    tm = torch.tensor([[0, 1], [3, -1], [-1, -1], [1 << 33, 2]], device=DEV)
    dp = torch.full((6, 64), torch.nan, device=DEV)
    dp[:4] = torch.arange(4.0, device=DEV)[:, None]
    dx = moe.dispatch_backward(dp, tm)
    assert dx[:, 0].tolist() == [1.0, 3.0, 0.0, 2.0]


def test_adjoint_of_the_forward_calls():
    """<dout, combine(y)> and <dpacked, dispatch(x)> are bilinear: the gradients must give the
    same numbers.  f32 throughout; sums in f64, each side off by its operators' f32 roundings."""
    note("adjoint")
    T, H, E, K = 150, 512, 16, 4
    g = _gen(21)
    idx, d0, rows = _routing(g, T, E, K, 0)
    x = _randn(g, (T, H))
    d = moe.dispatch(x, idx, E)
    dp = _randn(g, (rows, H))
    owned = torch.zeros(rows, dtype=torch.bool, device=DEV)
    owned[d.tok_map[d.tok_map >= 0]] = True
    lhs = (dp.double() * d.packed.double())[owned].sum()
    dx = moe.dispatch_backward(dp, d.tok_map)
    rhs = (dx.double() * x.double()).sum()
    mag = (dp.double().abs() * d.packed.double().abs())[owned].sum()
    assert (lhs - rhs).abs() <= mag * (K + 1) * U
    y, w, dout = _randn(g, (rows, H)), torch.rand((T, K), generator=g).to(DEV), _randn(g, (T, H))
    out, _ = moe.combine(y, d.tok_map, w, out_dtype=F32)
    dy, dw = moe.combine_backward(dout, y, d.tok_map, w, packed_cnt=d.packed_cnt, packed_off=d.packed_off)
    lhs = (dout.double() * out.double()).sum()
    mag = (dy.double().abs() * y.double().abs())[owned].sum()
    assert (lhs - (dy.double() * y.double())[owned].sum()).abs() <= mag * (2 * K + 3) * U
    assert (lhs - (dw.double() * w.double()).sum()).abs() <= mag * (2 * K + H / 8 + 20) * U


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------

def _ids(g, N, V, kind, idt):
    if kind == "zipf":
        p = 1.0 / torch.arange(1, V + 1, dtype=torch.float64)
        ids = torch.multinomial(p, N, replacement=True, generator=g) if N else torch.zeros(0)
    elif kind == "same":
        ids = torch.full((N,), V // 2)
    elif kind == "distinct":
        ids = torch.randperm(V, generator=g)[:N] if N <= V else torch.arange(N) % V
    elif kind == "runs":                       # a few tokens, each many times, far apart
        ids = torch.randint(0, min(V, 5), (N,), generator=g) * max(1, V // 5 - 1)
    else:
        ids = torch.randint(0, V, (N,), generator=g)
    ids = ids.to(idt)
    if kind == "padded" and N:
        ids[torch.rand(N, generator=g) < 0.4] = -1
        ids[N // 2:N // 2 + 2] = V
        ids[0] = -7
        if idt == torch.int64:
            ids[N // 3] = (1 << 32) + 1        # a valid id in its low 32 bits
    return ids.to(DEV)


@pytest.mark.parametrize("tdt,odt", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("N,V,H,kind,idt", [
    (0, 5, 8, "uniform", torch.int32), (1, 1, 8, "uniform", torch.int64), (1, 100, 7168, "uniform", torch.int32),
    (33, 7, 2056, "padded", torch.int64), (1000, 300, 1000, "padded", torch.int32),
    (129, 5000, 4096, "zipf", torch.int64)])
def test_embedding(N, V, H, kind, idt, tdt, odt):
    note(f"embedding {N} {V} {H} {kind} {idt} {tdt} {odt}")
    g = _gen(N + V + H)
    table = _randn(g, (V, H), tdt)
    ids = _ids(g, N, V, kind, idt)
    stats = torch.full((1,), 99, dtype=torch.int32, device=DEV)
    got = moe.embedding(ids, table, scale=1.7, out_dtype=odt, stats=stats)
    ok = (ids >= 0) & (ids < V)
    want = table[torch.where(ok, ids, 0).long()].float() * torch.tensor(1.7, dtype=F32, device=DEV)
    _same(got, torch.where(ok[:, None], want, 0.0).to(odt), "out")
    assert stats.item() == ((~ok) & (ids != -1)).sum().item()


GRAD = [(1, 1, 8, "uniform"), (0, 9, 16, "uniform"), (1, 600, 7168, "uniform"), (2, 2, 64, "same"),
        (63, 10, 520, "zipf"), (64, 513, 8, "distinct"), (255, 3, 128, "zipf"), (256, 300, 256, "same"),
        (257, 300, 256, "same"), (300, 5000, 1000, "padded"), (777, 65537, 64, "zipf"),
        (1024, 200, 2048, "padded"), (1025, 40, 4104, "runs"), (2500, 2, 72, "runs"), (3000, 131072, 16, "zipf"),
        (4099, 1000, 136, "same"), (5000, 262145, 8, "zipf"), (9000, 50, 64, "runs"), (20000, 3000, 48, "zipf"),
        (4096, 700, 64, "zipf"), (4097, 512, 8, "padded"), (4100, 500, 33016, "padded"),
        (5000, 6001, 4104, "zipf"), (4608, 9, 24, "same"), (70000, 200, 8, "zipf"),
        (300000, 5000, 8, "runs"), (262144, 3000, 8, "zipf"), (262145, 700, 16, "padded")]


def _grad_ref(dout, ids, V, scale):
    ok = (ids >= 0) & (ids < V)
    at = ids[ok].long()
    ref = torch.zeros((V, dout.shape[1]), dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(ref)
    ref.index_put_((at,), dout[ok].double(), accumulate=True)
    mag.index_put_((at,), dout[ok].double().abs(), accumulate=True)
    cnt = torch.bincount(at, minlength=V)[:, None].double()
    return ref * scale, mag * scale * (cnt + 3) * U, cnt[:, 0] > 0      # cnt additions, the scale, the base


@pytest.mark.parametrize("ddt,tdt", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("N,V,H,kind", GRAD)
def test_embedding_backward(N, V, H, kind, ddt, tdt):
    note(f"embedding_backward {N} {V} {H} {kind} {ddt} {tdt}")
    g = _gen(N * 3 + V + H)
    idt = torch.int64 if N % 2 else torch.int32
    dout, ids = _randn(g, (N, H), ddt), _ids(g, N, V, kind, idt)
    ref, tol, present = _grad_ref(dout, ids, V, 3.25)
    ws = moe.embedding_workspace(N, V, H)
    ws.fill_(0xA5)
    got = torch.full((V, H), torch.nan, dtype=tdt, device=DEV)
    assert moe.embedding_backward(dout, ids, V, scale=3.25, dtable=got, ws=ws) is got
    _near(got, ref, tol, "dtable")
    assert (got[~present] == 0).all()
    again = moe.embedding_backward(dout, ids, V, scale=3.25, dtable_dtype=tdt, ws=ws)
    _same(again, got, "second call on the same workspace")
    base = _randn(g, (V, H), tdt)
    base[~present] = torch.nan                  # rows that must be neither read nor written
    acc = base.clone()
    moe.embedding_backward(dout, ids, V, scale=3.25, accumulate=True, dtable=acc, ws=ws)
    _same(acc[~present], base[~present], "rows of absent tokens")
    want = base.double()[present] + ref[present]
    _near(acc[present], want, tol[present] + want.abs() * U, "accumulated")


def test_embedding_backward_ignores_rows_without_token():
    note("embedding_backward padding rows")
    dout = torch.full((40, 64), torch.nan, device=DEV)
    ids = torch.full((40,), -1, dtype=torch.int64, device=DEV)
    ids[[3, 17, 39]] = torch.tensor([5, 0, 5], device=DEV)
    dout[[3, 17, 39]] = torch.tensor([1.0, 2.0, 4.0], device=DEV)[:, None]
    got = moe.embedding_backward(dout, ids, 8)
    assert got[:, 0].tolist() == [2.0, 0, 0, 0, 0, 5.0, 0, 0]
    ids.fill_(-1)
    assert (moe.embedding_backward(dout, ids, 8) == 0).all()


def test_embedding_gradient_against_the_lookup():
    """<dout, embedding(table)> is linear in the table: its gradient gives the same number."""
    note("embedding adjoint")
    N, V, H = 500, 90, 256
    g = _gen(6)
    ids, table, dout = _ids(g, N, V, "padded", torch.int64), _randn(g, (V, H)), _randn(g, (N, H))
    out = moe.embedding(ids, table, scale=2.0)
    dt = moe.embedding_backward(dout, ids, V, scale=2.0)
    lhs, rhs = (out.double() * dout.double()).sum(), (dt.double() * table.double()).sum()
    mag = (out.double() * dout.double()).abs().sum()
    assert (lhs - rhs).abs() <= mag * (N + 4) * U


# ---------------------------------------------------------------------------
# as they are used: together, captured, on other streams, refused
# ---------------------------------------------------------------------------

def test_training_step_of_a_moe_layer():
    """tokens -> embedding -> gate -> dispatch -> experts -> combine -> loss, and back: every
    gradient against torch's autograd of the same layer in 64 bits.  Experts are one scale per
    expert; the logits come from a matrix that the test owns.  Each value passes through about
    H + K + 50 f32 roundings of terms whose magnitudes the test sums; the bound is taken from the
    largest magnitude of each gradient, 4 (H + K + 50) u times it, plus the runs of the table."""
    note("training step")
    T, H, E, K, V = 300, 256, 16, 4, 120
    g = _gen(99)
    ids = _ids(g, T, V, "zipf", torch.int64)
    table, wg = _randn(g, (V, H), F32, 0.5), _randn(g, (H, E), F32, H ** -0.5)
    c, target = torch.rand(E, generator=g).to(DEV) + 0.5, _randn(g, (T, H))

    x = moe.embedding(ids, table, scale=2.0)
    logits = (x.double() @ wg.double()).float()
    idx, w = moe.gate(logits, K)
    d = moe.dispatch(x, idx, E)
    e_of = torch.repeat_interleave(torch.arange(E, device=DEV), d.packed_cnt.long())
    y = d.packed * c[e_of, None]
    out, _ = moe.combine(y, d.tok_map, w, out_dtype=F32)
    dout = out - target
    dy, dw = moe.combine_backward(dout, y, d.tok_map, w, packed_cnt=d.packed_cnt, packed_off=d.packed_off)
    dpk = dy * c[e_of, None]
    dlogits = moe.gate_backward(logits, idx, dw)
    through_gate = (dlogits.double() @ wg.double().T).float()
    dx = moe.dispatch_backward(dpk, d.tok_map, residual=through_gate)
    dtable = moe.embedding_backward(dx, ids, V, scale=2.0)

    t64 = table.double().requires_grad_()
    x64 = t64[ids] * 2.0
    l64 = x64 @ wg.double()
    l64.retain_grad()
    w64 = torch.softmax(l64.gather(1, idx.long()), 1)
    o64 = (w64.unsqueeze(-1) * (x64.unsqueeze(1) * c.double()[idx.long()].unsqueeze(-1))).sum(1)
    (0.5 * (o64 - target.double()).square().sum()).backward()
    n = 4 * (H + K + 50)
    for got, want, what, more in ((dlogits, l64.grad, "dlogits", 0), (dtable, t64.grad, "dtable", T)):
        err = (got.double() - want).abs().max().item()
        lim = (n + more) * U * want.abs().max().item() * K
        assert err <= lim, (what, err, lim)


def _everything(c, o):
    moe.gate(c["logits"], c["K"], renormalize=False, idx=o["idx"], w=o["w"])
    moe.gate_backward(c["logits"], c["idx"], c["dw"], renormalize=False, dlogits=o["dl"])
    moe.combine_backward(c["dout"], c["y"], c["tm"], c["w"], packed_cnt=c["pc"], packed_off=c["po"],
                         dy=o["dy"], dw=o["dw"])
    moe.dispatch_backward(c["y"], c["tm"], residual=c["dout"], dx=o["dx"])
    moe.embedding(c["ids"], c["table"], scale=0.5, out=o["emb"], stats=o["st"])
    moe.embedding_backward(c["dout"], c["ids"], c["V"], scale=0.5, dtable=o["dt"], ws=c["ws"])
    moe.embedding_backward(c["dout"][:100], c["ids"][:100], c["V"], dtable=o["dt2"], ws=c["ws"])


def _everything_inputs(seed):
    T, H, E, K, V = 6000, 520, 32, 4, 700      # past 4096 positions: sorted by digits
    g = _gen(seed)
    idx, d, rows = _routing(g, T, E, K, 1000)
    c = dict(K=K, V=V, logits=_randn(g, (T, E)), idx=idx, dw=_randn(g, (T, K)), dout=_randn(g, (T, H), BF16),
             y=_randn(g, (rows, H), BF16), tm=d.tok_map, w=torch.rand((T, K), generator=g).to(DEV),
             pc=d.packed_cnt, po=d.packed_off, ids=_ids(g, T, V, "zipf", torch.int64),
             table=_randn(g, (V, H), BF16), ws=moe.embedding_workspace(T, V, H))
    e = lambda *s, dt=F32: torch.empty(s, dtype=dt, device=DEV)                     # noqa: E731
    def outs():
        return dict(idx=e(T, K, dt=torch.int32), w=e(T, K), dl=e(T, E), dy=e(rows, H, dt=BF16), dw=e(T, K),
                    dx=e(T, H, dt=BF16), emb=e(T, H, dt=BF16), st=e(1, dt=torch.int32), dt=e(V, H), dt2=e(V, H))
    return c, outs


def _fill(o):
    for t in o.values():
        t.view(torch.uint8).fill_(0xA5)


def test_captured_in_a_graph():
    """One graph of every call, replayed four times; the same calls run eagerly on the same
    workspace between the replays."""
    note("graph")
    c, outs = _everything_inputs(31)
    ref, o, other = outs(), outs(), outs()
    _everything(c, ref)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _everything(c, o)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _everything(c, o)
    for i in range(4):
        _fill(o)
        _fill(other)
        graph.replay()
        _everything(c, other)
        torch.cuda.synchronize()
        for k in ref:
            _same(o[k], ref[k], f"replay {i}: {k}")
            _same(other[k], ref[k], f"eager {i}: {k}")


def test_two_graphs_on_one_workspace():
    """Two captured graphs whose sorts take other sizes and numbers of passes, replayed in turn on
    one stream with one workspace between them."""
    note("two graphs")
    g = _gen(61)
    a = dict(V=700, ids=_ids(g, 6000, 700, "zipf", torch.int64), dout=_randn(g, (6000, 264), BF16))
    b = dict(V=300001, ids=_ids(g, 9000, 300001, "zipf", torch.int32), dout=_randn(g, (9000, 8), BF16))
    size = max(moe.embedding_workspace_size(c["dout"].shape[0], c["V"], c["dout"].shape[1]) for c in (a, b))
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    graphs = []
    for c in (a, b):
        c["ref"] = moe.embedding_backward(c["dout"], c["ids"], c["V"])
        c["out"] = torch.empty_like(c["ref"])
        moe.embedding_backward(c["dout"], c["ids"], c["V"], dtable=c["out"], ws=ws)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            moe.embedding_backward(c["dout"], c["ids"], c["V"], dtable=c["out"], ws=ws)
        graphs.append(gr)
    for i in range(4):
        for c in (a, b):
            c["out"].fill_(float("nan"))
        for gr in graphs:
            gr.replay()
        for c in (a, b):
            _same(c["out"], c["ref"], f"replay {i}")


def test_two_streams():
    """The same calls on two streams at once, each with its own workspace and buffers."""
    note("streams")
    pair = [_everything_inputs(s) for s in (41, 42)]
    refs = []
    for c, outs in pair:
        r = outs()
        _everything(c, r)
        refs.append(r)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pair]
    got = [outs() for _, outs in pair]
    for o in got:
        _fill(o)
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (c, _), o in zip(streams, pair, got):
            with torch.cuda.stream(s):
                _everything(c, o)
    torch.cuda.synchronize()
    for r, o in zip(refs, got):
        for k in r:
            _same(o[k], r[k], k)


def test_rows_past_four_gib():
    """Row offsets past 2^32 bytes: the last rows of a 5 GiB buffer, in every row mover."""
    note("5 GiB")
    H = 8192
    rows = (5 << 30) // (2 * H)
    big = torch.empty((rows, H), dtype=BF16, device=DEV)
    g = _gen(12)
    last = torch.tensor([rows - 1, rows - 2, 3, rows // 2 + 1], device=DEV)
    vals = _randn(g, (4, H), BF16)
    big[last] = vals
    out = moe.embedding(last, big)
    _same(out, vals, "embedding")
    dx = moe.dispatch_backward(big, last.view(2, 2))
    _same(dx, (vals[0::2].float() + vals[1::2].float()).to(BF16), "dispatch_backward")
    dout, w = _randn(g, (2, H), BF16), torch.ones((2, 2), device=DEV)
    _, dw = moe.combine_backward(dout, big, last.view(2, 2), w, want_dy=False)
    ref = (dout.double()[:, None] * vals.double().view(2, 2, H)).sum(-1)
    mag = (dout.double()[:, None] * vals.double().view(2, 2, H)).abs().sum(-1)
    _near(dw, ref, mag * (H / 8 + 17) * U, "dw")
    moe.combine_backward(dout, None, last.view(2, 2), w, dy=big, want_dw=False)
    _same(big[last].view(2, 2, H), dout[:, None].expand(2, 2, H).contiguous(), "dy")
    moe.embedding_backward(vals, last, rows, dtable=big)
    _same(big[last], vals, "dtable")
    assert (big[[0, rows // 2, rows - 3]] == 0).all()


def test_more_workgroups_than_one_launch_holds():
    """2^22 + 37 tokens: the row movers' grids are capped there and loop over the rest."""
    note("2^22 + 37 tokens")
    T, H = (1 << 22) + 37, 8
    g = _gen(70)
    rows = _randn(g, (T, H), BF16)
    tm = torch.randperm(T, generator=g).to(DEV).view(T, 1)
    _same(moe.dispatch_backward(rows, tm), rows[tm[:, 0]], "dx")
    w = torch.full((T, 1), 0.5, device=DEV)
    dy, dw = moe.combine_backward(rows, rows, tm, w)
    want = torch.empty_like(rows)
    want[tm[:, 0]] = rows * 0.5
    _same(dy, want, "dy")
    prod = rows.double() * rows[tm[:, 0]].double()
    _near(dw, prod.sum(1, keepdim=True), prod.abs().sum(1, keepdim=True) * (H / 8 + 17) * U, "dw")
    _same(moe.embedding(tm[:, 0], rows, scale=2.0), rows[tm[:, 0]] * 2.0, "embedding")
    _same(moe.embedding_backward(rows, tm[:, 0], T, dtable_dtype=BF16)[tm[:, 0]], rows, "dtable")


def test_refusals():
    """What the tensors show is refused before the call, and no buffer changes."""
    note("refusals")
    c, outs = _everything_inputs(51)
    o = outs()
    _fill(o)
    before = {k: v.clone() for k, v in o.items()}
    T, E = c["logits"].shape
    H = c["dout"].shape[1]
    bad = [
        lambda: moe.gate(c["logits"].cpu(), 2), lambda: moe.gate(c["logits"].half(), 2),
        lambda: moe.gate(c["logits"][:, ::2], 2), lambda: moe.gate(c["logits"], 4, idx=o["w"]),
        lambda: moe.gate(c["logits"], 3, w=o["w"]), lambda: moe.gate(c["logits"][0], 2),
        lambda: moe.gate_backward(c["logits"], c["idx"].long(), c["dw"]),
        lambda: moe.gate_backward(c["logits"], c["idx"], c["dw"][:-1]),
        lambda: moe.gate_backward(c["logits"], c["idx"], c["dw"], dlogits=o["dl"].to(BF16)),
        lambda: moe.combine_backward(c["dout"].t(), c["y"], c["tm"], c["w"]),
        lambda: moe.combine_backward(c["dout"], c["y"].cpu(), c["tm"], c["w"]),
        lambda: moe.combine_backward(c["dout"], c["y"][:, :-8], c["tm"], c["w"]),
        lambda: moe.combine_backward(c["dout"], c["y"], c["tm"].int(), c["w"]),
        lambda: moe.combine_backward(c["dout"], c["y"], c["tm"], c["w"].double()),
        lambda: moe.combine_backward(c["dout"], c["y"], c["tm"], None),
        lambda: moe.combine_backward(c["dout"], None, c["tm"], c["w"]),
        lambda: moe.combine_backward(c["dout"], c["y"], c["tm"], c["w"], fp4=True),
        lambda: moe.combine_backward(c["dout"], c["y"], c["tm"], c["w"], packed_cnt=c["pc"]),
        lambda: moe.combine_backward(c["dout"], c["y"], c["tm"], c["w"], packed_cnt=c["pc"],
                                     packed_off=c["po"][:-1]),
        lambda: moe.combine_backward(c["dout"], c["y"], c["tm"], c["w"], dy=o["dx"]),
        lambda: moe.combine_backward(c["dout"], c["y"], c["tm"], c["w"], want_dy=False, want_dw=False),
        lambda: moe.dispatch_backward(c["y"], c["tm"], residual=c["dout"][:-1]),
        lambda: moe.dispatch_backward(c["y"], c["tm"], residual=c["dout"], dx_dtype=F32),
        lambda: moe.dispatch_backward(c["y"][:, ::2], c["tm"]),
        lambda: moe.embedding(c["ids"].to(torch.int16), c["table"]), lambda: moe.embedding(c["ids"][::2], c["table"]),
        lambda: moe.embedding(c["ids"], c["table"].t()), lambda: moe.embedding(c["ids"].cpu(), c["table"]),
        lambda: moe.embedding(c["ids"], c["table"], out=o["dx"][:-1]),
        lambda: moe.embedding_backward(c["dout"], c["ids"], c["V"], accumulate=True),
        lambda: moe.embedding_backward(c["dout"], c["ids"][:-1], c["V"]),
        lambda: moe.embedding_backward(c["dout"], c["ids"], c["V"] + 1, dtable=o["dt"]),
        lambda: moe.embedding_backward(c["dout"], c["ids"], c["V"], ws=c["ws"].view(torch.int8)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("accepted:", i)
    refused = [
        lambda: moe.gate(c["logits"], 17), lambda: moe.gate(c["logits"][:, :4].contiguous(), 5),
        lambda: moe.gate_backward(c["logits"], c["idx"], c["dw"], dlogits=c["logits"]),
        lambda: moe.combine_backward(c["dout"], c["y"], c["tm"], c["w"], dy=c["y"]),
        lambda: moe.dispatch_backward(c["y"], c["tm"], dx=c["y"][:T]),
        lambda: moe.dispatch_backward(c["y"][:, :4].contiguous(), c["tm"]),
        lambda: moe.embedding(c["ids"][:c["V"]], c["table"], out=c["table"]),
        lambda: moe.embedding_backward(c["dout"], c["ids"], c["V"], dtable=o["dt"], ws=c["ws"][:-256]),
        lambda: moe.embedding_backward(c["dout"][:c["V"]], c["ids"][:c["V"]], c["V"],
                                       dtable=c["dout"][:c["V"]], ws=c["ws"]),
    ]
    saved = {k: v.clone() for k, v in c.items() if isinstance(v, torch.Tensor)}
    for f in refused:
        with pytest.raises(moe.MoeError):
            f()
    torch.cuda.synchronize()
    for k, v in saved.items():
        if k != "ws":
            _same(c[k], v, k)
    for k in o:
        _same(o[k], before[k], k)
