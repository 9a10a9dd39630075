"""GPU tests of the row operators of the experts' step against plain torch in 64 bits:
MXFP4 quantization, SwiGLU with its 8-bit checkpoint, and its gradient.

Tolerances.  u = 2^-24 is the most that one f32 rounding is off, relative to its result.
Quantization has one rounding, to codes, and is compared bit for bit.  SwiGLU: t =
exp(-|g|) is off by at most 6u (the two parts of its argument 1u each, exp2 2u, the
correction 2u), 1 + t by u more than half of that (t / (1 + t) <= 1/2), its reciprocal
by 2u more: r 6u, t*r 13u; the products that follow add 1u each.  exp2's result has no
subnormals: t below 2^-126 comes out 0, which moves s by at most MIN = 2^-126, an
absolute error that the factors beside s scale."""
import numpy as np
import pytest
import torch

import combine_moe_route_count_amd as moe
from _gpu_util import DEV, note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
MIN = 2.0 ** -126
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _pow2(e):
    return torch.from_numpy(np.ldexp(1.0, e.numpy().astype(np.int64)))


# ---------------------------------------------------------------------------
# MXFP4
# ---------------------------------------------------------------------------

def _mx_ref(x):
    """(codes [R,H/2], scales [R,H/32]) of x (CPU), element by element in 64 bits."""
    b = x.double().unflatten(-1, (-1, 32))
    fin = torch.where(torch.isfinite(b), b.abs(), 0.0)
    amax = fin.amax(-1)
    _, ex = np.frexp(amax.numpy())
    e = torch.from_numpy(ex.astype(np.int64)) - 2          # amax / 2^e in [2, 4)
    e = torch.where(amax / _pow2(e) >= 3.5, e, e - 1)
    e = torch.where(amax == 0, 0, e.clamp(min=-127))
    v = (b / _pow2(e).unsqueeze(-1)).abs().clamp(max=6.0)
    v = torch.where(torch.isinf(b), 6.0, v)
    nan = torch.isnan(b).any(-1)
    v = torch.where(nan.unsqueeze(-1), 0.0, v)
    d = (v.unsqueeze(-1) - E2M1).abs()
    best = d.amin(-1, keepdim=True)
    # nearest value; of two equally near the even code
    odd = torch.arange(8) % 2
    code = torch.where(d == best, odd, 2).argmin(-1)
    code = code + 8 * torch.signbit(b)
    code = torch.where(nan.unsqueeze(-1), 0, code).flatten(-2).to(torch.uint8)
    scale = torch.where(nan, 255, e + 127).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _mx_values(codes, scales):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    v = torch.where(c >= 8, -E2M1[c & 7], E2M1[c & 7]).unflatten(-1, (-1, 32))
    s = torch.where(scales == 255, torch.tensor(NAN, dtype=torch.float64), _pow2(scales.long() - 127))
    return (v * s.unsqueeze(-1)).flatten(-2)


def _check_quantize(x, what):
    codes, scales = moe.mxfp4_quantize(x.to(DEV))
    torch.cuda.synchronize()
    rc, rs = _mx_ref(x)
    assert torch.equal(scales.cpu(), rs), f"{what}: {(scales.cpu() != rs).sum()} scales differ"
    assert torch.equal(codes.cpu(), rc), f"{what}: {(codes.cpu() != rc).sum()} code bytes differ"
    return codes, scales


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("rows,H", [(1, 32), (1, 96), (3, 1056), (257, 64), (40, 7168), (1031, 992)])
def test_quantize_matches_definition(rows, H, dt):
    note(f"quantize {rows}x{H} {dt}")
    g = _gen(rows * 7 + H)
    x = torch.randn((rows, H), generator=g) * torch.exp2(6 * torch.randn((rows, 1), generator=g))
    codes, scales = _check_quantize(x.to(dt), "normal")
    for out in (F32, BF16):
        y = moe.mxfp4_dequantize(codes, scales, out_dtype=out)
        torch.cuda.synchronize()
        want = _mx_values(codes.cpu(), scales.cpu())
        assert torch.equal(y.cpu().double(), want.to(out).double()), out


@pytest.mark.parametrize("dt", [BF16, F32])
def test_quantize_borders(dt):
    """Ties, the border of the scale, signs of zero, tiny and huge blocks, infinities, NaN."""
    note(f"quantize borders {dt}")
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 6.5, 6.96875]
    rows = []
    for top in (3.5, 4.0, 6.0, 6.96875):              # largest of the block, in units of the scale
        for e in (-126, -20, 0, 90, 124):
            v = [top, -top] + mids[:8] + [-m for m in mids[:8]] + [0.0, -0.0]
            v = [max(-top, min(top, a)) for a in v] + [0.1] * (32 - len(v))
            rows.append([a * 2.0 ** e for a in v])
    rows.append([0.0] * 32)
    rows.append([-0.0] * 32)
    rows.append([INF] + [0.0] * 31)
    rows.append([-INF, 3.0, -1.0, 0.75] + [0.5] * 28)
    rows.append([NAN] + [1.0] * 31)
    rows.append([1.0] * 30 + [-NAN, INF])
    rows.append([1e-40] * 16 + [-3e-39] * 16)          # subnormal in both types
    rows.append([3.38e38, -3.38e38] + [1e38] * 30)
    x = torch.tensor(rows, dtype=torch.float64).to(dt)
    codes, scales = _check_quantize(x, "borders")
    y = moe.mxfp4_dequantize(codes, scales, out_dtype=F32).cpu()
    want = _mx_values(codes.cpu(), scales.cpu()).to(F32)
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(y[~torch.isnan(y)], want[~torch.isnan(want)])


@pytest.mark.parametrize("out", [BF16, F32])
def test_dequantize_every_code_and_scale(out):
    note(f"dequantize all {out}")
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)[:16 * 16].view(16, 16)
    codes = codes.repeat(256, 1).contiguous()             # [4096, 16]: every byte under every scale
    scales = torch.arange(256).repeat_interleave(16).to(torch.uint8).view(-1, 1).contiguous()
    y = moe.mxfp4_dequantize(codes.to(DEV), scales.to(DEV), out_dtype=out).cpu()
    want = _mx_values(codes, scales).to(F32).to(out)     # 6 * 2^127 and the like are infinite
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(y[ok], want[ok])
    assert torch.equal(torch.signbit(y[ok]), torch.signbit(want[ok]))


def test_quantize_past_32_bit_offsets():
    """More than 2^32 bytes of input; only the last rows are compared."""
    rows, H = 310000, 7168
    note("quantize long")
    x = torch.zeros((rows, H), dtype=BF16, device=DEV)
    tail = torch.randn((64, H), generator=_gen(5)).to(BF16)
    x[-64:] = tail.to(DEV)
    codes, scales = moe.mxfp4_quantize(x)
    y = moe.mxfp4_dequantize(codes, scales)
    torch.cuda.synchronize()
    rc, rs = _mx_ref(tail)
    assert torch.equal(codes[-64:].cpu(), rc) and torch.equal(scales[-64:].cpu(), rs)
    assert torch.equal(y[-64:].cpu().double(), _mx_values(rc, rs))
    assert not y[:-64].any()


def test_quantize_empty():
    x = torch.empty((0, 64), dtype=BF16, device=DEV)
    codes, scales = moe.mxfp4_quantize(x)
    assert codes.shape == (0, 32) and scales.shape == (0, 2)
    assert moe.mxfp4_dequantize(codes, scales).shape == (0, 64)


# ---------------------------------------------------------------------------
# SwiGLU
# ---------------------------------------------------------------------------

def _near(got, want, tol, what):
    """|got - want| <= tol, plus the rounding of got's own type; NaN and infinities in place."""
    g = got.cpu().double()
    assert torch.equal(torch.isnan(g), torch.isnan(want)), f"{what}: NaN in other places"
    fin = torch.isfinite(want)
    assert torch.equal(g[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)]), what
    lim = (tol + want.abs() * (torch.finfo(got.dtype).eps / 2)) * (1 + 2.0 ** -7) + 1e-37
    over = ((g - want).abs() > lim) & fin
    assert not over.any(), f"{what}: {over.sum().item()} of {over.numel()} past the bound"


def _parts(gu):
    g, u = gu.double().chunk(2, -1)
    return g, u, torch.sigmoid(g), torch.sigmoid(-g)


def _h_tol(g, u, s):
    """Bound of g * s * u."""
    return (g * s * u).abs() * 15 * U + (g * u).abs() * MIN


def _owned(cnt, off, rows):
    keep = torch.zeros(rows, dtype=torch.bool)
    for c, o in zip(cnt.tolist(), off.tolist()):
        keep[max(0, o):max(0, min(rows, o + c))] = True
    return keep


SEGMENTS = {
    "all": None,
    "compact": ([3, 0, 5, 1, 0], [0, 3, 3, 8, 9, 9]),
    "padded": ([2, 4, 0, 3], [0, 4, 8, 12, 16]),
    "late": ([2, 1], [5, 9, 12]),                # rows before the first segment
    "one": ([7], [0, 7]),
    "outside": ([2, 1 << 30], [0, 10, 1 << 30]),   # reaches past the buffer
}


def _segments(name):
    if SEGMENTS[name] is None:
        return None, None
    return tuple(torch.tensor(v, dtype=torch.int32) for v in SEGMENTS[name])


def _dev(t):
    return None if t is None else t.to(DEV)


def _gu(rows, I, dt, seed, keep=None):
    gu = (torch.randn((rows, 2 * I), generator=_gen(seed)) * 2).to(dt)
    gu[:, ::7] *= 20
    if keep is not None:           # whatever stands in rows that nobody owns is not looked at
        gu[~keep] = NAN
        gu[~keep, ::3] = INF
    return gu


def _e4m3_ref(x):
    """(codes, scales) of the checkpoint of x (CPU, finite)."""
    b = x.double().unflatten(-1, (-1, 128))
    amax = b.abs().amax(-1)
    _, ex = np.frexp(amax.numpy())
    k = torch.from_numpy(ex.astype(np.int64)) - 9
    k = torch.where(amax > 448.0 * _pow2(k), k + 1, k)
    k = torch.where(amax == 0, 0, k.clamp(min=-126))
    s = _pow2(k)
    q = (b / s.unsqueeze(-1)).float().to(torch.float8_e4m3fn)
    return q.flatten(-2).view(torch.uint8), s.float()


@pytest.mark.parametrize("segs", list(SEGMENTS))
@pytest.mark.parametrize("gu_dt,h_dt", [(BF16, BF16), (F32, F32), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("I,save", [(8, False), (40, False), (776, False), (128, True),
                                    (640, True), (2176, True), (4104, False)])
def test_swiglu(I, save, gu_dt, h_dt, segs):
    rows = 17
    cnt, off = _segments(segs)
    keep = torch.ones(rows, dtype=torch.bool) if cnt is None else _owned(cnt, off, rows)
    note(f"swiglu {I} {save} {gu_dt} {h_dt} {segs}")
    gu = _gu(rows, I, gu_dt, I, keep)
    h = torch.full((rows, I), 7.0, dtype=h_dt, device=DEV)
    codes = scales = None
    if save:
        codes = torch.full((rows, 2 * I), 0xA5, dtype=torch.uint8, device=DEV)
        scales = torch.full((rows, I // 64), 7.0, device=DEV)
    moe.swiglu(gu.to(DEV), _dev(cnt), _dev(off), save=save, h=h, codes=codes, scales=scales)
    torch.cuda.synchronize()
    g, u, s, _ = _parts(gu[keep])
    _near(h[keep.to(DEV)], g * s * u, _h_tol(g, u, s), "h")
    assert (h.cpu()[~keep] == 7).all()
    if save:
        rc, rs = _e4m3_ref(gu[keep])
        assert torch.equal(scales.cpu()[keep], rs) and torch.equal(codes.cpu()[keep], rc)
        assert (codes.cpu()[~keep] == 0xA5).all() and (scales.cpu()[~keep] == 7).all()


@pytest.mark.parametrize("segs", list(SEGMENTS))
@pytest.mark.parametrize("kind", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("dh_dt,out_dt", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("I", [8, 776, 128, 1920, 2304])
def test_swiglu_backward(I, dh_dt, out_dt, kind, segs):
    if kind == "fp8" and I % 128:
        I = 256
    rows = 17
    cnt, off = _segments(segs)
    keep = torch.ones(rows, dtype=torch.bool) if cnt is None else _owned(cnt, off, rows)
    note(f"swiglu_backward {I} {kind} {dh_dt} {out_dt} {segs}")
    gu = _gu(rows, I, F32 if kind != "bf16" else BF16, I + 1)
    scales = None
    if kind == "fp8":
        q, scales = _e4m3_ref(gu)
        gu = q.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(128, 1)
        given = q
    else:
        given = gu
    dh = torch.randn((rows, I), generator=_gen(9)).to(dh_dt)
    dh[~keep] = NAN
    dgu = torch.full((rows, 2 * I), 7.0, dtype=out_dt, device=DEV)
    h = torch.full((rows, I), 7.0, dtype=out_dt, device=DEV)
    moe.swiglu_backward(dh.to(DEV), given.to(DEV), scales=_dev(scales), packed_cnt=_dev(cnt),
                        packed_off=_dev(off), dgu=dgu, h=h)
    torch.cuda.synchronize()
    g, u, s, c = _parts(gu[keep])
    d = dh[keep].double()
    want = d * u * s * (1 + g * c)
    # s 13u, c 13u; g*c, the sum, s*(...), d*u, the last product: 1u each of what they make
    tol = (d * u * s).abs() * (1 + (g * c).abs()) * (13 + 14 + 4) * U
    tol = tol + (d * u).abs() * (1 + g.abs()) * MIN
    _near(dgu[keep.to(DEV)][:, :I], want, tol, "dg")
    _near(dgu[keep.to(DEV)][:, I:], d * g * s, _h_tol(g, d, s), "du")
    _near(h[keep.to(DEV)], g * s * u, _h_tol(g, u, s), "h")
    assert (dgu.cpu()[~keep] == 7).all() and (h.cpu()[~keep] == 7).all()


def test_swiglu_backward_without_h():
    gu = _gu(5, 64, BF16, 3)
    dh = torch.randn((5, 64), generator=_gen(4)).to(BF16)
    a, h = moe.swiglu_backward(dh.to(DEV), gu.to(DEV))
    b, none = moe.swiglu_backward(dh.to(DEV), gu.to(DEV), want_h=False)
    torch.cuda.synchronize()
    assert none is None and h is not None and torch.equal(a, b)


def test_swiglu_far_values():
    """Gates far out, where exp overflows or vanishes, zeros, infinities and NaN."""
    g = torch.tensor([0.0, -0.0, 1e4, -1e4, 200.0, -200.0, 88.0, -88.0, -103.0, INF, NAN, 1e-30,
                      -1e-30, 30.0, -30.0, -50.0])
    u = torch.tensor([1.5, 2.0, 3.0, 3.0, -1.0, 2.0, 0.5, 4.0, 4.0, 1.0, 1.0, 2.0, 2.0, 1.0, 1.0, -3.0])
    gu = torch.cat((g, u)).unsqueeze(0)
    h = moe.swiglu(gu.to(DEV))
    dgu, h2 = moe.swiglu_backward(torch.ones((1, 16), device=DEV), gu.to(DEV))
    torch.cuda.synchronize()
    gd, ud = g.double(), u.double()
    s, c = torch.sigmoid(gd), torch.sigmoid(-gd)
    # an infinite gate: silu' is inf * 0 in the formula
    want_h = gd * s * ud
    _near(h[0], want_h, _h_tol(gd, ud, s), "h")
    _near(h2[0], want_h, _h_tol(gd, ud, s), "h again")
    want = ud * s * (1 + gd * c)
    tol = (ud * s).abs() * (1 + (gd * c).abs()) * 31 * U + ud.abs() * (1 + gd.abs()) * MIN
    _near(dgu[0, :16], want, tol, "dg")
    _near(dgu[0, 16:], gd * s, _h_tol(gd, torch.ones(()), s), "du")


@pytest.mark.parametrize("dt", [BF16, F32])
def test_checkpoint_borders(dt):
    """The border of the scale (1.75 in the largest value's mantissa), tiny, zero and huge blocks,
    infinities and NaN."""
    note(f"checkpoint borders {dt}")
    rows = []
    for e in (-126, -110, -9, 0, 60, 119):
        for top in (1.75, 1.7578125, 1.0, 1.9921875):
            v = torch.linspace(-top, top, 128, dtype=torch.float64) * 2.0 ** e
            rows.append(v)
    rows.append(torch.zeros(128, dtype=torch.float64))
    x = torch.stack(rows)
    gu = torch.cat((x, x.flip(0)), 1).to(dt)
    _, codes, scales = moe.swiglu(gu.to(DEV), save=True)
    torch.cuda.synchronize()
    rc, rs = _e4m3_ref(gu)
    assert torch.equal(scales.cpu(), rs)
    assert torch.equal(codes.cpu(), rc)
    odd = torch.ones((1, 256))
    odd[0, 3], odd[0, 5], odd[0, 130], odd[0, 131] = INF, -INF, NAN, -NAN
    odd[0, 7] = 1.25
    _, codes, scales = moe.swiglu(odd.to(dt).to(DEV), save=True)
    v = moe.fp8_dequant(codes, scales).cpu().float()
    assert scales.cpu().tolist() == [[2.0 ** -8, 2.0 ** -8]]
    assert v[0, 3] == 1.75 and v[0, 5] == -1.75 and v[0, 7] == 1.25 and (v[0, 8:128] == 1).all()
    assert torch.isnan(v[0, 130]) and torch.isnan(v[0, 131]) and (v[0, 132:] == 1).all()


def test_checkpoint_keeps_values_to_half_a_step():
    gu = (torch.randn((64, 512), generator=_gen(1)) * 3).to(BF16)
    _, codes, scales = moe.swiglu(gu.to(DEV), save=True)
    kept = moe.fp8_dequant(codes, scales).cpu().double()
    blk = scales.cpu().double().repeat_interleave(128, 1)
    # relative 2^-4 for normal codes, half of the smallest step 2^-9 for the rest
    lim = torch.maximum(gu.double().abs() * 2.0 ** -4, blk * 2.0 ** -10)
    assert ((kept - gu.double()).abs() <= lim).all()


def test_swiglu_gradient_against_differences():
    g = _gen(11)
    gu = torch.randn((3, 32), generator=g, dtype=torch.float64)
    dh = torch.randn((3, 16), generator=g, dtype=torch.float64)
    dgu, _ = moe.swiglu_backward(dh.float().to(DEV), gu.float().to(DEV))
    gu, dh = gu.float().double(), dh.float().double()

    def f(z):
        a, b = z.chunk(2, -1)
        return (torch.nn.functional.silu(a) * b * dh).sum()
    eps = 1e-5
    for r in range(3):
        for c in range(32):
            d = torch.zeros_like(gu)
            d[r, c] = eps
            num = (f(gu + d) - f(gu - d)) / (2 * eps)
            # central difference: eps^2 / 6 times a third derivative below 10, and f's rounding
            assert abs(num - dgu[r, c].item()) < 1e-8 + 32 * U * (1 + abs(num)), (r, c)


def test_swiglu_long_rows_of_a_big_buffer():
    """Rows past 2^32 bytes of the buffer."""
    rows, I = 300000, 4096
    note("swiglu long")
    gu = torch.zeros((rows, 2 * I), dtype=BF16, device=DEV)
    tail = _gu(8, I, BF16, 2)
    gu[-8:] = tail.to(DEV)
    h, codes, scales = moe.swiglu(gu, save=True)
    dgu, h2 = moe.swiglu_backward(h, codes, scales=scales)
    torch.cuda.synchronize()
    g, u, s, _ = _parts(tail)
    _near(h[-8:], g * s * u, _h_tol(g, u, s), "h")
    rc, rs = _e4m3_ref(tail)
    assert torch.equal(codes[-8:].cpu(), rc) and torch.equal(scales[-8:].cpu(), rs)
    assert not h[:-8].any() and not dgu[:-8].any()
    g, u, s, _ = _parts(rc.view(torch.float8_e4m3fn).double() * rs.double().repeat_interleave(128, 1))
    _near(h2[-8:], g * s * u, _h_tol(g, u, s), "h of the checkpoint")


def test_swiglu_empty():
    gu = torch.empty((0, 256), dtype=BF16, device=DEV)
    h, codes, scales = moe.swiglu(gu, save=True)
    assert h.shape == (0, 128) and codes.shape == (0, 256) and scales.shape == (0, 2)
    dgu, h = moe.swiglu_backward(h, codes, scales=scales)
    assert dgu.shape == (0, 256) and h.shape == (0, 128)
