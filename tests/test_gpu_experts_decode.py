"""GPU tests of the experts' step of a few tokens against its definition in 64 bits.

Tolerances.  u = 2^-24; a sum of n products is off by at most 2*n*u times the sum of their
magnitudes (an addition inside the matrix instruction may cut instead of round, which
costs twice as much; products of bf16 values are exact).  g and u of h = silu(g) * u are
off by dg and du: 1.1*dg*|u| + |silu(g)|*du + dg*du, silu' being at most 1.1 in magnitude,
and (20 + |g|)*u of h for its own steps (exp2's argument is rounded once).  h is then held
in P bf16 parts, off by 2^(-9P) of itself; the second product's sum runs over P*I products
whose magnitudes are at most (1 + 2^-8) of those of h; the sum over k adds K*u."""
import numpy as np
import pytest
import torch

import combine_moe_route_count_amd as moe
from _gpu_util import DEV, note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _values(codes, scales):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    v = torch.where(c >= 8, -E2M1[c & 7], E2M1[c & 7]).unflatten(-1, (-1, 32))
    s = torch.from_numpy(np.ldexp(1.0, scales.numpy().astype(np.int64) - 127))
    s = torch.where(scales == 255, torch.tensor(NAN, dtype=torch.float64), s)
    return (v * s.unsqueeze(-1)).flatten(-2)


def _weights(g, E, rows, cols, mx):
    """(as given, scales or None, values in 64 bits)"""
    if mx:
        c = torch.randint(0, 256, (E, rows, cols // 2), generator=g, dtype=torch.uint8)
        s = torch.randint(119, 125, (E, rows, cols // 32), generator=g, dtype=torch.uint8)
        return c, s, _values(c, s)
    w = (torch.randn((E, rows, cols), generator=g) * cols ** -0.5).to(BF16)
    return w, None, w.double()


def _ref(x, idx, w, v13, v2, P):
    """(out, bound of its error before the rounding to its type)."""
    T, H = x.shape
    E, _, I = v2.shape
    out, tol = (torch.zeros((T, H), dtype=torch.float64) for _ in range(2))
    for t in range(T):
        for k in range(idx.shape[1]):
            e = int(idx[t, k])
            if not 0 <= e < E:
                continue
            z = v13[e] @ x[t]
            d = (v13[e].abs() @ x[t].abs()) * (2 * H * U)
            (g, u), (dg, du) = z.chunk(2), d.chunk(2)
            act = g * torch.sigmoid(g)
            h = act * u
            dh = 1.1 * dg * u.abs() + act.abs() * du + dg * du + h.abs() * (20 + g.abs()) * U
            y = v2[e] @ h
            dy = v2[e].abs() @ (dh + h.abs() * (2.0 ** (-9 * P) + 2 * P * I * U * (1 + 2.0 ** -8)))
            c = float(w[t, k])
            out[t] += c * y
            tol[t] += abs(c) * dy + (c * y).abs() * (idx.shape[1] + 10) * U
    return out, tol


def _check(got, ref, what):
    out, tol = ref
    g = got.cpu().double()
    nan = torch.isnan(out)
    assert torch.equal(torch.isnan(g), nan), f"{what}: NaN in other places"
    lim = (tol + out.abs() * (torch.finfo(got.dtype).eps / 2)) * (1 + 2.0 ** -7) + 1e-37
    over = ((g - out).abs() > lim) & ~nan
    assert not over.any(), f"{what}: {over.sum().item()} of {over.numel()} past the bound"


def _inputs(T, H, I, E, K, mx, seed, none=0.2, same=False):
    g = _gen(seed)
    x = torch.randn((T, H), generator=g).to(BF16)
    idx = torch.stack([torch.randperm(max(E, K), generator=g)[:K] % E for _ in range(T)]) if T else \
        torch.zeros((0, K))
    if same:
        idx = torch.zeros((T, K)) + E // 2
    idx = idx.int()
    idx[torch.rand((T, K), generator=g) < none] = -1
    w = torch.softmax(torch.randn((T, K), generator=g), -1)
    return x, idx, w, _weights(g, E, 2 * I, H, mx), _weights(g, E, H, I, mx)


def _dev(t):
    return None if t is None else t.to(DEV)


def _call(x, idx, w, w13, w2, out, ws=None):
    y = torch.full(x.shape, 7.0, dtype=out, device=DEV)
    moe.experts_decode(x.to(DEV), idx.to(DEV), w.to(DEV), _dev(w13[0]), _dev(w2[0]),
                       w13_scales=_dev(w13[1]), w2_scales=_dev(w2[1]), out=y, ws=ws)
    torch.cuda.synchronize()
    return y


SHAPES = [  # T, H, I, E, K, and whether all entries name one expert
    (1, 32, 32, 1, 1, False), (1, 160, 96, 16, 8, False), (2, 64, 32, 3, 3, False),
    (5, 544, 288, 4, 2, False), (16, 256, 64, 2, 1, False), (17, 96, 160, 1, 1, False),
    (33, 128, 64, 300, 7, False), (40, 64, 96, 6, 2, True), (130, 64, 64, 2, 1, True),
    (64, 96, 32, 1024, 16, False), (3, 1056, 1120, 8, 4, False)]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,H,I,E,K,same", SHAPES)
def test_matches_definition(T, H, I, E, K, same, mx, out):
    note(f"decode T={T} H={H} I={I} E={E} K={K} same={same} mx={mx} {out}")
    x, idx, w, w13, w2 = _inputs(T, H, I, E, K, mx, T + H + I, same=same)
    y = _call(x, idx, w, w13, w2, out)
    _check(y, _ref(x.double(), idx, w, w13[2], w2[2], 3 if out == F32 else 2), "decode")


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("H,I", [(8, 8), (24, 40), (1000, 264), (104, 1336), (2056, 72)])
def test_odd_sizes_in_bf16(H, I, out):
    note(f"decode odd H={H} I={I}")
    x, idx, w, w13, w2 = _inputs(6, H, I, 5, 3, False, H + I)
    y = _call(x, idx, w, w13, w2, out)
    _check(y, _ref(x.double(), idx, w, w13[2], w2[2], 3 if out == F32 else 2), "odd")


@pytest.mark.parametrize("T,H,I,E,K", [(14, 3040, 352, 6, 4), (1, 672, 1984, 18, 2), (9, 992, 2080, 3, 1)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_scale_rows_at_any_byte(T, H, I, E, K, out):
    """Rows of 95, 11, 21, 62, 31 and 65 scales, read 16 bytes at a time."""
    note(f"decode scales T={T} H={H} I={I}")
    x, idx, w, w13, w2 = _inputs(T, H, I, E, K, True, H + I)
    y = _call(x, idx, w, w13, w2, out)
    _check(y, _ref(x.double(), idx, w, w13[2], w2[2], 3 if out == F32 else 2), "scales")


@pytest.mark.parametrize("H,I", [(1024, 128), (96, 800), (2144, 1056)])
@pytest.mark.parametrize("at", [1, 2, 3])
def test_scales_that_begin_anywhere(at, H, I):
    note(f"decode scales at {at} H={H} I={I}")
    x, idx, w, w13, w2 = _inputs(5, H, I, 6, 2, True, H + at)

    def shifted(t):
        flat = torch.full((t.numel() + 8,), 255, dtype=torch.uint8, device=DEV)    # NaN around it
        flat[at:at + t.numel()] = t.to(DEV).flatten()
        return flat[at:at + t.numel()].view(t.shape)
    y = moe.experts_decode(x.to(DEV), idx.to(DEV), w.to(DEV), w13[0].to(DEV), w2[0].to(DEV),
                           shifted(w13[1]), shifted(w2[1]), out_dtype=F32)
    torch.cuda.synchronize()
    _check(y, _ref(x.double(), idx, w, w13[2], w2[2], 3), "shifted")


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T,K", [(5, 1), (11, 1), (20, 4), (33, 2)])
def test_many_entries_of_one_expert_among_many(T, K, out):
    """Few entries per expert on average, all of them on one: more than one pass over its weights."""
    note(f"decode crowd T={T} K={K} {out}")
    x, idx, w, w13, w2 = _inputs(T, 192, 96, 40, K, True, T, none=0.1, same=True)
    y = _call(x, idx, w, w13, w2, out)
    _check(y, _ref(x.double(), idx, w, w13[2], w2[2], 3 if out == F32 else 2), "crowd")


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,E,K", [(1024, 1024, 1), (64, 5, 16), (1024, 1, 1)])
def test_as_many_entries_as_are_allowed(T, E, K, mx):
    note(f"decode full T={T} E={E} K={K} mx={mx}")
    x, idx, w, w13, w2 = _inputs(T, 64, 32, E, K, mx, T + E, none=0.0)
    y = _call(x, idx, w, w13, w2, F32)
    _check(y, _ref(x.double(), idx, w, w13[2], w2[2], 3), "full")


@pytest.mark.parametrize("mx", [False, True])
def test_entries_that_count_for_nothing(mx):
    """Ids outside the experts with weights that must not be read as numbers, an expert named
    twice, tokens without any expert, NaN and infinities in one token only."""
    x, idx, w, w13, w2 = _inputs(6, 64, 32, 4, 4, mx, 9, none=0.0)
    idx[0] = torch.tensor([-1, 4, 1 << 30, -7])
    w[0] = torch.tensor([NAN, INF, -INF, NAN])
    idx[1] = torch.tensor([2, 2, -1, 2])
    w[1, 2] = NAN
    x[2, 5], x[3, 1] = NAN, INF
    y = _call(x, idx, w, w13, w2, F32)
    keep = torch.tensor([0, 1, 4, 5])
    ref = _ref(x.double()[keep], idx[keep], w[keep], w13[2], w2[2], 3)
    _check(y[keep.to(DEV)], ref, "others")
    assert (y[0] == 0).all()
    assert torch.isnan(y[2]).all() and not torch.isfinite(y[3]).any()


def test_no_entry_at_all():
    x, idx, w, w13, w2 = _inputs(3, 64, 32, 4, 2, False, 9)
    idx[:] = -1
    assert (_call(x, idx, w, w13, w2, BF16) == 0).all()


def test_no_tokens():
    x, idx, w, w13, w2 = _inputs(0, 64, 32, 4, 2, False, 9)
    assert _call(x, idx, w, w13, w2, BF16).shape == (0, 64)


def test_every_scale_of_the_weights():
    """One-hot tokens pick weight columns out: block scales from 2^-100 to 2^100 come through, and a
    NaN scale reaches the rows of its block."""
    H = I = 32
    g = _gen(4)
    E = 251
    x = torch.zeros((E, H), dtype=BF16)
    x[torch.arange(E), torch.arange(E) % H] = 1.0
    w13 = torch.randint(0, 256, (E, 2 * I, H // 2), generator=g, dtype=torch.uint8)
    s13 = torch.full((E, 2 * I, 1), 127, dtype=torch.uint8)
    s13[:, I:, 0] = (torch.arange(E) + 3).to(torch.uint8).unsqueeze(1)      # 2^-124 .. 2^126
    w2 = torch.zeros((E, H, I // 2), dtype=torch.uint8)
    for i in range(H):                                  # the identity: h comes out
        w2[:, i, i // 2] = 2 << (4 * (i % 2))
    s2 = torch.full((E, H, 1), 127, dtype=torch.uint8)
    s13[250, I + 4, 0] = 255
    idx, w = torch.arange(E, dtype=torch.int32).unsqueeze(1), torch.ones((E, 1))
    y = _call(x, idx, w, (w13, s13), (w2, s2), F32)
    ref = _ref(x.double(), idx, w, _values(w13, s13), _values(w2, s2), 3)
    # NaN times the identity's zeros: the whole row of that token
    assert torch.isnan(ref[0][250]).all() and torch.isnan(y[250]).all()
    # h is the identity's input: where one of a token's passes f32's largest value it is infinite
    # there, and infinity times the identity's zeros is NaN in the token's whole row
    past = (ref[0].abs() >= 2.0 ** 128).any(1)
    assert past.sum() < 8 and torch.isnan(y.cpu())[past].any(1).all()
    tiny = torch.isnan(ref[0]) | (ref[0].abs() < 2.0 ** -100) | past.unsqueeze(1)
    lim = ref[1] + ref[0].abs() * 2.0 ** -23
    bad = ((y.cpu().double() - ref[0]).abs() > lim) & ~tiny | (torch.isnan(y.cpu()) & ~tiny)
    assert not bad.any(), (bad.any(1).nonzero().flatten().tolist(), y.cpu()[bad][:8], ref[0][bad][:8])
    small = (ref[0].abs() < 2.0 ** -100) & ~past.unsqueeze(1)      # the parts of h are near bf16's subnormals there
    assert ((y.cpu().double() - ref[0]).abs() <= 2.0 ** -110)[small].all()


def test_every_scale_of_the_second_product():
    """The scales of w2 alone, with h of ordinary size."""
    H = I = 32
    g = _gen(5)
    E = 255
    x = torch.randn((E, H), generator=g).to(BF16)
    w13, s13, v13 = _weights(g, E, 2 * I, H, True)
    w2 = torch.randint(0, 256, (E, H, I // 2), generator=g, dtype=torch.uint8)
    s2 = torch.arange(E).to(torch.uint8).view(E, 1, 1).repeat(1, H, 1).contiguous()  # 2^-127 .. 2^127
    idx, w = torch.arange(E, dtype=torch.int32).unsqueeze(1), torch.ones((E, 1))
    y = _call(x, idx, w, (w13, s13), (w2, s2), F32)
    out, tol = _ref(x.double(), idx, w, v13, _values(w2, s2), 3)
    # a code of 4 or 6 times 2^126 and more is past bf16's (and f32's) largest value: infinite
    big = (out.abs() > 2.0 ** 126) | (_values(w2, s2).abs() >= 2.0 ** 128).any(2)
    assert not big[:240].any()
    assert not (~torch.isfinite(y.cpu()) & ~big).any()
    lim = tol + out.abs() * 2.0 ** -23 + 2.0 ** -126      # values of w2 at the subnormal border
    assert ((y.cpu().double() - out).abs() <= lim)[~big].all()


def test_workspace_is_reused_and_bits_do_not_change():
    ws = moe.experts_decode_workspace(64, 4, 96)
    a = _inputs(64, 64, 96, 12, 4, False, 1)
    b = _inputs(2, 1000, 40, 5, 3, False, 2)
    c = _inputs(9, 96, 32, 200, 5, True, 3)
    first = [_call(*i, F32) for i in (a, b, c)]
    for _ in range(3):
        for i, want in zip((a, c, b), (first[0], first[2], first[1])):
            assert torch.equal(_call(*i, F32, ws=ws), want)


def test_captured_and_replayed():
    """Two graphs on one workspace, replayed in turn between eager calls."""
    dev = lambda i: [t.to(DEV) for t in (i[0], i[1], i[2], i[3][0], i[4][0])]
    a, b = _inputs(8, 256, 64, 6, 2, False, 4), _inputs(3, 256, 64, 6, 2, False, 5)
    ws = moe.experts_decode_workspace(8, 2, 64)
    graphs = []
    for i in (a, b):
        d = dev(i)
        out = torch.zeros_like(d[0])
        moe.experts_decode(*d, out=out, ws=ws)
        torch.cuda.synchronize()
        want = out.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.experts_decode(*d, out=out, ws=ws)
        graphs.append((g, d, out, want))
    for r in range(4):
        for g, d, out, want in graphs:
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), r
            assert torch.equal(moe.experts_decode(*d, ws=ws), want)


def test_weights_past_32_bit_offsets():
    """Experts behind 4 GiB of weights."""
    E, H, I = 33, 8192, 8192
    note("decode long")
    w13 = torch.zeros((E, 2 * I, H // 2), dtype=torch.uint8, device=DEV)
    s13 = torch.full((E, 2 * I, H // 32), 127, dtype=torch.uint8, device=DEV)
    w2 = torch.zeros((E, H, I // 2), dtype=torch.uint8, device=DEV)
    s2 = torch.full((E, H, I // 32), 127, dtype=torch.uint8, device=DEV)
    x = torch.zeros((1, H), dtype=BF16, device=DEV)
    x[0, -1] = 2.0
    w13[-1, I - 1, -1], w13[-1, 2 * I - 1, -1] = 0x20, 0x40       # 1 and 2 in the last column
    w2[-1, -1, -1] = 0x50                                          # 3 in the last corner
    idx = torch.tensor([[E - 1, 0]], dtype=torch.int32, device=DEV)
    y = moe.experts_decode(x, idx, torch.ones((1, 2), device=DEV), w13, w2, s13, s2, out_dtype=F32)
    torch.cuda.synchronize()
    want = 2 / (1 + np.exp(-2.0)) * 4 * 3
    assert abs(y[0, -1].item() - want) < want * 40 * U and not y[0, :-1].any()
