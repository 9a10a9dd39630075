"""The gradients behind every form of the dispatch and the combine that they are documented for:
plain, padded, no-allocation, replayed and deduplicated dispatches, quantizing ones, and the combines
plain, deduplicated (both ways) and of e4m3 and e2m1 rows.

A dispatch is linear in the token rows and a combine in the expert rows and in the weights, so
<dpacked, dispatch(x)> = <dx, x> and <dout, combine(y, w)> = <dy, y> = <dw, w>.  The payload is f32
and the products are summed in 64 bits.  u = 2^-24.  A dispatch copies, and dx is a sum of at most K
rows: K u of the terms' magnitudes.  A combine rounds K products and K sums (2 K u, and R u more
where R ranks' parts are joined), dy is one product (u), dw sums H products over at least 8 partial
sums ((H / 8 + 17) u); a code times its scale is rounded once on each side (2 u)."""
import pytest
import torch

import combine_moe_route_count_amd as moe
from _gpu_util import DEV, note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
T, H, E, K, R = 157, 384, 16, 5, 4
SLACK = 1 + 2.0 ** -7


def _ids(g):
    idx = torch.argsort(torch.rand((T, E), generator=g), 1)[:, :K].int()
    idx[torch.rand((T, K), generator=g) < 0.1] = -1
    idx[T // 2] = -1
    return idx.to(DEV)


def _randn(g, *shape):
    return torch.randn(shape, generator=g).to(DEV)


def _owned(tok_map, rows):
    owned = torch.zeros(rows, dtype=torch.bool, device=DEV)
    owned[tok_map[tok_map >= 0]] = True
    return owned


DISPATCHES = {
    "plain": lambda x, idx: moe.dispatch(x, idx, E),
    "padded": lambda x, idx: moe.dispatch(x, idx, E, cap=40),
    "few rows": lambda x, idx: moe.dispatch(x, idx, E, packed_rows=T * K // 2),
    "no allocation": lambda x, idx: moe.dispatch_noalloc(x, idx, E),
    "no allocation, padded": lambda x, idx: moe.dispatch_noalloc(x, idx, E, cap=33),
    "dedup": lambda x, idx: moe.dedup_dispatch(x, idx, E, R),
    "dedup, padded": lambda x, idx: moe.dedup_dispatch(x, idx, E, R, cap=40),
    "dedup, few recv rows": lambda x, idx: moe.dedup_dispatch(x, idx, E, R, recv_rows=T),
}


@pytest.mark.parametrize("form", DISPATCHES)
def test_dispatch_forms(form):
    note(f"dispatch gradient of {form}")
    g = torch.Generator().manual_seed(5)
    x, idx = _randn(g, T, H), _ids(g)
    d = DISPATCHES[form](x, idx)
    rows = d.packed.shape[0]
    owned = _owned(d.tok_map, rows)
    assert 0 < owned.sum().item() and (d.tok_map < 0).any()
    dp = _randn(g, rows, H)
    dx = moe.dispatch_backward(dp, d.tok_map)
    a, b = dp.double()[owned], d.packed.double()[owned]
    assert ((a * b).sum() - (dx.double() * x.double()).sum()).abs() <= (a * b).abs().sum() * K * U * SLACK
    # what the dispatch wrote about its segments describes the rows that no entry owns
    w, dout = torch.rand((T, K), generator=g).to(DEV), _randn(g, T, H)
    dy = torch.full((rows, H), torch.nan, device=DEV)
    moe.combine_backward(dout, None, d.tok_map, w, dy=dy, want_dw=False, packed_cnt=d.packed_cnt,
                         packed_off=d.packed_off)
    assert torch.isfinite(dy).all() and (dy[~owned] == 0).all() and (dy[owned] != 0).any(1).all()


def test_replayed_dispatch():
    note("dispatch gradient of a replay")
    g = torch.Generator().manual_seed(6)
    idx = _ids(g)
    first = moe.dispatch(_randn(g, T, H), idx, E)
    x = _randn(g, T, H)
    packed = moe.dispatch_replay(x, first.tok_map, torch.zeros_like(first.packed))
    owned = _owned(first.tok_map, packed.shape[0])
    dp = _randn(g, packed.shape[0], H)
    dx = moe.dispatch_backward(dp, first.tok_map)
    a, b = dp.double()[owned], packed.double()[owned]
    assert ((a * b).sum() - (dx.double() * x.double()).sum()).abs() <= (a * b).abs().sum() * K * U * SLACK


@pytest.mark.parametrize("fp4", [False, True])
def test_quantizing_dispatch_is_passed_straight_through(fp4):
    """The packed rows are codes, and their gradient is that of the rows before the rounding."""
    note(f"dispatch gradient, quantizing, fp4={fp4}")
    g = torch.Generator().manual_seed(7)
    idx, x = _ids(g), _randn(g, T, H).bfloat16()
    q, plain = moe.dispatch(x, idx, E, fp8=not fp4, fp4=fp4), moe.dispatch(x, idx, E)
    assert torch.equal(q.tok_map, plain.tok_map)
    dp = _randn(g, T * K, H)
    dx = moe.dispatch_backward(dp, q.tok_map)
    ref, mag = torch.zeros((2, T, H), dtype=torch.float64, device=DEV)
    for k in range(K):
        t = (q.tok_map[:, k] >= 0).nonzero().flatten()
        ref[t] += dp[q.tok_map[t, k]].double()
        mag[t] += dp[q.tok_map[t, k]].double().abs()
    assert ((dx.double() - ref).abs() <= mag * K * U * SLACK).all()


def _adjoint(dout, out, dow, out_weights, dy, y, dw, w, tok_map, more):
    """out = sum w y and out_weights = sum w, against the gradients of both."""
    owned = _owned(tok_map, y.shape[0])
    a, b = dy.double()[owned], y[owned]
    mag = (a * b).abs().sum()
    rows = (dout.double() * out.double()).sum()
    assert (rows - (a * b).sum()).abs() <= mag * (2 * K + 1 + more) * U * SLACK
    through = (dow.double() * out_weights.double()).sum()
    mag = mag + ((dow.double()[:, None] * w.double()).abs() * (tok_map >= 0)).sum()
    assert (rows + through - (dw.double() * w.double()).sum()).abs() <= mag * (2 * K + H / 8 + 18 + more) * U * SLACK


@pytest.mark.parametrize("staged", [False, True])
@pytest.mark.parametrize("recv_rows", [None, T])
def test_deduplicated_combine(staged, recv_rows):
    note(f"combine gradient of the dedup form, staged={staged} recv_rows={recv_rows}")
    g = torch.Generator().manual_seed(8)
    idx = _ids(g)
    d = moe.dedup_dispatch(_randn(g, T, H), idx, E, R, recv_rows=recv_rows)
    recv = d.recv_x.shape[0]
    y, w, dout, dow = _randn(g, T * K, H), torch.rand((T, K), generator=g).to(DEV), _randn(g, T, H), _randn(g, T)
    plan = dict(R=R, idx=idx, rank_slot=d.rank_slot, recv_rows=recv)
    if staged:
        plan["partial"] = torch.empty((recv, H), dtype=torch.float32, device=DEV)
    out, ow = moe.combine(y, d.tok_map, w, E=E, out_dtype=torch.float32, dedup=plan)
    dy, dw = moe.combine_backward(dout, y, d.tok_map, w, dout_weights=dow, packed_cnt=d.packed_cnt,
                                  packed_off=d.packed_off)
    _adjoint(dout, out, dow, ow, dy, y.double(), dw, w, d.tok_map, R)


E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


@pytest.mark.parametrize("kind", ["plain", "fp8", "fp8 without scales", "fp4", "fp4 without scales"])
def test_combines_of_every_row_type(kind):
    note(f"combine gradient of {kind}")
    g = torch.Generator().manual_seed(9)
    d = moe.dispatch_noalloc(_randn(g, T, H), _ids(g), E, cap=40)
    rows = E * 40
    w, dout, dow = torch.rand((T, K), generator=g).to(DEV), _randn(g, T, H), _randn(g, T)
    fp4 = kind.startswith("fp4")
    sc = None if "without" in kind else (torch.rand((rows, H // 128), generator=g) + 0.5).to(DEV)
    if kind == "plain":
        y, sc = _randn(g, rows, H), None
        yv = y.double()
        out, ow = moe.combine(y, d.tok_map, w, out_dtype=torch.float32)
    elif fp4:
        y = torch.randint(0, 256, (rows, H // 2), generator=g, dtype=torch.uint8).to(DEV)
        yv = E2M1.to(DEV)[torch.stack((y & 15, y >> 4), -1).view(rows, H).long()]
        out, ow = moe.combine_fp4(y, sc, d.tok_map, w, out_dtype=torch.float32)
    else:
        codes = _randn(g, rows, H).to(torch.float8_e4m3fn)
        y, yv = codes.view(torch.uint8), codes.double()
        out, ow = moe.combine_fp8(y, sc, d.tok_map, w, out_dtype=torch.float32)
    if sc is not None:
        yv = yv * sc.double().repeat_interleave(128, 1)
    dy, dw = moe.combine_backward(dout, y, d.tok_map, w, y_scales=sc, fp4=fp4, dout_weights=dow,
                                  packed_cnt=d.packed_cnt, packed_off=d.packed_off)
    _adjoint(dout, out, dow, ow, dy, yv, dw, w, d.tok_map, 2)
