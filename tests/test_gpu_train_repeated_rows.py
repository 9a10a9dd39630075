"""tok_map with rows named more than once, which no dispatch writes but a caller may: dw of every
entry, and in dy one of the row's products at each element; the dispatch's gradient adds the row for
each entry that names it."""
import pytest
import torch

import combine_moe_route_count_amd as moe
from _gpu_util import DEV, note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("T,H,K,rows", [(2, 64, 1, 1), (40, 1032, 4, 30), (300, 4104, 3, 50)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_repeated_rows(T, H, K, rows, dt):
    note(f"repeated rows {T} {H} {K} {rows} {dt}")
    g = torch.Generator().manual_seed(T)
    tm = torch.randint(0, rows, (T, K), generator=g).to(DEV)
    tm[0] = 0                                    # one token names a row K times
    y, dout = torch.randn((rows + 3, H), generator=g).to(dt).to(DEV), torch.randn((T, H), generator=g).to(dt).to(DEV)
    w = torch.rand((T, K), generator=g).to(DEV)
    dy = torch.full((rows + 3, H), 7.0, dtype=dt, device=DEV)
    _, dw = moe.combine_backward(dout, y, tm, w, dy=dy)
    prod = dout.double()[:, None] * y.double()[tm]
    # products over at least 8 partial sums a row
    assert ((dw.double() - prod.sum(-1)).abs() <= prod.abs().sum(-1) * (H / 8 + 17) * U * (1 + 2.0 ** -7)).all()
    could = torch.zeros((rows + 3, H), dtype=torch.bool, device=DEV)
    for t in range(T):
        for k in range(K):
            r = tm[t, k]
            could[r] |= dy[r] == (w[t, k] * dout[t].float()).to(dt)
    named = torch.zeros(rows + 3, dtype=torch.bool, device=DEV)
    named[tm.flatten()] = True
    assert could[named].all() and (dy[~named] == 7.0).all() and not named[rows:].any()
    acc = torch.zeros((T, H), device=DEV)
    for k in range(K):
        acc = acc + y[tm[:, k]].float()
    assert torch.equal(moe.dispatch_backward(y, tm), acc.to(dt))
