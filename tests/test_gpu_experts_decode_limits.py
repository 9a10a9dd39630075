"""GPU tests of experts_decode where its numbers end: an h between the products that bf16
does not reach, and infinities among the weights.

h goes through the second product in bf16 parts.  Every h here is a sum of few powers of
two, so each is known exactly: with silu(g) = g for g >= 64 (1 / (1 + exp(-64)) rounds to 1
in f32) an h is a product of exact numbers, and results are compared with what the formula
gives for it, after one rounding to the result's type."""
import pytest
import torch

import combine_moe_route_count_amd as moe
from _gpu_util import DEV, note

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
INF = float("inf")
H = 64


class Weights:
    """[E,rows,cols] of zeros with single entries of +-2^e, in bf16 or MXFP4 (one entry's scale per
    block of 32)."""

    def __init__(self, E, rows, cols, mx):
        self.mx = mx
        if mx:
            self.w = torch.zeros((E, rows, cols // 2), dtype=torch.uint8)
            self.s = torch.full((E, rows, cols // 32), 127, dtype=torch.uint8)
        else:
            self.w, self.s = torch.zeros((E, rows, cols), dtype=BF16), None

    def put(self, row, col, e, sign=1):
        if not self.mx:
            self.w[:, row, col] = sign * (INF if e == INF else 2.0 ** e)
            return
        code, e = (7, 127) if e == INF else (2, e)              # 6 * 2^127 is past bf16's largest
        self.w[:, row, col // 2] |= (code + 8 * (sign < 0)) << 4 * (col % 2)      # (a place is put once)
        self.s[:, row, col // 32] = e + 127

    def on(self):
        return self.w.to(DEV), None if self.s is None else self.s.to(DEV)


def _call(x, idx, w, w13, w2, out):
    a, sa = w13.on()
    b, sb = w2.on()
    y = moe.experts_decode(x.to(DEV), idx.to(DEV), w.to(DEV), a, b, sa, sb, out_dtype=out)
    torch.cuda.synchronize()
    return y.cpu()


# tokens, experts, I: one entry per expert; several; more than 16 with many weight rows
SIZES = [(1, 2, 64), (20, 2, 64), (40, 2, 1664)]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("T,E,I", SIZES)
@pytest.mark.parametrize("mx", [False, True])
def test_h_past_the_largest_bf16(mx, T, E, I, sign, out):
    """h = +-2^128 (1 - 2^-10), an f32 number that rounds to an infinity in bf16."""
    note(f"decode top of the range mx={mx} T={T} I={I} {out}")
    x = torch.zeros((T, H), dtype=BF16)
    x[:, 0] = x[:, 32] = 1
    w13, w2 = Weights(E, 2 * I, H, mx), Weights(E, H, I, mx)
    w13.put(0, 0, 64)
    w13.put(I, 0, 64, sign)
    w13.put(I, 32, 54, -sign)
    for r in range(H):
        w2.put(r, 0, -34 - r % 8, 1 if r % 3 else -1)
    idx = (torch.arange(T) % E).int().unsqueeze(1)
    got = _call(x, idx, torch.ones((T, 1)), w13, w2, out)
    want = torch.tensor([sign * (1 if r % 3 else -1) * 2.0 ** (94 - r % 8) * (1 - 2.0 ** -10) for r in range(H)])
    assert torch.equal(got, want.to(out).expand(T, H))


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T,E,I", SIZES)
@pytest.mark.parametrize("mx", [False, True])
def test_infinite_weights_of_the_second_product(mx, T, E, I, out):
    """A weight that is infinite gives an infinity of its and h's sign, whether h is a bf16 number
    (1: its further parts are 0) or lies above or below one (1 +- 2^-10); with h = 0 a NaN.  Rows
    without such a weight are what they are."""
    note(f"decode infinite weights mx={mx} T={T} I={I} {out}")
    x = torch.zeros((T, H), dtype=BF16)
    x[:, 0] = x[:, 32] = 1
    w13, w2 = Weights(E, 2 * I, H, mx), Weights(E, H, I, mx)
    h = [1.0, 1 + 2.0 ** -10, 1 - 2.0 ** -10, -1.0, -1 - 2.0 ** -10, -1 + 2.0 ** -10, 0.0]
    for i, v in enumerate(h):
        w13.put(i, 0, 6)                                        # g = 64
        if v:
            w13.put(I + i, 0, -6, 1 if v > 0 else -1)
        if abs(v) not in (0.0, 1.0):
            w13.put(I + i, 32, -16, 1 if v > 1 or -1 < v < 0 else -1)
    want = torch.zeros(H)
    for i, v in enumerate(h):
        for j, sign in enumerate((1, -1)):
            w2.put(2 * i + j, i, INF, sign)
            want[2 * i + j] = sign * v * INF                    # 0 * infinity is NaN here too
    w2.put(20, 0, 3)
    want[20] = 8
    w2.put(21, 4, 1, -1)
    want[21] = 2 + 2.0 ** -9
    idx = (torch.arange(T) % E).int().unsqueeze(1)
    got = _call(x, idx, torch.ones((T, 1)), w13, w2, out)
    assert torch.equal(got.nan_to_num(nan=7.0, posinf=INF, neginf=-INF),
                       want.to(out).nan_to_num(nan=7.0, posinf=INF, neginf=-INF).expand(T, H))


@pytest.mark.parametrize("T,E,I", SIZES)
@pytest.mark.parametrize("mx", [False, True])
def test_infinite_h(mx, T, E, I):
    """Every third token's h is 2^136, infinite in f32, the others' 2^12: its sign goes with the
    weight's, and 0 times it is NaN."""
    note(f"decode infinite h mx={mx} T={T} I={I}")
    x = torch.zeros((T, H), dtype=BF16)
    x[:, 0] = 2.0
    x[::3, 0] = 2.0 ** 63
    w13, w2 = Weights(E, 2 * I, H, mx), Weights(E, H, I, mx)
    w13.put(0, 0, 5)
    w13.put(I, 0, 5)
    sign = torch.tensor([(0.0, 1.0, -1.0, 1.0)[r % 4] for r in range(H)])
    for r in range(H):
        if sign[r]:
            w2.put(r, 0, -3, sign[r])
    idx = (torch.arange(T) % E).int().unsqueeze(1)
    got = _call(x, idx, torch.ones((T, 1)), w13, w2, F32)
    for t in range(T):
        want = sign * (INF if t % 3 == 0 else 2.0 ** 9)
        assert torch.equal(got[t].nan_to_num(nan=7.0, posinf=INF, neginf=-INF),
                           want.nan_to_num(nan=7.0, posinf=INF, neginf=-INF)), t
