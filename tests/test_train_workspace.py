"""The table gradient's workspace over calls of different sizes: one sized for the largest batch
and table serves every smaller call of the same row length, and no call writes past what it asked
for."""
import random

import pytest
import torch

import combine_moe_route_count_amd as moe

WIDTHS = [8, 64, 264, 512, 520, 1024, 1032, 4096, 33016, 1 << 24]
# both sides of the small sort's last size, of each window length at some width, and of the sizes
# where digits get shorter (181 and 256 tiles of 1024 positions when workgroups scan for themselves,
# 256 and 512 past that)
POSITIONS = sorted({n + d for n in (1, 64, 512, 1024, 4032, 4096, 8192, 16384, 32768, 65536, 131008, 131072,
                                    181 * 1024, 256 * 1024, 512 * 1024, 1 << 20, (1 << 31) - 2)
                    for d in (-1, 0, 1)})
TABLES = sorted({v + d for v in (1, 16, 32, 512, 1 << 10, 1 << 14, 1 << 18, 1 << 20, 1 << 27, (1 << 31) - 2)
                 for d in (-1, 0, 1)} - {0})


@pytest.mark.parametrize("H", WIDTHS)
def test_size_does_not_shrink_with_more_positions(H):
    rng = random.Random(H)
    positions = sorted(POSITIONS + [rng.randrange(1, 1 << rng.randint(4, 24)) for _ in range(400)])
    for V in (1, 300, 5000, 262145, 1 << 30):
        sizes = [moe.embedding_workspace_size(n, V, H) for n in positions]
        for (a, b), (n, m) in zip(zip(sizes, sizes[1:]), zip(positions, positions[1:])):
            assert 0 < a <= b, (H, V, n, a, m, b)


@pytest.mark.parametrize("H", WIDTHS)
def test_size_does_not_shrink_with_a_larger_table(H):
    for N in POSITIONS:
        sizes = [moe.embedding_workspace_size(N, v, H) for v in TABLES]
        for (a, b), (v, u) in zip(zip(sizes, sizes[1:]), zip(TABLES, TABLES[1:])):
            assert a <= b, (H, N, v, a, u, b)


def _input(g, N, V, H):
    ids = (torch.rand(N, generator=g) ** 3 * V).long().clamp(max=V - 1)    # low ids more often
    return ids.cuda(), torch.randn((N, H), generator=g).cuda()


def _serve(sizes, H, seed):
    """Every size of one workspace for the largest, against workspaces of their own; the bytes behind
    the size a call asked for keep their value."""
    g = torch.Generator().manual_seed(seed)
    N, V = max(n for n, _ in sizes), max(v for _, v in sizes)
    ws = moe.embedding_workspace(N, V, H)
    for n, v in sizes:
        print(f"[case] table gradient {n} {v} {H} on the workspace of {N} {V}", flush=True)
        ids, dout = _input(g, n, v, H)
        ws.fill_(0xA5)
        got = moe.embedding_backward(dout, ids, v, ws=ws)
        need = moe.embedding_workspace_size(n, v, H)
        assert (ws[need:] == 0xA5).all()
        want = moe.embedding_backward(dout, ids, v)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int32), want.view(torch.int32)), (n, v, H)


@pytest.mark.gpu
def test_one_workspace_for_shorter_batches():
    _serve([(4096, 3000), (4032, 3000), (2048, 3000), (2047, 2999), (511, 3000), (65, 17), (1, 1)], 4096, 1)
    _serve([(20000, 262145), (19000, 262144), (4097, 513), (4097, 512), (4096, 262145), (33, 5)], 520, 2)


@pytest.mark.gpu
def test_one_workspace_across_the_digit_borders():
    _serve([(530000, 5000), (300000, 5000), (262145, 700), (262144, 5000), (185345, 5000), (185344, 512),
            (131072, 5000), (4097, 5000), (100, 5000)], 8, 3)
