"""Table gradients past 262144 positions, whose sorts take the one-launch routing and with it the
arrival counter at the head of the workspace, the only part of the training side that a call leaves
for the next one: captured and replayed, alternating with sorts of other kinds on one workspace, and
on two streams at once.  All results must be the bits of an eager call on a workspace of its own."""
import pytest
import torch

import combine_moe_route_count_amd as moe
from _gpu_util import DEV, note

pytestmark = pytest.mark.gpu

# (positions, table rows, row length): the one-launch routing with digits of 5 and of 4 bits, a sort
# whose workgroups scan for themselves, with one and with several digits, and a sort by counting
ROUTED = (262145, 700, 8)
ROUTED_SHORT = (530001, 5000, 8)
OWN_SCAN = (9001, 300001, 8)
ONE_DIGIT = (5000, 500, 8)
COUNTED = (900, 3000, 8)


class Call:
    def __init__(self, size, seed, accumulate=False):
        N, self.V, H = size
        g = torch.Generator().manual_seed(seed)
        ids = (torch.rand(N, generator=g) ** 3 * self.V).long().clamp(max=self.V - 1)
        ids[torch.rand(N, generator=g) < 0.1] = -1
        self.ids, self.size, self.accumulate = ids.to(DEV), size, accumulate
        self.dout = torch.randn((N, H), generator=g).to(torch.bfloat16).to(DEV)
        self.base = torch.randn((self.V, H), generator=g).to(DEV)
        own = moe.embedding_workspace(*size)
        own.fill_(0x5A)
        self.want = self.run(own, self.base.clone())
        torch.cuda.synchronize()
        ok = ids >= 0
        ref = torch.zeros((self.V, H), dtype=torch.float64)
        ref.index_add_(0, ids[ok], self.dout.double().cpu()[ok])
        mag = torch.zeros_like(ref).index_add_(0, ids[ok], self.dout.double().cpu()[ok].abs())
        cnt = torch.bincount(ids[ok], minlength=self.V)[:, None].double()
        if accumulate:
            ref, mag = ref + self.base.double().cpu(), mag + self.base.double().cpu().abs()
        # at most cnt additions of terms rounded by 2^-24 each, the scale and the base
        assert ((self.want.double().cpu() - ref).abs() <= mag * (cnt + 3) * 2.0 ** -24 * (1 + 2.0 ** -7)).all(), size
        self.out = torch.empty_like(self.base)

    def run(self, ws, out):
        return moe.embedding_backward(self.dout, self.ids, self.V, accumulate=self.accumulate, dtable=out, ws=ws)

    def reset(self):
        if self.accumulate:
            self.out.copy_(self.base)
        else:
            self.out.fill_(float("nan"))

    def check(self, what):
        assert torch.equal(self.out.view(torch.int32), self.want.view(torch.int32)), (self.size, what)


def _room(calls):
    """A workspace for the largest of the calls, filled with what a program might have left there."""
    ws = torch.empty(max(moe.embedding_workspace_size(*c.size) for c in calls), dtype=torch.uint8, device=DEV)
    ws.fill_(0xA5)
    return ws


def _captured(call, ws):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run(ws, call.out)
    return graph


@pytest.mark.parametrize("size", [ROUTED, ROUTED_SHORT])
@pytest.mark.parametrize("accumulate", [False, True])
def test_replayed_between_eager_calls(size, accumulate):
    note(f"long sort in a graph {size} {accumulate}")
    a, b = Call(size, 1, accumulate), Call(size, 2)
    ws = _room([a, b])
    graph = _captured(a, ws)              # the first run on this workspace is a replay
    for i in range(4):
        a.reset()
        b.reset()
        graph.replay()
        b.run(ws, b.out)
        torch.cuda.synchronize()
        a.check(f"replay {i}")
        b.check(f"eager {i}")


def test_sorts_of_every_kind_on_one_workspace():
    """Graphs of all kinds in several orders on one workspace, then the same calls eagerly."""
    note("sorts of every kind on one workspace")
    calls = [Call(s, 10 + i, i == 3) for i, s in enumerate((ROUTED, OWN_SCAN, COUNTED, ROUTED_SHORT, ONE_DIGIT))]
    ws = _room(calls)
    graphs = [_captured(c, ws) for c in calls]
    orders = [(0, 1, 2, 3, 4), (3, 0, 3, 2, 0), (4, 3, 2, 1, 0), (2, 3, 1, 0, 4)]
    for i, order in enumerate(orders):
        for c in calls:
            c.reset()
        for j, n in enumerate(order):
            if n in order[:j]:
                calls[n].reset()
            graphs[n].replay()
        torch.cuda.synchronize()
        for n in set(order):
            calls[n].check(f"replay {i}")
        for c in calls:
            c.reset()
        for n in dict.fromkeys(order):
            calls[n].run(ws, calls[n].out)
        torch.cuda.synchronize()
        for n in set(order):
            calls[n].check(f"eager {i}")


def test_two_streams_with_workspaces_of_their_own():
    note("long sorts on two streams")
    calls = [Call(ROUTED, 21), Call(ROUTED_SHORT, 22)]
    rooms = [_room(calls) for _ in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    for c in calls:
        c.reset()
    torch.cuda.synchronize()
    for _ in range(5):
        for c, ws, s in zip(calls, rooms, streams):
            with torch.cuda.stream(s):
                c.run(ws, c.out)
    torch.cuda.synchronize()
    for c in calls:
        c.check("two streams")
