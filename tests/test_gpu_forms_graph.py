"""Decode steps over an 8-bit pool as a captured graph: append with a norm, attend with a window, the values into a bf16
pool and back into another 8-bit one, replayed with lengths that grow and inputs that change."""
import pytest
import torch

import paged_kv_movement_amd as kvm
import pool8_util as pu
from gpu_util import say
from test_gpu_append_heads import BF, FL

pytestmark = pytest.mark.gpu

STEPS = 40


class State:
    """A batch's pools, tables and inputs, and one step on them; every State made of one batch holds the same values."""

    def __init__(self, b, rep, window):
        H, D, n = b.heads, b.dim, len(b.lens)
        self.bytes8, self.scales = b.bytes8.cuda(), b.scales.cuda()
        self.p8 = kvm.Paged8.from_pool(self.bytes8, self.scales)
        self.wide = torch.zeros(b.pool.shape, dtype=BF, device="cuda")
        self.p16 = kvm.Paged.from_pool(self.wide, chunk_size=b.page)
        self.other, self.other_scales = torch.zeros_like(self.bytes8), torch.ones_like(self.scales)
        self.p8b = kvm.Paged8.from_pool(self.other, self.other_scales)
        self.lens = torch.tensor(b.lens, dtype=torch.int32).cuda()
        self.own = kvm.Tables(b.own_table.cuda(), self.lens, max(b.lens) + STEPS)
        pre = kvm.Tables(b.prefix_table.cuda(), torch.tensor(b.prefix, dtype=torch.int32).cuda(), max(b.prefix))
        self.step = kvm.Step(self.p8, self.own, [1] * n, prefix=pre, group_sizes=b.sizes)
        self.q, self.k, self.v = (torch.zeros((n, h, D), dtype=BF, device="cuda") for h in (H * rep, H, H))
        self.pos = torch.zeros(n, dtype=torch.int32, device="cuda")
        g = torch.Generator().manual_seed(1)
        self.rope = kvm.Rope(D)
        self.norm = kvm.Norm(1 + torch.randn(D, generator=g), 1 + torch.randn(H, D, generator=g))
        self.seen = {"window": window, "sinks": 3}
        self.qr, self.out = torch.zeros_like(self.q), torch.zeros_like(self.q)
        self.lse = torch.zeros((n, H * rep), dtype=FL, device="cuda")
        self.ws = self.step.new_attend_workspace(H * rep, **self.seen)

    def take(self, x):
        for t, y in zip((self.q, self.k, self.v), x):
            t.copy_(y)

    def run(self):
        self.lens += 1
        self.pos.copy_(self.lens)
        kvm.append(self.p8, self.step, 0, self.q, self.k, self.v, self.pos, self.rope, q_out=self.qr, norm=self.norm)
        kvm.attend(self.p8, self.step, 0, self.qr, out=self.out, lse=self.lse, workspace=self.ws, **self.seen)
        kvm.unpack8(self.p8, self.own, self.p16)
        kvm.pack8(self.p16, self.own, self.p8b)

    def results(self):
        return (self.qr, self.out, self.lse, self.bytes8, self.scales, self.wide, self.other, self.other_scales)


@pytest.mark.parametrize("rep,window", [(1, 50), (8, 300)])
def test_decode_steps_as_a_graph(rep, window):
    say("graph", rep, window)
    b = pu.Batch8(13, 2, 64, 16, [40, 17, 200, 15], [1] * 4, [130], [3], table_room=-(-STEPS // 16) + 1)
    eager, graph = State(b, rep, window), State(b, rep, window)
    x = [b.normal(*t.shape).cuda() for t in (eager.q, eager.k, eager.v)]
    # one step of each outside a graph: what a first call makes is made
    for s in (eager, graph):
        s.take(x)
        s.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graph.run()
    for i in range(STEPS - 1):
        x = [b.normal(*t.shape, gain=1.0 + 3.0 * (i % 5 == 4)).cuda() for t in (eager.q, eager.k, eager.v)]
        for s in (eager, graph):
            s.take(x)
        graph.ws.fill_(0xFF)
        g.replay()
        eager.run()
        if i % 3 == 0:
            torch.cuda.synchronize()
        for n, (y, z) in enumerate(zip(graph.results(), eager.results())):
            assert torch.equal(y.view(torch.uint8), z.view(torch.uint8)), (i, n)
    assert int(graph.lens.max()) == 200 + STEPS and kvm.take_faults() == 0
