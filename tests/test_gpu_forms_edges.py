"""Windows, normalised heads and the 8-bit pool where they can go wrong at the edges: pools past 4 GiB, several streams and
graphs, empty batches, rows of no sequence, layouts, values that are not finite in every form of the attention."""
import math

import pytest
import torch

import paged_kv_movement_amd as kvm
import pool8_util as pu
import step_util as su
from gpu_util import say
from test_gpu_append_heads import BF, FL, check_blocks, device8
from test_gpu_attend_forms import batch, on_gpu
from test_gpu_step import device, within

pytestmark = pytest.mark.gpu


def test_8bit_calls_in_a_pool_past_4_gib():
    """Pages whose bytes lie beyond 32 bits: append, attend (narrow, wide, with a window), pack8 and unpack8 on a slab of
    4.6 GB of bytes, its bf16 twin of 9.2 GB."""
    H, rep, D, P, pages = 8, 4, 128, 16, 280000
    b = pu.Batch8(29, H, D, P, [40, 90, 33], [1, 70, 1], [100], [3], layers=1, table_room=1)
    at = torch.linspace(pages - 9000, pages - 1, b.pages).long()
    bytes8 = torch.full((1, 2, pages, P, H, D), 0x7F, dtype=torch.uint8, device="cuda")
    scales = torch.full((1, 2, pages, H), math.nan, device="cuda")
    bytes8[:, :, at.cuda()], scales[:, :, at.cuda()] = b.bytes8.cuda(), b.scales.cuda()
    wide = torch.empty((1, 2, pages, P, H, D), dtype=BF, device="cuda")

    def up(t):
        return torch.where(t >= 0, at[t.clamp(min=0).long()].int(), t).cuda()
    lens = torch.tensor(b.lens, dtype=torch.int32).cuda()
    own = kvm.Tables(up(b.own_table), lens, max(b.lens))
    pre = kvm.Tables(up(b.prefix_table), torch.tensor(b.prefix, dtype=torch.int32).cuda(), 100)
    big = kvm.Paged8.from_pool(bytes8, scales)
    big_step = kvm.Step(big, own, b.new, prefix=pre, group_sizes=[3])
    small_bytes, small_scales, small, small_step = device8(b)
    small_wide = torch.zeros(b.pool.shape, dtype=BF, device="cuda")
    wide[:, :, at.cuda()] = 0
    rope, norm = kvm.Rope(D), kvm.Norm()
    rows = b.q_start[-1]
    q, k, v = (b.normal(rows, h, D).cuda() for h in (H * rep, H, H))
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    results = []
    for pg, st, pl, sc, wd in ((big, big_step, bytes8, scales, wide), (small, small_step, small_bytes, small_scales, small_wide)):
        qr = kvm.append(pg, st, 0, q, k, v, pos, rope, norm=norm)
        res = [qr, *kvm.attend(pg, st, 0, qr), *kvm.attend(pg, st, 0, qr, window=30, sinks=2)]
        bf = kvm.Paged.from_pool(wd, chunk_size=P)
        kvm.unpack8(pg, st.own, bf)
        kvm.pack8(bf, st.own, pg)
        torch.cuda.synchronize()
        assert kvm.take_faults() == 0
        res += [x[:, :, at.cuda()] if pg is big else x for x in (pl, sc, wd)]
        results.append(res)
    for i, (x, y) in enumerate(zip(*results)):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)), i
    assert torch.all(bytes8[0, :, :pages - 9001].flatten(1)[:, ::997] == 0x7F)


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("where", ["k", "v", "q"])
@pytest.mark.parametrize("form", ["narrow", "wide"])
def test_window_follows_the_formula_where_a_value_is_not_finite(form, where, value):
    """In the bf16 pool; a row whose scores are all -infinity weighs nothing."""
    new = [1, 1] if form == "narrow" else [90, 40]
    b, q = batch((1, 2, 128, 16, [140, 60], new, [150], [2]), 16)
    x = b.rows(b.own_table, 0, 101, 100)[0]
    if where == "q":
        q[0, 1, 7] = value
    else:
        b.flat()[1, 0 if where == "k" else 1, x, 0, 3] = value
    paged, step = on_gpu(b, 16)
    for window, sinks in ((60, 0), (30, 4)):
        out, lse = kvm.attend(paged, step, 1, q.cuda(), window=window, sinks=sinks)
        wo, wl, eo, el = pu.attend_window64(b, q, 128 ** -0.5, window, sinks, layer=1)
        # where lse is infinite or NaN the formula's out is NaN (+infinity, NaN) or 0 (-infinity); finite rows as ever
        ok = torch.isfinite(wl)
        within(lse, wl, el, "lse")
        if where == "v":
            fine = torch.isfinite(wo)
            assert torch.equal(torch.isfinite(out.cpu()), fine)
            within(torch.where(fine, out.cpu().double(), 0.0), torch.where(fine, wo, 0.0), eo.nan_to_num(0.0), "out")
        else:
            within(out.cpu()[ok], wo[ok], eo[ok], "out")
            assert torch.isnan(out.cpu()[~ok & (wl != -math.inf)]).all()


def test_a_step_serves_pools_of_either_kind():
    """Steps know shapes only: one made for a bf16 pool works on an 8-bit pool of its shape and the other way round."""
    b, q = batch((2, 4, 128, 16, [300, 40], [1, 1], [90], [2]), 8)
    bytes8, scales, p8, step8 = device8(b)
    pool, p16, step16 = device(b)
    for seen in ({}, {"window": 50, "sinks": 3}):
        a = kvm.attend(p8, step16, 1, q.cuda(), **seen)
        c = kvm.attend(p8, step8, 1, q.cuda(), **seen)
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
        a = kvm.attend(p16, step8, 1, q.cuda(), **seen)
        d = kvm.attend(p16, step16, 1, q.cuda(), **seen)
        assert torch.equal(a[0], d[0]) and torch.equal(a[1], d[1])
        # one set of values: scores are the same products, so the sums are those of the same terms
        assert float((c[1] - d[1]).abs().max()) < 1e-5
    k = b.normal(2, 2, 128).cuda()
    pos = torch.zeros(2, dtype=torch.int32).cuda()
    with pytest.raises(kvm.KvError, match="another shape"):
        other = pu.Batch8(1, 2, 64, 16, [3, 3], [1, 1])
        kvm.append(device8(other)[2], step16, 0, None, k, k, pos, kvm.Rope(0))
    with pytest.raises(kvm.KvError, match="eviction state"):
        w = torch.zeros((2, 2, 304), device="cuda")
        kvm.append(p8, step8, 0, None, k, k, pos, kvm.Rope(0), weights=w, slot_positions=w.int())
    with pytest.raises(kvm.KvError, match="workspace"):
        kvm.attend(p8, step8, 1, q.cuda(), workspace=torch.empty(256, dtype=torch.uint8, device="cuda"), window=50)
    with pytest.raises(kvm.KvError, match="q_weight"):
        kvm.append(p8, step8, 0, q.cuda(), k, k, pos, kvm.Rope(0), norm=kvm.Norm(torch.ones(2, 128)))


@pytest.mark.parametrize("lens", [[], [0], [0, 0, 0]])
@pytest.mark.parametrize("bits", [16, 8])
def test_a_batch_of_nothing(lens, bits):
    b = (pu.Batch8 if bits == 8 else su.Batch)(1, 2, 64, 16, lens, [0] * len(lens))
    paged, step = on_gpu(b, bits, max_len=0)
    e = torch.empty((0, 8, 64), dtype=BF, device="cuda")
    k = torch.empty((0, 2, 64), dtype=BF, device="cuda")
    out, lse = kvm.attend(paged, step, 0, e, window=5, sinks=1)
    assert out.shape == e.shape and lse.shape == (0, 8)
    kvm.append(paged, step, 0, e, k, k, torch.empty(0, dtype=torch.int32, device="cuda"), kvm.Rope(64), norm=kvm.Norm())
    other = torch.zeros((1, 2, b.pages, 16, 2, 64), dtype=BF if bits == 8 else torch.uint8, device="cuda")
    if bits == 8:
        kvm.unpack8(paged, step.own, kvm.Paged.from_pool(other, chunk_size=16))
    else:
        kvm.pack8(paged, step.own, kvm.Paged8.from_pool(other, torch.zeros((1, 2, b.pages, 2), device="cuda")))
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0


@pytest.mark.parametrize("bits", [16, 8])
def test_rows_of_no_sequence_and_layouts(bits):
    """Rows that the step gives to nobody: their q is rotated, nothing of theirs is cached, their out is left alone; q and
    out as parts of wider rows."""
    b, q = batch((2, 2, 64, 16, [30, 17], [3, 2], [21], [1]), bits)
    paged, step = on_gpu(b, bits)
    pool = [t.clone() for t in paged._keep]
    want = kvm.attend(paged, step, 1, q.cuda(), window=9, sinks=1)
    wide = torch.zeros((5, 7, 96), dtype=BF, device="cuda")
    qs = wide[:, 1:5, 16:80]
    qs.copy_(q)
    out = torch.full((5, 4, 80), 3.0, dtype=BF, device="cuda")
    o, lse = kvm.attend(paged, step, 1, qs, out=out[:, :, 8:72], window=9, sinks=1)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert torch.all(out[:, :, :8] == 3.0) and torch.all(out[:, :, 72:] == 3.0)
    step.q_start.copy_(torch.tensor([0, 3, 4], dtype=torch.int32))       # row 4 is nobody's
    o, l = torch.full((5, 4, 64), 3.0, dtype=BF, device="cuda"), torch.full((5, 4), 3.0, device="cuda")
    kvm.attend(paged, step, 1, q.cuda(), out=o, lse=l, window=9, sinks=1)
    assert torch.all(o[4] == 3.0) and torch.all(l[4] == 3.0) and torch.equal(o[:3], want[0][:3])
    for t, s in zip(paged._keep, pool):
        assert torch.equal(t.contiguous().view(torch.uint8), s.contiguous().view(torch.uint8))
    k = b.normal(5, 2, 64).cuda()
    pos = torch.arange(5, dtype=torch.int32).cuda()
    q_all = kvm.append(paged, step, 0, q.cuda(), k, k, pos, kvm.Rope(64), norm=kvm.Norm())
    b.lens, b.new = [30, 17], [3, 1]
    if bits == 8:
        ke, ee = pu.rotated64(*pu.norm64(k.cpu(), None, 1e-6, False), pos.cpu(), *kvm.Rope.frequencies(64), 64, False)
        # the two arrays are views of one: what the pool holds now
        bytes8 = torch.stack([torch.stack(paged._keep[:2]), torch.stack(paged._keep[2:4])], 1)
        scales = torch.stack([torch.stack(paged._keep[4:6]), torch.stack(paged._keep[6:8])], 1)
        check_blocks(b, 0, (ke, k.cpu().double()), (ee, torch.zeros_like(ke)), b.bytes8, b.scales, bytes8, scales, [0, 3])
    assert torch.isfinite(q_all).all() and float(q_all[4].abs().max()) > 0
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0


def test_streams_with_pools_of_their_own():
    """Three streams at once, each with its own 8-bit pool, step and graph-less decode: as one after the other."""
    jobs = []
    for s in range(3):
        b, q = batch((2, 4, 128, 16, [300 + 50 * s, 40, 7 + s], [1, 1, 1], [90], [3]), 8, seed=s)
        paged, step = on_gpu(b, 8)
        k, v = b.normal(3, 2, 128).cuda(), b.normal(3, 2, 128).cuda()
        jobs.append((b, q.cuda(), k, v, paged, step, torch.arange(3, dtype=torch.int32).cuda()))
    rope, norm = kvm.Rope(128), kvm.Norm()
    saved = [[t.clone() for t in j[4]._keep] for j in jobs]

    def decode(j, stream=None):
        b, q, k, v, paged, step, pos = j
        res = []
        for _ in range(8):
            q = kvm.append(paged, step, 1, q, k, v, pos, rope, norm=norm, stream=stream)
            q, lse = kvm.attend(paged, step, 1, q, window=60, sinks=4, stream=stream)
            res += [q, lse]
        return res
    want = []
    for j in jobs:
        want.append([x.clone() for x in decode(j)] + [t.clone() for t in j[4]._keep])
    for j, s in zip(jobs, saved):
        for t, x in zip(j[4]._keep, s):
            t.copy_(x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [decode(j, st) for j, st in zip(jobs, streams)]
    torch.cuda.synchronize()
    for j, g, w in zip(jobs, got, want):
        for x, y in zip(g + list(j[4]._keep), w):
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
    assert kvm.take_faults() == 0


def test_two_graphs_share_a_workspace():
    """Attention with a window over a bf16 and over an 8-bit pool, captured apart with one workspace, replayed in turn."""
    made = []
    ws = None
    for bits in (16, 8):
        b, q = batch((2, 4, 128, 16, [700, 40, 7], [1, 1, 1], [90], [3]), bits)
        paged, step = on_gpu(b, bits)
        q = q.cuda()
        size = step.attend_workspace_bytes(8, 300, 4)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda") if ws is None or ws.numel() < size else ws
        made.append([paged, step, q, torch.empty_like(q), torch.empty((3, 8), device="cuda")])
    graphs = []
    for paged, step, q, out, lse in made:
        want = [x.clone() for x in kvm.attend(paged, step, 1, q, window=300, sinks=4)]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvm.attend(paged, step, 1, q, out=out, lse=lse, workspace=ws, window=300, sinks=4)
        graphs.append((g, out, lse, want))
    for _ in range(4):
        for g, out, lse, want in graphs:
            out.zero_()
            lse.zero_()
            ws.fill_(0xFF)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert kvm.take_faults() == 0


def test_pages_of_one_head_and_many_groups_of_heads():
    """pack8 and append8 where a page's heads take several workgroups, and heads of the largest and smallest size."""
    for H, D, P, lens, new in ((40, 128, 4, [9], [5]), (64, 16, 2, [5, 2], [3, 2]), (3, 256, 16, [40], [40]),
                               (1, 16, 16, [17], [17])):
        say("heads", H, D, P)
        b = pu.Batch8(3, H, D, P, lens, new)
        bytes8, scales, paged, step = device8(b)
        k, v = b.normal(b.q_start[-1], H, D, dtype=BF), b.normal(b.q_start[-1], H, D, dtype=BF)
        pos = torch.zeros(b.q_start[-1], dtype=torch.int32).cuda()
        kvm.append(paged, step, 0, None, k.cuda(), v.cuda(), pos, kvm.Rope(0))
        zero = torch.zeros(k.shape, dtype=torch.float64)
        check_blocks(b, 0, (k.double(), v.double()), (zero, zero), b.bytes8, b.scales, bytes8, scales, b.q_start)
        wide = torch.zeros(b.pool.shape, dtype=BF, device="cuda")
        p16 = kvm.Paged.from_pool(wide, chunk_size=P)
        kvm.unpack8(paged, step.own, p16)
        before = bytes8.clone(), scales.clone()
        held = pu.values(before[0].cpu(), before[1].cpu())
        for s, n in enumerate(lens):
            rows = b.rows(b.own_table, s, n)
            assert torch.equal(wide.cpu().view(1, 2, -1, H, D)[:, :, rows].double(), held.view(1, 2, -1, H, D)[:, :, rows])
        bytes8.fill_(1)
        scales.fill_(1.0)
        kvm.pack8(p16, step.own, paged)
        torch.cuda.synchronize()
        # held values are held again exactly, under a scale no larger
        again = pu.values(bytes8.cpu(), scales.cpu())
        for s, n in enumerate(lens):
            rows = b.rows(b.own_table, s, n)
            assert torch.equal(again.view(1, 2, -1, H, D)[:, :, rows], held.view(1, 2, -1, H, D)[:, :, rows])
    assert kvm.take_faults() == 0
