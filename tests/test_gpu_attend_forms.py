"""attend with a window and over an 8-bit pool, pack8 and unpack8, on the GPU against plain 64-bit implementations; and a
run of the calls together."""
import math

import pytest
import torch

import paged_kv_movement_amd as kvm
import pool8_util as pu
import step_util as su
from gpu_util import say
from test_gpu_append_heads import BF, FL, device8
from test_gpu_step import ATTEND, device, within

pytestmark = pytest.mark.gpu


def batch(case, bits, seed=5):
    H, rep, D, P, lens, new, prefix, sizes = case
    b = (pu.Batch8 if bits == 8 else su.Batch)(seed, H, D, P, lens, new, prefix, sizes, layers=2)
    return b, b.normal(b.q_start[-1], H * rep, D, gain=2.0)


def on_gpu(b, bits, **kw):
    """(paged, step)."""
    return (device8(b, **kw) if bits == 8 else device(b, **kw))[-2:]


def compare(b, q, bits, window, sinks, **kw):
    paged, step = on_gpu(b, bits, **kw)
    seen = {} if window is None else {"window": window, "sinks": sinks}
    out, lse = kvm.attend(paged, step, 1, q.cuda(), **seen)
    again = kvm.attend(paged, step, 1, q.cuda(), workspace=step.new_attend_workspace(q.shape[1], **seen).fill_(0xFF), **seen)
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    assert torch.equal(out.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse, again[1])
    wo, wl, eo, el = pu.attend_window64(b, q, b.dim ** -0.5, window, sinks, layer=1)
    within(lse, wl, el, "lse")
    within(out, wo, eo, "out")


EIGHT = [c for c in ATTEND if c[2] % 16 == 0 and len(c[4]) < 1000]


@pytest.mark.parametrize("case", EIGHT, ids=[str(i) for i in range(len(EIGHT))])
@pytest.mark.parametrize("loose", [0, 137])
def test_attend8(case, loose):
    say("attend8", case, loose)
    b, q = batch(case, 8)
    room = b.own_table.shape[1] * b.page
    compare(b, q, 8, None, 0, max_len=min(room, max(b.lens) + loose))


WINDOWS = [
    # heads, rep, dim, page, lens, new, prefix, sizes; then (window, sinks)
    ((1, 1, 128, 16, [1], [1], [], []), [(1, 0), (5, 3)]),
    ((8, 4, 128, 16, [1000], [1], [], []), [(1, 0), (64, 0), (100, 4), (300, 130), (999, 1), (1000, 0), (5000, 9)]),
    ((2, 4, 128, 16, [5, 0, 130, 64], [1, 1, 1, 1], [257], [3]), [(1, 0), (7, 2), (70, 200), (130, 300), (257, 0)]),
    ((2, 1, 64, 16, [33, 16, 1], [1, 1, 1], [40, 1], [1, 2]), [(3, 0), (20, 5), (41, 2)]),
    ((1, 5, 80, 12, [29, 3], [29, 2], [100], [2]), [(1, 1), (10, 0), (50, 64)]),
    ((2, 8, 128, 16, [200, 70, 3], [150, 70, 3], [300], [3]), [(1, 0), (33, 1), (129, 65), (250, 0), (600, 3)]),
    ((1, 2, 256, 16, [77, 40], [5, 40], [33], [2]), [(2, 2), (40, 0)]),
    ((1, 4, 256, 16, [150, 9], [75, 9], [40], [2]), [(17, 3), (100, 0)]),
    ((2, 2, 192, 32, [100, 12], [40, 12], [500], [2]), [(64, 64), (200, 1)]),
    ((1, 4, 128, 16, [3, 7, 9], [6, 0, 4], [], []), [(2, 1), (100, 0)]),       # more new tokens than cached ones
    ((1, 4, 128, 16, [3, 7, 9], [6, 0, 4], [90], [3]), [(2, 1), (8, 0)]),
    ((1, 1, 128, 16, [20] * 70, [1] * 70, [90], [70]), [(1, 0), (25, 3), (60, 100)]),   # more sequences than lanes
    ((2, 4, 128, 16, [12, 500] * 10, [1] * 20, [2000, 900], [11, 9]), [(13, 0), (100, 4), (1000, 64), (501, 66)]),
    ((1, 1, 64, 16, [1100, 20], [1100, 3], [130], [2]), [(1, 0), (64, 0), (200, 70), (1300, 2)]),   # a join by rows
    ((2, 1, 16, 16, [1, 40], [1030, 20], [70], [2]), [(9, 1), (200, 0)]),
    ((1, 2, 128, 16, [3, 3, 3], [1, 1, 1], [5, 0], [1, 1]), [(2, 1), (4, 7)]),
    ((1, 5, 32, 16, [796, 322], [9, 7], [40], [0]), [(100, 10), (321, 0)]),
    ((1, 2, 16, 4, [9, 5] * 100, [1, 2] * 100, [6, 11] * 35, [3, 2] * 35), [(6, 2), (15, 0)]),
    ((1, 4, 128, 16, [2600, 900], [1, 1], [], []), [(1024, 4), (2500, 64), (2000, 500)]),
    ((2, 2, 64, 16, [700], [700], [64], [1]), [(63, 64), (65, 1), (64, 63), (128, 128)]),
]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("case,seen", WINDOWS, ids=[str(i) for i in range(len(WINDOWS))])
def test_window(case, seen, bits):
    b, q = batch(case, bits)
    room = b.own_table.shape[1] * b.page
    for n, (window, sinks) in enumerate(seen):
        say("window", case, bits, window, sinks)
        compare(b, q, bits, window, sinks, max_len=min(room, max(b.lens) + 137 * (n % 2)))


@pytest.mark.parametrize("bits", [16, 8])
def test_a_window_past_everything_is_none(bits):
    """Bit for bit where the pieces are cut alike."""
    for case in (ATTEND[2], ATTEND[5], ATTEND[14]):
        b, q = batch(case, bits)
        paged, step = on_gpu(b, bits)
        out, lse = kvm.attend(paged, step, 1, q.cuda())
        for window, sinks in (((1 << 31) - 1, 0), ((1 << 31) - 1, (1 << 31) - 1), (1 << 30, 5)):
            o, l = kvm.attend(paged, step, 1, q.cuda(), window=window, sinks=sinks)
            assert torch.equal(o.view(torch.int16), out.view(torch.int16)) and torch.equal(l, lse)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("where", ["k", "v"])
def test_what_the_window_hides_does_not_reach_a_row(where, bits):
    """NaN keys or values in tokens that only some rows see, in a prefix and in own pages, wide and narrow forms."""
    for case in ((1, 2, 128, 16, [140, 20], [90, 9], [150], [2]), (2, 1, 64, 16, [140, 20], [1, 1], [150], [2])):
        b, q = batch(case, bits)
        hide = [(b.prefix_table, 0, 100), (b.own_table, 0, 60), (b.own_table, 1, 3)]
        for table, i, t in hide:
            b.flat()[1, 0 if where == "k" else 1, b.rows(table, i, t + 1, t)[0], 0, 3] = math.nan
        if bits == 8:
            b.quantise()
        paged, step = on_gpu(b, bits)
        for window, sinks in ((20, 2), (60, 101)):
            out, lse = kvm.attend(paged, step, 1, q.cuda(), window=window, sinks=sinks)
            wo, wl, eo, el = pu.attend_window64(b, q, b.dim ** -0.5, window, sinks, layer=1)
            assert sinks > 100 or not torch.isnan(wo).all()        # 101 sinks show every row a hidden token
            within(out, wo, eo, "out")
            within(lse, wl, el, "lse")


@pytest.mark.parametrize("spread", [6, 30, 60])
def test_attend8_blocks_far_apart(spread):
    """V blocks of magnitudes from 2^-spread to 2^spread, in an order that begins small, large or anywhere; the window
    leaves some rows only small ones.  What the larger ones add to an output bounds what a row that sees them may be off;
    a row that does not see them is as exact as without them."""
    for seed in range(3):
        for case in ((1, 4, 128, 16, [300, 70], [150, 70], [200], [2]), (2, 2, 64, 16, [260, 33], [100, 20], [150], [2]),
                     (1, 2, 256, 16, [150, 9], [75, 9], [40], [2]), (1, 1, 128, 16, [300], [1], [], [])):
            b = su.Batch(seed, *case[:1], *case[2:], layers=2)
            for table, lens in ((b.own_table, b.lens), (b.prefix_table, b.prefix)):
                for i, n in enumerate(lens):
                    for p in range(-(-n // b.page)):
                        e = int(torch.randint(-spread, spread + 1, (1,), generator=b.g)) if p or seed else -spread
                        rows = b.rows(table, i, min(n, (p + 1) * b.page), p * b.page)
                        b.flat()[:, 1, rows] *= 2.0 ** e
            b.__class__ = pu.Batch8
            b.quantise()
            q = b.normal(b.q_start[-1], case[0] * case[1], case[2], gain=2.0)
            compare(b, q, 8, None, 0)
            compare(b, q, 8, 20, 3)


def test_lengths_and_rows_that_change_on_the_device():
    """Lengths past their bound are cut, row ranges out of order touch nothing outside."""
    b, q = batch((2, 2, 128, 16, [64, 48], [1, 1], [32], [2]), 8)
    paged, step = on_gpu(b, 8)
    ref = kvm.attend(paged, step, 1, q.cuda(), window=20, sinks=3)
    step.own.lens.copy_(torch.tensor([1 << 30, -5], dtype=torch.int32))
    out, lse = kvm.attend(paged, step, 1, q.cuda(), window=20, sinks=3)
    assert torch.equal(out[0], ref[0][0]) and torch.isfinite(out.float()).all()
    step.q_start.copy_(torch.tensor([-3, 1 << 30, 2], dtype=torch.int32))
    kvm.attend(paged, step, 1, q.cuda(), window=20, sinks=3)
    k = b.normal(2, 2, 128).cuda()
    kvm.append(paged, step, 1, q.cuda(), k, k, torch.zeros(2, dtype=torch.int32).cuda(), kvm.Rope(128))
    torch.cuda.synchronize()
    kvm.take_faults()


def test_bad_pages_are_not_seen_and_reported():
    b, q = batch((2, 4, 128, 16, [100], [1], [200], [1]), 8)
    good = b.pool.clone()
    bad = b.own_table.clone()
    b.own_table[0, 2], b.prefix_table[0, 4] = -1, b.pages
    paged, step = on_gpu(b, 8)
    out, lse = kvm.attend(paged, step, 1, q.cuda(), window=290)
    assert kvm.take_faults() == 1
    b.own_table = bad
    b.prefix_table[0, 4] = 0
    keep = [t for t in range(200) if t > 9 and not 64 <= t < 80]
    k = torch.cat([good.view(2, 2, -1, 2, 128)[1, :, b.rows(b.prefix_table, 0, 200)][:, keep],
                   good.view(2, 2, -1, 2, 128)[1, :, b.rows(b.own_table, 0, 100)]
                   [:, [t for t in range(100) if not 32 <= t < 48]]], 1).double()
    for h in range(8):
        s = k[0, :, h // 4] @ q[0, h].double() * 128 ** -0.5
        want = torch.softmax(s, 0) @ k[1, :, h // 4]
        assert float((out[0, h].cpu().double() - want).abs().max()) <= 2.0 ** -7 * float(want.abs().max())
        assert abs(float(lse[0, h]) - float(torch.logsumexp(s, 0))) < 1e-5


# ------------------------------------------------------------------ pages between pools

PACKS = [
    # heads, dim, page, lens, layers, range
    (8, 128, 16, [1, 16, 33, 0], 3, (1, 3)),
    (1, 16, 1, [5, 2], 1, (0, 1)),
    (3, 80, 12, [30, 12, 11], 2, (0, 2)),
    (5, 256, 8, [17], 2, (1, 2)),
    (2, 64, 300, [299, 301], 1, (0, 1)),
    (4, 48, 64, [64, 200, 3], 2, (0, 2)),
]


@pytest.mark.parametrize("case", PACKS, ids=[str(i) for i in range(len(PACKS))])
@pytest.mark.parametrize("moved", [False, True])
def test_pack8_and_unpack8(case, moved):
    H, D, P, lens, L, (l0, l1) = case
    say("pack8", case, moved)
    b = su.Batch(8, H, D, P, lens, [0] * len(lens), layers=L)
    b.flat()[:, 1] *= 1e3
    x = b.rows(b.own_table, 0, 1)[0]
    b.flat()[:, 0, x, 0, :5] = torch.tensor([math.inf, -math.inf, math.nan, 0.0, -0.0]).bfloat16()
    pool, paged, step = device(b)
    extra = 2
    shape = (L, 2, b.pages + extra, P, H, D)
    bytes8 = torch.full(shape, 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full(shape[:3] + (H,), 123.0, device="cuda")
    p8 = kvm.Paged8.from_pool(bytes8, scales)
    to, table = None, b.own_table
    if moved:
        table = torch.where(b.own_table < 0, b.own_table, b.pages + extra - 1 - b.own_table)
        to = torch.full((len(lens), table.shape[1] + 3), -9, dtype=torch.int32)[:, 1:1 + table.shape[1]]
        to.copy_(table)
        to = to.cuda()
    kvm.pack8(paged, step.own, p8, to_table=to, layer_begin=l0, layer_end=l1)
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    eb, es = torch.full(shape, 0x55, dtype=torch.uint8), torch.full(shape[:3] + (H,), 123.0)
    back = torch.full(b.pool.shape, 7.0, dtype=BF)
    for s, n in enumerate(lens):
        for p in range(-(-n // P)):
            m = min(P, n - p * P)
            v = b.pool[l0:l1, :, int(b.own_table[s, p]), :m].double()
            sc = pu.scales_of(v, (2, 4))
            y = pu.e4m3(v / sc[:, :, None, :, None])
            eb[l0:l1, :, int(table[s, p]), :m] = pu.to_bytes(y)
            es[l0:l1, :, int(table[s, p])] = sc.float()
            back[l0:l1, :, int(b.own_table[s, p]), :m] = (y * sc[:, :, None, :, None]).bfloat16()
    got = bytes8.cpu()
    nan = (eb & 0x7F) == 0x7F
    assert torch.equal(nan, (got & 0x7F) == 0x7F) and torch.equal(got[~nan], eb[~nan])
    assert torch.equal(scales.cpu(), es)
    # and back, into a pool of its own
    out = torch.full(b.pool.shape, 7.0, dtype=BF, device="cuda")
    here = kvm.Tables(to, step.own.lens, step.own.max_len) if moved else step.own
    kvm.unpack8(p8, here, kvm.Paged.from_pool(out, chunk_size=P), to_table=step.own.table if moved else None,
                layer_begin=l0, layer_end=l1)
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    assert torch.equal(out.cpu().double().nan_to_num(7.7e33), back.double().nan_to_num(7.7e33))


def test_pack8_bad_pages_are_left_out_and_reported():
    b = su.Batch(8, 2, 64, 16, [40, 20], [0, 0])
    pool, paged, step = device(b)
    bytes8 = torch.full((1, 2, b.pages, 16, 2, 64), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((1, 2, b.pages, 2), 123.0, device="cuda")
    p8 = kvm.Paged8.from_pool(bytes8, scales)
    kvm.pack8(paged, step.own, p8)
    torch.cuda.synchronize()
    whole, whole_s = bytes8.clone(), scales.clone()
    bytes8.fill_(0x55)
    scales.fill_(123.0)
    to = b.own_table.clone()
    to[0, 1] = b.pages
    step.own.table[1, 0] = -1
    kvm.pack8(paged, step.own, p8, to_table=to.cuda())
    assert kvm.take_faults() == 1
    for page in (int(b.own_table[0, 1]), int(b.own_table[1, 0])):
        whole[:, :, page] = 0x55
        whole_s[:, :, page] = 123.0
    assert torch.equal(bytes8, whole) and torch.equal(scales, whole_s)
    target = kvm.Paged.from_pool(torch.zeros_like(pool), chunk_size=16)
    kvm.unpack8(p8, step.own, target, to_table=to.cuda())
    assert kvm.take_faults() == 1


# ------------------------------------------------------------------ together

def test_an_8bit_cache_from_chunks_to_decoding():
    """Chunks retrieved into bf16 pages, packed, then a decode loop on the 8-bit pool with normalised heads and a window;
    at the end unpacked.  Each attention is checked against the values the pool holds."""
    H, rep, D, P, steps, layers = 2, 4, 128, 16, 20, 2
    start = [100, 37, 250]
    room = [-(-(n + steps) // P) for n in start]
    b = su.Batch(9, H, D, P, [r * P for r in room], [1, 1, 1], layers=layers)
    pool, staging, _ = device(b)
    seqs = [kvm.Seq(b.own_table[s, :room[s]].contiguous().cuda(), 0, n,
                    [torch.zeros(staging.chunk_bytes(min(staging.chunk_size, n - c)), dtype=torch.uint8, device="cuda")
                     for c in range(0, n, staging.chunk_size)]) for s, n in enumerate(start)]
    kvm.store(staging, seqs)
    pool.zero_()
    got = kvm.retrieve(staging, seqs, masks=[[1] * len(s._chunks) for s in seqs])
    assert got == start
    bytes8 = torch.zeros(pool.shape, dtype=torch.uint8, device="cuda")
    scales = torch.ones(pool.shape[:3] + (H,), device="cuda")
    p8 = kvm.Paged8.from_pool(bytes8, scales)
    lens = torch.tensor(start, dtype=torch.int32).cuda()
    own = kvm.Tables(b.own_table.cuda(), lens, max(r * P for r in room))
    kvm.pack8(staging, own, p8)
    step = kvm.Step(p8, own, [1, 1, 1])
    rope, norm = kvm.Rope(D), kvm.Norm(b.normal(D, dtype=FL) + 1, b.normal(D, dtype=FL) + 1)
    lens += 1
    b.lens = [n + 1 for n in start]
    for i in range(steps):
        for layer in range(layers):
            q, k, v = (b.normal(3, h, D).cuda() for h in (H * rep, H, H))
            q = kvm.append(p8, step, layer, q, k, v, lens - 1, rope, norm=norm)
            out, lse = kvm.attend(p8, step, layer, q, window=64, sinks=4)
            if i % 9 == 0:
                b.pool = pu.values(bytes8.cpu(), scales.cpu()).bfloat16()
                wo, wl, eo, el = pu.attend_window64(b, q.cpu(), D ** -0.5, 64, 4, layer=layer)
                within(out, wo, eo, "out")
                within(lse, wl, el, "lse")
        if i + 1 < steps:
            lens += 1
            b.lens = [n + 1 for n in b.lens]
    kvm.unpack8(p8, own, staging)
    want = pu.values(bytes8.cpu(), scales.cpu()).bfloat16().view(layers, 2, -1, H, D)
    flat = pool.cpu().view(layers, 2, -1, H, D)
    for s, n in enumerate(b.lens):
        rows = b.rows(b.own_table, s, n)
        assert torch.equal(flat[:, :, rows], want[:, :, rows])
    assert kvm.take_faults() == 0


def _side_by_side(bits):
    b, q = batch((2, 4, 128, 16, [300, 40, 7], [1, 1, 1], [90], [3]), bits)
    paged, step = on_gpu(b, bits, max_len=304)
    return b, q.cuda(), paged, step


@pytest.mark.parametrize("bits", [16, 8])
def test_captured_and_replayed(bits):
    """A decode step in a graph, replayed with other lengths and inputs between eager calls."""
    b, q, paged, step = _side_by_side(bits)
    k = b.normal(3, 2, 128).cuda()
    v = b.normal(3, 2, 128).cuda()
    pos = torch.tensor([389, 129, 96], dtype=torch.int32).cuda()
    rope, norm = kvm.Rope(128), kvm.Norm(eps=1e-6)
    ws = step.new_attend_workspace(8, window=50, sinks=4)
    out, lse = torch.empty_like(q), torch.empty((3, 8), device="cuda")
    q_out = torch.empty_like(q)

    def decode(out, lse, q_out):
        kvm.append(paged, step, 1, q, k, v, pos, rope, q_out=q_out, norm=norm)
        kvm.attend(paged, step, 1, q_out, out=out, lse=lse, workspace=ws, window=50, sinks=4)
    pool = paged._keep                                     # the caller's tensors
    saved = [t.clone() for t in pool]

    def reset():
        for t, s in zip(pool, saved):
            t.copy_(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode(out, lse, q_out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode(out, lse, q_out)
    for n in ([300, 40, 7], [298, 33, 7], [300, 17, 1], [200, 40, 6]):
        step.own.lens.copy_(torch.tensor(n, dtype=torch.int32))
        q.copy_(b.normal(3, 8, 128))
        k.copy_(b.normal(3, 2, 128))
        reset()
        graph.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in (out, lse, q_out, *pool)]
        reset()
        eager = [torch.empty_like(out), torch.empty_like(lse), torch.empty_like(q_out)]
        decode(*eager)
        torch.cuda.synchronize()
        for x, y in zip(first, [*eager, *pool]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert kvm.take_faults() == 0


@pytest.mark.parametrize("bits", [16, 8])
def test_on_another_stream(bits):
    """Outputs and workspaces made for the call's stream, and the binding's arrays dropped while it is still busy."""
    b, q, paged, step = _side_by_side(bits)
    want = kvm.attend(paged, step, 1, q, window=50, sinks=4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.randn(2048, 2048, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):
            busy = busy @ busy * 1e-3
    got = kvm.attend(paged, step, 1, q, window=50, sinks=4, stream=side)
    keep = paged._keep
    del paged, step
    junk = [torch.full((256,), 0x7F, dtype=torch.int64, device="cuda") for _ in range(64)]
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert kvm.take_faults() == 0 and len(junk) == 64 and keep
