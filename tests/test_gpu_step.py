"""append, attend, add_weights and evict on the GPU against plain 64-bit
implementations (step_util).  Every pool row that no token is in holds NaN."""
import math

import pytest
import torch

import paged_kv_movement_amd as kvm
import step_util as su
from gpu_util import say

pytestmark = pytest.mark.gpu


def device(b, max_len=None, prefix_max=None):
    """(pool, paged, step) of a batch on the GPU."""
    pool = b.pool.cuda()
    paged = kvm.Paged.from_pool(pool, chunk_size=b.page)
    own = kvm.Tables(b.own_table.cuda(), torch.tensor(b.lens, dtype=torch.int32).cuda(),
                     max(b.lens, default=0) if max_len is None else max_len)
    pre = None
    if b.prefix:
        pre = kvm.Tables(b.prefix_table.cuda(), torch.tensor(b.prefix, dtype=torch.int32).cuda(),
                         max(b.prefix) if prefix_max is None else prefix_max)
    return pool, paged, kvm.Step(paged, own, b.new, prefix=pre, group_sizes=b.sizes)


def within(got, want, bound, what):
    """|got - want| <= bound where want is finite; NaN and infinities equal."""
    got, want = got.double().cpu(), want.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what
    over = ((got - want).abs() - bound)[fine]
    if over.numel():
        worst = float(over.max())
        assert worst <= 0, (what, "over the bound by", worst, "largest error",
                            float((got - want).abs()[fine].max()))


# ------------------------------------------------------------------ append

APPEND = [
    # heads, rep, dim, page, lens, new, rot, interleaved, scaling, type, q type, start
    (8, 4, 128, 16, [5, 33, 1], [1, 1, 1], 128, False, "none", torch.bfloat16, None, 0),
    (2, 4, 64, 16, [40, 17], [40, 3], 32, True, "yarn", torch.float16, None, 5000),
    (1, 1, 80, 12, [13, 0, 25], [1, 0, 25], 48, False, "linear", torch.float32, None, 100000),
    (3, 5, 72, 8, [9, 2], [2, 2], 20, False, "ntk", torch.float32, torch.bfloat16, 1 << 20),
    (2, 2, 36, 3, [7, 11], [7, 1], 36, True, "wavelength", torch.float16, torch.bfloat16, 77),
    (1, 8, 256, 256, [300], [260], 256, True, "none", torch.bfloat16, None, (1 << 31) - 400),
    (4, 1, 8, 1, [4, 4], [4, 1], 0, False, "none", torch.bfloat16, None, 3),
    (1, 2, 40, 16, [2], [5], 16, False, "none", torch.float32, None, -9),       # more new tokens than slots
]


@pytest.mark.parametrize("case", APPEND, ids=[str(i) for i in range(len(APPEND))])
@pytest.mark.parametrize("fused", [True, False])
def test_append(case, fused):
    H, rep, D, P, lens, new, rot, il, scaling, dt, qdt, start = case
    say("append", case, fused)
    b = su.Batch(1, H, D, P, lens, new, layers=3)
    pool, paged, step = device(b)
    rows = b.q_start[-1]
    qkv = b.normal(rows, (rep + 2) * H * D + (0 if fused else 1), dtype=dt).cuda()      # odd row stride: by elements
    q = qkv[:, :rep * H * D].unflatten(1, (rep * H, D))
    k = qkv[:, rep * H * D:(rep + 1) * H * D].unflatten(1, (H, D))
    v = qkv[:, (rep + 1) * H * D:(rep + 2) * H * D].unflatten(1, (H, D))
    pos = torch.tensor([start + i for m in new for i in range(m)], dtype=torch.int32)
    rope = kvm.Rope(rot, base=10000.0, interleaved=il, scaling=scaling, factor=4.0)
    f, gain = kvm.Rope.frequencies(rot, 10000.0, scaling, 4.0)
    cap = max(lens) + 3
    w = torch.full((len(lens), H, cap), 5.0, device="cuda")
    sp = torch.full((len(lens), H, cap), -5, dtype=torch.int32, device="cuda")
    q_out = None if qdt is None else torch.empty((rows, rep * H, D), dtype=qdt, device="cuda")
    got = kvm.append(paged, step, 1, q, k, v, pos.cuda(), rope, q_out=q_out, weights=w, slot_positions=sp)
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    # float32: sin and cos off by 2 u of the angle (as turns, rounded once) times 2 pi and 4 u of their own, the products
    # and their sum 3 u: 2^-20 of |x| + |y| covers all (u = 2^-24); then half a step of the output's type
    def bound(want, size, t):
        return size * 2.0 ** -20 + (want.abs() + size * 2.0 ** -20) * torch.finfo(t).eps / 2 + 2.0 ** -25
    want, size = su.rope64(q.cpu(), pos, f, gain, rot, il)
    within(got, want, bound(want, size, got.dtype), "q")
    exp = b.pool.clone().double()
    err = torch.zeros_like(exp)
    wk, size = su.rope64(k.cpu(), pos, f, gain, rot, il)
    we, pe = torch.full(w.shape, 5.0), torch.full(sp.shape, -5, dtype=torch.int32)
    e, ee = exp.view(3, 2, -1, H, D), err.view(3, 2, -1, H, D)
    for s, (n, m) in enumerate(zip(lens, new)):
        for i in range(m):
            slot = n - m + i
            if slot < 0:
                continue
            r, x = b.q_start[s] + i, b.rows(b.own_table, s, slot + 1, slot)[0]
            e[1, 0, x], ee[1, 0, x] = wk[r], bound(wk[r], size[r], torch.bfloat16)
            e[1, 1, x], ee[1, 1, x] = v[r].cpu().double(), v[r].cpu().double().abs() * 2.0 ** -8
            we[s, :, slot], pe[s, :, slot] = 0.0, pos[r]
    within(pool, exp, err, "pool")
    assert torch.equal(w.cpu(), we) and torch.equal(sp.cpu(), pe)


def test_append_in_place_and_without_q():
    b = su.Batch(2, 2, 64, 16, [20, 3], [4, 1])
    pool, paged, step = device(b)
    pos = torch.arange(5, dtype=torch.int32).cuda()
    rope = kvm.Rope(64)
    q, k, v = (b.normal(5, h, 64).cuda() for h in (8, 2, 2))
    apart = kvm.append(paged, step, 0, q, k, v, pos, rope)
    first = pool.clone()
    pool.copy_(b.pool)
    assert kvm.append(paged, step, 0, None, k, v, pos, rope) is None
    assert torch.equal(pool.view(torch.int16), first.view(torch.int16))
    same = kvm.append(paged, step, 0, q, k, v, pos, rope, q_out=q)
    assert same is q and torch.equal(q, apart)
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0


def test_append_bad_page_is_left_out_and_reported():
    b = su.Batch(3, 2, 64, 16, [20, 18], [2, 3])
    b.own_table[1, 1] = b.pages + 5
    pool, paged, step = device(b)
    pos = torch.arange(5, dtype=torch.int32).cuda()
    q, k, v = (b.normal(5, h, 64).cuda() for h in (2, 2, 2))
    kvm.append(paged, step, 0, q, k, v, pos, kvm.Rope(0))
    assert kvm.take_faults() == 1
    exp = b.pool.clone()
    e = exp.view(1, 2, -1, 2, 64)
    for slot, s, r in ((18, 0, 0), (19, 0, 1), (15, 1, 2)):
        x = b.rows(b.own_table, s, slot + 1, slot)[0]
        e[0, 0, x], e[0, 1, x] = k[r].cpu(), v[r].cpu()
    assert torch.equal(pool.cpu().view(torch.int16), exp.view(torch.int16))


# ------------------------------------------------------------------ attend, add_weights

ATTEND = [
    # heads, rep, dim, page, lens, new, prefix, sizes
    (1, 1, 128, 16, [1], [1], [], []),
    (8, 4, 128, 16, [1000], [1], [], []),
    (2, 4, 128, 16, [5, 0, 130, 64], [1, 1, 1, 1], [257], [3]),            # a sequence with no own token at all
    (2, 1, 64, 16, [33, 16, 1], [1, 1, 1], [40, 1], [1, 2]),
    (1, 5, 80, 12, [29, 3], [29, 2], [100], [2]),
    (2, 8, 128, 16, [200, 70, 3], [150, 70, 3], [300], [3]),
    (1, 2, 256, 8, [77, 40], [5, 40], [33], [2]),
    (3, 1, 8, 1, [9, 4], [3, 4], [7], [1]),
    (1, 16, 24, 3, [50], [20], [], []),
    (2, 2, 192, 32, [100, 12], [40, 12], [500], [2]),
    (1, 1, 128, 256, [700, 511], [1, 33], [], []),
    (1, 4, 128, 16, [3, 7, 9], [6, 0, 4], [], []),                          # more new tokens than cached ones: empty rows
    (1, 1, 128, 16, [20] * 70, [1] * 70, [90], [70]),                       # more sequences than a wave has lanes
    (2, 4, 128, 16, [12] * 20, [1] * 20, [2000, 900], [11, 9]),
    (1, 3, 128, 48, [600, 90], [300, 2], [1100], [2]),
    (1, 4, 256, 16, [150, 9], [75, 9], [40], [2]),                          # many rows of the widest heads
    (1, 5, 192, 32, [130], [60], [], []),
    (1, 1, 64, 16, [1100, 20], [1100, 3], [130], [2]),                      # rows enough for a join by rows
    (2, 1, 16, 16, [1, 40], [1030, 20], [70], [2]),                         # most rows see nothing of their own
    (1, 2, 128, 16, [3, 3, 3], [1, 1, 1], [5, 0], [1, 1]),                  # an empty prefix, and a sequence of no group
    (1, 5, 32, 16, [796, 322], [9, 7], [40], [0]),                          # a prefix of a group without sequences
    (1, 2, 16, 4, [9, 5] * 100, [1, 2] * 100, [6, 11] * 35, [3, 2] * 35),   # more groups than a wave has lanes
    (1, 1, 8, 1, [2, 0, 3] * 1400, [1, 1, 0] * 1400, [1] * 4200, [1] * 4200),   # more of both than 64 times its lanes
]


def _attend_case(case, seed=5, gain=1.0):
    H, rep, D, P, lens, new, prefix, sizes = case
    b = su.Batch(seed, H, D, P, lens, new, prefix, sizes, layers=2)
    q = b.normal(b.q_start[-1], H * rep, D, gain=gain)
    return b, q


@pytest.mark.parametrize("case", ATTEND, ids=[str(i) for i in range(len(ATTEND))])
@pytest.mark.parametrize("gain,loose", [(1.0, 0), (6.0, 137)])
def test_attend_and_weights(case, gain, loose):
    say("attend", case, gain)
    b, q = _attend_case(case, gain=gain)
    H, rep, D = case[0], case[1], case[2]
    room = b.own_table.shape[1] * b.page                  # the bound may be larger than every length
    pool, paged, step = device(b, max_len=min(room, max(b.lens) + loose))
    qd = q.cuda()
    out, lse = kvm.attend(paged, step, 1, qd)
    again = kvm.attend(paged, step, 1, qd, workspace=step.new_attend_workspace(H * rep).fill_(0xFF))
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    assert torch.equal(out.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse, again[1])
    wo, wl, eo, el = su.attend64(b, q, D ** -0.5, layer=1)
    within(lse, wl, el, "lse")
    within(out, wo, eo, "out")

    cap = max(b.lens) + loose + 3
    w = torch.rand((len(b.lens), H, cap), generator=b.g)
    p = torch.rand((len(b.prefix), H, max(b.prefix) + 2), generator=b.g) if b.prefix else None
    lse = wl.float()
    gw, gp = kvm.add_weights(paged, step, 1, qd, lse.cuda(), w.cuda(), p.cuda() if b.prefix else None)
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    ww, wp, ew, ep = su.weights64(b, q, lse, D ** -0.5, w, p, layer=1)
    within(gw, ww, ew, "weights")
    if b.prefix:
        within(gp, wp, ep, "prefix weights")
    # from zero, into another tensor, entries behind the lengths left alone
    o = torch.full((len(b.lens), H, cap), 9.0, device="cuda")
    kvm.add_weights(paged, step, 1, qd, lse.cuda(), None, out=o)
    for s, n in enumerate(b.lens):
        assert torch.all(o[s, :, n:] == 9.0)
        # from-zero sums differ from the others by the start value's own rounding
        assert torch.all((o[s, :, :n].cpu().double() - (ww - w.double())[s, :, :n]).abs() <= ew[s, :, :n] * 2 + 2.0 ** -22)


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_attend_what_is_not_seen_does_not_reach_a_row(where, value):
    """A non-finite key or value of a new token: the earlier rows of the same tile stay finite, the later ones follow
    the formula."""
    b, q = _attend_case((1, 2, 128, 16, [40, 20], [12, 9], [50], [2]))
    x = b.rows(b.own_table, 0, 36, 35)[0]                 # own token 35: seen by the rows of tokens 35..39
    b.flat()[1, 0 if where == "k" else 1, x, 0, 3] = value
    pool, paged, step = device(b)
    out, lse = kvm.attend(paged, step, 1, q.cuda())
    wo, wl, eo, el = su.attend64(b, q, 128 ** -0.5, layer=1)
    first = 35 - (40 - 12)
    blind = [r for r in range(21) if not first <= r < 12]
    within(out[blind], wo[blind], eo[blind], "rows that do not see it")
    within(lse[blind], wl[blind], el[blind], "rows that do not see it")
    seen = list(range(first, 12))
    if where == "v":
        within(lse[seen], wl[seen], el[seen], "lse does not read v")
        assert torch.equal(torch.isfinite(out[seen].cpu()), torch.isfinite(wo[seen]))
        assert not torch.isfinite(out[seen][:, :, 3].float()).any()
    elif value != value:
        assert torch.isnan(out[seen].float()).all() and torch.isnan(lse[seen]).all()


def test_attend_strides_and_untouched_rows():
    """q and out as parts of wider rows, and a step that gives some rows to nobody."""
    b, q = _attend_case((2, 2, 64, 16, [30, 17], [3, 2], [21], [1]))
    pool, paged, step = device(b)
    wide = torch.zeros((5, 7, 96), dtype=torch.bfloat16, device="cuda")
    qs = wide[:, 1:5, 16:80]
    qs.copy_(q)
    out = torch.full((5, 4, 80), 3.0, dtype=torch.bfloat16, device="cuda")
    o, lse = kvm.attend(paged, step, 1, qs, out=out[:, :, 8:72])
    ref, ref_lse = kvm.attend(paged, step, 1, q.cuda())
    assert torch.equal(o, ref) and torch.equal(lse, ref_lse)
    assert torch.all(out[:, :, :8] == 3.0) and torch.all(out[:, :, 72:] == 3.0)
    # row 4 is taken from the second sequence: on the device it ends one row earlier
    step.q_start.copy_(torch.tensor([0, 3, 4], dtype=torch.int32))
    o = torch.full((5, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full((5, 4), 3.0, device="cuda")
    kvm.attend(paged, step, 1, q.cuda(), out=o, lse=l)
    torch.cuda.synchronize()
    assert torch.all(o[4] == 3.0) and torch.all(l[4] == 3.0)
    assert torch.equal(o[:3], ref[:3])
    assert kvm.take_faults() == 0


def test_attend_bad_page_is_not_seen_and_reported():
    b, q = _attend_case((2, 4, 128, 16, [100], [1], [200], [1]))
    good = su.Batch(5, 2, 128, 16, [100], [1], [200], [1], layers=2)
    b.own_table[0, 2], b.prefix_table[0, 4] = -1, b.pages
    pool, paged, step = device(b)
    out, lse = kvm.attend(paged, step, 1, q.cuda())
    assert kvm.take_faults() == 1
    w = torch.zeros((1, 2, 100), device="cuda")
    kvm.add_weights(paged, step, 1, q.cuda(), lse, w)
    assert kvm.take_faults() == 1 and torch.all(w[:, :, 32:48] == 0)
    # the same without those tokens
    keep = [t for t in range(100) if not 32 <= t < 48]
    keep_p = [t for t in range(200) if not 64 <= t < 80]
    k = torch.cat([good.flat()[1, :, good.rows(good.prefix_table, 0, 200)][:, keep_p],
                   good.flat()[1, :, good.rows(good.own_table, 0, 100)][:, keep]], 1).double()
    for h in range(8):
        s = k[0, :, h // 4] @ q[0, h].double() * 128 ** -0.5
        p = torch.softmax(s, 0)
        want = p @ k[1, :, h // 4]
        assert float((out[0, h].cpu().double() - want).abs().max()) <= 2.0 ** -7 * float(want.abs().max())
        assert abs(float(lse[0, h]) - float(torch.logsumexp(s, 0))) < 1e-5


def test_lengths_beyond_the_bound_are_cut():
    """Device lengths past max_len and row ranges past their bounds: cut, nothing outside is touched."""
    b, q = _attend_case((2, 2, 128, 16, [64, 48], [1, 1], [32], [2]))
    pool, paged, step = device(b)
    ref = kvm.attend(paged, step, 1, q.cuda())
    step.own.lens.copy_(torch.tensor([1 << 30, -5], dtype=torch.int32))
    out, lse = kvm.attend(paged, step, 1, q.cuda())
    torch.cuda.synchronize()
    assert torch.equal(out[0], ref[0][0])                  # cut to max_len = 64, its true length
    only, _ = kvm.attend(paged, step, 1, q.cuda())
    assert torch.isfinite(only.float()).all() and kvm.take_faults() == 0
    step.q_start.copy_(torch.tensor([-3, 1 << 30, 2], dtype=torch.int32))
    kvm.attend(paged, step, 1, q.cuda())
    torch.cuda.synchronize()


# ------------------------------------------------------------------ evict

EVICT = [
    # heads, by head, dim, page, lens, keep, recent, layers
    (2, True, 64, 16, [100, 40, 41, 7], 40, 8, 2),
    (3, False, 40, 12, [50, 1, 0], 3, 3, 1),
    (1, True, 128, 16, [2050], 2049, 16, 1),
    (2, True, 8, 1, [30, 12], 12, 0, 3),
    (1, False, 256, 256, [5000], 1030, 1030, 1),
    (4, True, 128, 16, [1025, 3000], 1024, 100, 1),
    (2, True, 64, 16, [33], 0, 0, 1),                     # nothing stays
    (1, True, 64, 8, [9], 1, 1, 2),
    (2, True, 64, 16, [70, 71, 72, 73, 74, 75], 70, 0, 1),     # a few too many
    (1, False, 16, 16, [40000, 33000], 20000, 500, 1),   # more keys than LDS takes
    (1, True, 8, 256, [33000], 32997, 3, 1),
    (1, True, 128, 16, [13000], 12000, 1, 1),
]


@pytest.mark.parametrize("case", EVICT, ids=[str(i) for i in range(len(EVICT))])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind", ["random", "ties"])
def test_evict(case, in_place, kind):
    H, by_head, D, P, lens, keep, recent, layers = case
    say("evict", case, in_place, kind)
    b = su.Batch(7, H, D, P, lens, [0] * len(lens), layers=layers + 1, table_room=0 if in_place else 8)
    # a bound above the lengths takes other kernels than one that says how few moves there can be
    room = b.own_table.shape[1] * P
    pool, paged, step = device(b, max_len=max(lens) if in_place else min(room, max(lens) + 300))
    hs, cap = (H if by_head else 1), max(lens) + 305
    w = torch.rand((layers, len(lens), hs, cap), generator=b.g)
    if kind == "ties":
        w = torch.randint(0, 3, w.shape, generator=b.g).float()
        w[w == 0] = -0.0
        pick = torch.rand(w.shape, generator=b.g)
        w[pick < 0.05], w[pick > 0.97] = float("nan"), float("inf")
        w[(pick > 0.9) & (pick < 0.93)] = -float("inf")
        w[(pick > 0.5) & (pick < 0.55)] = 0.0
    p = torch.stack([torch.randperm(cap, generator=b.g) for _ in range(layers * len(lens) * hs)])
    p = (p * 5 - 2000).to(torch.int32).view(w.shape)
    wd, pd = w.cuda(), p.cuda()
    kw = {}
    if not in_place:
        kw = {"out_weights": torch.full((layers, len(lens), hs, keep + 1), 8.0, device="cuda"),
              "out_positions": torch.full((layers, len(lens), hs, keep + 1), 8, dtype=torch.int32, device="cuda")}
    span = recent * 5 if recent * 5 <= keep else recent          # positions are 5 apart
    new = kvm.evict(paged, step.own, 1, 1 + layers, wd, pd, keep, recent=span, **kw)
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    assert new.tolist() == [min(n, keep) for n in lens]
    gw, gp = (wd, pd) if in_place else (kw["out_weights"], kw["out_positions"])
    gw, gp = gw.cpu(), gp.cpu()
    exp = b.pool.clone()
    e = exp.view(layers + 1, 2, -1, hs, H // hs * D)
    for l in range(layers):
        for s, n in enumerate(lens):
            rows = b.rows(b.own_table, s, n)
            for h in range(hs):
                ew, epos, moves = su.evict_row(w[l, s, h, :n].tolist(), p[l, s, h, :n].tolist(), keep, span)
                k = min(n, keep)
                assert gp[l, s, h, :k].tolist() == epos[:k]
                assert torch.equal(gw[l, s, h, :k].view(torch.int32), torch.tensor(ew[:k]).view(torch.int32)) or \
                    torch.equal(torch.nan_to_num(gw[l, s, h, :k], 77.0), torch.nan_to_num(torch.tensor(ew[:k]), 77.0))
                for to, src in moves:
                    e[1 + l, :, rows[to], h] = e[1 + l, :, rows[src], h].clone()
                if in_place:
                    assert torch.equal(gp[l, s, h, k:], p[l, s, h, k:])
                else:
                    assert torch.all(gp[l, s, h, k:] == 8) and torch.all(gw[l, s, h, k:] == 8.0)
    assert torch.equal(pool.cpu().view(torch.int16), exp.view(torch.int16))


def test_evict_bad_page_is_reported():
    b = su.Batch(8, 1, 64, 16, [40], [0])
    b.own_table[0, 2] = -3
    pool, paged, step = device(b)
    w = torch.zeros((1, 1, 1, 40), device="cuda")
    w[..., 33] = 1.0                                       # sits on the bad page
    p = torch.arange(40, dtype=torch.int32, device="cuda").view(1, 1, 1, 40)
    kvm.evict(paged, step.own, 0, 1, w, p, 4, recent=0)
    assert kvm.take_faults() == 1
    assert torch.equal(pool.cpu().view(torch.int16), b.pool.view(torch.int16))
    assert int(p[0, 0, 0, 3]) == 33


# ------------------------------------------------------------------ together

def test_decode_with_a_retrieved_prefix_and_eviction():
    """A shared prefix comes back from chunks (retrieve), two sequences decode behind it: append, attend, add_weights,
    and an eviction once the budget is passed, followed in 64 bits with the cache the library holds."""
    H, rep, D, P, keep, recent = 2, 2, 64, 16, 24, 6
    b = su.Batch(11, H, D, P, [20, 9], [1, 1], [70], [2], layers=2, table_room=2)
    pool, paged, step = device(b, max_len=b.own_table.shape[1] * P)
    # chunk_size = page: one chunk a page
    chunks = [torch.zeros(paged.chunk_bytes(min(16, 70 - 16 * c)), dtype=torch.uint8, device="cuda") for c in range(5)]
    seq = kvm.Seq(b.prefix_table[0].contiguous().cuda(), 0, 70, chunks)
    kvm.store(paged, [seq])
    prefix_rows = b.rows(b.prefix_table, 0, 70).cuda()
    pool.view(2, 2, -1, H, D)[:, :, prefix_rows] = float("nan")
    assert kvm.retrieve(paged, [seq], masks=[[1] * 5]) == [70]
    torch.cuda.synchronize()
    assert torch.equal(pool.cpu().view(torch.int16), b.pool.view(torch.int16))

    rope = kvm.Rope(D)
    f, _ = kvm.Rope.frequencies(D)
    cap = b.own_table.shape[1] * P
    w = torch.zeros((2, 2, H, cap), device="cuda")
    sp = torch.arange(cap, dtype=torch.int32, device="cuda").expand(2, 2, H, cap).contiguous()
    pw = torch.zeros((2, 1, H, 70), device="cuda")
    for t in range(18):
        pos = torch.tensor([90 + t, 79 + t], dtype=torch.int32)
        step.own.lens += 1
        b.lens = [n + 1 for n in b.lens]
        for layer in range(2):
            q, k, v = (b.normal(2, h, D) for h in (H * rep, H, H))
            qr = kvm.append(paged, step, layer, q.cuda(), k.cuda(), v.cuda(), pos.cuda(), rope, weights=w[layer],
                            slot_positions=sp[layer])
            out, lse = kvm.attend(paged, step, layer, qr)
            before, pbefore = w[layer].cpu(), pw[layer].cpu()
            kvm.add_weights(paged, step, layer, qr, lse, w[layer], pw[layer])
            b.pool = pool.cpu()
            kk, size = su.rope64(k, pos, f, 1.0, D, False)
            for s in range(2):
                x = b.rows(b.own_table, s, b.lens[s], b.lens[s] - 1)[0]
                within(b.flat()[layer, 0, x], kk[s], size[s] * 2.0 ** -20 + kk[s].abs() * (2.0 ** -8 + 2.0 ** -20), "k")
                assert torch.equal(b.flat()[layer, 1, x], v[s])
            wo, wl, eo, el = su.attend64(b, qr.cpu(), D ** -0.5, layer=layer)
            within(lse, wl, el, "lse")
            within(out, wo, eo, "out")
            ww, wp, ew, ep = su.weights64(b, qr.cpu(), lse.cpu(), D ** -0.5, before, pbefore, layer=layer)
            within(w[layer], ww, ew, "weights")
            within(pw[layer], wp, ep, "prefix weights")
        if max(b.lens) > keep:
            w0, p0, pool0 = w.cpu(), sp.cpu(), pool.cpu().view(2, 2, -1, H, D)
            new = kvm.evict(paged, step.own, 0, 2, w, sp, keep, recent=recent)
            for layer in range(2):
                for s in range(2):
                    rows = b.rows(b.own_table, s, b.lens[s])
                    for h in range(H):
                        n = b.lens[s]
                        ew, ep_, moves = su.evict_row(w0[layer, s, h, :n].tolist(), p0[layer, s, h, :n].tolist(), keep, recent)
                        kept = min(n, keep)
                        assert w[layer, s, h, :kept].tolist() == ew[:kept] and sp[layer, s, h, :kept].tolist() == ep_[:kept]
                        for to, src in moves:
                            pool0[layer, :, rows[to], h] = pool0[layer, :, rows[src], h].clone()
            assert torch.equal(pool.cpu().view(torch.int16), pool0.view(b.pool.shape).view(torch.int16))
            step.own.lens.copy_(new)
            b.lens = new.tolist()
    assert max(b.lens) == keep and kvm.take_faults() == 0


def test_step_captured_in_a_graph_follows_the_lengths():
    """One decode step captured once and replayed as the sequences grow, with eager work between the replays; every
    replay equals the eager calls on a copy."""
    H, rep, D, P = 2, 4, 128, 16
    b = su.Batch(12, H, D, P, [20, 37, 5], [1, 1, 1], [150], [3], layers=1, table_room=1)
    cap = b.own_table.shape[1] * P
    sides = []
    for _ in range(2):
        pool, paged, step = device(b, max_len=cap)
        st = {"pool": pool, "paged": paged, "step": step, "w": torch.zeros((1, 3, H, cap), device="cuda"),
              "p": torch.arange(cap, dtype=torch.int32, device="cuda").expand(1, 3, H, cap).contiguous(),
              "q": torch.zeros((3, H * rep, D), dtype=torch.bfloat16, device="cuda"),
              "k": torch.zeros((3, H, D), dtype=torch.bfloat16, device="cuda"),
              "v": torch.zeros((3, H, D), dtype=torch.bfloat16, device="cuda"),
              "pos": torch.zeros(3, dtype=torch.int32, device="cuda"), "ws": step.new_attend_workspace(H * rep),
              "es": step.own.new_evict_workspace(paged, 1, H, 30), "rope": kvm.Rope(D),
              "out": torch.zeros((3, H * rep, D), dtype=torch.bfloat16, device="cuda"),
              "lse": torch.zeros((3, H * rep), device="cuda"), "qr": torch.zeros((3, H * rep, D), dtype=torch.bfloat16, device="cuda"),
              "lens": torch.zeros(3, dtype=torch.int32, device="cuda")}
        sides.append(st)

    def once(st):
        kvm.append(st["paged"], st["step"], 0, st["q"], st["k"], st["v"], st["pos"], st["rope"], q_out=st["qr"],
                   weights=st["w"][0], slot_positions=st["p"][0])
        kvm.attend(st["paged"], st["step"], 0, st["qr"], out=st["out"], lse=st["lse"], workspace=st["ws"])
        kvm.add_weights(st["paged"], st["step"], 0, st["qr"], st["lse"], st["w"][0])
        kvm.evict(st["paged"], st["step"].own, 0, 1, st["w"], st["p"], 30, recent=4, out_lens=st["lens"],
                  workspace=st["es"])

    eager, graphed = sides
    once(eager)                                        # loads the code before the capture
    eager["pool"].copy_(b.pool)
    eager["w"].zero_()
    eager["p"].copy_(graphed["p"])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        once(graphed)
    for t in range(6):
        for st in sides:
            gen = torch.Generator(device="cuda").manual_seed(100 + t)
            for x in ("q", "k", "v"):
                st[x].copy_(torch.randn(st[x].shape, generator=gen, device="cuda"))
            st["pos"].fill_(200 + t)
            st["step"].own.lens.add_(1)
        once(eager)
        g.replay()
        torch.cuda.synchronize()
        for x in ("qr", "out", "lse", "w", "p", "lens", "pool"):
            a, c = eager[x], graphed[x]
            assert torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a,
                               c.view(torch.int16) if c.dtype == torch.bfloat16 else c), (t, x)
        for st in sides:
            st["step"].own.lens.copy_(st["lens"])
        (torch.randn(512, 512, device="cuda") @ torch.randn(512, 512, device="cuda")).sum().item()
    assert kvm.take_faults() == 0


def test_rows_of_one_token_with_any_stride():
    """Dimensions of one may have any stride: q of one row and one head cut out of odd places."""
    b, q = _attend_case((1, 1, 64, 16, [30], [1], [], []))
    pool, paged, step = device(b)
    wide = torch.zeros((3, 5, 72), dtype=torch.bfloat16, device="cuda")
    odd = wide.as_strided((1, 1, 64), (77, 13, 1), 0)
    odd.copy_(q)
    out, lse = kvm.attend(paged, step, 1, odd)
    ref, ref_lse = kvm.attend(paged, step, 1, q.cuda())
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


def test_python_refusals():
    b, q = _attend_case((2, 2, 64, 16, [30, 17], [3, 2], [21], [1]))
    pool, paged, step = device(b)
    qd, lse = q.cuda(), torch.zeros((5, 4), device="cuda")
    rope, pos = kvm.Rope(64), torch.zeros(5, dtype=torch.int32, device="cuda")
    k = torch.zeros((5, 2, 64), dtype=torch.bfloat16, device="cuda")
    raw = torch.cuda.current_stream().cuda_stream or 1
    w = torch.zeros((2, 2, 30), device="cuda")
    sp = torch.zeros((2, 2, 30), dtype=torch.int32, device="cuda")
    for call in (lambda: kvm.attend(paged, step, 1, qd.float()), lambda: kvm.attend(paged, step, 1, qd[:4]),
                 lambda: kvm.attend(paged, step, 1, qd[:, :3]), lambda: kvm.attend(paged, step, 2, qd),
                 lambda: kvm.attend(paged, step, 1, qd, scale=0.0), lambda: kvm.attend(paged, step, 1, q),
                 lambda: kvm.attend(paged, step, 1, qd.transpose(1, 2).contiguous().transpose(1, 2)),
                 lambda: kvm.attend(paged, step, 1, qd, lse=lse.half()), lambda: kvm.attend(paged, step, 1, qd, stream=raw),
                 lambda: kvm.attend(paged, step, 1, qd, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")),
                 lambda: kvm.append(paged, step, 0, qd, k, k, pos.long(), rope), lambda: kvm.append(paged, step, 0, qd, k, k.half(), pos, rope),
                 lambda: kvm.append(paged, step, 0, qd, k, k, pos[:4], rope), lambda: kvm.append(paged, step, 0, None, k, k, pos, rope, q_out=qd),
                 lambda: kvm.append(paged, step, 0, qd, k, k, pos, kvm.Rope(66)), lambda: kvm.append(paged, step, 0, qd, k, k, pos, rope, weights=w),
                 lambda: kvm.append(paged, step, 0, qd, k, k, pos, rope, weights=w[:, :, :20], slot_positions=sp[:, :, :20]),
                 lambda: kvm.add_weights(paged, step, 0, qd, lse, w[:1]), lambda: kvm.add_weights(paged, step, 0, qd, lse),
                 lambda: kvm.add_weights(paged, step, 0, qd, lse, w[:, :, :29].contiguous()),
                 lambda: kvm.evict(paged, step.own, 0, 1, w[None], sp[None], 40, recent=41),
                 lambda: kvm.evict(paged, step.own, 0, 2, w[None], sp[None], 10),
                 lambda: kvm.evict(paged, step.own, 0, 1, w[None], sp[None].float(), 10),
                 lambda: kvm.evict(paged, step.own, 0, 1, w[None], sp[None], 10, out_lens=step.own.lens),
                 lambda: kvm.evict(paged, step.own, 0, 1, w[None], sp[None], 10, out_weights=w[None]),
                 lambda: kvm.Step(paged, step.own, [1]), lambda: kvm.Step(paged, step.own, [1, 1], group_sizes=[1]),
                 lambda: kvm.Step(paged, step.own, [1, 1], prefix=step.prefix, group_sizes=[3]),
                 lambda: kvm.Step(paged, kvm.Tables(step.own.table, step.own.lens, 1000), [1, 1]),
                 lambda: kvm.Tables(step.own.table.long(), step.own.lens, 10), lambda: kvm.Tables(step.own.table, step.own.lens[:1], 10),
                 lambda: kvm.Tables(step.own.table.cpu(), step.own.lens, 10)):
        with pytest.raises(kvm.KvError):
            call()
    torch.cuda.synchronize()
    assert torch.equal(pool.cpu().view(torch.int16), b.pool.view(torch.int16)) and kvm.take_faults() == 0


def test_calls_on_a_side_stream():
    """Two streams at once, each with its own workspace, ordered after the current stream's work."""
    b, q = _attend_case((2, 4, 128, 16, [300, 170], [1, 1], [400], [2]))
    pool, paged, step = device(b)
    qd = q.cuda()
    ref = kvm.attend(paged, step, 1, qd)
    torch.cuda.synchronize()
    outs = []
    for st in (torch.cuda.Stream(), torch.cuda.Stream()):
        st.wait_stream(torch.cuda.current_stream())
        ws = step.new_attend_workspace(8)
        outs.append(kvm.attend(paged, step, 1, qd, workspace=ws, stream=st))
        outs.append(kvm.attend(paged, step, 1, qd, stream=st))       # allocates for that stream
    torch.cuda.synchronize()
    for o, l in outs:
        assert torch.equal(o, ref[0]) and torch.equal(l, ref[1])
