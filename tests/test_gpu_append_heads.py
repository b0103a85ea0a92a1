"""append with normalised heads, and into an 8-bit pool, on the GPU against plain 64-bit implementations."""
import math

import pytest
import torch

import paged_kv_movement_amd as kvm
import pool8_util as pu
import step_util as su
from gpu_util import say
from test_gpu_step import device, within

pytestmark = pytest.mark.gpu

BF, HF, FL = torch.bfloat16, torch.float16, torch.float32


def device8(b, max_len=None, prefix_max=None):
    """(bytes, scales, paged8, step) of a Batch8 on the GPU."""
    bytes8, scales = b.bytes8.cuda(), b.scales.cuda()
    paged = kvm.Paged8.from_pool(bytes8, scales)
    own = kvm.Tables(b.own_table.cuda(), torch.tensor(b.lens, dtype=torch.int32).cuda(),
                     max(b.lens, default=0) if max_len is None else max_len)
    pre = None
    if b.prefix:
        pre = kvm.Tables(b.prefix_table.cuda(), torch.tensor(b.prefix, dtype=torch.int32).cuda(),
                         max(b.prefix) if prefix_max is None else prefix_max)
    return bytes8, scales, paged, kvm.Step(paged, own, b.new, prefix=pre, group_sizes=b.sizes)


def projections(b, rep, dtype, fused):
    """q, k, v: parts of one projection's rows; not fused: rows an odd number of elements apart."""
    H, D, rows = b.heads, b.dim, b.q_start[-1]
    qkv = b.normal(rows, (rep + 2) * H * D + (0 if fused else 1), dtype=dtype).cuda()
    return (qkv[:, :rep * H * D].unflatten(1, (rep * H, D)), qkv[:, rep * H * D:(rep + 1) * H * D].unflatten(1, (H, D)),
            qkv[:, (rep + 1) * H * D:(rep + 2) * H * D].unflatten(1, (H, D)))


def positions_of(new, start):
    return torch.tensor([start + i for m in new for i in range(m)], dtype=torch.int32)


NORMS = [
    # heads, rep, dim, page, lens, new, rot, interleaved, type, q type, start, centered, weights by head, eps
    (8, 4, 128, 16, [5, 33, 1], [1, 1, 1], 128, False, BF, None, 0, False, False, 1e-6),
    (2, 4, 64, 16, [40, 17], [40, 3], 32, True, HF, None, 5000, False, True, 1e-5),
    (1, 1, 80, 12, [13, 0, 25], [1, 0, 25], 48, False, FL, None, 100000, True, True, 1e-6),
    (3, 5, 72, 8, [9, 2], [2, 2], 20, False, FL, BF, 1 << 20, False, False, 0.0),
    (2, 2, 36, 3, [7, 11], [7, 1], 36, True, HF, BF, 77, True, False, 1e-6),
    (1, 8, 256, 256, [300], [260], 256, True, BF, None, (1 << 31) - 400, False, True, 1e-6),
    (4, 1, 8, 1, [4, 4], [4, 1], 0, False, BF, None, 3, True, False, 1e-3),
    (1, 2, 40, 16, [2], [5], 16, False, FL, None, -9, False, True, 1e-6),       # more new tokens than slots
    (1, 2, 264, 16, [9], [4], 264, False, BF, None, 1000, True, True, 1e-6),    # more units than a wave has lanes
    (2, 1, 520, 4, [6, 5], [2, 5], 500, True, FL, None, 10, False, False, 1e-6),
    (5, 7, 112, 16, [70], [3], 112, False, HF, None, 200, True, True, 1e-6),
    (1, 1, 2, 4, [3], [3], 2, False, BF, None, 0, False, False, 1e-6),
    (4, 2, 128, 16, [20, 9], [3, 9], 46, True, BF, None, 500, False, False, 1e-6),   # pairs that end inside a vector
    (2, 3, 80, 16, [20, 9], [3, 9], 2, True, HF, None, 500, True, True, 1e-6),
]


@pytest.mark.parametrize("case", NORMS, ids=[str(i) for i in range(len(NORMS))])
@pytest.mark.parametrize("fused", [True, False])
def test_append_normed(case, fused):
    H, rep, D, P, lens, new, rot, il, dt, qdt, start, centered, by_head, eps = case
    if H * D % 8:
        H = 8 // math.gcd(8, D)
    say("append normed", case, fused)
    b = su.Batch(1, H, D, P, lens, new, layers=3)
    pool, paged, step = device(b)
    q, k, v = projections(b, rep, dt, fused)
    pos = positions_of(new, start)
    rope = kvm.Rope(rot, base=10000.0, interleaved=il)
    f, gain = kvm.Rope.frequencies(rot, 10000.0)
    qw = b.normal(*((rep * H, D) if by_head else (D,)), dtype=FL) + 1
    kw = b.normal(*((H, D) if by_head else (D,)), dtype=FL) + 1
    norm = kvm.Norm(qw, kw, eps=eps, centered=centered)
    cap = max(lens) + 3
    w = torch.full((len(lens), H, cap), 5.0, device="cuda")
    sp = torch.full((len(lens), H, cap), -5, dtype=torch.int32, device="cuda")
    q_out = None if qdt is None else torch.empty((q.shape[0], rep * H, D), dtype=qdt, device="cuda")
    got = kvm.append(paged, step, 1, q, k, v, pos.cuda(), rope, q_out=q_out, weights=w, slot_positions=sp, norm=norm)
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    want, err = pu.rotated64(*pu.norm64(q.cpu(), qw, eps, centered), pos, f, gain, rot, il)
    within(got, want, pu.rounded(want, err, got.dtype), "q")
    exp = b.pool.clone().double()
    off = torch.zeros_like(exp)
    wk, ek = pu.rotated64(*pu.norm64(k.cpu(), kw, eps, centered), pos, f, gain, rot, il)
    we, pe = torch.full(w.shape, 5.0), torch.full(sp.shape, -5, dtype=torch.int32)
    e, ee = exp.view(3, 2, -1, H, D), off.view(3, 2, -1, H, D)
    for s, (n, m) in enumerate(zip(lens, new)):
        for i in range(m):
            slot, r = n - m + i, b.q_start[s] + i
            if slot < 0:
                continue
            x = b.rows(b.own_table, s, slot + 1, slot)[0]
            e[1, 0, x], ee[1, 0, x] = wk[r], pu.rounded(wk[r], ek[r], BF)
            e[1, 1, x], ee[1, 1, x] = v[r].cpu().double(), v[r].cpu().double().abs() * 2.0 ** -8 + 2.0 ** -133
            we[s, :, slot], pe[s, :, slot] = 0.0, pos[r]
    within(pool, exp, off, "pool")
    assert torch.equal(w.cpu(), we) and torch.equal(sp.cpu(), pe)


@pytest.mark.parametrize("centered", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30, 1e-38])
def test_norm_of_heads_far_from_one(centered, eps):
    """Heads whose squares leave float32, one of zeros, one with an infinity, one with a NaN: each as the formula has it,
    none reaching another."""
    H, D = 12, 64
    b = su.Batch(3, H, D, 16, [2], [2])
    pool, paged, step = device(b)
    k = b.normal(2, H, D, dtype=FL) + 0.5
    for h, size in enumerate((3e37, 1e30, 1e19, 1.0, 1e-12, 1e-19, 1e-30, 2e-38, 0.0)):
        k[:, h] *= size
    k[:, 9, 5], k[:, 10, 63] = math.inf, math.nan
    q = k.clone()
    rope = kvm.Rope(0)
    pos = torch.arange(2, dtype=torch.int32).cuda()
    q_out = kvm.append(paged, step, 0, q.cuda(), k.cuda(), k.cuda(), pos, rope,
                       norm=kvm.Norm(eps=eps, centered=centered))
    torch.cuda.synchronize()
    want, err = pu.norm64(k, None, float(torch.tensor(eps, dtype=FL)), centered)
    ok = [0, 1, 2, 3, 4, 5, 6, 7, 8, 11]
    if eps == 0.0:
        ok.remove(8)                                       # 0 / 0
        assert torch.isnan(q_out[:, 8]).all()
    # where eps outweighs squares that are below float32, what is lost is below 2^-126 over the root
    slack = 2.0 ** -60 * want.abs() + 2.0 ** -100
    if eps > 0.0:
        slack[:, 7] += want[:, 7].abs() * 2.0 ** -20 + 2.0 ** -40
    within(q_out[:, ok], want[:, ok], (pu.rounded(want, err, FL) + slack)[:, ok], "q")
    assert not torch.isfinite(q_out[:, 9, 5]).any() and torch.isnan(q_out[:, 10]).all()
    if not centered:
        assert torch.all(q_out[:, 9, :5] == 0)


@pytest.mark.parametrize("interleaved,rot", [(True, 40), (True, 42), (False, 32)])
@pytest.mark.parametrize("bits", [16, 8])
def test_what_does_not_turn_passes(interleaved, rot, bits):
    """An infinity or a NaN behind the elements that turn stays where it is."""
    b = (pu.Batch8 if bits == 8 else su.Batch)(3, 2, 64, 16, [4], [4])
    paged, step = (device8 if bits == 8 else device)(b)[-2:]
    x = b.normal(4, 2, 64, dtype=BF)
    x[0, 0, rot], x[1, 1, 63], x[2, 0, 62], x[3, 1, rot + 1] = math.inf, -math.inf, math.nan, math.inf
    pos = torch.arange(7, 11, dtype=torch.int32).cuda()
    rope = kvm.Rope(rot, interleaved=interleaved)
    norm = None if bits == 8 else kvm.Norm(torch.ones(64))
    got = kvm.append(paged, step, 0, x.cuda(), x.cuda(), x.cuda(), pos, rope, norm=norm).cpu()
    if bits == 8:
        assert torch.equal(got[:, :, rot:].view(torch.int16), x[:, :, rot:].view(torch.int16))
    assert torch.isfinite(got[:, :, :rot]).all() or bits == 16
    for r, h, d in ((0, 0, rot), (1, 1, 63), (2, 0, 62), (3, 1, rot + 1)):
        assert torch.isfinite(torch.cat([got[r, h, :d], got[r, h, d + 1:]])).all() or r == 2 or bits == 16
        assert not torch.isfinite(got[r, h, d])
    assert kvm.take_faults() == 0


def test_append_normed_in_place_without_q_and_without_norm():
    b = su.Batch(2, 2, 64, 16, [20, 3], [4, 1])
    pool, paged, step = device(b)
    pos = torch.arange(5, dtype=torch.int32).cuda()
    rope = kvm.Rope(64)
    q, k, v = (b.normal(5, h, 64).cuda() for h in (8, 2, 2))
    norm = kvm.Norm(None, b.normal(64, dtype=FL), eps=1e-5)
    apart = kvm.append(paged, step, 0, q, k, v, pos, rope, norm=norm)
    first = pool.clone()
    pool.copy_(b.pool)
    assert kvm.append(paged, step, 0, None, k, v, pos, rope, norm=norm) is None
    assert torch.equal(pool.view(torch.int16), first.view(torch.int16))
    assert kvm.append(paged, step, 0, q, k, v, pos, rope, q_out=q, norm=norm) is q and torch.equal(q, apart)
    # the weights are read at each call
    w = torch.ones(64, device="cuda")
    norm = kvm.Norm(w, w)
    one = kvm.append(paged, step, 0, apart, k, v, pos, rope, norm=norm)
    w.fill_(2.0)
    assert torch.equal(kvm.append(paged, step, 0, apart, k, v, pos, rope, norm=norm), one * 2)
    assert kvm.take_faults() == 0


# ------------------------------------------------------------------ an 8-bit pool

EIGHT = [
    # heads, rep, dim, page, lens, new, rot, interleaved, type, q type, start, norm
    (8, 4, 128, 16, [5, 33, 1, 16, 17], [1, 1, 1, 1, 1], 128, False, BF, None, 0, False),
    (8, 4, 128, 16, [100, 47, 32], [90, 20, 32], 128, False, BF, None, 9, True),
    (2, 4, 64, 16, [40, 17], [40, 3], 32, True, HF, None, 5000, True),
    (1, 1, 80, 12, [13, 0, 25], [1, 0, 25], 48, False, FL, None, 100000, False),
    (3, 2, 48, 8, [9, 2], [2, 2], 20, False, FL, BF, 1 << 20, True),
    (2, 2, 16, 3, [7, 11], [7, 1], 16, True, HF, BF, 77, False),
    (1, 8, 256, 256, [300], [260], 256, True, BF, None, (1 << 31) - 400, True),
    (4, 1, 16, 1, [4, 4], [4, 1], 0, False, BF, None, 3, False),
    (1, 2, 32, 16, [2], [5], 16, False, FL, None, -9, False),               # more new tokens than slots
    (2, 1, 272, 16, [9, 30], [4, 30], 272, False, BF, None, 1000, True),     # more units than a wave has lanes
    (1, 1, 128, 64, [150, 64], [149, 1], 128, False, HF, None, 10, False),
    (3, 1, 128, 128, [300], [299], 128, False, FL, None, 10, True),          # more angles than a workgroup keeps
    (1, 3, 96, 300, [299], [299], 96, True, BF, None, 0, False),
    (8, 8, 128, 16, [78, 204, 90], [5, 5, 17], 122, True, BF, None, 40, True),   # pairs that end inside a vector
    (70, 1, 128, 64, [130], [129], 128, False, BF, None, 7, True),           # the same of more heads than a workgroup takes
    (2, 1, 256, 32, [70, 40], [66, 40], 256, True, HF, None, 7, False),
]


def check_blocks(b, layer, want, err, before_bytes, before_scales, bytes8, scales, q_start):
    """The pool after an append8 of K and V values `want` [2][rows, H, D], each off by at most `err`."""
    got_b, got_s = bytes8.cpu(), scales.cpu().double()
    left_b, left_s = before_bytes.clone(), before_scales.clone()
    for s, (n, m) in enumerate(zip(b.lens, b.new)):
        first = max(0, n - m)
        if m == 0 or n == 0:
            continue
        for p in range(first // b.page, -(-n // b.page)):
            page = int(b.own_table[s, p])
            lo, hi = max(first, p * b.page) - p * b.page, min(n, (p + 1) * b.page) - p * b.page
            r = q_start[s] + p * b.page + lo - (n - m)
            for kv in range(2):
                x, e = want[kv][r:r + hi - lo], err[kv][r:r + hi - lo]
                fin = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
                least, most = pu.scales_of((fin - e).clamp(min=0), (0, 2)), pu.scales_of(fin + e, (0, 2))
                sc, was = got_s[layer, kv, page], before_scales[layer, kv, page].double()
                if lo > 0:
                    least, most = torch.maximum(least, was), torch.maximum(most, was)
                    old = pu.values(before_bytes[layer, kv, page, :lo], was)
                    assert torch.equal(pu.values(got_b[layer, kv, page, :lo], sc).nan_to_num(7.7e33),
                                       (pu.e4m3(old / sc[:, None]) * sc[:, None]).nan_to_num(7.7e33)), "old tokens"
                assert torch.all((least <= sc) & (sc <= most)), ("scale", least, sc, most)
                got = pu.values(got_b[layer, kv, page, lo:hi], sc)
                # scales end at 2^119: what is beyond 448 2^119 (float32 goes on to 1.14 times that) is held as that
                x = torch.where(torch.isfinite(x), x.clamp(-448 * 2.0 ** 119, 448 * 2.0 ** 119), x)
                # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale below 2^-6 of it
                half = torch.maximum((x.abs() + e) * 2.0 ** -4, (sc * 2.0 ** -10)[:, None].expand_as(x))
                within(got, torch.where(torch.isfinite(x), x, torch.full_like(x, math.nan)), e + half, "new tokens")
                # every value that is not within its error of a border is the formula's
                low, high = (pu.e4m3((x + d * e) / sc[:, None]) * sc[:, None] for d in (-1, 1))
                exact = torch.isfinite(x) & (low == high)
                assert torch.equal(got[exact], low[exact]) and exact.double().mean() > 0.4
            left_b[layer, :, page, :hi] = got_b[layer, :, page, :hi]
            left_s[layer, :, page] = got_s[layer, :, page].float()
    assert torch.equal(got_b, left_b), "bytes that hold no token of the call"
    assert torch.equal(got_s.float().view(torch.int32), left_s.view(torch.int32)), "scales of other blocks"


@pytest.mark.parametrize("case", EIGHT, ids=[str(i) for i in range(len(EIGHT))])
@pytest.mark.parametrize("fused", [True, False])
def test_append8(case, fused):
    H, rep, D, P, lens, new, rot, il, dt, qdt, start, normed = case
    say("append8", case, fused)
    b = pu.Batch8(1, H, D, P, lens, new, layers=3, gain=0.7)
    bytes8, scales, paged, step = device8(b)
    q, k, v = projections(b, rep, dt, fused)
    pos = positions_of(new, start)
    rope = kvm.Rope(rot, base=10000.0, interleaved=il)
    f, gain = kvm.Rope.frequencies(rot, 10000.0)
    qw, kw = b.normal(rep * H, D, dtype=FL) + 1, b.normal(H, D, dtype=FL) + 1
    norm = kvm.Norm(qw, kw) if normed else None
    q_out = None if qdt is None else torch.empty((q.shape[0], rep * H, D), dtype=qdt, device="cuda")
    got = kvm.append(paged, step, 1, q, k, v, pos.cuda(), rope, q_out=q_out, norm=norm)
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0

    def ready(x, w):
        y, e = pu.norm64(x, w, float(torch.tensor(1e-6)), False) if normed else (x.double(), torch.zeros(x.shape).double())
        return pu.rotated64(y, e, pos, f, gain, rot, il)
    want, err = ready(q.cpu(), qw)
    within(got, want, pu.rounded(want, err, got.dtype), "q")
    # k goes through 64 bits: off by the angle's rounding, 2^-53 of it in either formula, and some roundings of 2^-53
    wk, _ = ready(k.cpu(), kw)
    y = pu.norm64(k.cpu(), kw, float(torch.tensor(1e-6)), False)[0] if normed else k.cpu().double()
    ek = (su.rope64(y, pos, f, gain, rot, il)[1] + y.abs()) * (2.0 ** -46 + float(pos.abs().max()) * 2.0 ** -51)
    check_blocks(b, 1, (wk, v.cpu().double()), (ek, torch.zeros(v.shape).double()), b.bytes8, b.scales, bytes8, scales,
                 b.q_start)


def test_append8_of_odd_values():
    """Not rotated: exact.  Infinities and NaN are held as NaN and do not touch their block; zeros, subnormals, float32's
    largest, values on the borders of the scale and of the bytes."""
    H, D, P = 3, 16, 4
    b = pu.Batch8(4, H, D, P, [4, 4, 7, 4, 4, 4], [4, 4, 3, 4, 4, 4])
    bytes8, scales, paged, step = device8(b)
    rows = b.q_start[-1]
    x = b.normal(rows, H, D, dtype=FL)
    x[0:4] = 0.0
    x[0, 1, 0] = 1e-42
    x[4, 0, 3], x[5, 0, 4], x[6, 1, 0] = math.inf, -math.inf, math.nan
    x[7, 2, :] = math.inf
    x[4:8, 2, :] = math.nan
    x[8:11] *= 1e-33
    x[11, 0, 0], x[12, 1, 1], x[13, 2, 2] = 448.0, 448.0000305, 3.4028234e38
    x[15] = torch.tensor([i * 0.0625 + 0.03125 for i in range(H * D)]).view(H, D)      # ties
    x[19] = torch.tensor([(2 * i + 1) * 2.0 ** -10 for i in range(H * D)]).view(H, D)
    x[20, :, 0] = 448.0
    pos = torch.zeros(rows, dtype=torch.int32).cuda()
    kvm.append(paged, step, 0, None, x.cuda(), (-x).cuda(), pos, kvm.Rope(0))
    torch.cuda.synchronize()
    zero = torch.zeros(x.shape, dtype=torch.float64)
    check_blocks(b, 0, (x.double(), -x.double()), (zero, zero), b.bytes8, b.scales, bytes8, scales, b.q_start)
    assert kvm.take_faults() == 0


def test_append8_token_by_token():
    """A page filled one token at a time, each larger than the last: the scale ends where it would if all had come at
    once, and each token is off by its rounding and one half step for each time the block grew (none of which is larger
    than the last scale's)."""
    H, D, P, n = 2, 64, 16, 40
    b = pu.Batch8(5, H, D, P, [n], [n], layers=1)
    x = b.normal(n, H, D, dtype=BF)
    x *= torch.exp2(torch.arange(n).float() / 3)[:, None, None].bfloat16()
    rope = kvm.Rope(0)
    pos = torch.zeros(n, dtype=torch.int32).cuda()
    bytes8, scales, paged, step = device8(b)
    kvm.append(paged, step, 0, None, x.cuda(), x.cuda(), pos, rope)
    once = scales.clone()
    bytes8.copy_(b.bytes8)
    scales.fill_(math.nan)
    own = step.own
    one = kvm.Step(paged, own, [1])
    for i in range(n):
        own.lens.fill_(i + 1)
        kvm.append(paged, one, 0, None, x[i:i + 1].cuda(), x[i:i + 1].cuda(), pos[:1], rope)
    torch.cuda.synchronize()
    assert torch.equal(scales[0, :, b.own_table[0, :3].long()], once[0, :, b.own_table[0, :3].long()])
    got = pu.values(bytes8.cpu(), scales.cpu()).view(1, 2, -1, H, D)[0, 0, b.rows(b.own_table, 0, n)]
    sc = scales.cpu().double()[0, 0, b.own_table[0, :3].long()].repeat_interleave(P, 0)[:n]
    half = torch.maximum(x.double().abs() * 2.0 ** -4, 16 * sc[..., None] * 2.0 ** -10)
    within(got, x.double(), half, "values")
    assert kvm.take_faults() == 0


def test_append8_bad_pages_and_pools():
    b = pu.Batch8(6, 2, 64, 16, [20, 18], [2, 3])
    b.own_table[1, 1] = b.pages + 5
    bytes8, scales, paged, step = device8(b)
    pos = torch.arange(5, dtype=torch.int32).cuda()
    q, k, v = (b.normal(5, h, 64).cuda() for h in (2, 2, 2))
    got = kvm.append(paged, step, 0, q, k, v, pos, kvm.Rope(0))
    assert kvm.take_faults() == 1 and torch.equal(got, q)
    b.new, b.lens = [2, 1], [20, 16]
    zero = torch.zeros(k.shape, dtype=torch.float64)
    check_blocks(b, 0, (k.cpu().double(), v.cpu().double()), (zero, zero), b.bytes8, b.scales, bytes8, scales, [0, 2])
    # a scale array at an odd address: nothing is written
    bytes8.copy_(b.bytes8)
    paged.v_scale_addrs += 2
    kvm.append(paged, step, 0, q, k, v, pos, kvm.Rope(0))
    assert kvm.take_faults() & 4 and torch.equal(bytes8.cpu(), b.bytes8)
