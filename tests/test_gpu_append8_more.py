"""append, into both pools, of heads that turn in part and hold values that are not finite, and of rotations with a gain:
what the pool holds afterwards."""
import math

import pytest
import torch

import paged_kv_movement_amd as kvm
import pool8_util as pu
import step_util as su
from gpu_util import say
from test_gpu_append_heads import BF, FL, HF, check_blocks, device8
from test_gpu_step import device

pytestmark = pytest.mark.gpu

TURNS = [(True, 40), (True, 42), (False, 32), (True, 2), (False, 64)]


def odd_rows(b, rot):
    """Rows with one value each, behind what turns, that is not finite: (x, where they are)."""
    x = b.normal(4, 2, 64, dtype=BF)
    at = ((0, 0, min(rot, 63), math.inf), (1, 1, 63, -math.inf), (2, 0, max(rot, 62), math.nan),
          (3, 1, min(rot + 1, 63), math.inf)) if rot < 64 else ()
    for r, h, d, value in at:
        x[r, h, d] = value
    return x, at


def float_bound(y, pos, f, gain, rot, il):
    """Of a key that went through 64 bits, as test_gpu_append_heads has it: the angle's rounding in either formula and some
    roundings of 2^-53."""
    return (su.rope64(y, pos, f, gain, rot, il)[1] + y.abs()).nan_to_num(0.0, 0.0, 0.0) * (
        2.0 ** -46 + float(pos.abs().max()) * 2.0 ** -51)


@pytest.mark.parametrize("interleaved,rot", TURNS)
def test_bytes_beside_what_does_not_turn(interleaved, rot):
    """Only the value itself is NaN in the pool; its pair, its neighbours and the block's scale are the formula's."""
    say("bytes beside", interleaved, rot)
    b = pu.Batch8(3, 2, 64, 16, [4], [4])
    bytes8, scales, paged, step = device8(b)
    x, at = odd_rows(b, rot)
    pos = torch.arange(7, 11, dtype=torch.int32)
    rope = kvm.Rope(rot, interleaved=interleaved)
    f, gain = kvm.Rope.frequencies(rot)
    kvm.append(paged, step, 0, None, x.cuda(), x.cuda(), pos.cuda(), rope)
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    k = su.rope64(x, pos, f, gain, rot, interleaved)[0]
    assert int((~torch.isfinite(k)).sum()) == len(at)
    check_blocks(b, 0, (k, x.double()), (float_bound(x.double(), pos, f, gain, rot, interleaved),
                                         torch.zeros(x.shape, dtype=torch.float64)), b.bytes8, b.scales, bytes8, scales,
                 b.q_start)
    held = pu.values(bytes8.cpu(), scales.cpu()).view(1, 2, -1, 2, 64)[0][:, b.rows(b.own_table, 0, 4)]
    for kv in range(2):
        assert torch.equal(torch.isnan(held[kv]), ~torch.isfinite(k if kv == 0 else x.double()))


@pytest.mark.parametrize("interleaved,rot", TURNS[:4])
def test_normed_rows_with_a_value_that_is_not_finite(interleaved, rot):
    """As the formula has it: beside an infinity a head is 0 and the infinity NaN, beside a NaN all of it is NaN; another
    head and V are what they are without."""
    say("normed rows", interleaved, rot)
    b = su.Batch(3, 2, 64, 16, [4], [4])
    pool, paged, step = device(b)
    x, at = odd_rows(b, rot)
    pos = torch.arange(7, 11, dtype=torch.int32).cuda()
    rope, norm = kvm.Rope(rot, interleaved=interleaved), kvm.Norm(torch.ones(64))
    q = kvm.append(paged, step, 0, x.cuda(), x.cuda(), x.cuda(), pos, rope, norm=norm).cpu()
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    k, v = (pool.cpu().view(1, 2, -1, 2, 64)[0, i][b.rows(b.own_table, 0, 4)] for i in range(2))
    assert torch.equal(v.view(torch.int16)[torch.isfinite(x)], x.view(torch.int16)[torch.isfinite(x)])
    assert torch.equal(v.float().nan_to_num(7.0), x.float().nan_to_num(7.0))
    odd = {(r, h): (d, value) for r, h, d, value in at}
    for got in (q, k):
        for r in range(4):
            for h in range(2):
                y = got[r, h].float()
                if (r, h) not in odd:
                    assert torch.isfinite(y).all() and torch.any(y != 0)
                    continue
                d, value = odd[r, h]
                if math.isnan(value):
                    assert torch.isnan(y).all()
                else:
                    assert math.isnan(float(y[d])) and torch.all(torch.cat([y[:d], y[d + 1:]]) == 0)


@pytest.mark.parametrize("dim,rot,interleaved,page,lens,new,dtype", [
    (128, 128, False, 16, [100, 47, 5], [90, 20, 1], BF),
    (64, 32, True, 16, [40, 17], [40, 3], HF),
    (80, 48, False, 12, [13, 25], [1, 25], FL),
    (128, 128, False, 128, [300], [299], BF),              # more angles than a workgroup keeps
])
@pytest.mark.parametrize("gain", [None, 0.375, 3.0])
def test_append8_of_a_rotation_with_a_gain(dim, rot, interleaved, page, lens, new, dtype, gain):
    """Positions that follow one another, as an angle turned on, and others; what does not turn has no gain."""
    say("gain", dim, rot, interleaved, page, gain)
    b = pu.Batch8(9, 2, dim, page, lens, new, layers=2)
    bytes8, scales, paged, step = device8(b)
    rows = b.q_start[-1]
    pos = torch.arange(rows, dtype=torch.int32) + 1000
    pos[rows // 2:] += 5000
    pos[rows // 3] = 70000
    rope = kvm.Rope(rot, interleaved=interleaved, scaling="yarn", factor=4.0, gain=gain)
    f, g = kvm.Rope.frequencies(rot, scaling="yarn", factor=4.0)
    g = float(torch.tensor(g if gain is None else gain, dtype=FL))
    assert g != 1.0
    k, v = b.normal(rows, 2, dim, dtype=dtype), b.normal(rows, 2, dim, dtype=dtype)
    kvm.append(paged, step, 1, None, k.cuda(), v.cuda(), pos.cuda(), rope)
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    want = su.rope64(k, pos, f, g, rot, interleaved)[0]
    check_blocks(b, 1, (want, v.double()), (float_bound(k.double(), pos, f, g, rot, interleaved),
                                            torch.zeros(v.shape, dtype=torch.float64)), b.bytes8, b.scales, bytes8, scales,
                 b.q_start)


def test_append8_of_many_rows_is_that_of_few():
    """New tokens enough for q to have a launch of its own: q and the pool as from calls of one sequence each."""
    H, rep, D, P, n = 2, 2, 64, 16, 2700
    b = pu.Batch8(11, H, D, P, [n, n + 5, n, 30], [n, n, n - 9, 30], layers=1)
    bytes8, scales, paged, step = device8(b)
    rows = b.q_start[-1]
    assert rows > 8000
    q, k, v = (b.normal(rows, h, D).cuda() for h in (H * rep, H, H))
    pos = torch.arange(rows, dtype=torch.int32).cuda()
    rope, norm = kvm.Rope(D), kvm.Norm(b.normal(D, dtype=FL) + 1, b.normal(D, dtype=FL) + 1)
    got = kvm.append(paged, step, 0, q, k, v, pos, rope, norm=norm)
    many = [x.clone() for x in (bytes8, scales)]
    bytes8.copy_(b.bytes8)
    scales.copy_(b.scales)
    own = step.own
    for s, m in enumerate(b.new):
        one = kvm.Step(paged, kvm.Tables(own.table[s:s + 1], own.lens[s:s + 1], b.lens[s]), [m])
        r = slice(b.q_start[s], b.q_start[s] + m)
        part = kvm.append(paged, one, 0, q[r], k[r], v[r], pos[r], rope, norm=norm)
        assert torch.equal(part, got[r])
    torch.cuda.synchronize()
    assert torch.equal(many[0], bytes8) and torch.equal(many[1].view(torch.int32), scales.view(torch.int32))
    assert kvm.take_faults() == 0
