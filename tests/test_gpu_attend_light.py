"""attend where a few tokens draw the attention and weigh nothing in the output: what is left of it is the sum of many
light weights, which must not be lost beside the heavy ones."""
import pytest
import torch

import paged_kv_movement_amd as kvm
import pool8_util as pu
import step_util as su
from gpu_util import say
from test_gpu_append_heads import device8
from test_gpu_step import device, within

pytestmark = pytest.mark.gpu

CASES = [
    # heads, rep, dim, page, lens, new, prefix, sizes; window
    ((1, 4, 128, 16, [30, 9], [20, 6], [4096], [2]), None),          # many rows of a group over its prefix
    ((2, 2, 64, 16, [3000], [40], [], []), None),                    # a prompt's end over its own pages
    ((1, 2, 256, 32, [2050], [12], [], []), None),
    ((1, 4, 128, 16, [3000], [1], [], []), None),                    # a single token
    ((1, 4, 128, 16, [2600], [24], [900], [1]), 2000),
]


@pytest.mark.parametrize("case,window", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("nats", [12.0, 17.4, 20.0, 60.0])
def test_light_weights_beside_heavy_ones(case, window, bits, nats):
    """Every 64th token's score is `nats` above the others', and its V is 0.  The bounds are those of float32 sums with
    the weights as two bf16 parts, 2^-16 of each weight however light it is (step_util.attend64): they are relative to
    sum w |v|, which here is the light tokens' alone."""
    say("light", case, window, bits, nats)
    H, rep, D, P, lens, new, prefix, sizes = case
    b = su.Batch(7, H, D, P, lens, new, prefix, sizes, layers=2)
    top = nats * D ** 0.5 / 8.0
    for table, ns in ((b.own_table, b.lens), (b.prefix_table, b.prefix)):
        for i, n in enumerate(ns):
            rows = b.rows(table, i, n)
            heavy = torch.arange(n) % 64 == 5
            k, v = b.flat()[:, 0, rows].float() * 0.05, b.flat()[:, 1, rows].float().abs() + 0.5
            k[..., 0] = torch.where(heavy, top, 0.0)[None, :, None]
            v[:, heavy] = 0.0
            b.flat()[:, 0, rows], b.flat()[:, 1, rows] = k.bfloat16(), v.bfloat16()
    q = b.normal(b.q_start[-1], H * rep, D, gain=0.5)
    q[..., 0] = 8.0
    if bits == 8:
        b.__class__ = pu.Batch8
        b.quantise()
    paged, step = (device8(b) if bits == 8 else device(b))[-2:]
    seen = {} if window is None else {"window": window, "sinks": 4}
    out, lse = kvm.attend(paged, step, 1, q.cuda(), **seen)
    torch.cuda.synchronize()
    assert kvm.take_faults() == 0
    b.__class__ = su.Batch                       # the bound that knows no fp16
    wo, wl, eo, el = pu.attend_window64(b, q, D ** -0.5, window, seen.get("sinks", 0), layer=1)
    within(lse, wl, el, "lse")
    within(out, wo, eo, "out")
    assert float((eo / wo.abs()).nan_to_num(0.0).max()) < 2.0 ** -6        # what is asked is relative to the output
