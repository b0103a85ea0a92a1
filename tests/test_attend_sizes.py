"""Workspaces of attend where an 8-bit pool is cut into other pieces than a bf16 one: they are those of the pool that the
call is given, whichever pool the step was made for."""
import pytest
import torch

import paged_kv_movement_amd as kvm
import pool8_util as pu
from gpu_util import say
from test_abi_host import _lib, _paged
from test_gpu_append_heads import device8
from test_gpu_step import device, within
from test_step_forms_host import paged8, ref, window
from test_step_host import step, tables



def pool(c, kind):
    p = object.__new__(kind)
    p.c = c
    return p


def step_of(c, paged):
    s = object.__new__(kvm.Step)
    s.c, s.paged = c, paged
    return s


# wide pieces of a prefix beside narrow own ones, where the pools' cuts differ
def descriptors():
    c = step(own=tables(n=17, max_len=454, stride=64), prefix=tables(n=1, max_len=3683, stride=256), n_rows=17,
             max_new=1, max_group_rows=17)
    return c, pool(_paged(H=8, D=64, n=4096), kvm.Paged), pool(paged8(H=8, D=64, n=4096), kvm.Paged8)


@pytest.mark.parametrize("seen", [None, (1926, 4)])
def test_sizes_are_those_of_the_pool_that_is_asked_for(seen):
    c, p16, p8 = descriptors()
    L, w = _lib(), None if seen is None else window(*seen)
    of16 = L.kv_attend_window_workspace_bytes(ref(p16.c), ref(c), 8, ref(w))
    of8 = L.kv_attend8_workspace_bytes(ref(p8.c), ref(c), 8, ref(w))
    assert of16 > 0 and (seen is not None or of8 > of16)     # the shape is one where it matters
    args = (8,) if seen is None else (8, *seen)
    more = {} if seen is not None else {"window": None}
    for made_for in (p16, p8):
        s = step_of(c, made_for)
        assert s.attend_workspace_bytes(*args, paged=p16, **more) == of16
        assert s.attend_workspace_bytes(*args, paged=p8, **more) == of8
        assert s.attend_workspace_bytes(*args, **more) == (of16 if made_for is p16 else of8)


@pytest.mark.gpu
@pytest.mark.parametrize("seen", [{}, {"window": 1000, "sinks": 4}])
def test_a_step_of_one_pool_on_the_other(seen):
    """The call allocates, and new_attend_workspace gives, what the pool of the call needs."""
    say("a step of one pool on the other", seen)
    b = pu.Batch8(3, 8, 64, 16, [454 - 7 * i for i in range(17)], [1] * 17, [3683], [17], layers=1)
    bytes8, scales, p8, step8 = device8(b)
    pl, p16, step16 = device(b)
    q = b.normal(17, 8, 64, gain=2.0)
    sizes = [step16.attend_workspace_bytes(8, *seen.values(), paged=p) for p in (p16, p8)]
    if not seen:
        assert sizes[1] > sizes[0]
    wo, wl, eo, el = pu.attend_window64(b, q, 64 ** -0.5, seen.get("window"), seen.get("sinks", 0))
    for paged in (p8, p16):
        got = []
        for s in (step16, step8):
            out, lse = kvm.attend(paged, s, 0, q.cuda(), **seen)
            within(lse, wl, el, "lse")
            within(out, wo, eo, "out")
            ws = s.new_attend_workspace(8, *seen.values(), paged=paged).fill_(0xFF)
            again = kvm.attend(paged, s, 0, q.cuda(), workspace=ws, **seen)
            got += [(out, lse), again]
        for out, lse in got[1:]:
            assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    if not seen:
        with pytest.raises(kvm.KvError, match="workspace"):
            kvm.attend(p8, step8, 0, q.cuda(), workspace=step8.new_attend_workspace(8, paged=p16))
    assert kvm.take_faults() == 0


def test_a_window_can_need_more_than_none():
    """Sizes are not ordered by the window; the largest of those asked for serves them all, as the header says."""
    L, p = _lib(), _paged(n=1 << 20)
    c = step(own=tables(n=32, max_len=6000, stride=512), prefix=tables(n=1, max_len=8192, stride=512), n_rows=32,
             max_new=1, max_group_rows=32)
    none = L.kv_attend_workspace_bytes(ref(p), ref(c), 32)
    sizes = [L.kv_attend_window_workspace_bytes(ref(p), ref(c), 32, ref(window(w, 4))) for w in (64, 4096, 1 << 30)]
    assert 0 < none < sizes[1] < sizes[2] and sizes[0] < none
    # a workspace of one call's size is refused where another one's is larger, before anything is launched
    q, out = kvm._KvRows(0x10000, 32 * 128, 128), kvm._KvRows(0x1000000, 32 * 128, 128)

    def call(ws_bytes, w):
        return L.kv_attend_window(ref(p), ref(c), 0, ref(q), 32, 0.1, ref(w), ref(out), 0x10000, 0x10000, ws_bytes, None)
    assert call(none, window(4096, 4)) == kvm.KV_EINVAL and "workspace" in L.kv_last_error().decode()
