"""The model-step entry points without a GPU: the host refuses malformed calls
before any HIP call, sizes workspaces from the bounds, and the rotary
frequencies follow their formulas."""
import ctypes
import math

import pytest

import paged_kv_movement_amd as kvm
from test_abi_host import _lib, _paged

A = 0x10000          # an address that is never followed


def tables(n=2, max_len=100, table=A, stride=7, lens=A):
    return kvm._KvTables(n, max_len, table, stride, lens)


def step(own=None, prefix=None, q_start=A, group_start=A, n_rows=2, max_new=1, max_group_rows=2):
    return kvm._KvStep(own or tables(), prefix or kvm._KvTables(), q_start, group_start, n_rows, max_new, max_group_rows)


def rows(data=A, row=32 * 128, head=128):
    return kvm._KvRows(data, row, head)


def ref(x):
    return None if x is None else ctypes.byref(x)


def attend(p=None, s=None, layer=0, q=None, heads=32, scale=0.1, out=None, lse=A, ws=A, ws_bytes=1 << 40):
    L = _lib()
    return L.kv_attend(ref(p or _paged()), ref(s or step()), layer, ref(q or rows()), heads, scale, ref(out or rows()), lse,
                       ws, ws_bytes, None)


EINVAL, ERANGE = kvm.KV_EINVAL, kvm.KV_ERANGE


@pytest.mark.parametrize("kw,code,word", [
    (dict(layer=-1), EINVAL, "layers"), (dict(layer=32), EINVAL, "layers"),
    (dict(heads=0), EINVAL, "q_heads"), (dict(heads=12), EINVAL, "multiple"),
    (dict(p=_paged(D=12, H=2), heads=2), EINVAL, "head_dim"), (dict(p=_paged(D=264, H=1), heads=1), EINVAL, "head_dim"),
    (dict(p=_paged(n=1 << 30)), EINVAL, "2^31"),
    (dict(s=step(own=tables(stride=6))), ERANGE, "block table"),
    (dict(s=step(own=tables(n=-1))), EINVAL, "sequences"), (dict(s=step(own=tables(max_len=-1))), EINVAL, "max_len"),
    (dict(s=step(own=tables(lens=None))), EINVAL, "lens"), (dict(s=step(own=tables(table=None))), EINVAL, "table"),
    (dict(s=step(own=tables(stride=1 << 31))), EINVAL, "stride"),
    (dict(s=step(prefix=tables(n=1, stride=1))), ERANGE, "prefix"),
    (dict(s=step(prefix=tables(n=1), group_start=None)), EINVAL, "group_start"),
    (dict(s=step(q_start=None)), EINVAL, "q_start"), (dict(s=step(n_rows=-1)), EINVAL, "n_rows"),
    (dict(q=rows(data=None)), EINVAL, "q is NULL"), (dict(q=rows(data=A + 8)), EINVAL, "16 bytes"),
    (dict(q=rows(head=132)), EINVAL, "16 bytes"), (dict(out=rows(data=A + 4)), EINVAL, "8 bytes"),
    (dict(out=rows(row=1026)), EINVAL, "8 bytes"), (dict(lse=None), EINVAL, "lse"),
    (dict(scale=0.0), EINVAL, "scale"), (dict(scale=-1.0), EINVAL, "scale"), (dict(scale=float("nan")), EINVAL, "scale"),
    (dict(scale=float("inf")), EINVAL, "scale"),
    (dict(ws=None), EINVAL, "workspace"), (dict(ws=A + 128), EINVAL, "workspace"), (dict(ws_bytes=100), EINVAL, "workspace"),
    (dict(s=step(n_rows=1 << 30)), EINVAL, "too many"),
    (dict(s=step(own=tables(n=1 << 24, max_len=16), max_new=1 << 20)), EINVAL, "too many"),
])
def test_attend_refusals(kw, code, word):
    assert attend(**kw) == code
    assert word in _lib().kv_last_error().decode()


def test_attend_with_nothing_to_do_launches_nothing():
    assert attend(s=step(n_rows=0)) == kvm.KV_OK
    assert attend(s=step(own=tables(n=0))) == kvm.KV_OK


def test_attend_workspace_grows_with_the_bounds_only():
    L = _lib()

    def size(**kw):
        return L.kv_attend_workspace_bytes(ref(_paged()), ref(step(**kw)), 32)
    assert size() >= 256 and size() % 256 == 0
    assert size(n_rows=64) > size()
    assert size(own=tables(max_len=9000, stride=600)) > size()
    assert L.kv_attend_workspace_bytes(ref(_paged()), ref(step()), 12) == 0
    assert b"multiple" in L.kv_last_error()


@pytest.mark.timeout(60, method="signal")
@pytest.mark.parametrize("group_rows", [0, 1, 5, 700, 1 << 20])
@pytest.mark.parametrize("new", [0, 1, 5, 700, 1 << 20])
def test_attend_workspace_of_any_bounds(group_rows, new):
    """A size, or a refusal with its reason, in bounded time: empty groups, groups of few rows over one token, long tables."""
    L = _lib()
    for own_len in (0, 1, 64, 65, 5000, 1 << 30):
        for prefix_len in (None, 0, 1, 40, 64, 65, 100000, 1 << 30):
            for dim in (8, 128, 256):
                own = tables(n=3, max_len=own_len, stride=1 << 26)
                prefix = None if prefix_len is None else tables(n=2, max_len=prefix_len, stride=1 << 26)
                s = step(own=own, prefix=prefix, n_rows=min(3 * new, 1 << 20), max_new=new, max_group_rows=group_rows)
                size = L.kv_attend_workspace_bytes(ref(_paged(D=dim)), ref(s), 32)
                assert size % 256 == 0 and (size > 0 or b"too many" in L.kv_last_error())


def append(p=None, s=None, layer=0, q=1, k=1, v=1, o=1, heads=32, t=0, ot=0, pos=A, rope=1, slots=None):
    def r(x):
        return ref(rows()) if x == 1 else ref(x)
    rp = kvm._KvRope(A, 128, 0, 1.0) if rope == 1 else rope
    return _lib().kv_append(ref(p or _paged()), ref(s or step()), layer, r(q), r(k), r(v), r(o), heads, t, ot, pos, ref(rp),
                            ref(slots), None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(layer=32), EINVAL, "layers"), (dict(k=None), EINVAL, "NULL"), (dict(rope=None), EINVAL, "NULL"),
    (dict(q=None), EINVAL, "together"), (dict(o=None), EINVAL, "together"), (dict(t=3), EINVAL, "type"),
    (dict(t=1, ot=2), EINVAL, "q_out"), (dict(heads=0), EINVAL, "q_heads"), (dict(pos=None), EINVAL, "positions"),
    (dict(rope=kvm._KvRope(A, 3, 0, 1.0)), EINVAL, "rot"), (dict(rope=kvm._KvRope(A, 130, 0, 1.0)), EINVAL, "rot"),
    (dict(rope=kvm._KvRope(A, -2, 0, 1.0)), EINVAL, "rot"), (dict(rope=kvm._KvRope(None, 64, 0, 1.0)), EINVAL, "freqs"),
    (dict(k=rows(data=A + 1)), EINVAL, "aligned"), (dict(o=rows(data=A + 2), ot=0, t=0, q=rows(data=None)), EINVAL, "NULL"),
    (dict(slots=kvm._KvSlots(A, None, 8, 100)), EINVAL, "slots"), (dict(slots=kvm._KvSlots(A, A, 2, 100)), EINVAL, "heads"),
    (dict(slots=kvm._KvSlots(A, A, 8, 99)), ERANGE, "cap"), (dict(s=step(own=tables(stride=6))), ERANGE, "block table"),
])
def test_append_refusals(kw, code, word):
    assert append(**kw) == code
    assert word in _lib().kv_last_error().decode()


@pytest.mark.parametrize("own,prefix,code,word", [
    (None, None, EINVAL, "needed"), (kvm._KvSums(None, None, 100), None, EINVAL, "own"),
    (kvm._KvSums(None, A, 99), None, ERANGE, "own"), (None, kvm._KvSums(None, None, 9), EINVAL, "prefix"),
])
def test_add_weights_refusals(own, prefix, code, word):
    assert _lib().kv_add_weights(ref(_paged()), ref(step()), 0, ref(rows()), A, 32, 0.1, ref(own), ref(prefix), None) == code
    assert word in _lib().kv_last_error().decode()


def evict(t=None, l0=0, l1=1, i=None, o=None, keep=50, recent=5, lens=2 * A, ws=A, n_ws=1 << 30):
    i = i or kvm._KvSlots(A, A, 8, 100)
    return _lib().kv_evict(ref(_paged()), ref(t or tables()), l0, l1, ref(i), ref(o or i), keep, recent, lens, ws, n_ws, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(l1=0), EINVAL, "layers"), (dict(l1=33), EINVAL, "layers"), (dict(keep=-1), EINVAL, "keep"),
    (dict(recent=51), EINVAL, "recent"), (dict(recent=-1), EINVAL, "recent"),
    (dict(i=kvm._KvSlots(A, A, 3, 100)), EINVAL, "heads"), (dict(i=kvm._KvSlots(A, A, 8, 99)), ERANGE, "cap"),
    (dict(o=kvm._KvSlots(2 * A, 2 * A, 8, 49)), ERANGE, "out"), (dict(o=kvm._KvSlots(2 * A, 2 * A, 1, 60)), EINVAL, "heads"),
    (dict(o=kvm._KvSlots(A, 2 * A, 8, 100)), EINVAL, "in place"), (dict(o=kvm._KvSlots(A, A, 8, 101)), EINVAL, "cap"),
    (dict(i=kvm._KvSlots(None, A, 8, 100)), EINVAL, "NULL"), (dict(lens=None), EINVAL, "NULL"),
    (dict(lens=A), EINVAL, "out_lens"), (dict(ws=None), EINVAL, "workspace"), (dict(n_ws=10), EINVAL, "workspace"),
    (dict(t=tables(stride=6)), ERANGE, "block table"),
])
def test_evict_refusals(kw, code, word):
    assert evict(**kw) == code
    assert word in _lib().kv_last_error().decode()


def test_evict_workspace():
    L = _lib()
    n = [L.kv_evict_workspace_bytes(ref(_paged()), ref(tables()), layers, heads, keep)
         for layers, heads, keep in ((1, 8, 50), (4, 8, 50), (1, 1, 50), (1, 8, 100), (1, 8, 0))]
    assert n[1] > n[0] > n[2] and n[3] < n[0] and n[4] >= 256
    assert L.kv_evict_workspace_bytes(ref(_paged()), ref(tables()), 33, 8, 50) == 0


def test_rope_frequencies():
    f, g = kvm.Rope.frequencies(8, 10000.0)
    assert g == 1.0 and f == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-15)
    assert kvm.Rope.frequencies(8, 10000.0, "linear", 4.0)[0] == pytest.approx([x / 4 for x in f], rel=1e-15)
    n, _ = kvm.Rope.frequencies(8, 10000.0, "ntk", 4.0)
    assert n[0] == 1.0 and n[3] == pytest.approx(f[3] / 4.0, rel=1e-12)        # the slowest pair is interpolated in full
    for scaling in ("yarn", "wavelength"):
        y, gain = kvm.Rope.frequencies(128, 10000.0, scaling, 8.0, 4096)
        b, _ = kvm.Rope.frequencies(128, 10000.0)
        assert y[0] == b[0] and y[-1] == pytest.approx(b[-1] / 8, rel=1e-15)    # fast pairs stay, slow ones are divided
        assert all(b[j] / 8 * (1 - 1e-12) <= y[j] <= b[j] * (1 + 1e-12) for j in range(64))
        assert gain == (pytest.approx(0.1 * math.log(8.0) + 1.0) if scaling == "yarn" else 1.0)
    assert kvm.Rope.frequencies(0) == ([], 1.0)
    for bad in (dict(rot=3), dict(rot=4, base=1.0), dict(rot=4, factor=0.0), dict(rot=4, scaling="other"),
                dict(rot=2, scaling="ntk"), dict(rot=4, scaling="yarn", fast=1.0, slow=2.0),
                dict(rot=4, scaling="wavelength", low=4.0, high=4.0), dict(rot=4, original_length=0)):
        with pytest.raises(kvm.KvError):
            kvm.Rope.frequencies(**bad)
