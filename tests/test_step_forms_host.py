"""Windows, normalised heads and the 8-bit pool without a GPU: what the host refuses before any HIP call, and the sizes
of workspaces."""
import ctypes

import pytest

import paged_kv_movement_amd as kvm
from test_abi_host import _lib, _paged
from test_step_host import A, EINVAL, ERANGE, ref, rows, step, tables


def paged8(k_scales=A, v_scales=A, **kw):
    return kvm._KvPaged8(_paged(**kw), k_scales, v_scales)


def window(w=64, s=4):
    return kvm._KvWindow(w, s)


def norm(q=A, k=A, qs=0, ks=0, eps=1e-6, centered=0):
    return kvm._KvNorm(q, k, qs, ks, eps, centered)


def last_error():
    return _lib().kv_last_error().decode()


def attend(bits, p=None, s=None, layer=0, q=None, heads=32, scale=0.1, w=None, out=None, lse=A, ws=A, ws_bytes=1 << 40):
    L = _lib()
    f, p = (L.kv_attend8, p or paged8()) if bits == 8 else (L.kv_attend_window, p or _paged())
    return f(ref(p), ref(s or step()), layer, ref(q or rows()), heads, scale, ref(w), ref(out or rows()), lse, ws,
             ws_bytes, None)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("kw,code,word", [
    (dict(w=window(0, 0)), EINVAL, "window"), (dict(w=window(-1, 0)), EINVAL, "window"),
    (dict(w=window(5, -1)), EINVAL, "sinks"),
    (dict(layer=-1), EINVAL, "layers"), (dict(layer=32), EINVAL, "layers"), (dict(heads=12), EINVAL, "multiple"),
    (dict(s=step(own=tables(stride=6))), ERANGE, "block table"), (dict(s=step(q_start=None)), EINVAL, "q_start"),
    (dict(q=rows(data=None)), EINVAL, "q is NULL"), (dict(q=rows(head=132)), EINVAL, "16 bytes"),
    (dict(out=rows(data=A + 4)), EINVAL, "8 bytes"), (dict(lse=None), EINVAL, "lse"),
    (dict(scale=0.0), EINVAL, "scale"), (dict(ws_bytes=100), EINVAL, "workspace"), (dict(out=rows()), EINVAL, "out must"),
])
def test_attend_refuses(bits, kw, code, word):
    kw.setdefault("w", window())
    assert attend(bits, **{"out": rows(data=A << 8), **kw}) == code and word in last_error(), last_error()


@pytest.mark.parametrize("p,word", [
    (paged8(k_scales=None), "scales"), (paged8(v_scales=None), "scales"), (paged8(D=72, H=8), "multiple of 16"),
    (paged8(D=264, H=2), "multiple of 16"), (paged8(D=272, H=1), "head_dim"), (paged8(n=1 << 30), "2^31"),
])
def test_attend_refuses_8bit_pools(p, word):
    assert attend(8, p=p) == EINVAL and word in last_error(), last_error()


def test_null_pools():
    L = _lib()
    s = step()
    assert L.kv_attend8(None, ref(s), 0, ref(rows()), 32, 0.1, None, ref(rows()), A, A, 1 << 40, None) == EINVAL
    assert L.kv_attend8_workspace_bytes(None, ref(s), 32, None) == 0 and "paged8" in last_error()
    assert L.kv_append8(None, ref(s), 0, None, ref(rows()), ref(rows()), None, 0, 0, 0, A, None, None, None) == EINVAL
    assert L.kv_pack8(ref(_paged()), ref(tables()), None, None, 0, 0, 1, None) == EINVAL
    assert L.kv_pack8(None, ref(tables()), ref(paged8()), None, 0, 0, 1, None) == EINVAL
    assert L.kv_unpack8(ref(paged8()), None, ref(_paged()), None, 0, 0, 1, None) == EINVAL
    assert "tables" in last_error()


def test_window_workspaces():
    """By what an item may see: a window makes the workspace no larger, a narrow one over a long table smaller; a window
    past everything asks for what none does; the two pools for the same."""
    L, p, p8 = _lib(), _paged(n=1 << 20), paged8(n=1 << 20)
    for s in (step(own=tables(n=4, max_len=100000, stride=6250), n_rows=4),
              step(own=tables(n=4, max_len=3000, stride=6250), n_rows=2400, max_new=600),
              step(own=tables(n=4, max_len=900, stride=6250), prefix=tables(n=1, max_len=50000, stride=6250), n_rows=4,
                   max_group_rows=4)):
        none = L.kv_attend_workspace_bytes(ref(p), ref(s), 32)
        sizes = [L.kv_attend_window_workspace_bytes(ref(p), ref(s), 32, ref(window(w, 4)))
                 for w in (1, 64, 1000, 1 << 30, (1 << 31) - 1)]
        assert none > 0 and sizes[-1] == sizes[-2] == none and all(0 < x <= 2 * none for x in sizes)
        assert [L.kv_attend8_workspace_bytes(ref(p8), ref(s), 32, ref(window(w, 4)))
                for w in (1, 64, 1000, 1 << 30, (1 << 31) - 1)] == sizes
        assert L.kv_attend8_workspace_bytes(ref(p8), ref(s), 32, None) == none
        assert L.kv_attend_window_workspace_bytes(ref(p), ref(s), 32, None) == none
        assert L.kv_attend_window_workspace_bytes(ref(p), ref(s), 32, ref(window((1 << 31) - 1, (1 << 31) - 1))) == none
    assert L.kv_attend_window_workspace_bytes(ref(p), ref(step()), 32, ref(window(0, 0))) == 0


def append(kind, p=None, s=None, k=None, v=None, q=None, out=None, heads=0, type=0, out_type=0, rope=None, n=None, slots=None):
    L = _lib()
    rope = rope or kvm._KvRope(A, 128, 0, 1.0)
    kv = rows(row=8 * 128)
    if kind == 8:
        return L.kv_append8(ref(p or paged8()), ref(s or step()), 0, ref(q), ref(k or kv), ref(v or kv), ref(out), heads,
                            type, out_type, A, ref(rope), ref(n), None)
    return L.kv_append_normed(ref(p or _paged()), ref(s or step()), 0, ref(q), ref(k or kv), ref(v or kv), ref(out), heads,
                              type, out_type, A, ref(rope), ref(n or norm()), ref(slots), None)


@pytest.mark.parametrize("kind", [16, 8])
@pytest.mark.parametrize("kw,word", [
    (dict(n=norm(eps=-1.0)), "eps"), (dict(n=norm(eps=float("nan"))), "eps"), (dict(n=norm(eps=float("inf"))), "eps"),
    (dict(n=norm(centered=2)), "centered"), (dict(n=norm(q=A + 4)), "aligned"), (dict(n=norm(k=A + 8)), "aligned"),
    (dict(n=norm(qs=130)), "multiples of 4"), (dict(n=norm(ks=-128)), "multiples of 4"),
    (dict(rope=kvm._KvRope(A, 7, 0, 1.0)), "rot"), (dict(rope=kvm._KvRope(A, 130, 0, 1.0)), "rot"),
    (dict(rope=kvm._KvRope(None, 64, 0, 1.0)), "freqs"), (dict(type=3), "type"),
    (dict(q=rows()), "together"), (dict(q=rows(), out=rows(row=64), heads=32), "overlap"),
    (dict(k=rows(data=None)), "NULL"), (dict(k=rows(data=A + 1)), "aligned"),
    (dict(s=step(q_start=None)), "q_start"), (dict(s=step(n_rows=-1)), "n_rows"),
])
def test_append_refuses(kind, kw, word):
    assert append(kind, **kw) == EINVAL and word in last_error(), last_error()


def test_append_of_nothing():
    empty = step(own=tables(n=0), n_rows=0)
    assert append(16, s=empty) == kvm.KV_OK and append(8, s=empty) == kvm.KV_OK
    assert append(8, p=paged8(D=72, H=8)) == EINVAL and append(8, p=paged8(v_scales=None)) == EINVAL


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,code,word", [
    (dict(t=tables(stride=6)), ERANGE, "block table"), (dict(t=tables(lens=None)), EINVAL, "lens"),
    (dict(to=A, stride=6), ERANGE, "to_table"), (dict(to=A, stride=-1), EINVAL, "to_stride"),
    (dict(to=A, stride=1 << 31), EINVAL, "to_stride"),
    (dict(layers=(0, 0)), EINVAL, "layers"), (dict(layers=(-1, 1)), EINVAL, "layers"), (dict(layers=(0, 33)), EINVAL, "layers"),
    (dict(p8=paged8(P=32)), EINVAL, "page size"), (dict(p8=paged8(H=4)), EINVAL, "page size"),
    (dict(p8=paged8(D=64)), EINVAL, "page size"), (dict(p8=paged8(L=3), layers=(0, 1)), EINVAL, "page size"),
    (dict(p8=paged8(k_scales=None)), EINVAL, "scales"),
    (dict(t=tables(n=1 << 24, max_len=1 << 20, stride=1 << 20)), EINVAL, "too many"),
])
def test_pack_refuses(back, kw, code, word):
    L = _lib()
    p, p8 = _paged(), kw.get("p8") or paged8()
    args = (kw.get("to"), kw.get("stride", 0), *kw.get("layers", (0, 1)), None)
    t = kw.get("t") or tables()
    rc = L.kv_unpack8(ref(p8), ref(t), ref(p), *args) if back else L.kv_pack8(ref(p), ref(t), ref(p8), *args)
    assert rc == code and word in last_error(), last_error()


def test_pack_of_nothing():
    L = _lib()
    for t in (tables(n=0), tables(max_len=0), tables(n=0, table=None, lens=None), tables(max_len=0, table=None)):
        assert L.kv_pack8(ref(_paged()), ref(t), ref(paged8()), None, 0, 0, 1, None) == kvm.KV_OK
        assert L.kv_unpack8(ref(paged8()), ref(t), ref(_paged()), None, 0, 0, 1, None) == kvm.KV_OK


# ---- the binding

class Stub:
    """Stands where a call must not get to."""
    def __getattr__(self, name):
        raise AssertionError(f"{name} was looked at")


@pytest.mark.parametrize("wrong", [1 << 32, (1 << 32) + 64, 1 << 31, -(1 << 31) - 1])
def test_windows_past_32_bits_are_refused_not_cut(wrong):
    for w, s in ((wrong, 0), (64, wrong)):
        with pytest.raises(kvm.KvError, match="32 bits"):
            kvm._window(w, s)


def test_sinks_need_a_window():
    with pytest.raises(kvm.KvError, match="without a window"):
        kvm._window(None, 4)
    assert kvm._window(None, 0) is None and kvm._window(7, 2).window == 7


def test_an_8bit_pool_is_refused_where_a_bf16_one_is_meant():
    p8, x = object.__new__(kvm.Paged8), Stub()
    for call in (lambda: kvm.add_weights(p8, x, 0, x, x), lambda: kvm.evict(p8, x, 0, 1, x, x, 5),
                 lambda: kvm.Batch(p8, []), lambda: kvm.store(p8, []), lambda: kvm.pack8(p8, x, x),
                 lambda: kvm.unpack8(x, x, p8)):
        with pytest.raises(kvm.KvError, match="bf16 pool"):
            call()
    p = object.__new__(kvm.Paged)
    for call in (lambda: kvm.pack8(p, x, p), lambda: kvm.unpack8(p, x, p)):
        with pytest.raises(kvm.KvError, match="Paged8"):
            call()


def test_struct_sizes():
    """The binding's structs lie as the header's: fields in order, C alignment."""
    assert ctypes.sizeof(kvm._KvPaged8) == ctypes.sizeof(kvm._KvPaged) + 16
    assert ctypes.sizeof(kvm._KvNorm) == 40 and ctypes.sizeof(kvm._KvWindow) == 8
