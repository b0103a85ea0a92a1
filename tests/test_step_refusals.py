"""Calls of a model step that the host refuses, or answers without a launch, before any HIP call (no GPU needed)."""
import ctypes

import pytest

import paged_kv_movement_amd as kvm
from test_abi_host import _lib, _paged
from test_step_host import A, EINVAL, append, attend, ref, rows, step, tables


def add_weights(s=None, q=None, lse=A, own=None, prefix=None):
    return _lib().kv_add_weights(ref(_paged()), ref(s or step()), 0, ref(q or rows()), lse, 32, 0.1, ref(own), ref(prefix),
                                 None)


def last_error():
    return _lib().kv_last_error().decode()


# ---- q_start is read for every group too

NO_ROWS = dict(own=tables(n=0), prefix=tables(n=1), q_start=None)


def test_groups_of_no_sequences_still_need_q_start():
    """With prefixes but no sequences the kernels read q_start[0]."""
    assert add_weights(s=step(**NO_ROWS), prefix=kvm._KvSums(None, A, 100)) == EINVAL
    assert "q_start" in last_error()
    assert append(s=step(**NO_ROWS)) == EINVAL and "q_start" in last_error()
    assert attend(s=step(**NO_ROWS)) == EINVAL and "q_start" in last_error()
    assert attend(s=step(own=tables(n=0), q_start=None, group_start=None)) == kvm.KV_OK     # neither: nothing reads it


# ---- nothing cached, nothing asked

def test_batches_of_nothing_may_have_no_memory():
    """An empty tensor's address is NULL: sequences that hold nothing, or none at all, are no error."""
    empty = step(own=tables(n=0), n_rows=0)
    none = kvm._KvSums(None, None, 0)
    assert add_weights(s=empty, own=kvm._KvSums(None, None, 100)) == kvm.KV_OK
    assert add_weights(s=step(own=tables(max_len=0), n_rows=0), own=none) == kvm.KV_OK
    assert add_weights(s=step(own=tables(max_len=0), prefix=tables(n=1, max_len=0), n_rows=0), own=none, prefix=none) == kvm.KV_OK
    assert append(s=empty, slots=kvm._KvSlots(None, None, 8, 100)) == kvm.KV_OK
    assert append(s=step(own=tables(max_len=0), n_rows=0), slots=kvm._KvSlots(None, None, 8, 0)) == kvm.KV_OK
    # where there is something to write, NULL stays refused
    assert add_weights(own=kvm._KvSums(None, None, 100)) == EINVAL and "own" in last_error()
    assert add_weights(s=step(prefix=tables(n=1)), prefix=kvm._KvSums(None, None, 100)) == EINVAL
    assert append(slots=kvm._KvSlots(None, None, 8, 100)) == EINVAL and "slots" in last_error()


# ---- numbers that a C int does not hold

class Stub:
    """Stands where a call must not get to."""
    def __getattr__(self, name):
        raise AssertionError(f"{name} was looked at")


@pytest.mark.parametrize("wrong", [1 << 32, (1 << 32) + 7, 1 << 31, -(1 << 31) - 1, 1 << 63])
def test_numbers_past_32_bits_are_refused_not_cut(wrong):
    """ctypes cuts an integer to its low bits: keep = 2^32 would evict everything, layer = 2^32 write into layer 0."""
    x = Stub()
    for call in (lambda: kvm.evict(x, x, 0, 1, x, x, wrong), lambda: kvm.evict(x, x, 0, 1, x, x, 5, recent=wrong),
                 lambda: kvm.evict(x, x, wrong, wrong + 1, x, x, 5), lambda: kvm.evict(x, x, 0, wrong, x, x, 5),
                 lambda: kvm.append(x, x, wrong, x, x, x, x, x), lambda: kvm.attend(x, x, wrong, x),
                 lambda: kvm.add_weights(x, x, wrong, x, x)):
        with pytest.raises(kvm.KvError, match="32 bits"):
            call()


@pytest.mark.parametrize("keep", [1 << 32, (1 << 32) + 50])
def test_sizes_past_32_bits_are_refused_not_cut(keep):
    t = object.__new__(kvm.Tables)
    t.c = tables()
    p = Stub()
    for args in ((p, 1, 8, keep), (p, 1 << 32, 8, 50), (p, 1, 1 << 32, 50)):
        with pytest.raises(kvm.KvError, match="32 bits"):
            t.evict_workspace_bytes(*args)
    s = object.__new__(kvm.Step)
    s.paged = Stub()
    with pytest.raises(kvm.KvError, match="32 bits"):
        s.attend_workspace_bytes(keep)


# ---- what the binding made itself stays while a kernel on the current stream reads it

class Recorded:
    """A device tensor that notes the streams it is said to be used on."""
    is_cuda = True

    def __init__(self):
        self.streams = []

    def get_device(self):
        return 0

    device = "cuda:0"

    def record_stream(self, stream):
        self.streams.append(stream.cuda_stream)


class FakeTorch:
    """Two streams of one device, by handle; ``current`` is the one that calls without a stream go to."""
    current = 7

    def __init__(self):
        outer = self

        class Stream:
            def __init__(self, handle):
                self.cuda_stream = handle

        class C:
            _cuda_getCurrentRawStream = staticmethod(lambda device: outer.current)

        class Cuda:
            current_device = staticmethod(lambda: 0)
            current_stream = staticmethod(lambda device=None: Stream(outer.current))
        self._C, self.cuda = C, Cuda


@pytest.fixture
def fake_torch(monkeypatch):
    t = FakeTorch()
    monkeypatch.setattr(kvm, "_t", lambda: t)
    return t


def test_a_step_is_recorded_on_the_current_stream(fake_torch):
    p = Stub()
    s = object.__new__(kvm.Step)
    s.paged, s._dim, s._device, s._tensors, s._on_streams = p, 64, 0, [Recorded(), Recorded()], set()
    for current, expect in ((7, [7]), (7, [7]), (9, [7, 9]), (7, [7, 9])):          # once per stream
        fake_torch.current = current
        assert s._call(p, None, Recorded()) == current
        assert all(t.streams == expect for t in s._tensors)


def test_a_batch_is_recorded_on_the_current_stream(fake_torch):
    b = object.__new__(kvm.Batch)
    b._dev_tensors, b._on_streams, b._checked_fmts = [Recorded(), Recorded()], set(), {kvm.FMT_BF16}
    for current, expect in ((7, [7]), (7, [7]), (9, [7, 9]), (7, [7, 9])):
        fake_torch.current = current
        assert kvm._batch(None, b, kvm.FMT_BF16, None) is b
        assert all(t.streams == expect for t in b._dev_tensors)


# ---- outputs whose rows lie on one another

@pytest.mark.parametrize("n,heads,row,head,overlap", [
    (2, 32, 32 * 128, 128, False), (2, 32, 0, 128, True), (2, 32, 32 * 128, 0, True), (2, 32, 32 * 128, 64, True),
    (2, 32, 128, 128, True),                    # row 1 is row 0's second head
    (2, 32, 31 * 128, 128, True),               # its first head is row 0's last
    (2, 32, 128, 256, False), (3, 32, 128, 256, True),         # heads outside, two or three rows in each
    (32, 32, 128, 32 * 128, False), (33, 32, 128, 32 * 128, True),
    (2, 32, -32 * 128, 128, False), (2, 32, -128, 128, True), (2, 32, 64, 1 << 40, True),
    (1, 32, 0, 128, False), (1, 32, 0, 0, True), (9, 8, 1 << 62, 1 << 62, True), (9, 8, 1 << 62, 128, False),
])
def test_outputs_whose_rows_overlap_are_refused(n, heads, row, head, overlap):
    """What two rows write into one place depends on their order: out and q_out of such strides are refused.  The calls
    that are not refused end at the workspace or at k's address, before any HIP call."""
    s = step(n_rows=n)
    out = rows(row=row, head=head)
    assert attend(s=s, heads=heads, out=out, ws=None) == EINVAL
    assert ("overlap" in last_error()) == overlap
    assert append(s=s, heads=heads, o=out, k=rows(data=A + 1)) == EINVAL
    assert ("overlap" in last_error()) == overlap
