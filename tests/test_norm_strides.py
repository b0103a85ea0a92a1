"""Weights of each head, of heads whose size is no multiple of 4: such heads go element by element, and so do their
weights."""
import pytest

import paged_kv_movement_amd as kvm
import test_gpu_append_heads as ah
from test_abi_host import _paged
from test_step_forms_host import append, last_error, norm
from test_step_host import rows, step, tables

BF, HF, FL = ah.BF, ah.HF, ah.FL


def test_strides_ask_for_vectors_only_where_heads_are_vectors():
    empty = step(own=tables(n=0), n_rows=0)
    for D, ok in ((6, True), (10, True), (36, True), (2, True), (128, False), (40, False)):
        for wrong in (norm(qs=D + 2 if D % 4 == 0 else D), norm(ks=D + 1)):
            rope = kvm._KvRope(0x10000, 2, 0, 1.0)
            rc = append(16, p=_paged(H=4, D=D), s=empty, k=rows(row=4 * D), n=wrong, rope=rope)
            assert rc == (kvm.KV_OK if ok else kvm.KV_EINVAL), (D, last_error())
    for wrong in (norm(qs=-6), norm(ks=-1), norm(q=0x10004), norm(k=0x10008)):
        assert append(16, p=_paged(H=4, D=6), s=empty, n=wrong) == kvm.KV_EINVAL and "aligned" in last_error()


CASES = [
    # as ah.NORMS: heads, rep, dim, page, lens, new, rot, interleaved, type, q type, start, centered, weights by head, eps
    (4, 3, 6, 16, [20, 9], [3, 9], 4, False, BF, None, 50, False, True, 1e-6),
    (4, 2, 10, 4, [7, 1], [7, 1], 10, True, FL, None, 9, True, True, 1e-5),
    (4, 1, 2, 4, [3], [3], 2, False, HF, BF, 0, False, True, 1e-6),
    (4, 2, 14, 16, [30], [30], 0, False, BF, None, 0, True, True, 1e-6),
    (8, 1, 70, 16, [30], [30], 70, False, FL, BF, 3, False, True, 1e-6),        # more units than lanes, none a vector
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=[str(c[2]) for c in CASES])
def test_weights_of_each_head_of_any_size(case):
    ah.test_append_normed(case, True)


@pytest.mark.gpu
def test_heads_of_one_element():
    ah.test_append_normed((8, 1, 1, 4, [5], [5], 0, False, BF, None, 0, False, True, 1e-6), True)
