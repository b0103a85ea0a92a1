"""Paged8 without a GPU: which tensors it takes."""
import pytest
import torch

import paged_kv_movement_amd as kvm


class DeviceTensor:
    """A tensor on a device as far as Paged8 looks at one: its memory is never touched."""
    is_cuda, device = True, torch.device("cpu")

    def __init__(self, shape, dtype, address):
        self.shape, self.dtype, self.address = torch.Size(shape), dtype, address

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.address


def made(dim=32, k=0x1000, v=0x20000, ks=0x30000, vs=0x40000):
    layers = [DeviceTensor((5, 16, 2, dim), torch.uint8, x) for x in (k, v)]
    scales = [DeviceTensor((5, 2), torch.float32, x) for x in (ks, vs)]
    return kvm.Paged8([layers[0]], [layers[1]], [scales[0]], [scales[1]])


def test_addresses_are_taken_as_they_are():
    p = made(ks=0x30004)
    assert [x.tolist() for x in p._arrays] == [[0x1000], [0x20000], [0x30004], [0x40000]]


@pytest.mark.parametrize("wrong", [dict(k=0x1001), dict(k=0x1008), dict(v=0x20004), dict(ks=0x30002), dict(vs=0x40001)])
def test_bytes_that_the_kernels_cannot_reach_are_refused(wrong):
    with pytest.raises(kvm.KvError, match="multiples of 16 bytes"):
        made(**wrong)
