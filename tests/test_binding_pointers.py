"""What the binding takes for an address."""
import torch

from moe_expert_grouped_split_gb300 import binding as B


class Address(int):
    pass


def test_addresses():
    t = torch.zeros(4)
    assert B._ptr(None) is None
    assert B._ptr(4096) == 4096 and B._ptr(Address(4096)) == 4096
    assert B._ptr(t) == t.data_ptr()


def test_streams():
    assert B._stream(0) == 0 and B._stream(Address(64)) == 64
    assert B._stream(type("S", (), {"cuda_stream": 7})()) == 7
