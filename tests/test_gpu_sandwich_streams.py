"""The workspace of the sandwich norm's gradients on streams other than the
current one: never memory that another stream may still be using."""
import pytest
import torch
from test_gpu_sandwich import Grads, Made

from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300.build import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def same_bits(a, b):
    return all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_made_on_the_calls_stream(raw):
    g = Grads(Made(300, 2048, groups=[0, 100, 300]))
    want = g.run()
    m = g.m
    m.norm = B.SandwichNorm(m.H, m.rows, m.pre, m.post, 1.25, 0.9, 1e-6, max_groups=m.G)
    o, s = g.outputs(), torch.cuda.Stream()
    torch.cuda.synchronize()
    # a block of its size that the current stream has just given back
    freed = torch.empty(max(256, m.norm.ws_bytes), dtype=torch.uint8, device="cuda")
    at = freed.data_ptr()
    del freed
    g.call(stream=s.cuda_stream if raw else s, **o)
    torch.cuda.synchronize()
    assert m.norm.ws.data_ptr() != at
    assert same_bits(want, o)


def test_given_back_when_every_stream_is_done():
    g = Grads(Made(300, 2048))
    want = g.run()  # makes the workspace on the current stream
    m, o, s = g.m, g.outputs(), torch.cuda.Stream()
    at, size = m.norm.ws.data_ptr(), m.norm.ws.numel()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)  # about 0.1 s
    g.call(stream=s, **o)
    m.norm = None
    other = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert not s.query()  # still at work
    assert other.data_ptr() != at
    other.fill_(0xFF)
    torch.cuda.synchronize()
    assert same_bits(want, o)


def test_default_stream_by_its_handle():
    g = Grads(Made(40, 512))
    want = g.run()
    m, o = g.m, g.outputs()
    m.norm = B.SandwichNorm(m.H, m.rows, m.pre, m.post, 1.25, 0.9, 1e-6)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        g.call(stream=0, **o)
    torch.cuda.synchronize()
    assert same_bits(want, o)
