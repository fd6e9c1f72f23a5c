"""Weights and tokens are written when their maker returns: other streams
copy from the pools and read the tokens without waiting for this one."""
import pytest
import torch

from moe_expert_grouped_split_gb300 import inputs as I

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("make", [I.make_layer, I.make_layer_fp8, I.make_layer_nvfp4])
def test_layers_are_written(make):
    shape = I.LayerShape(T=8, H=2048, I=1024, E=16, k=2, S=1)
    for _ in range(2):                      # the second from cached blocks: no allocation waits
        lw = make(shape, I.split_placement(16, 4, 3), 0, 0, device="cuda")
        assert torch.cuda.current_stream().query()
        del lw


def test_tokens_are_written():
    for step in range(4):
        x = I.make_tokens(16384, 7168, 0, step=step, device="cuda")
        assert torch.cuda.current_stream().query()
        del x
