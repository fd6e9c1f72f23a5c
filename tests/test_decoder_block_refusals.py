"""What the decoder block's tail refuses before any call of the library
(CPU tensors, no GPU)."""
import types

import pytest
import torch

from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300.build import build
from moe_expert_grouped_split_gb300.decoder_block import DecoderBlockTail

H, D, E, N, R, T = 64, 128, 8, 3, 16, 6


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def weights():
    return dict(w_o=bf16(H, D), a=bf16(N, R, D), b=bf16(N, H, R), scale=torch.ones(N), norm_weight=bf16(H),
                w_router=bf16(E, H), choice_bias=torch.zeros(E), how=B.scoring())


def runtime():
    return types.SimpleNamespace(ctx=None, cfg=dict(hidden=H, max_tokens=T, n_experts=E, top_k=2),
                                 weight_dtype=B.DTYPE_BF16)


@pytest.mark.parametrize("name, value", [
    ("w_o", bf16(D, H).t()), ("w_o", torch.zeros(H, D)), ("a", bf16(N, D, R).transpose(1, 2)), ("a", bf16(N, R, D - 8)),
    ("b", bf16(N, R, H)), ("b", torch.zeros(N, H, R)), ("scale", torch.ones(N, dtype=torch.bfloat16)),
    ("scale", torch.ones(N - 1)), ("norm_weight", torch.zeros(H)), ("norm_weight", bf16(2 * H)[::2]),
    ("w_router", bf16(H, E)), ("choice_bias", torch.zeros(E, dtype=torch.float64)), ("choice_bias", torch.zeros(E - 1))],
    ids=lambda v: v if isinstance(v, str) else "")
def test_weights(name, value):
    with pytest.raises(ValueError, match=name):
        DecoderBlockTail(runtime(), 0, **{**weights(), name: value})


@pytest.mark.parametrize("name, value", [
    ("attn", bf16(T, 2 * D)[:, :D]), ("attn", torch.zeros(T, D)), ("attn", bf16(T, D - 8)), ("tokens", bf16(T + 1, D)),
    ("adapter_ids", torch.zeros(T, dtype=torch.int64)), ("adapter_ids", torch.zeros(2 * T, dtype=torch.int32)[::2]),
    ("adapter_ids", torch.zeros(T - 1, dtype=torch.int32)),
    ("residual", bf16(T, 2 * H)[:, H:]), ("residual", bf16(T - 1, H)), ("residual", torch.zeros(T, H))],
    ids=lambda v: v if isinstance(v, str) else "")
def test_calls(name, value):
    block = DecoderBlockTail(runtime(), 0, **weights())
    args = dict(attn=bf16(T, D), adapter_ids=torch.zeros(T, dtype=torch.int32), residual=bf16(T, H))
    args["attn" if name == "tokens" else name] = value
    with pytest.raises(ValueError, match=name):
        block(**args)


def test_no_tokens():
    block = DecoderBlockTail(runtime(), 0, **weights())
    assert block(bf16(0, D), torch.zeros(0, dtype=torch.int32), bf16(0, H)).shape == (0, H)
