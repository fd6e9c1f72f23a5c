"""Runtime.lora_add looks at types, shapes and strides before the library gets
addresses (CPU tensors and a recording stand-in for the library)."""
import types

import pytest
import torch

from moe_expert_grouped_split_gb300 import binding as B

T, K, N, R, n = 5, 64, 128, 16, 3


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def good(T=T):
    return dict(x=bf16(T, K), a=bf16(n, R, K), b=bf16(n, N, R), adapter_scale=torch.ones(n),
                adapter_ids=torch.zeros(T, dtype=torch.int32), base=bf16(T, N), out=bf16(T, N))


@pytest.fixture
def call(monkeypatch):
    seen = []
    monkeypatch.setattr(B, "lib", lambda: types.SimpleNamespace(dwdp_lora_add=lambda *a: seen.append(a) or 0))
    rt = object.__new__(B.Runtime)
    rt.ctx, rt.ws, rt.ws_bytes = 0, torch.zeros(256, dtype=torch.uint8), 256

    def f(**args):
        B.Runtime.lora_add(rt, **args, stream=0)
        return seen[-1]
    f.seen = seen
    return f


@pytest.mark.parametrize("name, value", [
    ("x", torch.zeros(T, K)), ("x", bf16(T, K - 8)), ("x", bf16(K, T).t()), ("x", bf16(T, K).half()),
    ("a", bf16(n, R, K).float()), ("a", bf16(n, K, R).transpose(1, 2)), ("a", bf16(n, R + 8, K)), ("a", bf16(n + 1, R, K)),
    ("b", bf16(n, R, N)), ("b", bf16(n, N, 2 * R)[:, :, :R]),
    ("adapter_scale", torch.ones(n, dtype=torch.float64)), ("adapter_scale", torch.ones(n - 1)),
    ("adapter_scale", torch.ones(2 * n)[::2]),
    ("adapter_ids", torch.zeros(T, dtype=torch.int64)), ("adapter_ids", torch.zeros(T - 1, dtype=torch.int32)),
    ("adapter_ids", torch.zeros(2 * T, dtype=torch.int32)[::2]),
    ("base", bf16(T, N - 8)), ("base", torch.zeros(T, N)), ("base", bf16(N, T).t()),
    ("out", bf16(T - 1, N)), ("out", torch.zeros(T, N)), ("out", bf16(T, 2 * N)[:, ::2])],
    ids=lambda v: v if isinstance(v, str) else "")
def test_refused(call, name, value):
    with pytest.raises(ValueError, match="lora_add"):
        call(**{**good(), name: value})
    assert not call.seen


def test_row_strides_reach_the_library(call):
    x, base, out = bf16(T, K + 8), bf16(T, N + 16), bf16(T, N + 24)
    seen = call(**{**good(), "x": x[:, :K], "base": base[:, :N], "out": out[:, :N]})
    assert seen[2:6] == (K + 8, T, K, N) and seen[13] == N + 16 and seen[15] == N + 24


def test_one_row_has_any_stride(call):
    """A column seen as a row: its row stride, 1, means nothing."""
    x = bf16(K, 1).t()
    assert x.stride(0) == 1 and x.stride(1) == 1
    seen = call(**{**good(1), "x": x})
    assert seen[2] == K and seen[13] == N and seen[15] == N
