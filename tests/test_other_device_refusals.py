"""An object made on one device and called while another is current, with tensors
of that one: its weights, workspace and context are not there (CPU tensors that
say where they are, and a library that takes everything)."""
import types

import pytest
import torch

from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300.build import build

H, T, E, K = 64, 6, 8, 2


class On0(torch.Tensor):
    def get_device(self):
        return 0


class On1(torch.Tensor):
    def get_device(self):
        return 1


@pytest.fixture
def called(monkeypatch):
    build()
    sizes = {n: getattr(B.lib(), n) for n in ("dwdp_sandwich_grad_workspace_bytes", "dwdp_balance_workspace_bytes")}
    names = []
    calls = types.SimpleNamespace(**{n: (lambda *a, n=n: names.append(n) or 0) for n, _, _ in B.SIGNATURES})
    for n, f in sizes.items():
        setattr(calls, n, f)
    monkeypatch.setattr(B, "_lib", calls)
    monkeypatch.setattr(B, "lib", lambda: calls)
    monkeypatch.setattr(B, "_stream", lambda s: None)
    monkeypatch.setattr(B, "_device", lambda: 0)
    return names


def bf16(where, *s):
    return torch.zeros(s, dtype=torch.bfloat16).as_subclass(where)


def f32(where, *s):
    return torch.zeros(s).as_subclass(where)


def test_sandwich_norm(called, monkeypatch):
    norm = B.SandwichNorm(H, T, bf16(On0, H), bf16(On0, H), device="cpu")

    def forward(on):
        norm.forward(bf16(on, T, H), residual_out=bf16(on, T, H), out=bf16(on, T, H))

    def grad(on):
        norm.grad(bf16(on, T, H), bf16(on, T, H), f32(on, T, 2), bf16(on, T, H), dx=bf16(on, T, H))

    forward(On0), grad(On0)
    assert called == ["dwdp_sandwich_norm", "dwdp_sandwich_norm_grad"]
    monkeypatch.setattr(B, "_device", lambda: 1)
    for call in (forward, grad):
        for on in (On0, On1):
            with pytest.raises(ValueError):
                call(on)
    assert len(called) == 2


def test_the_routers_calls(called, monkeypatch):
    rt = object.__new__(B.Runtime)
    rt.ctx, rt.cfg, rt.ws, rt.ws_bytes = None, dict(n_experts=E, top_k=K), torch.empty(256, dtype=torch.uint8).as_subclass(On0), 256

    def losses(on):
        out = B.BalanceBuffers(1, E, device="cpu")
        out.counts = out.counts.as_subclass(on)
        rt.balance_loss(f32(on, T, E), torch.zeros((T, K), dtype=torch.int32).as_subclass(on), B.scoring(), out)

    def grad(on):
        rt.route_scored_grad(f32(on, T, E), torch.zeros((T, K), dtype=torch.int32).as_subclass(on), B.scoring(), f32(on, T, E))

    losses(On0), grad(On0)
    assert len(called) == 2
    monkeypatch.setattr(B, "_device", lambda: 1)
    for call in (losses, grad):
        for on in (On0, On1):
            with pytest.raises(ValueError):
                call(on)
    assert len(called) == 2
