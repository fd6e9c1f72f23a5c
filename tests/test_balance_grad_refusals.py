"""What DecoderBlockTail.balance_grad refuses before anything is enqueued (CPU
tensors stand for the device's, the library for a context that is not there)."""
import types

import pytest
import torch

from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300.build import build
from moe_expert_grouped_split_gb300.decoder_block import DecoderBlockTail, Kept

H, D, E, N, R, T = 64, 128, 8, 3, 16, 6


@pytest.fixture
def block(monkeypatch):
    build()
    monkeypatch.setattr(B, "_device", lambda: -1)  # where CPU tensors say they are
    monkeypatch.setattr(B, "_stream", lambda s: None)
    rt = object.__new__(B.Runtime)
    rt.ctx, rt.weight_dtype, rt.cfg = None, B.DTYPE_BF16, dict(hidden=H, max_tokens=T, n_experts=E, top_k=2)
    rt.ws, rt.ws_bytes = torch.empty(256, dtype=torch.uint8), 256
    bf16 = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    return DecoderBlockTail(rt, 0, bf16(H, D), bf16(N, R, D), bf16(N, H, R), torch.ones(N), bf16(H), bf16(E, H),
                            torch.zeros(E), B.scoring())


def offsets(*v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype)


@pytest.mark.parametrize("good", [None, offsets(0, T), offsets(0, 2, T)], ids=str)
def test_the_call_it_takes_reaches_the_library(block, good):
    with pytest.raises(B.DwdpError, match="ctx is NULL"):
        block.balance_grad(Kept(T, H, E, 2, "cpu"), seq_offsets=good)


@pytest.mark.parametrize("bad", [offsets(0, 2, T, dtype=torch.int64), offsets(0, 9, 2, 9, T, 9)[::2], offsets(0), offsets(),
                                 offsets(0, 2, T).view(1, 3), offsets(0, 2, T, dtype=torch.float32),
                                 torch.tensor(T, dtype=torch.int32)], ids=str)
def test_sequences_it_would_misread(block, bad, monkeypatch):
    def none(*a):
        raise AssertionError("the library was called")
    calls = types.SimpleNamespace(**{n: none for n, _, _ in B.SIGNATURES})
    calls.dwdp_balance_workspace_bytes = B.lib().dwdp_balance_workspace_bytes
    monkeypatch.setattr(B, "lib", lambda: calls)
    with pytest.raises(ValueError):
        block.balance_grad(Kept(T, H, E, 2, "cpu"), seq_offsets=bad)


def test_sequences_on_another_device(block, monkeypatch):
    class There(torch.Tensor):
        """On device 0, for those who ask."""
        def get_device(self):
            return 0
    here = Kept(T, H, E, 2, "cpu")
    with pytest.raises(ValueError, match="seq_offsets"):
        block.balance_grad(here, seq_offsets=offsets(0, T).as_subclass(There))


@pytest.mark.parametrize("bad", [Kept(T, H, E - 4, 2, "cpu"), Kept(T, H, E, 1, "cpu"), Kept(T, H, 2 * E, 2, "cpu")],
                         ids=["fewer experts", "fewer choices", "more experts"])
def test_rows_kept_for_another_router(block, bad):
    with pytest.raises(ValueError):
        block.balance_grad(bad, seq_offsets=None)


@pytest.mark.parametrize("bad", [torch.zeros(1 << 16), torch.zeros(1 << 16, dtype=torch.uint8)[::2]], ids=["type", "stride"])
def test_workspace(block, bad):
    logits, ids = torch.zeros(T, E), torch.zeros((T, 2), dtype=torch.int32)
    call = lambda ws: block.rt.balance_loss(logits, ids, B.scoring(), B.BalanceBuffers(1, E, device="cpu"), ws=ws)  # noqa: E731
    with pytest.raises(B.DwdpError, match="ctx is NULL"):
        call(torch.zeros(1 << 16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="ws"):
        call(bad)


@pytest.mark.parametrize("of", [(T - 1, H, E, 2), (T + 1, H, E, 2), (T, H // 2, E, 2), (T, H, E // 2, 2), (T, H, 2 * E, 2),
                                (T, H, E, 1), (T, H, E, 3)], ids=str)
def test_a_call_that_would_leave_its_rows_in_another_blocks(block, of, monkeypatch):
    """Refused before the first call of the library, which here takes everything."""
    called = []
    calls = types.SimpleNamespace(**{n: (lambda *a, n=n: called.append(n) or 0) for n, _, _ in B.SIGNATURES})
    block.norm  # asks for its workspace's size
    monkeypatch.setattr(B, "_lib", calls)
    monkeypatch.setattr(B, "lib", lambda: calls)
    args = (torch.zeros((T, D), dtype=torch.bfloat16), torch.zeros(T, dtype=torch.int32), torch.zeros((T, H), dtype=torch.bfloat16))
    block(*args, kept=block.keep(T))
    assert "dwdp_sandwich_norm" in called and "dwdp_route_scored" in called
    called.clear()
    with pytest.raises(ValueError, match="kept"):
        block(*args, kept=Kept(*of, "cpu"))
    assert not called
