"""What follows attention in a decoder block, on one context: the output
projection with its adapters, the residual addition and norm, the scored
router and the expert layer.

Every step is a call of the library (binding.py); this module only keeps the
buffers and the order, so it can be captured into a CUDA graph.  With E4M3
experts the norm's codes go straight to the expert layer
(dwdp_moe_layer_codes), which then quantizes nothing.

    python -m moe_expert_grouped_split_gb300.decoder_block [tokens]

runs a small E4M3 block and prints its time per step.
"""
from __future__ import annotations

import torch

from . import binding as B


def _dense(name, t, shape, dtype) -> None:
    """The library gets addresses only: what it would misread is refused here."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: {dtype} {list(shape)}, contiguous, is needed; "
                         f"got {t.dtype} {list(t.shape)} with strides {list(t.stride())}")


class DecoderBlockTail:
    """One layer's weights and buffers.  Tensors are contiguous, of the types
    and shapes named here; others are refused (ValueError).

    rt             Runtime whose layer `layer` is mapped (Runtime.set_layer)
    w_o            [H, D] bf16, the attention's output projection
    a, b, scale    adapters of w_o: [n, R, D], [n, H, R] bf16 and [n] fp32
    norm_weight    [H] bf16
    w_router       [E, H] bf16; choice_bias [E] fp32 or None; how: scoring()
    """

    def __init__(self, rt: B.Runtime, layer: int, w_o, a, b, scale, norm_weight, w_router, choice_bias, how,
                 eps: float = 1e-6):
        H, T = rt.cfg["hidden"], rt.cfg["max_tokens"]
        dev = w_o.device
        D, E, (n, R) = w_o.shape[1], rt.cfg["n_experts"], a.shape[:2]
        for name, t, shape, dtype in (("w_o", w_o, (H, D), torch.bfloat16), ("a", a, (n, R, D), torch.bfloat16),
                                      ("b", b, (n, H, R), torch.bfloat16), ("scale", scale, (n,), torch.float32),
                                      ("norm_weight", norm_weight, (H,), torch.bfloat16),
                                      ("w_router", w_router, (E, H), torch.bfloat16),
                                      ("choice_bias", choice_bias, (E,), torch.float32)):
            if t is not None:
                _dense(name, t, shape, dtype)
        self.rt, self.layer, self.eps = rt, layer, eps
        self.w_o = w_o.view(1, *w_o.shape)  # a buffer of one slot
        self.a, self.b, self.scale = a, b, scale
        self.norm_weight, self.w_router, self.choice_bias, self.how = norm_weight, w_router, choice_bias, how
        bf16 = dict(dtype=torch.bfloat16, device=dev)
        self.y, self.x, self.out = (torch.empty((T, H), **bf16) for _ in range(3))
        self.e4m3 = rt.weight_dtype == B.DTYPE_E4M3
        self.codes = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=dev) if self.e4m3 else None
        self.row_scale = torch.empty(T, dtype=torch.float32, device=dev) if self.e4m3 else None
        self.rb = B.RouteBuffers(T, rt.cfg["n_experts"], rt.cfg["top_k"], dev)
        # row_offsets [0, t] of the projection's one group, for every t
        self.rows = torch.zeros((T + 1, 4), dtype=torch.int32, device=dev)
        self.rows[:, 1] = torch.arange(T + 1, dtype=torch.int32, device=dev)
        need = B.dwdp_lora_workspace_bytes(T, a.shape[2], H, a.shape[1])
        self.lora_ws = torch.empty(need, dtype=torch.uint8, device=dev)

    def __call__(self, attn, adapter_ids, residual, stage: int = 0, stream=None):
        """attn [T, D]: the attention's output; adapter_ids [T] int32 (-1:
        none); residual [T, H] bf16, updated in place.  Returns the expert
        layer's output [T, H], to be added to the residual by the next
        block's norm."""
        T, H, D = attn.shape[0], self.y.shape[1], self.w_o.shape[2]
        if T > self.y.shape[0]:
            raise ValueError(f"{T} tokens in buffers for {self.y.shape[0]}")
        _dense("attn", attn, (T, D), torch.bfloat16)
        _dense("adapter_ids", adapter_ids, (T,), torch.int32)
        _dense("residual", residual, (T, H), torch.bfloat16)
        y, x, out = self.y[:T], self.x[:T], self.out[:T]
        if T == 0:
            return out
        n, R, _ = self.a.shape
        B.dwdp_grouped_gemm(self.rt.ctx, B.EPI_BF16, attn, T, D, H, self.rows[T], 1, [self.w_o], [0, 0], y, stream)
        B.dwdp_lora_add(self.rt.ctx, attn, D, T, D, H, self.a, self.b, self.scale, n, R, adapter_ids, y, H, y, H,
                        self.lora_ws, self.lora_ws.numel(), stream)
        B.dwdp_add_rmsnorm(y, T, H, self.norm_weight, self.eps, x, residual=residual, residual_out=residual,
                           codes=self.codes, row_scale=self.row_scale, stream=stream)
        self.rt.route_scored(x, self.w_router, self.choice_bias, self.how, self.rb, stream)
        if self.e4m3:
            self.rt.moe_codes(self.layer, stage, self.codes[:T], self.row_scale, self.rb, out, stream)
        else:
            self.rt.moe(self.layer, stage, x, self.rb, out, stream)
        return out


def main(tokens: int = 256) -> None:
    from . import inputs as I

    H, D, n, R = 2048, 2048, 8, 16
    shape = I.LayerShape(T=tokens, H=H, I=512, E=32, k=4, S=1)
    lw = I.make_layer_fp8(shape, I.split_placement(32, 32, 0), 0, 0, device="cuda")
    rt = B.Runtime(H, shape.I, shape.E, shape.k, shape.S, tokens, 1, 0, weight_dtype=B.DTYPE_E4M3)
    rt.set_layer(0, lw)
    rand = lambda name, std, *s: I.randn_bf16(s, std, I.seed_for(0, name), "cuda")
    block = DecoderBlockTail(rt, 0, rand("wo", I.sqrt_inv(D), H, D), rand("a", I.sqrt_inv(D), n, R, D),
                             rand("b", 0.1, n, H, R), torch.ones(n, device="cuda"),
                             torch.ones(H, dtype=torch.bfloat16, device="cuda"),
                             rand("wr", I.sqrt_inv(H), shape.E, H), torch.zeros(shape.E, device="cuda"),
                             B.scoring(B.SCORE_SIGMOID, 4, 2, B.GROUP_TOP2, True, 2.5))
    attn, residual = rand("attn", 1.0, tokens, D), rand("residual", 1.0, tokens, H)
    ids = torch.arange(tokens, device="cuda", dtype=torch.int32) * n // tokens
    for _ in range(10):
        out = block(attn, ids, residual)
    start, end = torch.cuda.Event(True), torch.cuda.Event(True)
    torch.cuda.synchronize()
    start.record()
    for _ in range(50):
        out = block(attn, ids, residual)
    end.record()
    torch.cuda.synchronize()
    assert rt.device_status() == 0
    print(f"{tokens} tokens, H {H}, {shape.E} E4M3 experts top-{shape.k}: {start.elapsed_time(end) / 50:.3f} ms a step, "
          f"output {tuple(out.shape)}, finite: {bool(torch.isfinite(out).all())}")
    rt.close()


if __name__ == "__main__":
    import sys
    main(*(int(v) for v in sys.argv[1:2]))
