"""What follows attention in a decoder block, on one context: the output
projection with its adapters, the residual addition and norm (with a norm
after the projection, a gate and the residual's scale, where a model has
them), the scored router and the expert layer.

Every step is a call of the library (binding.py); this module only keeps the
buffers and the order, so it can be captured into a CUDA graph.  With E4M3
experts the norm's codes go straight to the expert layer
(dwdp_moe_layer_codes), which then quantizes nothing.

The time of the expert layer, and what has to be staged for it, depend on how
evenly the router uses the experts.  DecoderBlockTail.balance_grad gives the
gradients of the router's balance and z losses (and of its weights) by the
router's weight, the norms', the gates, the projection's output and the
residual; the experts, the projection's weight and the adapters stay as they are.  A forward call
that is to be followed by it keeps its rows in 8 bits (Kept).

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


class Kept:
    """What a forward call of a DecoderBlockTail leaves for balance_grad: the
    projection's output and the residual stream as E4M3 rows with one scale
    each, 1 / rms of the norms, the router's input, logits and choices."""

    def __init__(self, T: int, H: int, E: int, k: int, device="cuda"):
        e4m3 = dict(dtype=torch.float8_e4m3fn, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        self.T, self.of = T, (T, H, E, k)
        self.y_codes, self.h_codes = torch.empty((T, H), **e4m3), torch.empty((T, H), **e4m3)
        self.y_scale, self.h_scale, self.rstd = torch.empty(T, **f32), torch.empty(T, **f32), torch.empty((T, 2), **f32)
        self.x = torch.empty((T, H), dtype=torch.bfloat16, device=device)
        self.rb = B.RouteBuffers(T, E, k, device, keep_logits=True)


class DecoderBlockTail:
    """One layer's weights and buffers.  Tensors are contiguous, of the types
    and shapes named here; others are refused (ValueError).

    rt             Runtime whose layer `layer` is mapped (Runtime.set_layer)
    w_o            [H, D] bf16, the attention's output projection
    a, b, scale    adapters of w_o: [n, R, D], [n, H, R] bf16 and [n] fp32
    norm_weight    [H] bf16
    w_router       [E, H] bf16; choice_bias [E] fp32 or None; how: scoring()
    post_weight    [H] bf16 or None: a norm after the projection
    block_scale, residual_scale  of the (normed, gated) projection and of the
                   residual in their sum
    max_gates      most gates of a call
    """

    def __init__(self, rt: B.Runtime, layer: int, w_o, a, b, scale, norm_weight, w_router, choice_bias, how,
                 eps: float = 1e-6, post_weight=None, block_scale: float = 1.0, residual_scale: float = 1.0,
                 max_gates: int = 1):
        H, T = rt.cfg["hidden"], rt.cfg["max_tokens"]
        dev = w_o.device
        D, E, (n, R) = w_o.shape[1], rt.cfg["n_experts"], a.shape[:2]
        for name, t, shape, dtype in (("w_o", w_o, (H, D), torch.bfloat16), ("a", a, (n, R, D), torch.bfloat16),
                                      ("b", b, (n, H, R), torch.bfloat16), ("scale", scale, (n,), torch.float32),
                                      ("norm_weight", norm_weight, (H,), torch.bfloat16),
                                      ("w_router", w_router, (E, H), torch.bfloat16),
                                      ("choice_bias", choice_bias, (E,), torch.float32),
                                      ("post_weight", post_weight, (H,), torch.bfloat16)):
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
        # row_offsets [0, t] of a product's one group, for every t
        most = max(T, E)
        self.rows = torch.zeros((most + 1, 4), dtype=torch.int32, device=dev)
        self.rows[:, 1] = torch.arange(most + 1, dtype=torch.int32, device=dev)
        need = B.dwdp_lora_workspace_bytes(T, a.shape[2], H, a.shape[1])
        self.lora_ws = torch.empty(need, dtype=torch.uint8, device=dev)
        self.plain = post_weight is None and block_scale == 1.0 and residual_scale == 1.0
        self._norm_of = (H, T, norm_weight, post_weight, block_scale, residual_scale, eps, max_gates)
        self._norm = None

    @property
    def norm(self) -> B.SandwichNorm:
        """The norms around the projection, made when first needed."""
        if self._norm is None:
            H, T, pre, post, block_scale, residual_scale, eps, max_gates = self._norm_of
            self._norm = B.SandwichNorm(H, T, pre, post, block_scale, residual_scale, eps, max_groups=max_gates,
                                        device=self.y.device)
        return self._norm

    def keep(self, T: int) -> Kept:
        """Room for what a call of T tokens leaves for balance_grad."""
        return Kept(T, self.y.shape[1], self.rt.cfg["n_experts"], self.rt.cfg["top_k"], self.y.device)

    def _kept_here(self, kept, T) -> None:
        of = (T, self.y.shape[1], self.rt.cfg["n_experts"], self.rt.cfg["top_k"])
        if kept is not None and (kept.of != of or kept.x.device != self.y.device):
            raise ValueError(f"kept is for tokens, width, experts, choices {kept.of} on {kept.x.device}; "
                             f"{of} on {self.y.device} are needed")

    def __call__(self, attn, adapter_ids, residual, stage: int = 0, stream=None, gate=None, row_offsets=None,
                 kept: Kept | None = None):
        """attn [T, D]: the attention's output; adapter_ids [T] int32 (-1:
        none); residual [T, H] bf16, updated in place.  gate [H] or [G, H] bf16,
        with row_offsets [G + 1] int32: dwdp_sandwich_norm's; together they cover
        all rows.  kept: filled for balance_grad.  Returns the expert layer's output
        [T, H], to be added to the residual by the next block's norm."""
        T, H, D = attn.shape[0], self.y.shape[1], self.w_o.shape[2]
        if T > self.y.shape[0]:
            raise ValueError(f"{T} tokens in buffers for {self.y.shape[0]}")
        _dense("attn", attn, (T, D), torch.bfloat16)
        _dense("adapter_ids", adapter_ids, (T,), torch.int32)
        _dense("residual", residual, (T, H), torch.bfloat16)
        self._kept_here(kept, T)
        y, x, out = self.y[:T], self.x[:T], self.out[:T]
        if T == 0:
            return out
        n, R, _ = self.a.shape
        B.dwdp_grouped_gemm(self.rt.ctx, B.EPI_BF16, attn, T, D, H, self.rows[T], 1, [self.w_o], [0, 0], y, stream)
        B.dwdp_lora_add(self.rt.ctx, attn, D, T, D, H, self.a, self.b, self.scale, n, R, adapter_ids, y, H, y, H,
                        self.lora_ws, self.lora_ws.numel(), stream)
        rb = self.rb
        if kept is not None:
            x, rb = kept.x, kept.rb
        if self.plain and gate is None and kept is None:
            B.dwdp_add_rmsnorm(y, T, H, self.norm_weight, self.eps, x, residual=residual, residual_out=residual,
                               codes=self.codes, row_scale=self.row_scale, stream=stream)
        else:
            rows8 = {} if not self.e4m3 else dict(codes=self.codes[:T], row_scale=self.row_scale[:T])
            if kept is not None:
                rows8.update(x_codes=kept.y_codes, x_scale=kept.y_scale, h_codes=kept.h_codes, h_scale=kept.h_scale,
                             rstd=kept.rstd)
            self.norm.forward(y, residual, residual, x, gate, row_offsets, stream=stream, **rows8)
        self.rt.route_scored(x, self.w_router, self.choice_bias, self.how, rb, stream)
        if self.e4m3:
            self.rt.moe_codes(self.layer, stage, self.codes[:T], self.row_scale, rb, out, stream)
        else:
            self.rt.moe(self.layer, stage, x, rb, out, stream)
        return out

    def balance_grad(self, kept: Kept, dbalance=None, dz=None, dtopk_w=None, seq_offsets=None, gate=None,
                     row_offsets=None, dresidual_out=None, stream=None) -> dict:
        """Of the call that filled `kept`, with the same gate and row_offsets: the
        router's losses, and the gradients of
          sum dbalance balance + sum dz z + sum dtopk_w topk_w
        (with dresidual_out [T, H] bf16, what else the residual's gradient is),
        each of dbalance and dz [S] fp32 and dtopk_w [T, k] fp32 or None;
        seq_offsets int32 [S + 1] or None (one sequence).  The choice, the counts
        and the experts are held fixed.  Returns new tensors: counts, mean_p, balance, z
        (BalanceBuffers'), dlogits [T, E] bf16, dw_router [E, H], dnorm_weight and
        dpost_weight [H], dgate fp32, dy (the projection's output) and dresidual
        [T, H] bf16; None for what there is not.  stream: a torch.cuda.Stream or None."""
        with torch.cuda.stream(stream):
            T, H, E, dev = kept.T, self.y.shape[1], self.rt.cfg["n_experts"], self.y.device
            if T == 0:
                raise ValueError("no tokens")
            self._kept_here(kept, T)
            bf16, f32 = dict(dtype=torch.bfloat16, device=dev), dict(dtype=torch.float32, device=dev)
            S = 1 if seq_offsets is None else seq_offsets.numel() - 1
            if S < 1:
                raise ValueError(f"seq_offsets: {seq_offsets.numel()} elements; two at least are needed")
            rb, losses = kept.rb, B.BalanceBuffers(S, E, device=dev)
            ws = torch.empty(B.dwdp_balance_workspace_bytes(T, E, S), dtype=torch.uint8, device=dev)
            self.rt.balance_loss(rb.logits, rb.topk_ids, self.how, losses, seq_offsets=seq_offsets, ws=ws)
            dlogits = torch.empty((T, E), **bf16)
            self.rt.route_scored_grad(rb.logits, rb.topk_ids, self.how, dlogits, dtopk_w=dtopk_w, counts=losses.counts,
                                      dbalance=dbalance, dz=dz, seq_offsets=seq_offsets, choice_bias=self.choice_bias)
            # the GEMM takes rows of multiples of 64 elements
            up = lambda n: -(-n // 64) * 64  # noqa: E731
            left, w_t = torch.zeros((T, up(E)), **bf16), torch.zeros((1, H, up(E)), **bf16)
            left[:, :E], w_t[0, :, :E] = dlogits, self.w_router.t()
            dx = torch.empty((T, H), **bf16)
            B.dwdp_grouped_gemm(self.rt.ctx, B.EPI_BF16, left, T, up(E), H, self.rows[T], 1, [w_t], [0, 0], dx)
            left_t, x_t = torch.zeros((E, up(T)), **bf16), torch.zeros((1, H, up(T)), **bf16)
            left_t[:, :T], x_t[0, :, :T] = dlogits.t(), kept.x.t()
            dw_router = torch.empty((E, H), **f32)
            B.dwdp_grouped_gemm(self.rt.ctx, B.EPI_F32, left_t, E, up(T), H, self.rows[E], 1, [x_t], [0, 0], dw_router)
            dy, dresidual = torch.empty((T, H), **bf16), torch.empty((T, H), **bf16)
            dnorm = torch.empty(H, **f32)
            dpost = torch.empty(H, **f32) if self.norm.post_weight is not None else None
            dgate = torch.empty(gate.shape, **f32) if gate is not None else None
            self.norm.grad(kept.y_codes, kept.h_codes, kept.rstd, dx, dresidual_out, dx=dy, dresidual=dresidual,
                           dpost_weight=dpost, dpre_weight=dnorm, dgate=dgate, gate=gate, row_offsets=row_offsets,
                           x_scale=kept.y_scale, h_scale=kept.h_scale)
        return dict(counts=losses.counts, mean_p=losses.mean_p, balance=losses.balance, z=losses.z, dlogits=dlogits,
                    dw_router=dw_router, dnorm_weight=dnorm, dpost_weight=dpost, dgate=dgate, dy=dy, dresidual=dresidual)


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
    kept = block.keep(tokens)
    block(attn, ids, residual, kept=kept)
    grads = block.balance_grad(kept, dbalance=torch.ones(1, device="cuda"))
    assert rt.device_status() == 0
    print(f"balance loss {float(grads['balance']):.4f}, its gradient by the router's weight {float(grads['dw_router'].norm()):.3e}")
    print(f"{tokens} tokens, H {H}, {shape.E} E4M3 experts top-{shape.k}: {start.elapsed_time(end) / 50:.3f} ms a step, "
          f"output {tuple(out.shape)}, finite: {bool(torch.isfinite(out).all())}")
    rt.close()


if __name__ == "__main__":
    import sys
    main(*(int(v) for v in sys.argv[1:2]))
