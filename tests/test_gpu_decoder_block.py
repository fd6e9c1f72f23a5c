"""The second half of a decoder block (decoder_block.py): its result is that
of the calls one by one, each checked on its own elsewhere; the whole is
near the formulas in 64 bits; it can be captured into a CUDA graph; and the
norm's codes are at least as good a feed for E4M3 experts as quantizing its
bf16 rows."""
import numpy as np
import pytest
import torch

from gpu_helpers import to_f64
from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300 import inputs as I
from moe_expert_grouped_split_gb300.build import build
from moe_expert_grouped_split_gb300.decoder_block import DecoderBlockTail

pytestmark = pytest.mark.gpu

H, D, INTER, E, K, N_AD, R = 512, 384, 128, 16, 4, 3, 16
HOW = dict(score=B.SCORE_SIGMOID, n_groups=4, top_groups=2, group_score=B.GROUP_TOP2, renormalize=True, scale=2.5)


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


class Made:
    def __init__(self, T, fmt):
        shape = I.LayerShape(T=T, H=H, I=INTER, E=E, k=K, S=1)
        make = I.make_layer_fp8 if fmt == B.DTYPE_E4M3 else I.make_layer
        self.lw = make(shape, I.split_placement(E, E, 0), 0, 0, device="cuda")
        self.rt = B.Runtime(H, INTER, E, K, 1, T, 1, 0, weight_dtype=fmt)
        self.rt.set_layer(0, self.lw)
        rand = lambda name, std, *s: I.randn_bf16(s, std, I.seed_for(5, name), "cuda")
        self.wo, self.a, self.b = rand("wo", I.sqrt_inv(D), H, D), rand("a", I.sqrt_inv(D), N_AD, R, D), rand("b", 0.3, N_AD, H, R)
        self.scale = torch.tensor([0.5, 1.0, 2.0], device="cuda")
        self.gamma = rand("gamma", 1.0, H)
        self.wr = rand("wr", I.sqrt_inv(H), E, H)
        self.bias = 0.1 * torch.randn(E, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
        self.block = DecoderBlockTail(self.rt, 0, self.wo, self.a, self.b, self.scale, self.gamma, self.wr, self.bias,
                                      B.scoring(**HOW))
        self.attn, self.residual = rand("attn", 1.0, T, D), rand("res", 1.0, T, H)
        self.ids = (torch.arange(T, device="cuda", dtype=torch.int32) * 7) % (N_AD + 1) - 1

    def run(self, T=None):
        res = self.residual[:T].clone()
        out = self.block(self.attn[:T], self.ids[:T], res).clone()
        torch.cuda.synchronize()
        assert self.rt.device_status() == 0
        return out, res


@pytest.mark.parametrize("fmt", [B.DTYPE_BF16, B.DTYPE_E4M3])
@pytest.mark.parametrize("T", [1, 65, 300, 1100])
def test_the_block_is_its_calls(T, fmt):
    m = Made(T, fmt)
    out, res = m.run()
    # the projection and its adapters, the residual and the norm, in 64 bits:
    # bf16 roundings of y0, v and y, then of the sum (2^-8 each)
    y0 = to_f64(m.attn) @ to_f64(m.wo).T
    v = to_f64(m.attn) @ to_f64(m.a).reshape(N_AD * R, D).T
    ids = m.ids.cpu().numpy()
    mine = np.stack([np.where(ids == i, float(m.scale[i]), 0.0) for i in range(N_AD)], axis=1)
    v = (v.reshape(T, N_AD, R) * mine[:, :, None]).reshape(T, N_AD * R)
    bt = np.concatenate([to_f64(m.b[i]) for i in range(N_AD)], axis=1).T
    y = y0 + v @ bt
    h = y + to_f64(m.residual)
    tol = 2.0 ** -8 * (2 * np.abs(y0) + np.abs(v) @ np.abs(bt) + np.abs(y) + np.abs(h)) + 1e-4
    assert (np.abs(to_f64(res) - h) <= tol).all()
    # and the rest call by call, on what the block's norm gave
    x = m.block.x[:T].clone()
    rb, again = B.RouteBuffers(T, E, K), torch.empty_like(out)
    m.rt.route_scored(x, m.wr, m.bias, B.scoring(**HOW), rb)
    if fmt == B.DTYPE_E4M3:
        m.rt.moe_codes(0, 0, m.block.codes[:T].clone(), m.block.row_scale.clone(), rb, again)
    else:
        m.rt.moe(0, 0, x, rb, again)
    torch.cuda.synchronize()
    assert torch.equal(again, out)
    m.rt.close()


def test_fewer_tokens_than_the_buffers_hold():
    m = Made(300, B.DTYPE_E4M3)
    whole, res = m.run()
    part, res_part = m.run(123)
    assert torch.equal(res_part, res[:123])
    d = (part.float() - whole[:123].float()).abs().max()
    assert float(d) <= 2e-2 * float(whole.float().abs().max())  # other expert tiles, the same rows
    assert m.run(0)[0].shape == (0, H)
    m.rt.close()


@pytest.mark.parametrize("T", [1, 200, 1100])
def test_captured_into_a_graph(T):
    m = Made(T, B.DTYPE_E4M3)
    out, res = m.run()
    buf = m.residual.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.block(m.attn, m.ids, buf, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = m.block(m.attn, m.ids, buf, stream=s)
    for _ in range(3):
        buf.copy_(m.residual)
        m.block.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and torch.equal(buf, res)
    # other inputs in the same buffers
    m.attn.mul_(0.5)
    m.ids.fill_(2)
    buf.copy_(m.residual)
    g.replay()
    torch.cuda.synchronize()
    replayed, res2 = got.clone(), buf.clone()
    out2, res3 = m.run()
    assert torch.equal(replayed, out2) and torch.equal(res2, res3)
    assert m.rt.device_status() == 0
    m.rt.close()


def test_codes_of_the_norm_against_codes_of_its_bf16_rows():
    """Both quantize the norm's rows with one scale per row; the norm's own
    codes are rounded once, from rows bf16 has not rounded."""
    T = 257
    x = I.randn_bf16((T, H), 1.0, 3, "cuda")
    r = I.randn_bf16((T, H), 3.0, 4, "cuda")
    w = I.randn_bf16((H,), 1.0, 5, "cuda")
    out, res = torch.empty_like(x), torch.empty_like(x)
    codes = torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(T, device="cuda")
    B.dwdp_add_rmsnorm(x, T, H, w, 1e-6, out, residual=r, residual_out=res, codes=codes, row_scale=s)
    codes2, s2 = torch.empty_like(codes), torch.empty_like(s)
    B.dwdp_quantize_rows(B.DTYPE_E4M3, out, T, H, codes2, None, s2)
    torch.cuda.synchronize()
    h = to_f64(x) + to_f64(r)
    y = h / np.sqrt((h * h).mean(axis=1) + 1e-6)[:, None] * to_f64(w)
    err = lambda c, sc: np.sqrt((((to_f64(c) * to_f64(sc)[:, None]) - y) ** 2).sum(axis=1) / (y * y).sum(axis=1))
    assert err(codes, s).mean() <= err(codes2, s2).mean()
    assert err(codes, s).max() <= 2.0 ** -4
