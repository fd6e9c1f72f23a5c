"""dwdp_moe_layer_codes: the E4M3 layer on rows that are codes already.  On
the codes dwdp_quantize_rows makes of x it must give dwdp_moe_layer's bits
on x (the same codes, the same GEMMs)."""
import pytest
import torch

from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300 import inputs as I
from moe_expert_grouped_split_gb300.build import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


@pytest.mark.parametrize("T, H, k, S", [(1, 256, 2, 1), (64, 256, 2, 0), (333, 512, 4, 1), (300, 256, 3, 1),
                                        (130, 1024, 8, 1)])
def test_same_bits_as_the_layer_on_bf16_rows(T, H, k, S):
    shape = I.LayerShape(T=T, H=H, I=128, E=8, k=k, S=S)
    placement = I.split_placement(8, 4, 1)
    lw = I.make_layer_fp8(shape, placement, 0, 0, device="cuda")
    x = I.make_tokens(T, H, 3).cuda()
    rt = B.Runtime(H, 128, 8, k, S, T, 1, 4, weight_dtype=B.DTYPE_E4M3)
    try:
        rt.set_layer(0, lw)
        rt.prefetch(0, 0, 64 << 10, [torch.cuda.Stream()])
        rb = B.RouteBuffers(T, 8, k)
        rt.route(x, lw.wr, None, rb)
        want = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        rt.moe(0, 0, x, rb, want)
        codes = torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda")
        scale = torch.empty(T, device="cuda")
        B.dwdp_quantize_rows(B.DTYPE_E4M3, x, T, H, codes, None, scale)
        got = torch.full_like(want, float("nan"))
        rt.moe_codes(0, 0, codes, scale, rb, got)
        torch.cuda.synchronize()
        assert rt.device_status() == 0
        assert torch.equal(got, want)
    finally:
        rt.close()


def test_refusals():
    T, H = 8, 256
    x = torch.zeros((T, H), dtype=torch.uint8, device="cuda")
    sx = torch.ones(T, device="cuda")
    out = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    rb = B.RouteBuffers(T, 8, 2)
    bf16 = B.Runtime(H, 128, 8, 2, 0, T, 1, 0)
    try:
        with pytest.raises(B.DwdpError) as ei:
            bf16.moe_codes(0, 0, x, sx, rb, out)
        assert ei.value.code == -1 and "E4M3" in str(ei.value)
    finally:
        bf16.close()
    rt = B.Runtime(H, 128, 8, 2, 0, T, 1, 0, weight_dtype=B.DTYPE_E4M3)
    try:
        with pytest.raises(B.DwdpError) as ei:
            rt.moe_codes(0, 0, x, sx, rb, out)              # no expert map yet
        assert ei.value.code == -2
        placement = I.split_placement(8, 8, 1)
        lw = I.make_layer_fp8(I.LayerShape(T=T, H=H, I=128, E=8, k=2), placement, 0, 0, device="cuda")
        rt.set_layer(0, lw)
        for a, s in ((x, None), (None, sx), (x, sx.data_ptr() + 4), (x.cpu().pin_memory(), sx)):
            with pytest.raises(B.DwdpError) as ei:
                B.dwdp_moe_layer_codes(rt.ctx, 0, 0, a, s, T, rb.c, out, rt.ws, rt.ws_bytes)
            assert ei.value.code == -1
        B.dwdp_moe_layer_codes(rt.ctx, 0, 0, x, sx, 0, rb.c, out, rt.ws, rt.ws_bytes)   # no tokens: nothing to do
        torch.cuda.synchronize()
        assert rt.device_status() == 0 and (out == 0).all()
    finally:
        rt.close()
