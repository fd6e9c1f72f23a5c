"""Calls from a host thread that has not used CUDA yet give what they give
from any other: tensor maps need a context, which such a thread has not got."""
import threading

import pytest
import torch

from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300 import inputs as I
from moe_expert_grouped_split_gb300.build import build

pytestmark = pytest.mark.gpu

T, H, E, K = 2100, 256, 64, 4


@pytest.fixture(scope="module")
def rt():
    build()
    r = B.Runtime(H, 128, E, K, 0, T, 1, 0, min_ws_bytes=B.dwdp_lora_workspace_bytes(T, H, H, 16))
    r.set_layer(0, I.make_layer(I.LayerShape(T=T, H=H, I=128, E=E, k=K), I.split_placement(E, E, 0), 0, 0, device="cuda"))
    yield r
    r.close()


def routing(rb):
    return [rb.topk_ids, rb.topk_w, rb.counts, rb.offsets, rb.perm, rb.inv_perm]


def calls(rt):
    x, wr = I.make_tokens(T, H, 1, device="cuda"), I.randn_bf16((E, H), 0.1, 2, "cuda")
    a, b = I.randn_bf16((2, 16, H), 0.1, 3, "cuda"), I.randn_bf16((2, H, 16), 0.1, 4, "cuda")
    ids, scale = (torch.arange(T, device="cuda") // 700 - 1).int(), torch.ones(2, device="cuda")
    base = I.randn_bf16((T, H), 1.0, 5, "cuda")
    rows = torch.tensor([0, T, 0, 0], dtype=torch.int32, device="cuda")
    rb0 = B.RouteBuffers(T, E, K)
    rt.route(x, wr, None, rb0)
    torch.cuda.synchronize()

    def fresh(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")

    def route(s, rb):
        rt.route(x, wr, None, rb, s)

    def route_scored(s, rb):
        rt.route_scored(x, wr, None, B.scoring(B.SCORE_SIGMOID), rb, s)

    def lora_add(s, out):
        rt.lora_add(x, a, b, scale, ids, base, out, s)

    def grouped_gemm(s, out):
        B.dwdp_grouped_gemm(rt.ctx, B.EPI_BF16, x, T, H, H, rows, 1, [fresh_w], [0, 0], out, s)

    def moe(s, out):
        rt.moe(0, 0, x, rb0, out, s)

    fresh_w = I.randn_bf16((1, H, H), 0.1, 6, "cuda")
    made = {"route": (route, lambda: B.RouteBuffers(T, E, K)), "route_scored": (route_scored, lambda: B.RouteBuffers(T, E, K))}
    made.update({f.__name__: (f, lambda: fresh(T, H)) for f in (lora_add, grouped_gemm, moe)})
    return made


@pytest.mark.parametrize("name", ["route", "route_scored", "lora_add", "grouped_gemm", "moe"])
def test_same_as_from_the_main_thread(rt, name):
    call, out = calls(rt)[name]
    stream, failed = torch.cuda.Stream(), []
    here, there = out(), out()
    torch.cuda.synchronize()
    call(stream, here)
    torch.cuda.synchronize()

    def work():
        try:
            call(stream, there)
        except B.DwdpError as e:
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed[0]
    assert rt.device_status() == 0
    pairs = zip(routing(here), routing(there)) if isinstance(here, B.RouteBuffers) else [(here, there)]
    assert all(torch.equal(u, v) for u, v in pairs)
