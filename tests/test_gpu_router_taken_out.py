"""The router's gradient where a bias of -inf takes experts out and some of them
fill a choice up: their weight is 0 (dwdp_route_scored), so they are in no sum
and get no gradient from it.  Against torch's derivative of the weights that the
routing gave, tolerances as in test_gpu_balance."""
import ctypes

import pytest
import torch
from test_gpu_balance import HOWS, Made, near
from test_gpu_block_training import K
from test_gpu_block_training import Made as Block

from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300.build import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def weights(z, ids, out, sigmoid, renorm, scale):
    """topk_w in z's type; out [E]: experts taken out."""
    s = torch.sigmoid(z) if sigmoid else torch.softmax(z, 1)
    w = torch.where(out[ids], 0.0, s.gather(1, ids))
    total = w.sum(1, keepdim=True)
    return scale * (torch.where(total > 0, w / torch.where(total > 0, total, 1.0), 0.0) if renorm else w)


@pytest.mark.parametrize("how", HOWS, ids=str)
@pytest.mark.parametrize("E, k, left", [(16, 4, 2), (9, 9, 4), (64, 6, 1), (64, 6, 0), (256, 8, 7), (256, 8, 200), (300, 32, 5)])
def test_experts_that_fill_a_choice_up(E, k, left, how):
    T, H = 70, 64
    m = Made(T, E, k, [0, 30, 70], how, seed=E + left)
    g = torch.Generator("cuda").manual_seed(left)
    x, wr = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((T, H), (E, H)))
    wr *= 0.25
    bias = torch.full((E,), -float("inf"), device="cuda")
    bias[torch.randperm(E, generator=g, device="cuda")[:left]] = 0.1
    rb = B.RouteBuffers(T, E, k, keep_logits=True)
    m.rt.route_scored(x, wr, bias, m.how, rb)
    torch.cuda.synchronize()
    m.z, m.ids, out = rb.logits[:T].clone(), rb.topk_ids[:T].clone(), torch.isinf(bias)
    assert int((~out[m.ids.long()]).sum(1).max()) == min(left, k)
    z = m.z.double().requires_grad_(True)
    w = weights(z, m.ids.long(), out, m.sigmoid, m.renorm, m.scale)
    near(rb.topk_w[:T], w.detach(), 2.0 ** -14 * w.detach())  # the formula is the routing's
    counts = m.losses().counts
    for half in (False, True):
        dl = torch.full((T, E), float("nan"), dtype=torch.bfloat16 if half else torch.float32, device="cuda")
        m.rt.route_scored_grad(m.z, m.ids, m.how, dl, dtopk_w=m.dw, seq_offsets=m.offsets, choice_bias=bias)
        torch.cuda.synchronize()
        want = torch.autograd.grad((w * m.dw.double()).sum(), z, retain_graph=True)[0]
        # shares q of the sum are at most 1: |q (dw - sum q dw)| <= 2 max|dw|; not renormalised, p for q
        p = torch.sigmoid(m.z.double()) if m.sigmoid else torch.softmax(m.z.double(), 1)
        mag = 2 * m.scale * m.dw.double().abs().amax(1, keepdim=True) * (torch.ones_like(p) if m.renorm else p)
        tol = (2 * m.rel(m.z.double()) + (E / 16 + 32) * 2.0 ** -23) * mag + 1e-37
        near(dl, want, tol + (2.0 ** -8 * want.abs() if half else 0.0))
        assert left > 0 or (dl == 0).all()
    # beside the losses, which see all choices
    dl = torch.empty((T, E), device="cuda")
    with_losses = dict(counts=counts, dbalance=m.db, dz=m.dz, seq_offsets=m.offsets)
    m.rt.route_scored_grad(m.z, m.ids, m.how, dl, dtopk_w=m.dw, choice_bias=bias, **with_losses)
    losses, tol2 = m.formula(counts, w=False)
    near(dl, losses + want, tol + tol2)
    # a bias that takes nobody out changes nothing
    a, b = torch.empty_like(dl), torch.empty_like(dl)
    m.rt.route_scored_grad(m.z, m.ids, m.how, a, dtopk_w=m.dw, choice_bias=torch.zeros(E, device="cuda"), **with_losses)
    m.rt.route_scored_grad(m.z, m.ids, m.how, b, dtopk_w=m.dw, **with_losses)
    assert torch.equal(a, b)
    m.close()


def test_the_block_hands_its_bias_on():
    m = Block(130, E=16, post=True)
    m.bias[3:] = -float("inf")  # the block's own tensor: three experts for four choices
    kept = m.block.keep(130)
    m.run(kept)
    assert int((kept.rb.topk_w[:130] == 0).sum()) == 130
    dw = torch.randn((130, K), generator=torch.Generator("cuda").manual_seed(2), device="cuda")
    got = m.block.balance_grad(kept, dtopk_w=dw)
    z = kept.rb.logits[:130].double().requires_grad_(True)
    w = weights(z, kept.rb.topk_ids[:130].long(), torch.isinf(m.bias), True, True, m.how.scale)
    want = torch.autograd.grad((w * dw.double()).sum(), z)[0]
    # a rounding to bf16, and binary32 relative to the terms (shares of at most 1)
    near(got["dlogits"], want, 2.0 ** -8 * want.abs() + 2.0 ** -14 * m.how.scale * dw.double().abs().amax(1, keepdim=True))
    m.close()


def test_refuses_a_bias_it_would_misread():
    m = Made(16, 64, 4)
    dl, bias = torch.empty((16, 64), device="cuda"), torch.zeros(64, device="cuda")
    c = lambda b: m.rt.route_scored_grad(m.z, m.ids, m.how, dl, dtopk_w=m.dw, choice_bias=b)  # noqa: E731
    c(bias)
    for bad in (bias.bfloat16(), bias[:32], bias.cpu(), torch.zeros(128, device="cuda")[::2]):
        with pytest.raises(ValueError):
            c(bad)
    P = 4096
    assert B.lib().dwdp_route_scored_biased_grad(m.rt.ctx, P, P, P, P + 4, 4, None, 1, ctypes.byref(m.how), None, None,
                                                 None, P, 0, None) == -1
    m.close()
