"""The decoder block's second half with norms on both sides, gates and scales,
and the gradients of its router's losses: the block is its calls one by one,
each checked on its own elsewhere; the gradients are near the derivative of
the whole in 64 bits; and a run of them together, captured into a graph.

The whole's error: the kept rows are E4M3 (2^-4 of a value at most, either
way, so a product of many is off by about 2^-4 / sqrt(3) in the 2-norm), their
gradients' two terms are that much off each, and bf16 roundings are 2^-8; so
2^-3 in the 2-norm for what goes through kept rows, 2^-5 for what sees bf16 only
(four roundings of 2^-8 and a GEMM's operands)."""
import pytest
import torch

from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300 import inputs as I
from moe_expert_grouped_split_gb300.build import build
from moe_expert_grouped_split_gb300.decoder_block import DecoderBlockTail

pytestmark = pytest.mark.gpu

H, D, INTER, K, N_AD, R = 512, 384, 128, 4, 3, 16
EPS = 1e-6
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


class Made:
    def __init__(self, T, fmt=B.DTYPE_E4M3, E=16, post=True, gates=0, scales=(0.75, 1.25), how=None, most=None):
        shape = I.LayerShape(T=most or T, H=H, I=INTER, E=E, k=K, S=1)
        make = I.make_layer_fp8 if fmt == B.DTYPE_E4M3 else I.make_layer
        self.lw = make(shape, I.split_placement(E, E, 0), 0, 0, device="cuda")
        self.rt = B.Runtime(H, INTER, E, K, 1, most or T, 1, 0, weight_dtype=fmt)
        self.rt.set_layer(0, self.lw)
        rand = lambda name, std, *s: I.randn_bf16(s, std, I.seed_for(77, name), "cuda")  # noqa: E731
        self.wo, self.a, self.b = rand("wo", I.sqrt_inv(D), H, D), rand("a", I.sqrt_inv(D), N_AD, R, D), rand("b", 0.3, N_AD, H, R)
        self.scale = torch.tensor([0.5, 1.0, 2.0], device="cuda")
        self.pre, self.post = 1 + rand("pre", 0.2, H), 1 + rand("post", 0.2, H) if post else None
        self.wr = rand("wr", 2 * I.sqrt_inv(H), E, H)
        self.bias = 0.1 * torch.randn(E, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
        self.how = how or B.scoring(B.SCORE_SIGMOID, 4, 2, B.GROUP_TOP2, True, 2.5)
        self.c, self.a_res = scales
        self.block = DecoderBlockTail(self.rt, 0, self.wo, self.a, self.b, self.scale, self.pre, self.wr, self.bias, self.how,
                                      eps=EPS, post_weight=self.post, block_scale=self.c, residual_scale=self.a_res,
                                      max_gates=max(1, gates))
        self.T, self.E = T, E
        self.attn, self.residual = rand("attn", 1.0, T, D), rand("res", 1.0, T, H)
        self.ids = (torch.arange(T, device="cuda", dtype=torch.int32) * 7) % (N_AD + 1) - 1
        self.gate = 1 + rand("gate", 0.3, gates, H) if gates else None
        ends = [0] + [T * (i + 1) // gates for i in range(gates)] if gates else None
        self.row_offsets = torch.tensor(ends, dtype=torch.int32, device="cuda") if gates > 1 else None
        self.of = torch.zeros(T, dtype=torch.int64, device="cuda")
        if gates > 1:
            self.of = torch.searchsorted(self.row_offsets[1:].contiguous(), torch.arange(T, device="cuda"), right=True)

    def run(self, kept=None, stream=None):
        res = self.residual.clone()
        out = self.block(self.attn, self.ids, res, stream=stream, gate=self.gate, row_offsets=self.row_offsets, kept=kept)
        torch.cuda.synchronize()
        assert self.rt.device_status() == 0
        return out.clone(), res

    def close(self):
        self.rt.close()


@pytest.mark.parametrize("fmt", [B.DTYPE_BF16, B.DTYPE_E4M3])
@pytest.mark.parametrize("T, gates", [(1, 1), (65, 0), (300, 3)])
def test_the_block_is_its_calls(T, gates, fmt):
    m = Made(T, fmt, gates=gates)
    out, res = m.run()
    y = m.block.y[:T].clone()
    n = B.SandwichNorm(H, T, m.pre, m.post, m.c, m.a_res, EPS, max_groups=max(1, gates))
    x, res2, rb, again = torch.empty_like(y), torch.empty_like(y), B.RouteBuffers(T, m.E, K), torch.empty_like(out)
    o = {}
    if fmt == B.DTYPE_E4M3:
        o = dict(codes=torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda"), row_scale=torch.empty(T, device="cuda"))
    n.forward(y, m.residual, res2, x, m.gate, m.row_offsets, **o)
    m.rt.route_scored(x, m.wr, m.bias, m.how, rb)
    if fmt == B.DTYPE_E4M3:
        m.rt.moe_codes(0, 0, o["codes"], o["row_scale"], rb, again)
    else:
        m.rt.moe(0, 0, x, rb, again)
    torch.cuda.synchronize()
    assert torch.equal(res2, res) and torch.equal(x, m.block.x[:T]) and torch.equal(again, out)
    kept = m.block.keep(T)
    out2, res3 = m.run(kept)
    assert torch.equal(out2, out) and torch.equal(res3, res) and torch.equal(kept.x, x)
    assert torch.equal(kept.rb.topk_ids, rb.topk_ids)
    m.close()


def test_without_extras_it_is_the_block_it_was():
    """The plain block still takes dwdp_add_rmsnorm; with rows kept, the same to a rounding."""
    m = Made(130, post=False, scales=(1.0, 1.0))
    assert m.block.plain
    out, res = m.run()
    assert m.block._norm is None
    x = m.block.x[:130].clone()
    kept = m.block.keep(130)
    _, res2 = m.run(kept)
    assert torch.equal(res2, res)
    assert float((kept.x.float() - x.float()).abs().max()) <= 2.0 ** -7 * float(x.float().abs().max())
    m.close()


def whole(m, kept, counts, db, dz, dw, dres, seqs):
    """The sum of losses in 64 bits from the projection's output on, and its derivative."""
    leaf = {n: t.double().requires_grad_(True) for n, t in dict(
        y=m.block.y[:m.T], residual=m.residual, pre=m.pre, wr=m.wr,
        **({"post": m.post} if m.post is not None else {}), **({"gate": m.gate} if m.gate is not None else {})).items()}
    n = leaf["y"]
    if m.post is not None:
        n = n / torch.sqrt(n.square().mean(1, keepdim=True) + EPS) * leaf["post"]
    if m.gate is not None:
        n = n * leaf["gate"][m.of]
    h = m.a_res * leaf["residual"] + m.c * n
    x = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * leaf["pre"]
    z = x @ leaf["wr"].t()
    sigmoid = m.how.score == B.SCORE_SIGMOID
    s = torch.sigmoid(z) if sigmoid else torch.softmax(z, 1)
    loss = (h * dres.double()).sum() if dres is not None else 0.0
    for i, (lo, hi) in enumerate(zip(seqs[:-1], seqs[1:])):
        p = s[lo:hi] / s[lo:hi].sum(1, keepdim=True)
        loss = loss + float(db[i]) * (m.E / (K * (hi - lo)) * counts[i].double() * p.mean(0)).sum()
        if dz is not None:
            loss = loss + float(dz[i]) * torch.logsumexp(z[lo:hi], 1).square().mean()
    if dw is not None:
        w = s.gather(1, kept.rb.topk_ids.long())
        w = w / w.sum(1, keepdim=True) if m.how.renormalize else w
        loss = loss + (w * m.how.scale * dw.double()).sum()
    grads = torch.autograd.grad(loss, list(leaf.values()))
    return dict(zip(leaf, grads))


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


SOFT = dict(score=B.SCORE_SOFTMAX, renormalize=False)


@pytest.mark.parametrize("T, E, gates, post, soft", [(300, 16, 3, True, False), (130, 16, 0, False, True), (65, 128, 1, True, False),
                                                     (1100, 64, 5, True, True)])
def test_gradients_of_the_balance(T, E, gates, post, soft):
    m = Made(T, E=E, gates=gates, post=post, how=B.scoring(**SOFT) if soft else None)
    kept = m.block.keep(T)
    m.run(kept)
    y = m.block.y[:T].clone()
    seqs = [0, T // 3, T]
    offsets = torch.tensor(seqs, dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(5)
    db = torch.rand(2, generator=g, device="cuda") + 0.5
    dz = 0.1 * torch.rand(2, generator=g, device="cuda")
    dw = torch.randn((T, K), generator=g, device="cuda") / T
    dres = (torch.randn((T, H), generator=g, device="cuda") * 1e-4).to(BF16)
    for parts in (dict(), dict(dz=dz, dtopk_w=dw, dresidual_out=dres)):
        got = m.block.balance_grad(kept, dbalance=db, seq_offsets=offsets, gate=m.gate, row_offsets=m.row_offsets, **parts)
        torch.cuda.synchronize()
        assert m.rt.device_status() == 0
        assert torch.equal(m.block.y[:T], y)
        want = whole(m, kept, got["counts"], db, parts.get("dz"), parts.get("dtopk_w"), parts.get("dresidual_out"), seqs)
        for i, (lo, hi) in enumerate(zip(seqs[:-1], seqs[1:])):
            counts = torch.bincount(kept.rb.topk_ids[lo:hi].reshape(-1).long(), minlength=E)
            assert torch.equal(got["counts"][i].long(), counts)
        assert off(got["dw_router"], want["wr"]) <= 2.0 ** -5
        names = dict(dy="y", dresidual="residual", dnorm_weight="pre", dpost_weight="post", dgate="gate")
        for n, of in names.items():
            if of in want:
                assert off(got[n], want[of]) <= 2.0 ** -3, n
            else:
                assert got[n] is None
    m.close()


def test_a_step_against_the_gradient_evens_the_router():
    """Not how far a loss falls: only that its slope has the gradient's sign and
    size, by the block's own forward calls at router weights moved a little
    (choices may change, so shares are taken from the logits with the counts held)."""
    m = Made(257, E=16, post=True)
    kept = m.block.keep(257)
    m.run(kept)
    g = m.block.balance_grad(kept, dbalance=torch.ones(1, device="cuda"))
    f = g["counts"][0].double() * m.E / (K * 257)
    def loss(wr):  # noqa: E306
        s = torch.sigmoid(kept.x.double() @ wr.double().t())
        return float((f * (s / s.sum(1, keepdim=True)).mean(0)).sum())
    step = 1e-3 / float(g["dw_router"].norm())
    fall = loss(m.wr.double()) - loss(m.wr.double() - step * g["dw_router"].double())
    assert abs(fall / (step * float(g["dw_router"].norm()) ** 2) - 1) <= 2.0 ** -4
    m.close()


def test_captured_and_replayed():
    m = Made(200, gates=2, most=256)
    kept, res = m.block.keep(200), m.residual.clone()
    s = torch.cuda.Stream()
    db = torch.ones(1, device="cuda")
    args = dict(gate=m.gate, row_offsets=m.row_offsets)
    s.wait_stream(torch.cuda.current_stream())
    m.block(m.attn, m.ids, res, stream=s, kept=kept, **args)
    first = m.block.balance_grad(kept, dbalance=db, stream=s, **args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        m.block(m.attn, m.ids, res, stream=s, kept=kept, **args)
        got = m.block.balance_grad(kept, dbalance=db, stream=s, **args)
    for _ in range(2):
        res.copy_(m.residual)
        graph.replay()
        torch.cuda.synchronize()
        for n, t in first.items():
            assert t is None or torch.equal(t, got[n]), n
    assert m.rt.device_status() == 0
    m.close()


def test_refusals():
    m = Made(40, gates=2)
    kept = m.block.keep(40)
    for bad in (dict(gate=m.gate.float()), dict(row_offsets=None), dict(gate=None), dict(kept=m.block.keep(39)),
                dict(gate=torch.cat([m.gate, m.gate]))):
        with pytest.raises(ValueError):
            m.block(m.attn, m.ids, m.residual.clone(), **{**dict(gate=m.gate, row_offsets=m.row_offsets, kept=kept), **bad})
    with pytest.raises(ValueError):
        DecoderBlockTail(m.rt, 0, m.wo, m.a, m.b, m.scale, m.pre, m.wr, m.bias, m.how, post_weight=m.pre.float())
    with pytest.raises(ValueError):
        m.block.balance_grad(m.block.keep(0), dbalance=torch.ones(1, device="cuda"))
    m.close()
