"""dwdp_balance_loss and dwdp_route_scored_grad against their formulas in 64
bits; the gradient also against torch's derivative of the losses and weights,
and against differences.

Tolerances, relative to the sums of the terms' magnitudes: an exponential by
an approximate power of two is off by (|x| + 2) 2^-23, a share has two of
them, a sum and a reciprocal; a sum over a sequence adds at most 700 terms one
after the other (2^-24 each), over E experts E / 32 and a tree."""
import numpy as np
import pytest
import torch

from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300.build import build

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
TINY = 1e-37  # shares below 2^-126 may be 0
HOWS = [dict(score=s, renormalize=r) for s in (B.SCORE_SOFTMAX, B.SCORE_SIGMOID) for r in (True, False)]


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


class Made:
    """offsets: None (one sequence) or a list."""

    def __init__(self, T, E, k, offsets=None, how=HOWS[0], seed=0, spread=1.5, scale=2.5):
        g = torch.Generator("cuda").manual_seed(seed)
        self.T, self.E, self.k = T, E, k
        self.z = spread * torch.randn((T, E), generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
        pick = self.z + torch.randn((T, E), generator=g, device="cuda")
        self.ids = torch.sort(pick.topk(k, dim=1)[1], dim=1)[0].int()
        self.offsets = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
        self.ends = [0, T] if offsets is None else offsets
        self.S = len(self.ends) - 1
        self.dw = torch.randn((T, k), generator=g, device="cuda")
        self.db = torch.randn(self.S, generator=g, device="cuda")
        self.dz = torch.randn(self.S, generator=g, device="cuda")
        self.how = B.scoring(scale=scale, **how)
        self.sigmoid, self.renorm, self.scale = how["score"] == B.SCORE_SIGMOID, how["renormalize"], scale
        self.rt = B.Runtime(64, 64, E, k, 0, max(1, T), 1, 0, min_ws_bytes=B.dwdp_balance_workspace_bytes(T, E, self.S))

    def close(self):
        assert self.rt.device_status() == 0
        self.rt.close()

    def losses(self, z=True, stream=None):
        out = B.BalanceBuffers(self.S, self.E, z=z)
        for t in (out.mean_p, out.balance, out.z):
            if t is not None:
                t.fill_(float("nan"))
        out.counts.fill_(-7)
        self.rt.ws.fill_(0xFF)
        torch.cuda.synchronize()
        self.rt.balance_loss(self.z, self.ids, self.how, out, seq_offsets=self.offsets, stream=stream)
        torch.cuda.synchronize()
        return out

    def grad(self, half=False, w=True, b=True, z=True, counts=None, stream=None):
        dl = torch.full((self.T, self.E), float("nan"), dtype=torch.bfloat16 if half else torch.float32, device="cuda")
        counts = self.losses().counts if counts is None else counts
        torch.cuda.synchronize()
        self.rt.route_scored_grad(self.z, self.ids, self.how, dl, dtopk_w=self.dw if w else None, counts=counts,
                                  dbalance=self.db if b else None, dz=self.dz if z else None, seq_offsets=self.offsets,
                                  stream=stream)
        torch.cuda.synchronize()
        return dl

    # ---- the formulas ----
    def shares(self, z):
        if not self.sigmoid:
            return torch.softmax(z, 1)
        log_s = torch.nn.functional.logsigmoid(z)
        return torch.exp(log_s - torch.logsumexp(log_s, 1, keepdim=True))

    def seq(self, b):
        return slice(self.ends[b], self.ends[b + 1])

    def rel(self, z):
        """Of a share: its exponentials' arguments, and the sum."""
        m = z.max(1, keepdim=True)[0].clamp(max=0) if z.numel() else z
        most = float(torch.maximum(z.abs(), (z - m).abs()).clamp(max=90).max()) if z.numel() else 0.0
        return (4 * (most + 2) + self.E / 32 + 16) * U

    def check_losses(self, out):
        for b in range(self.S):
            z, ids = self.z[self.seq(b)].double(), self.ids[self.seq(b)]
            n = z.shape[0]
            counts = torch.bincount(ids.reshape(-1).long(), minlength=self.E)
            assert torch.equal(out.counts[b].long(), counts)
            if n == 0:
                assert (out.mean_p[b] == 0).all() and out.balance[b] == 0 and (out.z is None or out.z[b] == 0)
                continue
            p = self.shares(z).mean(0)
            rel = self.rel(z) + min(n, 700) * U / 2
            near(out.mean_p[b], p, rel * p + TINY)
            loss = self.E / (self.k * n) * (counts * p).sum()
            near(out.balance[b], loss, (rel + (self.E / 32 + 16) * U) * loss + TINY)
            if out.z is not None:
                lse = torch.logsumexp(z, 1)
                err = self.rel(z) + 4 * U * lse.abs()
                near(out.z[b], lse.square().mean(), (2 * lse.abs() * err + err ** 2).mean() + rel * lse.square().mean())

    def formula(self, counts, w=True, b=True, z=True):
        """(d loss / d logits, the bound of binary32's error), token by token."""
        zz = self.z.double()
        want, mag = torch.zeros_like(zz), torch.zeros_like(zz)
        p = self.shares(zz)
        back = torch.sigmoid(-zz) if self.sigmoid else torch.ones_like(zz)  # 1 - s, or softmax's 1

        def through(G):
            dot, adot = (p * G).sum(1, keepdim=True), (p * G.abs()).sum(1, keepdim=True)
            return p * back * (G - dot), p * back * (G.abs() + adot)

        for i in range(self.S):
            at, n = self.seq(i), self.ends[i + 1] - self.ends[i]
            if n == 0:
                continue
            if b:
                G = torch.zeros_like(zz)
                G[at] = float(self.db[i]) * self.E / (self.k * n) * counts[i].double() / n
                v, m = through(G)
                want, mag = want + v, mag + m
            if z:
                lse = torch.logsumexp(zz[at], 1, keepdim=True)
                v = 2 * float(self.dz[i]) / n * lse * torch.softmax(zz[at], 1)
                want[at] += v
                mag[at] += v.abs() + 2 * abs(float(self.dz[i])) / n * torch.softmax(zz[at], 1)
        if w:
            ids, dw = self.ids.long(), self.dw.double() * self.scale
            if self.renorm:
                logs = torch.nn.functional.logsigmoid(zz) if self.sigmoid else zz
                q = torch.softmax(logs.gather(1, ids), 1)
                dot, adot = (q * dw).sum(1, keepdim=True), (q * dw.abs()).sum(1, keepdim=True)
                f = q * back.gather(1, ids)
                want, mag = want.scatter_add(1, ids, f * (dw - dot)), mag.scatter_add(1, ids, f * (dw.abs() + adot))
            elif self.sigmoid:
                s = torch.sigmoid(zz).gather(1, ids)
                v = dw * s * back.gather(1, ids)
                want, mag = want.scatter_add(1, ids, v), mag.scatter_add(1, ids, v.abs())
            else:
                G = torch.zeros_like(zz).scatter_(1, ids, dw)
                v, m = through(G)
                want, mag = want + v, mag + m
        return want, (2 * self.rel(zz) + (self.E / 16 + 32) * U) * mag + TINY

    def check_grad(self, dl, counts, **parts):
        want, tol = self.formula(counts, **parts)
        near(dl, want, tol + (2.0 ** -8 * want.abs() if dl.dtype == torch.bfloat16 else 0.0))


def near(got, want, tol):
    off = (got.double() - want).abs() - tol
    assert torch.isfinite(off).all() and (off.numel() == 0 or float(off.max()) <= 0), float(off.max())


SIZES = [(1, 8, 1), (1, 1, 1), (5, 3, 3), (33, 16, 16), (64, 17, 2), (100, 32, 32), (77, 61, 6), (129, 64, 6), (200, 128, 8),
         (90, 131, 8), (65, 256, 8), (40, 257, 3), (70, 512, 10), (31, 777, 32), (66, 1024, 32)]


@pytest.mark.parametrize("how", HOWS, ids=str)
@pytest.mark.parametrize("T, E, k", SIZES)
def test_losses_and_gradients(T, E, k, how):
    m = Made(T, E, k, how=how, seed=E)
    out = m.losses()
    m.check_losses(out)
    none = m.losses(z=False)
    assert torch.equal(none.mean_p, out.mean_p) and torch.equal(none.counts, out.counts)
    assert torch.equal(none.balance, out.balance)
    for parts in (dict(), dict(w=False), dict(b=False), dict(z=False), dict(w=False, z=False), dict(b=False, z=False)):
        m.check_grad(m.grad(counts=out.counts, **parts), out.counts, **parts)
    m.check_grad(m.grad(half=True), out.counts)
    assert (m.grad(w=False, b=False, z=False) == 0).all()
    m.close()


OFFSETS = [[0, 300], [0, 0, 1, 1, 2, 300], [0, 8, 16, 24, 299, 300], [0] + list(range(1, 301)), [10, 20, 250], [0, 0, 0], [300, 300],
           [0, 100], [150, 150, 300]]


@pytest.mark.parametrize("offsets", OFFSETS, ids=lambda o: str(o[:6]))
@pytest.mark.parametrize("E, k", [(24, 3), (256, 8)])
def test_sequences(offsets, E, k):
    for how in HOWS[1:3]:
        m = Made(300, E, k, offsets, how)
        out = m.losses()
        m.check_losses(out)
        dl = m.grad()
        m.check_grad(dl, out.counts)
        outside = torch.ones(300, dtype=torch.bool, device="cuda")
        outside[offsets[0]:offsets[-1]] = False
        # a NaN in no sequence reaches no loss
        m.z[outside] = float("nan")
        again = m.losses()
        for n in ("counts", "mean_p", "balance", "z"):
            assert torch.equal(getattr(again, n), getattr(out, n)), n
        assert torch.equal(m.grad()[~outside], dl[~outside])
        m.close()


@pytest.mark.parametrize("T, E, k, S", [(4096, 64, 6, 7), (8192, 256, 8, 16), (20001, 256, 8, 1), (5000, 8, 2, 300), (70000, 16, 2, 3)])
def test_many_tokens(T, E, k, S):
    cuts = np.sort(np.random.default_rng(T).integers(0, T + 1, S - 1))
    for how in HOWS[:3:2]:
        m = Made(T, E, k, [0, *cuts.tolist(), T], how, seed=T)
        out = m.losses()
        m.check_losses(out)
        dl = m.grad(counts=out.counts)
        m.check_grad(dl, out.counts)
        again = m.losses()  # the same bits from run to run
        for n in ("counts", "mean_p", "balance", "z"):
            assert torch.equal(getattr(again, n), getattr(out, n)), n
        assert torch.equal(dl, m.grad(counts=out.counts))
        m.close()


@pytest.mark.parametrize("how", HOWS, ids=str)
@pytest.mark.parametrize("E", [40, 256])
def test_logits_far_from_zero(how, E):
    """Scores that vanish in binary32, scores next to 1, both in one token, and
    chosen experts far below the largest."""
    m = Made(12, E, 4, how=how)
    m.z[0] -= 200.0
    m.z[1] += 200.0
    m.z[2, ::2] -= 150.0
    m.z[3, 5] += 60.0
    m.z[4, :] = -1000.0
    m.z[5, :] = 80.0
    m.z[6, 7] = -300.0
    m.z[7] -= 60.0
    m.z[8] -= 44.0
    m.ids[2] = torch.arange(0, 8, 2)  # chosen against the scores, as a bias does
    m.ids[3] = torch.arange(8, 12)
    out = m.losses()
    m.check_losses(out)
    m.check_grad(m.grad(), out.counts)
    m.check_grad(m.grad(b=False, z=False), out.counts, b=False, z=False)
    m.close()


def test_minus_infinity_is_a_masked_expert():
    m = Made(20, 64, 4, how=HOWS[0])
    m.z[:, 60:] = -1e30
    near_inf = m.losses()
    m.z[:, 60:] = -float("inf")
    m.ids.clamp_(max=59)
    out = m.losses()
    assert torch.equal(out.mean_p, near_inf.mean_p) and (out.mean_p[:, 60:] == 0).all()
    dl = m.grad(z=False, w=False)
    assert (dl[:, 60:] == 0).all() and torch.isfinite(dl).all()
    m.rt.device_status()
    m.rt.close()


@pytest.mark.parametrize("how", HOWS, ids=str)
def test_a_nan_stays_in_its_token_and_sequence(how):
    m = Made(90, 64, 6, [0, 30, 60, 90], how)
    out, dl = m.losses(), m.grad()
    m.z[40, 3] = float("nan")
    bad, dbad = m.losses(), m.grad(counts=out.counts)
    for n in ("mean_p", "balance", "z"):
        a, b = getattr(out, n), getattr(bad, n)
        assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.isnan(b[1]).all(), n
    rest = torch.arange(90, device="cuda") != 40
    assert torch.equal(dl[rest], dbad[rest]) and torch.isnan(dbad[40]).all()
    m.close()


@pytest.mark.parametrize("how", HOWS, ids=str)
def test_gradient_is_torchs_derivative(how):
    m = Made(50, 64, 6, [0, 20, 50], how)
    counts = m.losses().counts
    z = m.z.double().requires_grad_(True)
    loss = 0.0
    for i in range(m.S):
        at = m.seq(i)
        n = m.ends[i + 1] - m.ends[i]
        s = torch.sigmoid(z[at]) if m.sigmoid else torch.softmax(z[at], 1)
        p = s / s.sum(1, keepdim=True)
        loss = loss + float(m.db[i]) * m.E / (m.k * n) * (counts[i].double() * p.mean(0)).sum()
        loss = loss + float(m.dz[i]) * torch.logsumexp(z[at], 1).square().mean()
    s = torch.sigmoid(z) if m.sigmoid else torch.softmax(z, 1)
    w = s.gather(1, m.ids.long())
    w = w / w.sum(1, keepdim=True) if m.renorm else w
    loss = loss + (w * m.scale * m.dw.double()).sum()
    want = torch.autograd.grad(loss, z)[0]
    tol = m.formula(counts)[1]
    near(m.grad(), want, tol)
    m.close()


def test_gradient_against_differences():
    """loss_b by the call itself at z +- step: its slope is the gradient's
    product with the direction, to within the losses' own error over the step
    (64 tokens' rounding, 2^-20 of the losses) and the step's square."""
    m = Made(64, 32, 4, [0, 24, 64], HOWS[2])
    counts = m.losses().counts
    m.dw.zero_()
    dl = m.grad(counts=counts).double()
    way = torch.randn(m.z.shape, generator=torch.Generator("cuda").manual_seed(9), device="cuda")
    kept, step, got = m.z, 2.0 ** -6, []
    for sign in (1, -1):
        m.z = kept + sign * step * way
        o = m.losses()  # the choice is held: ids are given
        got.append(float((m.db.double() * o.balance.double() + m.dz.double() * o.z.double()).sum()))
    slope, size = (got[0] - got[1]) / (2 * step), abs(got[0]) + abs(got[1]) + float(m.db.abs().sum())
    m.z = kept
    curve = float(m.db.abs().sum() + m.dz.abs().sum()) * 40 * step ** 2
    assert abs(float((dl * way.double()).sum()) - slope) <= 2.0 ** -20 * size / step + curve
    m.close()


def test_ids_outside_are_reported():
    m = Made(30, 64, 6)
    out = m.losses()
    dl = m.grad(counts=out.counts)
    was = m.ids[4, 2].item()
    for bad in (64, -1, 1 << 30):
        m.ids[4, 2] = bad
        o = m.losses()
        assert m.rt.device_status() == -6
        assert int(out.counts[0, was]) - int(o.counts[0, was]) == 1
        assert int(o.counts.sum()) == int(out.counts.sum()) - 1
        g = m.grad(counts=out.counts)
        assert m.rt.device_status() == -6
        rest = torch.arange(30, device="cuda") != 4
        assert torch.equal(g[rest], dl[rest]) and torch.isfinite(g).all()
    m.rt.close()


def test_no_tokens():
    m = Made(0, 16, 2, [0, 0, 0])
    m.check_losses(m.losses())
    assert m.grad().shape == (0, 16)
    m.close()


def test_captured_and_replayed_on_another_stream():
    m = Made(700, 256, 8, [0, 300, 700], HOWS[2])
    out, dl = m.losses(), m.grad()
    again, d2 = B.BalanceBuffers(m.S, m.E), torch.empty_like(dl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        m.rt.balance_loss(m.z, m.ids, m.how, again, seq_offsets=m.offsets)
        m.rt.route_scored_grad(m.z, m.ids, m.how, d2, dtopk_w=m.dw, counts=again.counts, dbalance=m.db, dz=m.dz,
                               seq_offsets=m.offsets)
    for _ in range(2):
        d2.fill_(float("nan")), again.mean_p.fill_(float("nan")), again.counts.fill_(-1)
        m.rt.ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d2, dl) and torch.equal(again.mean_p, out.mean_p) and torch.equal(again.counts, out.counts)
        assert torch.equal(again.balance, out.balance) and torch.equal(again.z, out.z)
    m.z.mul_(0.5)
    m.offsets.copy_(torch.tensor([0, 650, 700]))
    m.ends = [0, 650, 700]
    graph.replay()
    torch.cuda.synchronize()
    m.check_losses(again)
    m.check_grad(d2, again.counts)
    m.close()


def test_logits_beyond_2_to_the_31():
    T, E, k = 2_200_000, 1024, 2
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    part = Made(64, E, k, how=HOWS[2])
    want = part.losses()
    want_d = part.grad(counts=want.counts)
    z = torch.zeros((T, E), device="cuda")
    z[-64:] = part.z
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    ids[:, 1] = 1
    ids[-64:] = part.ids
    dw = torch.zeros((T, k), device="cuda")
    dw[-64:] = part.dw
    offsets = torch.tensor([0, T - 64, T], dtype=torch.int32, device="cuda")
    # a context for that many tokens, without the expert layer's workspace
    ctx = B.dwdp_create(64, 64, E, k, 0, T, 1, 0)
    ws = torch.empty(B.dwdp_balance_workspace_bytes(T, E, 2), dtype=torch.uint8, device="cuda")
    out, dl = B.BalanceBuffers(2, E), torch.empty((T, E), device="cuda")
    B.dwdp_balance_loss(ctx, z, ids, T, offsets, 2, part.how, out.counts, out.mean_p, out.balance, out.z, ws, ws.numel())
    B.dwdp_route_scored_grad(ctx, z, ids, dw, T, offsets, 2, part.how, out.counts,
                             torch.cat([part.db, part.db]), torch.cat([part.dz, part.dz]), dl)
    torch.cuda.synchronize()
    assert B.dwdp_device_status(ctx) == 0
    B.dwdp_destroy(ctx)
    assert torch.equal(out.counts[1], want.counts[0]) and torch.equal(dl[-64:], want_d)
    rel = part.rel(part.z.double()) + 128 * U
    near(out.mean_p[1], want.mean_p[0].double(), rel * want.mean_p[0].double())
    assert abs(float(out.mean_p[0].sum()) - 1.0) <= 1e-3
    part.close()


def test_refuses_what_it_would_misread():
    m = Made(16, 64, 4, [0, 4, 16])
    out, dl = B.BalanceBuffers(2, 64), torch.empty((16, 64), device="cuda")
    f = lambda **k: m.rt.balance_loss(**{**dict(logits=m.z, topk_ids=m.ids, how=m.how, out=out, seq_offsets=m.offsets), **k})  # noqa: E731
    f()
    for bad in (dict(logits=m.z.bfloat16()), dict(logits=m.z[:, :32]), dict(logits=m.z.cpu()), dict(topk_ids=m.ids.long()),
                dict(topk_ids=m.ids[:8]), dict(topk_ids=m.ids[:, :2]), dict(seq_offsets=m.offsets.long()), dict(seq_offsets=None),
                dict(seq_offsets=m.offsets[:2]), dict(out=B.BalanceBuffers(2, 32)), dict(out=B.BalanceBuffers(3, 64)), dict(out=B.BalanceBuffers(2, 64, device="cpu"))):
        with pytest.raises(ValueError):
            f(**bad)
    with pytest.raises(B.DwdpError):  # more than max_tokens
        f(logits=torch.zeros((17, 64), device="cuda"), topk_ids=torch.zeros((17, 4), dtype=torch.int32, device="cuda"))
    c = lambda **k: m.rt.route_scored_grad(**{**dict(logits=m.z, topk_ids=m.ids, how=m.how, dlogits=dl, dtopk_w=m.dw, counts=out.counts, dbalance=m.db, dz=m.dz, seq_offsets=m.offsets), **k})  # noqa: E731
    c()
    for bad in (dict(dlogits=dl.half()), dict(dlogits=dl[:8]), dict(dlogits=dl.t()), dict(dtopk_w=m.dw.bfloat16()), dict(dtopk_w=m.dw[:, :2]),
                dict(counts=out.counts[:1]), dict(counts=out.mean_p), dict(dbalance=m.db[:1]), dict(dz=m.dz.double())):
        with pytest.raises(ValueError):
            c(**bad)
    with pytest.raises(B.DwdpError):
        c(counts=None)
    L, P = B.lib(), 4096
    import ctypes
    call = lambda logits=P, ids=P, T=4, off=P, n=2, sc=m.how, counts=P, mean=P, bal=P, z=P, ws=P, nb=1 << 24: L.dwdp_balance_loss(  # noqa: E731
        m.rt.ctx, logits, ids, T, off, n, ctypes.byref(sc), counts, mean, bal, z, ws, nb, None)
    for bad in (dict(logits=None), dict(ids=None), dict(T=-1), dict(T=17), dict(n=0), dict(n=-1), dict(off=None), dict(sc=B.scoring(5)),
                dict(counts=None), dict(mean=None), dict(bal=None), dict(ws=None), dict(nb=64), dict(logits=P + 4), dict(ids=P + 4),
                dict(off=P + 4), dict(counts=P + 4), dict(mean=P + 8), dict(bal=P + 4), dict(z=P + 4), dict(ws=P + 8)):
        assert call(**bad) == -1, bad
    call = lambda logits=P, ids=P, dw=P, T=4, off=P, n=2, sc=m.how, counts=P, db=P, dz=P, out=P, half=0: L.dwdp_route_scored_grad(  # noqa: E731
        m.rt.ctx, logits, ids, dw, T, off, n, ctypes.byref(sc), counts, db, dz, out, half, None)
    for bad in (dict(logits=None), dict(ids=None), dict(T=-1), dict(T=17), dict(n=0), dict(off=None), dict(sc=B.scoring(5)),
                dict(sc=B.scoring(scale=0.0)), dict(sc=B.scoring(scale=float("nan"))), dict(counts=None), dict(out=None), dict(half=2),
                dict(dw=P + 4), dict(counts=P + 4), dict(db=P + 4), dict(dz=P + 4), dict(out=P + 8)):
        assert call(**bad) == -1, bad
    m.close()
