"""dwdp_sandwich_norm and its gradients against their formulas in 64 bits.

Tolerances: a rounding to bf16 is off by at most 2^-8 of the value, to E4M3 by
2^-4 of it or half a subnormal step (2^-10).  FP32 = 2^-17 bounds what one step
in binary32 does to a value (a tree sum of up to 32768 terms with at most 64
one after the other, a reciprocal square root and a few products), relative
to the sum of its terms' magnitudes; where a step's error enters the next one,
the bound is carried through the formula.  Sums over rows add up to `rows`
terms one after the other: rows 2^-24 of their magnitudes more."""
import numpy as np
import pytest
import torch

from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300 import inputs as I
from moe_expert_grouped_split_gb300.build import build

pytestmark = pytest.mark.gpu

FP32 = 2.0 ** -17
BF16_HALF, E4M3_HALF, E4M3_SUB = 2.0 ** -8, 2.0 ** -4, 2.0 ** -10
EPS = 1e-6
F8, BF16 = torch.float8_e4m3fn, torch.bfloat16
A, C = 0.9, 1.25  # residual_scale, block_scale


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def d(t):
    return t.double()


def randn(name, std, *shape):
    return I.randn_bf16(shape, std, I.seed_for(31, name, *shape), "cuda")


class Made:
    """Inputs of one case.  groups: None (no gate), 1, or a list of offsets."""

    def __init__(self, rows, H, post=True, pre=True, residual=True, groups=1, pad=0):
        self.rows, self.H = rows, H
        wide = randn("x", 1.0, rows, H + pad)
        self.x = wide[:, :H]
        self.residual = randn("residual", 3.0, rows, H) if residual else None
        self.post = randn("post", 1.0, H) if post else None
        self.pre = randn("pre", 1.0, H) if pre else None
        self.offsets, self.gate, self.of = None, None, None
        at = torch.arange(rows, device="cuda")
        if groups is not None:
            G = 1 if groups == 1 else len(groups) - 1
            self.gate = randn("gate", 1.0, G, H)
            self.of = torch.zeros(rows, dtype=torch.int64, device="cuda")
            if groups != 1:
                self.offsets = torch.tensor(groups, dtype=torch.int32, device="cuda")
                self.of = torch.searchsorted(self.offsets[1:].contiguous(), at, right=True)
                self.of[at < groups[0]] = G
        self.G = 0 if groups is None else self.gate.shape[0]
        self.inside = torch.ones(rows, dtype=torch.bool, device="cuda") if self.of is None else self.of < self.G
        self.norm = B.SandwichNorm(H, max(1, rows), self.pre, self.post, C, A, EPS, max_groups=max(1, self.G))

    def gates(self):
        """[rows, H] in 64 bits (1 where there is none)."""
        if self.gate is None:
            return torch.ones((self.rows, self.H), dtype=torch.float64, device="cuda")
        return torch.cat([d(self.gate), torch.zeros_like(d(self.gate[:1]))])[self.of]

    def outputs(self, codes=True, kept=True):
        full = lambda v, t: torch.full((self.rows, self.H), v, dtype=torch.float32, device="cuda").to(t)  # noqa: E731
        one = lambda *n: torch.full(n, float("nan"), device="cuda")  # noqa: E731
        o = dict(residual_out=full(float("nan"), BF16))
        if self.pre is not None:
            o["out"] = full(float("nan"), BF16)
            if codes:
                o.update(codes=full(3.0, F8), row_scale=one(self.rows))
        if kept:
            o.update(x_codes=full(3.0, F8), x_scale=one(self.rows), h_codes=full(3.0, F8), h_scale=one(self.rows),
                     rstd=one(self.rows, 2))
        return o

    def forward(self, codes=True, kept=True, stream=None):
        o = self.outputs(codes, kept)
        torch.cuda.synchronize()
        self.norm.forward(self.x, self.residual, gate=self.gate, row_offsets=self.offsets, stream=stream, **o)
        torch.cuda.synchronize()
        return o

    # ---- the formulas: values and how far binary32 may be from them ----
    def h(self):
        x = d(self.x)
        rx = 1 / torch.sqrt(x.square().mean(1, keepdim=True) + EPS) if self.post is not None else torch.ones_like(x[:, :1])
        n = x * rx * (d(self.post) if self.post is not None else 1.0)
        part = C * self.gates() * n
        res = A * d(self.residual) if self.residual is not None else torch.zeros_like(x)
        return part + res, FP32 * (part.abs() + res.abs()), rx

    def check_forward(self, o):
        i = self.inside
        h, eh, rx = self.h()
        near(o["residual_out"], h, BF16_HALF * h.abs() + eh, i)
        rh = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) if self.pre is not None else torch.ones_like(rx)
        erh = rh * FP32 + rh ** 2 * eh.square().mean(1, keepdim=True).sqrt()  # d rh <= rh^2 rms(error of h)
        if self.pre is not None:
            w = d(self.pre)
            y = h * rh * w
            ey = (eh * rh + h.abs() * erh) * w.abs() + FP32 * y.abs()
            near(o["out"], y, BF16_HALF * y.abs() + ey, i)
            if "codes" in o:
                rows8(o["codes"], o["row_scale"], y, ey, i)
        if "x_codes" in o:
            rows8(o["x_codes"], o["x_scale"], d(self.x), FP32 * d(self.x).abs(), i)
            rows8(o["h_codes"], o["h_scale"], h, eh, i)
            near(o["rstd"], torch.cat([rx, rh], 1), torch.cat([FP32 * rx, erh], 1), i)


def near(got, want, tol, rows=None):
    off = (d(got) - want).abs() - tol
    off = off if rows is None else off[rows]
    assert torch.isfinite(off).all() and (off.numel() == 0 or float(off.max()) <= 1e-38), float(off.max())


def rows8(codes, scale, v, ev, i):
    m = v.abs().amax(1)
    want = torch.where(m > 0, m / 448.0, torch.ones_like(m))
    em = ev.amax(1)
    near(scale, want, torch.where(m > 0, FP32 * want + em / 448.0, 0.0 * m), i)
    q = v / want[:, None]
    moved = ev / want[:, None] + q.abs() * (FP32 + (em / m.clamp(min=1e-300)))[:, None]
    near(codes, q, (E4M3_HALF) * q.abs() + E4M3_SUB + 2 * moved, i)


ENDS = [0, 0, 5, 5, 6, 40, 77]  # with groups of no rows
FORMS = [dict(), dict(groups=None), dict(groups=ENDS), dict(post=False, groups=None), dict(pre=False), dict(residual=False),
         dict(post=False, pre=False, groups=ENDS), dict(post=False, residual=False, groups=None)]


@pytest.mark.parametrize("H", [8, 64, 520, 1536, 7168, 8192, 8200, 32768])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_rows(H, form):
    m = Made(77, H, **form)
    m.check_forward(m.forward())
    m.check_forward(m.forward(codes=False, kept=False))


@pytest.mark.parametrize("rows, H", [(1, 7168), (2, 8), (1003, 2048), (5000, 512), (2500, 1024), (700, 7168), (160, 16384)])
def test_counts_of_rows(rows, H):
    m = Made(rows, H, groups=1 if rows < 3 else [0, rows // 3, rows - 1, rows], pad=64)
    m.check_forward(m.forward(kept=False))
    m.check_forward(m.forward(codes=False))


def test_many_groups():
    for G in (31, 32, 33, 1100):
        rng = np.random.default_rng(G)
        at = np.sort(rng.integers(0, 1201, G - 1))
        m = Made(1200, 64, groups=[0, *at.tolist(), 1200])
        m.check_forward(m.forward())


@pytest.mark.parametrize("groups", [[7, 20, 20, 60], [60, 60], [0, 0], [77, 77, 77]])
def test_rows_in_no_group_are_left_as_they_were(groups):
    m = Made(77, 512, groups=groups)
    o = m.forward()
    m.check_forward(o)
    out = ~m.inside
    for name, t in m.outputs().items():
        assert torch.equal(o[name][out].view(torch.uint8), t[out].view(torch.uint8)), name
    # and a NaN there reaches nobody
    m.x[out] = float("nan")
    again = m.forward()
    for name in o:
        assert torch.equal(again[name].view(torch.uint8), o[name].view(torch.uint8)), name


def test_row_stride_and_nothing_between_the_rows_is_touched():
    m = Made(33, 512, pad=576)
    whole = m.x.as_strided((33, 512 + 576), (512 + 576, 1))
    whole[:, 512:] = float("nan")
    before = whole.view(torch.int16).clone()
    m.check_forward(m.forward())
    assert torch.equal(whole.view(torch.int16), before)


@pytest.mark.parametrize("H", [7168, 16384])
def test_in_place(H):
    m = Made(50, H)
    apart = m.forward()
    x, r = m.x.clone(), m.residual.clone()
    m.norm.forward(x, r, gate=m.gate, residual_out=r, out=x)
    torch.cuda.synchronize()
    assert torch.equal(x, apart["out"]) and torch.equal(r, apart["residual_out"])


def test_in_place_with_rows_fetched_ahead():
    m = Made(1300, 7168, groups=[0, 5, 700, 1300])
    apart = m.forward(kept=False)
    x, r = m.x.clone(), m.residual.clone()
    m.norm.forward(x, r, gate=m.gate, row_offsets=m.offsets, residual_out=r, out=x)
    torch.cuda.synchronize()
    assert torch.equal(x, apart["out"]) and torch.equal(r, apart["residual_out"])
    g = Grads(m)
    o = g.run()
    g.call(dx=g.dout, dresidual=g.dres)
    torch.cuda.synchronize()
    assert torch.equal(g.dout, o["dx"]) and torch.equal(g.dres, o["dresidual"])


@pytest.mark.parametrize("H", [512, 7168, 8192, 12296])
@pytest.mark.parametrize("form", [dict(), dict(pre=False), dict(post=False), dict(post=False, pre=False)], ids=str)
def test_many_rows_of_which_some_are_in_no_group(H, form):
    """Blocks that pass over rows, at their start, at their end, and altogether."""
    rows = 6000 if H == 512 else 2500
    m = Made(rows, H, groups=[700, 705, 705, rows - 903, rows - 31], **form)
    o = m.forward()
    m.check_forward(o)
    out = ~m.inside
    for name, t in m.outputs().items():
        assert torch.equal(o[name][out].view(torch.uint8), t[out].view(torch.uint8)), name
    for x8 in (False, True):
        g = Grads(m, x8, x8 and m.pre is not None)
        b = g.run()
        g.check(b)
        for n in ("dx", "dresidual"):
            assert torch.isnan(b[n][out]).all()


@pytest.mark.parametrize("pad", [8, 16, 64])
@pytest.mark.parametrize("H", [64, 2048, 7168])
def test_gradients_from_codes_whose_rows_lie_apart(H, pad):
    g = Grads(Made(330, H, groups=[0, 100, 330]), True, True)
    o = g.run()
    wide = torch.full((330, H + pad), 3.0, device="cuda").to(F8)
    wide[:, :H] = g.x
    g.x = wide[:, :H]
    again = g.run()
    for n in o:
        near(again[n], *g.formula()[n], g.m.inside if n in ("dx", "dresidual") else None)


def test_is_add_rmsnorm_without_its_extras():
    m = Made(65, 1536, post=False, groups=None)
    m.norm = B.SandwichNorm(m.H, m.rows, m.pre, None, 1.0, 1.0, EPS)
    o = m.forward()
    out, res = torch.empty_like(m.residual), torch.empty_like(m.residual)
    codes, scale = torch.empty_like(o["codes"]), torch.empty(m.rows, device="cuda")
    B.dwdp_add_rmsnorm(m.x, m.rows, m.H, m.pre, EPS, out, residual=m.residual, residual_out=res, codes=codes,
                       row_scale=scale)
    torch.cuda.synchronize()
    assert torch.equal(res, o["residual_out"])
    near(o["out"], d(out), (2 * BF16_HALF) * d(out).abs())
    near(scale, d(o["row_scale"]), FP32 * d(scale))


def test_kept_rows_are_quantize_rows_rows():
    m = Made(65, 1536)
    o = m.forward()
    codes, scale = torch.empty_like(o["x_codes"]), torch.empty(m.rows, device="cuda")
    B.dwdp_quantize_rows(B.DTYPE_E4M3, m.x, m.rows, m.H, codes, None, scale)
    torch.cuda.synchronize()
    near(o["x_scale"], d(scale), FP32 * d(scale))
    differ = codes.view(torch.uint8) != o["x_codes"].view(torch.uint8)
    assert float(differ.float().mean()) <= 1e-3  # next to the middle of two codes


def test_zero_rows():
    m = Made(3, 256)
    m.x[1] = 0
    m.residual[1] = 0
    o = m.forward()
    m.check_forward(o)
    for n in ("codes", "x_codes", "h_codes", "out", "residual_out"):
        assert (o[n][1].float() == 0).all()
    for n in ("row_scale", "x_scale", "h_scale"):
        assert o[n][1] == 1.0


@pytest.mark.parametrize("H", [1024, 16384])
def test_squares_beyond_the_range(H):
    m = Made(6, H)
    m.x[0] *= 1e30
    m.x[1, 3] = -3e38
    m.x[2] *= 1e-30
    m.residual[3] *= 1e30
    m.residual[4, 5] = 1e35
    o = m.forward(codes=False)
    h, eh, rx = m.h()
    near(o["residual_out"], h, BF16_HALF * h.abs() + eh)
    rh = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
    near(o["rstd"][:, :1], rx, 2.0 ** -16 * rx)
    y = h * rh * d(m.pre)
    near(o["out"], y, (BF16_HALF + 2.0 ** -14) * y.abs() + 2.0 ** -14 * (eh * rh * d(m.pre).abs()) * 2.0 ** 17)


def test_a_nan_stays_in_its_row():
    m = Made(5, 512)
    clean = m.forward()
    m.x[2, 100] = float("nan")
    m.x[4, 0] = float("inf")
    o = m.forward()
    for n in clean:
        assert torch.equal(o[n][[0, 1, 3]].view(torch.uint8), clean[n][[0, 1, 3]].view(torch.uint8)), n
    assert torch.isnan(o["out"][2]).all() and torch.isnan(o["out"][4]).all()
    assert torch.isnan(o["row_scale"][2]) and torch.isnan(o["h_scale"][2]) and torch.isnan(o["rstd"][2]).all()


# -------------------------------------------------------------- gradients --
class Grads:
    """The gradients of a Made, from bf16 rows or rows in 8 bits."""

    def __init__(self, m: Made, x8=False, h8=False, dres=True):
        self.m = m
        rows, H = m.rows, m.H
        o = m.forward(codes=False)
        self.rstd = torch.where(m.inside[:, None], o["rstd"], torch.ones_like(o["rstd"]))
        fix = lambda t: torch.where(m.inside[:, None], t.float(), torch.zeros_like(t.float())).to(t.dtype)  # noqa: E731
        s = lambda t: torch.where(m.inside, t, torch.ones_like(t))  # noqa: E731
        self.x, self.x_scale = (fix(o["x_codes"]), s(o["x_scale"])) if x8 else (m.x, None)
        self.h, self.h_scale = (fix(o["h_codes"]), s(o["h_scale"])) if h8 else (fix(o["residual_out"]), None)
        self.dout = randn("dout", 1.0, rows, H) if m.pre is not None else None
        self.dres = randn("dres", 1.0, rows, H) if dres or m.pre is None else None
        if m.pre is None:
            self.h = self.h_scale = None

    def outputs(self):
        m = self.m
        bf = lambda: torch.full((m.rows, m.H), float("nan"), dtype=BF16, device="cuda")  # noqa: E731
        o = dict(dx=bf(), dresidual=bf())
        if m.post is not None:
            o["dpost_weight"] = torch.full((m.H,), float("nan"), device="cuda")
        if m.pre is not None:
            o["dpre_weight"] = torch.full((m.H,), float("nan"), device="cuda")
        if m.gate is not None:
            o["dgate"] = torch.full((m.G, m.H), float("nan"), device="cuda")
        return o

    def call(self, stream=None, **o):
        m = self.m
        m.norm.grad(self.x, self.h, self.rstd, self.dout, self.dres, gate=m.gate, row_offsets=m.offsets,
                    x_scale=self.x_scale, h_scale=self.h_scale, stream=stream, **o)

    def run(self):
        o = self.outputs()
        self.m.norm.ws.fill_(0xFF)  # NaN: what is read has to be written first
        torch.cuda.synchronize()
        self.call(**o)
        torch.cuda.synchronize()
        return o

    def formula(self):
        """{name: (value, bound of binary32's error)}"""
        m = self.m
        on = m.inside[:, None].double()
        val = lambda t, s: d(t) * (d(s)[:, None] if s is not None else 1.0)  # noqa: E731
        rx, rh = d(self.rstd)[:, :1], d(self.rstd)[:, 1:]
        zero = torch.zeros((m.rows, m.H), dtype=torch.float64, device="cuda")
        dres = d(self.dres) if self.dres is not None else zero
        r = {}
        if m.pre is not None:
            hhat, w, dout = val(self.h, self.h_scale) * rh, d(m.pre), d(self.dout) * on
            gy = dout * w
            mean, mag = (gy * hhat).mean(1, keepdim=True), (gy * hhat).abs().mean(1, keepdim=True)
            dh = dres + rh * (gy - hhat * mean)
            edh = FP32 * (dres.abs() + rh * (gy.abs() + hhat.abs() * mag))
            r["dpre_weight"] = self.total(dout * hhat, 0)
        else:
            dh, edh = dres, FP32 * dres.abs()
        dh, edh = dh * on, edh * on
        xhat = torch.nan_to_num(val(self.x, self.x_scale)) * rx
        post = d(m.post) if m.post is not None else torch.ones_like(xhat[0])
        g = C * m.gates()
        dn, edn = g * dh, g.abs() * (edh + FP32 * dh.abs())
        if m.gate is not None:
            each = C * dh * xhat * post
            err = C * edh * (xhat * post).abs()
            one = torch.nn.functional.one_hot(m.of, m.G + 1).double()[:, :m.G]
            r["dgate"] = tuple(one.t() @ v for v in (each, err + (FP32 + m.rows * 2.0 ** -24) * each.abs()))
        gn, egn = dn * post, edn * post.abs()
        if m.post is not None:
            r["dpost_weight"] = self.total(dn * xhat, edn * xhat.abs())
            mean, mag = (gn * xhat).mean(1, keepdim=True), (gn * xhat).abs().mean(1, keepdim=True)
            emean = (egn * xhat.abs()).mean(1, keepdim=True) + FP32 * mag
            dx = rx * (gn - xhat * mean)
            edx = rx * (egn + xhat.abs() * emean + FP32 * (gn.abs() + xhat.abs() * mag))
        else:
            dx, edx = dn, edn
        r["dx"] = dx, edx + BF16_HALF * dx.abs()
        r["dresidual"] = A * dh, A * edh + BF16_HALF * A * dh.abs() + 1e-40
        return r

    def total(self, v, err):
        return v.sum(0), ((FP32 + self.m.rows * 2.0 ** -24) * v.abs() + err).sum(0)

    def check(self, o):
        for name, (want, tol) in self.formula().items():
            near(o[name], want, tol, self.m.inside if name in ("dx", "dresidual") else None)


@pytest.mark.parametrize("H", [8, 64, 520, 1536, 4096, 4104, 7168, 8192, 8200, 20008, 32768])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_gradients(H, form):
    g = Grads(Made(77, H, **form))
    g.check(g.run())


@pytest.mark.parametrize("x8, h8", [(False, True), (True, False), (True, True)])
@pytest.mark.parametrize("H", [8, 520, 7168, 16392])
def test_gradients_from_rows_in_8_bits(H, x8, h8):
    g = Grads(Made(161, H, groups=[0, 3, 3, 100, 160, 161]), x8, h8)
    g.check(g.run())
    g = Grads(Made(9, H), x8, h8, dres=False)
    g.check(g.run())


@pytest.mark.parametrize("rows, H", [(1, 7168), (2, 8), (152, 7168), (153, 7168), (1003, 2048), (3000, 512), (20000, 256), (305, 8192), (700, 12296)])
@pytest.mark.parametrize("x8", [False, True])
def test_gradients_of_many_rows(rows, H, x8):
    g = Grads(Made(rows, H, groups=1 if rows < 3 else [0, rows // 3, rows - 1, rows], pad=0 if x8 else 64), x8, x8)
    o = g.run()
    g.check(o)
    again = g.run()
    for n in o:
        assert torch.equal(o[n], again[n]), n  # the same bits from run to run


def test_gradients_of_many_groups():
    for G in (33, 1100):
        at = np.sort(np.random.default_rng(G).integers(0, 1201, G - 1))
        g = Grads(Made(1200, 64, groups=[0, *at.tolist(), 1200]))
        g.check(g.run())


@pytest.mark.parametrize("groups", [[7, 20, 20, 60], [60, 60], [0, 0], [77, 77, 77], [0, 2, 3]])
def test_gradients_of_rows_in_no_group(groups):
    g = Grads(Made(77, 512, groups=groups))
    o = g.run()
    g.check(o)
    for n in ("dx", "dresidual"):
        assert torch.isnan(o[n][~g.m.inside]).all()
    g.dout[~g.m.inside] = float("nan")
    g.rstd[~g.m.inside] = float("nan")
    again = g.run()
    for n in ("dpost_weight", "dpre_weight", "dgate"):
        assert torch.equal(o[n], again[n])


def test_gradients_of_no_rows_are_zeros():
    m = Made(1, 512, groups=[0, 0, 0])
    o = Grads(m).outputs()
    e = torch.empty((0, 512), dtype=BF16, device="cuda")
    m.norm.grad(e, e, torch.empty((0, 2), device="cuda"), e, e, gate=m.gate, row_offsets=m.offsets, dx=e, dresidual=e,
                dpost_weight=o["dpost_weight"], dpre_weight=o["dpre_weight"], dgate=o["dgate"])
    torch.cuda.synchronize()
    for n in ("dpost_weight", "dpre_weight", "dgate"):
        assert (o[n] == 0).all()


def test_gradients_one_by_one_and_in_place():
    g = Grads(Made(200, 1536, groups=[0, 90, 200]))
    o = g.run()
    for n in o:  # each output alone
        one = {n: g.outputs()[n]}
        g.call(**one)
        torch.cuda.synchronize()
        assert torch.equal(one[n], o[n]), n
    dout, dres = g.dout, g.dres
    g.dout, g.dres = dout.clone(), dres.clone()
    g.call(dx=g.dout, dresidual=g.dres)
    torch.cuda.synchronize()
    assert torch.equal(g.dout, o["dx"]) and torch.equal(g.dres, o["dresidual"])


def test_gradients_without_what_they_do_not_need():
    """No post norm: x is needed for the gate's gradient alone."""
    g = Grads(Made(40, 512, post=False))
    o = g.run()
    x, g.x = g.x, None
    part = {n: t for n, t in g.outputs().items() if n != "dgate"}
    g.call(**part)
    torch.cuda.synchronize()
    for n in part:
        assert torch.equal(part[n], o[n]), n
    with pytest.raises(B.DwdpError):
        g.call(dgate=o["dgate"])


def test_gradients_against_differences():
    """The slope of loss = sum(h du + y dv) in 64 bits along random directions
    of every input is their gradients' product with the direction.  The call
    sees h rounded to bf16 (2^-8 of it), its outputs are rounded once more, and
    rounding errors of either sign leave about the root of their squares' sum:
    6 of those are allowed."""
    m = Made(6, 256, groups=[0, 2, 6])
    g = Grads(m)
    o = g.run()
    ins = dict(x=d(m.x), residual=d(m.residual), post=d(m.post), pre=d(m.pre), gate=d(m.gate))

    def loss(x, residual, post, pre, gate):
        n = x / torch.sqrt(x.square().mean(1, keepdim=True) + EPS) * post
        h = A * residual + C * gate[m.of] * n
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * pre
        return float((h * d(g.dres) + y * d(g.dout)).sum())

    grads = dict(x="dx", residual="dresidual", post="dpost_weight", pre="dpre_weight", gate="dgate")
    gen = torch.Generator("cuda").manual_seed(3)
    for name, of in grads.items():
        way = torch.randn(ins[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        eps = 1e-5
        hi, lo = ({**ins, name: ins[name] + s * eps * way} for s in (1, -1))
        slope = (loss(**hi) - loss(**lo)) / (2 * eps)
        terms = d(o[of]) * way
        assert abs(float(terms.sum()) - slope) <= 6 * 2 * BF16_HALF * float(terms.square().sum().sqrt()), name


def test_a_nan_gradient_stays_in_its_row():
    g = Grads(Made(300, 512))
    clean = g.run()
    g.dout[7, 3] = float("nan")
    o = g.run()
    rest = torch.arange(300, device="cuda") != 7
    for n in ("dx", "dresidual"):
        assert torch.isnan(o[n][7]).all() and torch.equal(o[n][rest], clean[n][rest])


# ------------------------------------------------------ streams and sizes --
def test_captured_and_replayed_on_another_stream():
    m = Made(333, 1536, groups=[0, 100, 333])
    g = Grads(m)
    fwd, bwd = m.forward(), g.run()
    s = torch.cuda.Stream()
    o, b = m.outputs(), g.outputs()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        m.norm.forward(m.x, m.residual, gate=m.gate, row_offsets=m.offsets, **o)
        g.call(**b)
    for _ in range(2):
        for t in (*o.values(), *b.values()):
            t.view(torch.uint8).fill_(0x55)
        graph.replay()
        torch.cuda.synchronize()
        for n in fwd:
            assert torch.equal(o[n].view(torch.uint8), fwd[n].view(torch.uint8)), n
        for n in bwd:
            assert torch.equal(b[n], bwd[n]), n
    # other inputs, and other groups, in the same tensors
    m.x.mul_(0.5)
    m.offsets.copy_(torch.tensor([0, 200, 333]))
    m.of = (torch.arange(333, device="cuda") >= 200).long()
    graph.replay()
    torch.cuda.synchronize()
    m.check_forward(o)
    g.check(b)


def test_elements_beyond_2_to_the_31():
    rows, H = 300_000, 7168
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    m = Made(64, H)
    g = Grads(m, True, True)
    big = lambda t: torch.empty((rows, H), dtype=t, device="cuda")  # noqa: E731
    x, r = big(BF16), big(BF16)
    x.zero_(), r.zero_()
    x[-64:], r[-64:] = m.x, m.residual
    norm = B.SandwichNorm(H, rows, m.pre, m.post, C, A, EPS)
    o = dict(residual_out=big(BF16), out=big(BF16), x_codes=big(F8), h_codes=big(F8), x_scale=torch.empty(rows, device="cuda"),
             h_scale=torch.empty(rows, device="cuda"), rstd=torch.empty((rows, 2), device="cuda"))
    norm.forward(x, r, gate=m.gate, **o)
    torch.cuda.synchronize()
    last = {n: t[-64:] for n, t in o.items()}
    m.check_forward(last)
    # rows of zero gradients before them: the sums are those of the last rows
    g.x, g.x_scale, g.h, g.h_scale, g.rstd = (last[n].clone() for n in ("x_codes", "x_scale", "h_codes", "h_scale", "rstd"))
    x.zero_(), r.zero_()
    x[-64:], r[-64:] = g.dout, g.dres
    b = dict(dx=o["out"], dresidual=o["residual_out"], dpost_weight=torch.empty(H, device="cuda"),
             dpre_weight=torch.empty(H, device="cuda"), dgate=torch.empty((1, H), device="cuda"))
    norm.grad(o["x_codes"], o["h_codes"], o["rstd"], x, r, gate=m.gate, x_scale=o["x_scale"], h_scale=o["h_scale"], **b)
    torch.cuda.synchronize()
    g.check({n: t[-64:] if n in ("dx", "dresidual") else t for n, t in b.items()})


def test_refuses_what_it_would_misread():
    m = Made(16, 512, groups=[0, 4, 16])
    g = Grads(m)
    o, b = m.outputs(), g.outputs()
    f = lambda **k: m.norm.forward(**{**dict(x=m.x, residual=m.residual, gate=m.gate, row_offsets=m.offsets), **o, **k})  # noqa: E731
    for bad in (dict(x=m.x.float()), dict(x=m.x[:, :256]), dict(x=m.x.t()), dict(x=m.x.cpu()), dict(residual=m.residual.float()),
                dict(residual=m.residual[:8]), dict(residual=m.residual.cpu()), dict(gate=m.gate.float()), dict(gate=m.gate[:, :256]),
                dict(row_offsets=m.offsets.long()), dict(row_offsets=m.offsets[:2]), dict(gate=None),
                dict(row_offsets=None), dict(out=o["out"].float()), dict(out=o["out"].t()), dict(codes=o["out"]),
                dict(rstd=o["rstd"][:, 0]), dict(rstd=o["rstd"].double()), dict(x_scale=o["x_scale"][:4]),
                dict(h_codes=o["h_codes"][:4])):
        with pytest.raises(ValueError):
            f(**bad)
    with pytest.raises(ValueError):
        m.norm.forward(torch.empty((17, 512), dtype=BF16, device="cuda"), out=o["out"])  # more than max_rows
    c = lambda **k: m.norm.grad(**{**dict(x=m.x, h=g.h, rstd=g.rstd, dout=g.dout, dresidual_out=g.dres, gate=m.gate, row_offsets=m.offsets), **b, **k})  # noqa: E731
    for bad in (dict(x=m.x.float()), dict(x_scale=o["x_scale"]), dict(h=g.h.float()), dict(h_scale=o["h_scale"]), dict(h=g.h[:4]),
                dict(rstd=g.rstd.double()), dict(dout=g.dout.float()), dict(dresidual_out=g.dres[:, :8]), dict(dx=g.dout.float()),
                dict(dpost_weight=b["dpost_weight"].bfloat16()), dict(dgate=b["dgate"][:1]), dict(dgate=b["dgate"].half())):
        with pytest.raises(ValueError):
            c(**bad)
    with pytest.raises(ValueError):
        B.SandwichNorm(512, 4, pre_weight=m.pre.float())
    with pytest.raises(B.DwdpError):
        B.SandwichNorm(512, 16, m.pre, m.post, eps=0.0).forward(m.x, out=o["out"])
