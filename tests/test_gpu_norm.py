"""dwdp_add_rmsnorm against the formula in 64 bits.

Tolerances: a rounding to bf16 is off by at most 2^-8 of the value, to E4M3 by
2^-4 of it or half a subnormal step (2^-10); what precedes it is binary32
(a tree sum of up to 32768 squares, a division, a square root and three
products: below 2^-17 together)."""
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


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def formula(x, r, w, eps=EPS):
    h = f64(x) + (f64(r) if r is not None else 0.0)
    y = h / np.sqrt((h * h).mean(axis=1) + eps)[:, None] * f64(w)
    m = np.abs(y).max(axis=1)
    return h, y, np.where(m > 0, m / 448.0, 1.0)


def call(x, w, r=None, codes=True, eps=EPS, stream=None):
    rows, H = x.shape
    o = dict(out=torch.full((rows, H), float("nan"), dtype=torch.bfloat16, device="cuda"))
    if r is not None:
        o["residual_out"] = torch.full_like(o["out"], float("nan"))
    if codes:
        o["codes"] = torch.full((rows, H), 0x7F, dtype=torch.uint8, device="cuda")
        o["row_scale"] = torch.full((rows,), float("nan"), device="cuda")
    torch.cuda.synchronize()
    B.dwdp_add_rmsnorm(x, rows, H, w, eps, residual=r, x_stride=x.stride(0), stream=stream, **o)
    torch.cuda.synchronize()
    return o


def check(o, x, w, r=None, eps=EPS):
    h, y, scale = formula(x, r, w, eps)
    assert (np.abs(f64(o["out"]) - y) <= (BF16_HALF + FP32) * np.abs(y) + 1e-38).all()
    if r is not None:
        assert (np.abs(f64(o["residual_out"]) - h) <= (BF16_HALF + FP32) * np.abs(h) + 1e-38).all()
    if "codes" in o:
        s = f64(o["row_scale"])
        assert (np.abs(s - scale) <= FP32 * scale).all()
        q = y / scale[:, None]
        c = f64(o["codes"].view(torch.float8_e4m3fn))
        assert (np.abs(c - q) <= (E4M3_HALF + FP32) * np.abs(q) + E4M3_SUB * (1 + FP32)).all()


@pytest.mark.parametrize("H", [8, 64, 520, 1536, 7168, 8200, 16384, 32768])
@pytest.mark.parametrize("rows", [1, 3, 333])
@pytest.mark.parametrize("residual, codes", [(False, False), (False, True), (True, False), (True, True)])
def test_rows(rows, H, residual, codes):
    x = I.randn_bf16((rows, H), 1.0, I.seed_for(1, rows, H), "cuda")
    r = I.randn_bf16((rows, H), 4.0, I.seed_for(2, rows, H), "cuda") if residual else None
    w = I.randn_bf16((H,), 1.0, I.seed_for(3, H), "cuda")
    check(call(x, w, r, codes), x, w, r)


@pytest.mark.parametrize("rows, H", [(5000, 1024), (2500, 512), (2501, 264), (2100, 7168), (2100, 6152), (2049, 8192)])
def test_many_rows(rows, H):
    x = I.randn_bf16((rows, H), 1.0, 5, "cuda")
    r = I.randn_bf16((rows, H), 4.0, 6, "cuda")
    w = I.randn_bf16((H,), 1.0, 7, "cuda")
    check(call(x, w, r), x, w, r)


def test_row_stride_and_nothing_between_the_rows_is_touched():
    rows, H, wide = 77, 512, 576 + 512
    buf = I.randn_bf16((rows, wide), 1.0, 8, "cuda")
    buf[:, H:] = float("nan")
    before = buf.view(torch.int16).clone()
    w = I.randn_bf16((H,), 1.0, 9, "cuda")
    check(call(buf[:, :H], w), buf[:, :H], w)
    assert torch.equal(buf.view(torch.int16), before)


def test_in_place():
    rows, H = 300, 7168
    x = I.randn_bf16((rows, H), 1.0, 10, "cuda")
    r = I.randn_bf16((rows, H), 4.0, 11, "cuda")
    w = I.randn_bf16((H,), 1.0, 12, "cuda")
    apart = call(x, w, r)
    x2, r2 = x.clone(), r.clone()
    codes, scale = torch.empty_like(apart["codes"]), torch.empty_like(apart["row_scale"])
    B.dwdp_add_rmsnorm(x2, rows, H, w, EPS, x2, residual=r2, residual_out=r2, codes=codes, row_scale=scale)
    torch.cuda.synchronize()
    assert torch.equal(x2, apart["out"]) and torch.equal(r2, apart["residual_out"])
    assert torch.equal(codes, apart["codes"]) and torch.equal(scale, apart["row_scale"])


def test_zero_rows_and_zero_weights():
    H = 256
    x = torch.zeros((3, H), dtype=torch.bfloat16, device="cuda")
    x[1] = 2.0
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    o = call(x, w)
    assert (o["out"][[0, 2]] == 0).all() and (o["codes"][[0, 2]] == 0).all()
    assert o["row_scale"][0] == 1.0 and o["row_scale"][2] == 1.0
    check(o, x, w)
    o = call(x, torch.zeros_like(w))
    assert (o["out"] == 0).all() and (o["row_scale"] == 1.0).all()


@pytest.mark.parametrize("rows, H", [(2200, 512), (2200, 7168), (3, 8), (40, 32768)])
def test_squares_beyond_the_range_in_every_kernel(rows, H):
    x = I.randn_bf16((rows, H), 1.0, 20, "cuda")
    x[::3] *= 1e30
    x[1::7, 0] = -3e38
    w = I.randn_bf16((H,), 1.0, 21, "cuda")
    o = call(x, w)
    h, y, scale = formula(x, None, w)
    assert (np.abs(f64(o["out"]) - y) <= (BF16_HALF + FP32) * np.abs(y) + 1e-38).all()
    assert (np.abs(f64(o["row_scale"]) - scale) <= FP32 * scale).all()


def test_range_ends():
    """Rows whose squares pass binary32's range, rows of tiny values (eps then
    decides), and one huge element among ordinary ones."""
    H = 1024
    x = I.randn_bf16((5, H), 1.0, 13, "cuda")
    x[0] *= 1e30
    x[1] = 3e38
    x[2] *= 1e-30
    x[3, 7] = 1e25
    w = I.randn_bf16((H,), 1.0, 14, "cuda")
    o = call(x, w)
    h, y, scale = formula(x, None, w)
    for row in (0, 1, 3, 4):
        got = f64(o["out"][row])
        assert (np.abs(got - y[row]) <= (BF16_HALF + FP32) * np.abs(y[row]) + 1e-38).all(), row
        assert abs(f64(o["row_scale"])[row] - scale[row]) <= FP32 * scale[row]
    # a row below 2^-100 times nothing: quantized with a scale of its own
    assert (np.abs(f64(o["out"][2]) - y[2]) <= (BF16_HALF + FP32) * np.abs(y[2]) + 1e-38).all()
    back = f64(o["codes"].view(torch.float8_e4m3fn))[2] * f64(o["row_scale"])[2]
    assert (np.abs(back - y[2]) <= (E4M3_HALF + FP32) * np.abs(y[2]) + (E4M3_SUB + FP32) * f64(o["row_scale"])[2]).all()


def test_nan_and_inf_stay_in_their_rows():
    H = 512
    x = I.randn_bf16((4, H), 1.0, 15, "cuda")
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    o = call(x, w)
    assert torch.isnan(o["out"][1]).all() and torch.isnan(o["row_scale"][1])
    assert torch.isnan(o["out"][2, 5])
    clean = call(x[[0, 3]].contiguous(), w)
    for name in ("out", "codes", "row_scale"):
        assert torch.equal(o[name][[0, 3]], clean[name])


def test_same_bits_every_time_and_on_another_stream():
    x = I.randn_bf16((513, 7168), 1.0, 16, "cuda")
    r = I.randn_bf16((513, 7168), 1.0, 17, "cuda")
    w = I.randn_bf16((7168,), 1.0, 18, "cuda")
    a, b = call(x, w, r), call(x, w, r, stream=torch.cuda.Stream())
    for name in a:
        assert torch.equal(a[name], b[name])


@pytest.mark.parametrize("H", [512, 4096, 8192])
def test_rows_beyond_2_to_31_elements(H):
    rows, last = (1 << 31) // H + 20, 30
    x, r = (torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[-last:] = I.randn_bf16((last, H), 1.0, 20, "cuda")
    r[-last:] = I.randn_bf16((last, H), 4.0, 21, "cuda")
    w = I.randn_bf16((H,), 1.0, 22, "cuda")
    o = call(x, w, r)
    check({name: t[-last:] for name, t in o.items()}, x[-last:], w, r[-last:])
    assert not o["out"][:100].any() and (o["row_scale"][:100] == 1).all()


def test_row_stride_beyond_2_to_31_elements():
    rows, H, stride = 9, 512, (1 << 28) + 8
    x = torch.empty(8 * stride + H, dtype=torch.bfloat16, device="cuda").as_strided((rows, H), (stride, 1))
    x.copy_(I.randn_bf16((rows, H), 1.0, 23, "cuda"))
    w = I.randn_bf16((H,), 1.0, 24, "cuda")
    check(call(x, w), x, w)


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("rows, H", [(5000, 1024), (2500, 512), (2501, 1000), (2100, 7168), (2100, 6152), (2049, 8192),
                                     (1300, 904), (2000, 1032)])
def test_many_rows_without_a_residual(rows, H, codes):
    x = I.randn_bf16((rows, H), 1.0, 25, "cuda")
    w = I.randn_bf16((H,), 1.0, 26, "cuda")
    check(call(x, w, codes=codes), x, w)


@pytest.mark.parametrize("rows, H", [(2200, 904), (2200, 7168), (2200, 8192)])
def test_squares_beyond_the_range_without_a_residual(rows, H):
    x = I.randn_bf16((rows, H), 1.0, 27, "cuda")
    x[3::7] *= 2.0 ** 100
    w = I.randn_bf16((H,), 1.0, 28, "cuda")
    check(call(x, w), x, w)


def test_nan_and_inf_stay_in_their_rows_of_many():
    rows, H = 2200, 7168
    x = I.randn_bf16((rows, H), 1.0, 29, "cuda")
    w = I.randn_bf16((H,), 1.0, 30, "cuda")
    clean = call(x, w)
    x[5, 17], x[2000, 3] = float("nan"), float("inf")
    o = call(x, w)
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[5] = rest[2000] = False
    assert torch.isnan(o["out"][5]).all() and torch.isnan(o["row_scale"][5])
    for name in o:
        a, b = o[name][rest], clean[name][rest]
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_two_threads_with_different_widths():
    """The same kernel with other sizes of shared memory from two host
    threads: neither call is refused."""
    import threading

    failed = []
    made = []
    for H in (6400, 8192):
        x = I.randn_bf16((2000, H), 1.0, H, "cuda")
        made.append((x, torch.ones(H, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(x, w, out, stream):
        try:
            for i in range(3000):
                B.dwdp_add_rmsnorm(x, x.shape[0], x.shape[1], w, EPS, out, stream=stream)
                if i % 500 == 499:
                    stream.synchronize()
        except B.DwdpError as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=m) for m in made]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed[0]


# rows and widths that run every kernel, with and without a residual
EVERY_KERNEL = [(2200, 512), (2200, 904), (2200, 7168), (3, 8), (130, 7168), (40, 32768)]


@pytest.mark.parametrize("rows, H", EVERY_KERNEL)
@pytest.mark.parametrize("residual, codes", [(False, False), (False, True), (True, True)])
def test_squares_below_the_range(rows, H, residual, codes):
    """Without an eps that carries them: rows whose squares binary32 does not
    hold, down to the smallest values of bf16, among ordinary ones."""
    x = I.randn_bf16((rows, H), 1.0, 31, "cuda")
    r = I.randn_bf16((rows, H), 1.0, 32, "cuda") if residual else None
    for t in (x, r) if residual else (x,):
        t[0] *= 2.0 ** -100
        t[1::4] *= 2.0 ** -75
        t[2::8] *= 2.0 ** -124          # the upper end of bf16's own subnormal values
    w = I.randn_bf16((H,), 1.0, 33, "cuda")
    for eps in (0.0, 1e-38):
        check(call(x, w, r, codes, eps), x, w, r, eps)


@pytest.mark.parametrize("rows, H", EVERY_KERNEL)
def test_codes_of_weights_at_the_ends_of_the_range(rows, H):
    """Rows and weights whose products leave binary32's range although their
    norm does not, and rows beyond the range of squares with small weights."""
    for x_exp, w_exp in ((65, -95), (40, 100), (-40, -55), (100, 20), (-90, 110)):
        x = I.randn_bf16((rows, H), 1.0, 34, "cuda") * 2.0 ** x_exp
        w = I.randn_bf16((H,), 1.0, 35, "cuda") * 2.0 ** w_exp
        check(call(x, w, eps=0.0), x, w, eps=0.0)


@pytest.mark.parametrize("rows, H", EVERY_KERNEL)
def test_zero_rows_without_eps(rows, H):
    x = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    x[1] = 2.0 ** -120
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    o = call(x, w, eps=0.0)
    zero = [t for t in range(rows) if t != 1]
    assert (o["codes"][zero] == 0).all() and (o["row_scale"][zero] == 1).all()
    assert torch.isnan(o["out"][zero].float()).all()        # 0 / 0
    assert (o["out"][1] == 1).all()
