"""dwdp_lora_add against the formula in 64 bits.

Tolerance, element by element: v = s x A^T is summed in binary32 (K products:
below 2^-20 of the sum of their magnitudes for K <= 8192) and rounded to bf16
(2^-8 of it), which the second product carries to the output with |B|; the
output's own sum is binary32 (2^-20 of its magnitudes) and is rounded to bf16
(2^-8 of the result)."""
import numpy as np
import pytest
import torch

from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300 import inputs as I
from moe_expert_grouped_split_gb300.build import build

pytestmark = pytest.mark.gpu

FP32, BF16_HALF = 2.0 ** -20, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def bank(n, K, N, R, seed=0):
    a = I.randn_bf16((n, R, K), I.sqrt_inv(K), I.seed_for(seed, "a"), "cuda")
    b = I.randn_bf16((n, N, R), I.sqrt_inv(R), I.seed_for(seed, "b"), "cuda")
    return a, b, torch.linspace(0.5, 2.0, n, device="cuda")


def run(x, a, b, scale, ids, base, out=None, stream=None, status=0):
    T, K = x.shape
    n, R, _ = a.shape
    rt = B.Runtime(64, 64, 1, 1, 0, max(T, 1), 1, 0, min_ws_bytes=B.dwdp_lora_workspace_bytes(T, K, b.shape[1], R))
    rt.ws.fill_(255)  # NaN patterns: nothing may be taken from a workspace that was not written
    out = torch.full_like(base, float("nan")) if out is None else out
    torch.cuda.synchronize()
    try:
        rt.lora_add(x, a, b, scale, ids, base, out, stream)
        torch.cuda.synchronize()
        assert rt.device_status() == status
    finally:
        rt.close()
    return out


def check(out, x, a, b, scale, ids, base):
    """out within the tolerance; rows without an adapter equal base."""
    n = a.shape[0]
    none = (ids < 0) | (ids >= n)
    assert torch.equal(out[none].view(torch.int16), base[none].view(torch.int16))
    for i in torch.unique(ids[~none]).tolist():
        at = torch.nonzero(ids == i)[:, 0]
        xs, A, W, s = x[at].double(), a[i].double(), b[i].double(), float(scale[i])
        v = s * (xs @ A.t())
        want = base[at].double() + v @ W.t()
        dv = FP32 * abs(s) * (xs.abs() @ A.abs().t()) + BF16_HALF * (1 + FP32) * v.abs()
        tol = dv @ W.abs().t() + FP32 * (base[at].double().abs() + v.abs() @ W.abs().t()) + BF16_HALF * want.abs()
        off = (out[at].double() - want).abs()
        assert bool((off <= tol * (1 + 2.0 ** -7) + 1e-37).all()), float((off / (tol + 1e-37)).max())


def case(T, K, N, R, n, ids, seed=0, pad=0):
    x = I.randn_bf16((T, K + pad), 1.0, I.seed_for(seed, "x"), "cuda")[:, :K]
    base = I.randn_bf16((T, N + pad), 1.0, I.seed_for(seed, "base"), "cuda")[:, :N]
    a, b, scale = bank(n, K, N, R, seed)
    ids = torch.as_tensor(np.asarray(ids), dtype=torch.int32, device="cuda")
    return x, a, b, scale, ids, base


SIZES = [(64, 64, 16), (8, 8, 8), (1024, 512, 16), (520, 1032, 24), (2048, 1536, 64), (7168, 264, 128), (136, 7168, 32),
         (72, 200, 40)]


@pytest.mark.parametrize("K, N, R", SIZES)
@pytest.mark.parametrize("T", [1, 7, 64, 129, 300])
@pytest.mark.parametrize("order", ["one", "runs", "mixed"])
def test_sizes(T, K, N, R, order):
    n = 5
    rng = np.random.default_rng(T + K)
    ids = {"one": np.full(T, 3), "runs": np.sort(rng.integers(-1, n, T)), "mixed": rng.integers(-1, n, T)}[order]
    args = case(T, K, N, R, n, ids, seed=T)
    check(run(*args), *args)


@pytest.mark.parametrize("K, N, R", SIZES + [(72, 264, 16), (7168, 520, 16), (1000, 1000, 32)])
@pytest.mark.parametrize("T", [1153, 2048])
@pytest.mark.parametrize("order", ["one", "runs", "mixed"])
def test_sizes_of_many_tokens(K, N, R, T, order):
    test_sizes(T, K, N, R, order)


@pytest.mark.parametrize("T", [64, 200, 1000, 1300])
def test_every_token_its_own_adapter(T):
    n = 300
    ids = np.random.default_rng(T).permutation(np.resize(np.arange(n), T))
    args = case(T, 512, 256, 16, n, ids)
    check(run(*args), *args)


def test_long_batch_of_ragged_requests():
    T, n = 5003, 9
    rng = np.random.default_rng(4)
    cuts = np.sort(rng.integers(1, T, 20))
    ids = np.repeat(rng.integers(-1, n, 21), np.diff(np.concatenate([[0], cuts, [T]])))
    for R in (8, 16, 64, 128):
        args = case(T, 1024, 520, R, n, ids, seed=R)
        check(run(*args), *args)


def test_nobody_has_an_adapter():
    args = case(150, 256, 264, 16, 2, np.full(150, -1))
    assert torch.equal(run(*args), args[-1])


@pytest.mark.parametrize("T", [200, 1537])
def test_row_strides_and_in_place(T):
    K, N = 512, 768
    ids = np.random.default_rng(5).integers(-1, 4, T)
    x, a, b, scale, ids, base = case(T, K, N, 16, 4, ids, pad=512)
    wide = torch.full((T, N + 64), 5.0, dtype=torch.bfloat16, device="cuda")
    out = run(x, a, b, scale, ids, base, out=wide[:, :N])
    check(out, x, a, b, scale, ids, base)
    assert (wide[:, N:] == 5.0).all()
    full = torch.cat([base, torch.full((T, 8), 3.0, dtype=torch.bfloat16, device="cuda")], dim=1)
    same = run(x, a, b, scale, ids, full[:, :N], out=full[:, :N])
    assert torch.equal(same, out) and (full[:, N:] == 3.0).all()


@pytest.mark.parametrize("T", [40, 1200])
def test_ids_outside_the_bank_are_reported_and_skipped(T):
    n = 3
    ids = np.random.default_rng(6).integers(-1, n, T)
    ids[5], ids[30] = n, -2
    args = case(T, 256, 256, 16, n, ids)
    check(run(*args, status=-6), *args)


@pytest.mark.parametrize("T", [70, 1100])
def test_nan_stays_with_its_token_and_adapter(T):
    """A NaN in one token's row, and adapters full of NaN that no token of
    the batch uses, or that its neighbours use."""
    n = 6
    ids = np.random.default_rng(7).integers(0, 4, T)
    ids[10], ids[11] = 4, 0
    x, a, b, scale, ids, base = case(T, 256, 256, 16, n, ids)
    clean = run(x, a, b, scale, ids, base)
    x = x.clone()
    x[20, 7] = float("nan")
    a[4:] = float("nan")
    b[5] = float("inf")
    out = run(x, a, b, scale, ids, base)
    assert torch.isnan(out[20]).all() and torch.isnan(out[10]).all()
    rest = torch.ones(T, dtype=torch.bool)
    rest[[10, 20]] = False
    assert torch.equal(out[rest.cuda()], clean[rest.cuda()])


@pytest.mark.parametrize("T", [777, 3000])
def test_same_bits_every_time_and_on_another_stream(T):
    ids = np.random.default_rng(8).integers(-1, 8, T)
    args = case(T, 1024, 1032, 32, 8, ids)
    first = run(*args)
    assert torch.equal(first, run(*args)) and torch.equal(first, run(*args, stream=torch.cuda.Stream()))


def test_no_tokens_and_refusals():
    T, K, N, R, n = 8, 64, 64, 16, 2
    x, a, b, scale, ids, base = case(T, K, N, R, n, np.zeros(T))
    out = torch.zeros_like(base)
    need = B.dwdp_lora_workspace_bytes(T, K, N, R)
    rt = B.Runtime(64, 64, 1, 1, 0, T, 1, 0, min_ws_bytes=need)
    good = dict(x=x, x_stride=K, T=T, K=K, N=N, a=a, b=b, adapter_scale=scale, n_adapters=n, R=R, adapter_ids=ids,
                base=base, base_stride=N, out=out, out_stride=N, ws=rt.ws, ws_bytes=need)
    try:
        B.dwdp_lora_add(rt.ctx, **dict(good, T=0))
        bad = [(dict(T=-1), -1), (dict(n_adapters=0), -1), (dict(K=60), -5), (dict(N=12), -5), (dict(R=12), -5),
               (dict(R=136), -5), (dict(R=0), -5), (dict(x_stride=56), -1), (dict(x_stride=68), -1),
               (dict(base_stride=32), -1), (dict(out_stride=65), -1), (dict(ws_bytes=need - 1), -1), (dict(ws=None), -1),
               (dict(out=base, out_stride=N + 8), -1)]
        bad += [({name: None}, -1) for name in ("x", "a", "b", "adapter_scale", "adapter_ids", "base", "out")]
        bad += [({name: good[name].data_ptr() + 4}, -1) for name in ("x", "a", "b", "adapter_ids", "base", "out", "ws")]
        for change, code in bad:
            with pytest.raises(B.DwdpError) as ei:
                B.dwdp_lora_add(rt.ctx, **dict(good, **change))
            assert ei.value.code == code, change
        torch.cuda.synchronize()
        assert rt.device_status() == 0 and (out == 0).all()
    finally:
        rt.close()


@pytest.mark.parametrize("T", [1, 40, 1100])
def test_row_strides_beyond_2_to_31_elements(T):
    K, N, n = 512, 520, 4
    stride = ((1 << 31) // max(T - 8, 1) + 7) // 8 * 8
    x, a, b, scale, ids, base = case(T, K, N, 16, n, np.random.default_rng(9).integers(-1, n, T))
    far = [torch.empty((T - 1) * stride + w, dtype=torch.bfloat16, device="cuda").as_strided((T, w), (stride, 1))
           for w in (K, N, N)]
    far[0].copy_(x)
    far[1].copy_(base)
    assert torch.equal(run(far[0], a, b, scale, ids, far[1], out=far[2]), run(x, a, b, scale, ids, base))
    check(far[2], x, a, b, scale, ids, base)


@pytest.mark.parametrize("T", [1, 40, 1100])
def test_bank_beyond_2_to_31_elements(T):
    K = N = 8192
    n, used = (1 << 31) // (16 * K) + 6, 4
    x, some_a, some_b, _, few, base = case(T, K, N, 16, used, np.random.default_rng(10).integers(0, used, T))
    a = torch.empty((n, 16, K), dtype=torch.bfloat16, device="cuda")
    b = torch.empty((n, N, 16), dtype=torch.bfloat16, device="cuda")
    a[-used:], b[-used:] = some_a, some_b
    scale, ids = torch.linspace(0.5, 2.0, n, device="cuda"), few + (n - used)
    check(run(x, a, b, scale, ids, base), x, a, b, scale, ids, base)


def test_bank_of_too_many_rows_is_refused():
    x, a, b, scale, ids, base = case(4, 64, 64, 16, 1, [0] * 4)
    rt = B.Runtime(64, 64, 1, 1, 0, 4, 1, 0, min_ws_bytes=B.dwdp_lora_workspace_bytes(4, 64, 64, 16))
    try:
        with pytest.raises(B.DwdpError) as ei:
            B.dwdp_lora_add(rt.ctx, x=x, x_stride=64, T=4, K=64, N=64, a=a, b=b, adapter_scale=scale,
                            n_adapters=1 << 27, R=16, adapter_ids=ids, base=base, base_stride=64,
                            out=torch.empty_like(base), out_stride=64, ws=rt.ws, ws_bytes=rt.ws.numel())
        assert ei.value.code == -5
    finally:
        rt.close()


@pytest.mark.parametrize("K, N, R", SIZES + [(72, 264, 16), (7168, 520, 16), (1000, 1000, 32)])
@pytest.mark.parametrize("T", [2049, 2200])
@pytest.mark.parametrize("order", ["one", "runs", "mixed"])
def test_sizes_of_more_tokens(K, N, R, T, order):
    test_sizes(T, K, N, R, order)


@pytest.mark.parametrize("T, K, N", [(1024, 8192, 8192), (1023, 8192, 8200), (1100, 8, 16384)])
@pytest.mark.parametrize("order", ["runs", "mixed"])
def test_wide_rows_around_a_thousand_tokens(T, K, N, order):
    test_sizes(T, K, N, 16, order)


def test_many_strided_tokens_in_place():
    test_row_strides_and_in_place(2500)


def test_many_tokens_with_bad_ids():
    test_ids_outside_the_bank_are_reported_and_skipped(2300)


def test_nan_among_many_tokens():
    test_nan_stays_with_its_token_and_adapter(2300)


def test_many_tokens_each_its_own_adapter():
    test_every_token_its_own_adapter(2100)


@pytest.mark.parametrize("n", [3, 255, 256])
@pytest.mark.parametrize("T", [39, 64, 65, 129, 257, 1000, 2047, 2048])
def test_any_order_of_tokens(T, n):
    ids = np.random.default_rng(T + n).integers(-1, n, T)
    ids[-1] = n - 1
    args = case(T, 520, 296, 16, n, ids, seed=T)
    check(run(*args), *args)
    base = args[-1].clone()
    assert torch.equal(run(*args[:-1], base, out=base), run(*args))


@pytest.mark.parametrize("N", [80000, 131072])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 17])
def test_few_tokens_of_a_vocabulary_projection(T, N):
    """Columns enough for the wide expand tiles although the tokens are few."""
    for R in (16, 64):
        args = case(T, 64, N, R, 4, np.random.default_rng(T).integers(-1, 4, T), seed=T + R)
        check(run(*args), *args)


@pytest.mark.parametrize("R", [8, 16, 24, 64, 128])
@pytest.mark.parametrize("T", [2049, 2100])
def test_lanes_of_a_warp_with_different_adapters(T, R):
    """Each of a warp's 32 rows keeps another adapter's columns than its
    neighbours, in every group of adapters the tile goes through."""
    for ids in (np.arange(T) % 32, np.where(np.arange(T) % 3 == 0, -1, np.arange(T) % 7)):
        args = case(T, 264, 136, R, 32, ids, seed=R)
        check(run(*args), *args)
