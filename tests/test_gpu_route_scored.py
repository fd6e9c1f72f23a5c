"""dwdp_route_scored: the logits against x W^T in 64 bits, and everything that
follows them against the formulas in 64 bits on the returned fp32 logits.

The chosen ids have to be equal for every token (the call promises the choice
of the formulas in binary64); weights are a few binary32 operations on the
chosen logits: within 2^-19 of their value, exponents of up to 2^7 adding
2^-24 * 2^7 = 2^-17 more."""
import numpy as np
import pytest
import torch

from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300 import inputs as I
from moe_expert_grouped_split_gb300.build import build

pytestmark = pytest.mark.gpu

W_TOL = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def formula(z, bias, how, k):
    """(ids ascending, weights, choice values) of fp32 logits z in 64 bits."""
    z = z.astype(np.float64)
    T, E = z.shape
    e = np.exp(-np.abs(z))
    if how.score == B.SCORE_SIGMOID:
        s = np.where(z >= 0, 1.0, e) / (1.0 + e)
    else:
        s = np.exp(z - z.max(axis=1, keepdims=True))
        s = s / s.sum(axis=1, keepdims=True)
    c = s if bias is None else s + bias.astype(np.float64)
    G = how.n_groups
    left = c
    if how.top_groups < G:
        by = np.sort(c.reshape(T, G, E // G), axis=2)
        v = by[:, :, -1]
        if how.group_score == B.GROUP_TOP2 and E // G > 1:
            v = by[:, :, -1] + by[:, :, -2]
        kept = np.argsort(-v, axis=1, kind="stable")[:, :how.top_groups]
        in_kept = np.zeros((T, G), bool)
        np.put_along_axis(in_kept, kept, True, axis=1)
        mask = np.repeat(in_kept, E // G, axis=1)
    else:
        mask = np.ones((T, E), bool)
    ids = np.empty((T, k), np.int64)
    for t in range(T):
        at = np.nonzero(mask[t])[0]
        ids[t] = np.sort(at[np.argsort(-left[t, at], kind="stable")[:k]])
    w = np.take_along_axis(s, ids, axis=1)
    if bias is not None:
        w = np.where(np.isneginf(bias[ids]), 0.0, w)
    if how.renormalize:
        total = w.sum(axis=1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return ids, w * np.float64(np.float32(how.scale)), c


def route(T, H, E, k, how, x=None, wr=None, bias=None, seed=0, std=None, keep_logits=True, status=0):
    rt = B.Runtime(H, 64, E, k, 0, T, 1, 0)
    try:
        if x is None:
            x = I.make_tokens(T, H, seed).cuda()
        if wr is None:
            wr = I.randn_bf16((E, H), std or I.sqrt_inv(H), I.seed_for(seed, "Wr")).cuda()
        rb = B.RouteBuffers(T, E, k, keep_logits=keep_logits)
        for t in (rb.topk_ids, rb.counts, rb.offsets, rb.perm, rb.inv_perm):
            t.fill_(-7)
        rb.topk_w.fill_(float("nan"))
        torch.cuda.synchronize()
        rt.route_scored(x, wr, torch.from_numpy(bias).cuda() if bias is not None else None, how, rb)
        torch.cuda.synchronize()
        assert rt.device_status() == status
        return x, wr, rb
    finally:
        rt.close()


def check(T, E, k, how, bias, rb):
    z = rb.logits.cpu().numpy()
    ids, w, _ = formula(z, bias, how, k)
    got = rb.topk_ids.cpu().numpy()
    bad = np.nonzero((got != ids).any(axis=1))[0]
    assert bad.size == 0, f"{bad.size} of {T} tokens, first {bad[0]}: {got[bad[0]]} for {ids[bad[0]]}"
    dw = np.abs(rb.topk_w.cpu().numpy().astype(np.float64) - w)
    assert (dw <= W_TOL * w + 1e-37).all(), dw.max()
    flat = ids.reshape(-1)
    counts = np.bincount(flat, minlength=E)
    perm = np.argsort(flat, kind="stable")
    inv = np.empty_like(perm)
    inv[perm] = np.arange(T * k)
    assert np.array_equal(rb.counts.cpu().numpy(), counts)
    assert np.array_equal(rb.offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(counts)]))
    assert np.array_equal(rb.perm.cpu().numpy(), perm) and np.array_equal(rb.inv_perm.cpu().numpy(), inv)


def how_of(score, G=1, top=1, gs=B.GROUP_MAX, renorm=True, scale=1.0):
    return B.scoring(score, G, top, gs, renorm, scale)


SIG, SOFT = B.SCORE_SIGMOID, B.SCORE_SOFTMAX
CASES = [
    # T, H, E, k, how, biased
    (1, 7168, 256, 8, how_of(SIG, 8, 4, B.GROUP_TOP2, True, 2.5), True),
    (2, 7168, 256, 8, how_of(SIG, 8, 4, B.GROUP_TOP2, True, 2.5), True),
    (17, 7168, 256, 8, how_of(SIG, 8, 4, B.GROUP_TOP2, True, 2.5), True),
    (64, 1024, 256, 8, how_of(SIG, 8, 4, B.GROUP_TOP2, True, 2.5), True),
    (129, 1024, 256, 8, how_of(SIG, 8, 4, B.GROUP_TOP2, True, 2.5), True),
    (1003, 512, 256, 8, how_of(SIG, 8, 4, B.GROUP_TOP2, True, 2.5), True),
    (4099, 256, 256, 8, how_of(SIG, 8, 4, B.GROUP_TOP2, False, 1.0), True),
    (300, 512, 160, 6, how_of(SOFT, 8, 3, B.GROUP_MAX, False, 16.0), False),
    (300, 512, 160, 6, how_of(SOFT, 8, 3, B.GROUP_TOP2, True, 1.0), True),
    (77, 128, 64, 6, how_of(SOFT), False),
    (77, 128, 64, 1, how_of(SOFT, renorm=False), False),
    (77, 128, 60, 4, how_of(SIG), True),
    (50, 128, 300, 16, how_of(SIG, 5, 2, B.GROUP_TOP2), True),
    (40, 128, 1020, 32, how_of(SIG, 17, 9, B.GROUP_TOP2), True),
    (40, 128, 1024, 32, how_of(SOFT, 32, 2, B.GROUP_MAX), True),
    (40, 128, 1024, 32, how_of(SOFT), False),
    (40, 128, 992, 3, how_of(SIG, 31, 1, B.GROUP_TOP2), False),
    (9, 64, 32, 2, how_of(SIG, 32, 2, B.GROUP_TOP2), True),      # groups of one expert
    (9, 64, 8, 8, how_of(SIG, 4, 4, B.GROUP_TOP2), True),        # everything is chosen
    (9, 64, 8, 4, how_of(SOFT, 4, 2, B.GROUP_TOP2), True),       # everything in the kept groups
    (5, 64, 1, 1, how_of(SIG), False),
    (17003, 64, 64, 8, how_of(SIG, 8, 4, B.GROUP_TOP2), True),   # more chunks of pairs than the placing blocks sum up
    (129, 7168, 256, 8, how_of(SIG, 8, 4, B.GROUP_TOP2), True),
    (255, 576, 40, 3, how_of(SOFT), True),
    (31, 7168, 24, 3, how_of(SIG), False),
    (700, 7168, 512, 8, how_of(SIG, 8, 4, B.GROUP_TOP2), True),
    (33, 64, 7, 3, how_of(SOFT, 7, 3, B.GROUP_MAX), False),
    (1100, 7168, 256, 8, how_of(SIG, 8, 4, B.GROUP_TOP2, True, 2.5), True),
    (1024, 64, 256, 8, how_of(SIG, 8, 4, B.GROUP_TOP2, True, 2.5), True),     # the most pairs one kernel takes
    (1025, 64, 256, 8, how_of(SIG, 8, 4, B.GROUP_TOP2, True, 2.5), True),
    (256, 64, 1024, 32, how_of(SOFT), True),
    (257, 64, 1024, 32, how_of(SOFT, 16, 9, B.GROUP_TOP2), True),
    (8191, 64, 48, 1, how_of(SIG, 3, 1, B.GROUP_MAX), True),
    (8193, 64, 48, 1, how_of(SIG, 3, 1, B.GROUP_MAX), True),
    (3, 64, 1020, 32, how_of(SIG, 17, 9, B.GROUP_TOP2), True),
    (3001, 576, 72, 6, how_of(SOFT, 8, 3, B.GROUP_MAX), True),
    (1030, 192, 300, 7, how_of(SIG, 3, 2, B.GROUP_TOP2), True),
    (2305, 128, 64, 6, how_of(SOFT, renorm=False), False),
    (9000, 64, 16, 2, how_of(SOFT, 4, 2, B.GROUP_TOP2), False),
]


@pytest.mark.parametrize("T, H, E, k, how, biased", CASES,
                         ids=[f"T{c[0]}_H{c[1]}_E{c[2]}_k{c[3]}_G{c[4].n_groups}" + f"_{i}" for i, c in enumerate(CASES)])
def test_routes_as_the_formulas_say(T, H, E, k, how, biased):
    bias = np.random.default_rng(E + k).normal(0, 0.1, E).astype(np.float32) if biased else None
    x, wr, rb = route(T, H, E, k, how, bias=bias, seed=T + E)
    z = rb.logits.cpu().numpy().astype(np.float64)
    ref = (x.double() @ wr.double().t()).cpu().numpy()
    # fp32 sums of H products: each step off by 2^-24 of a partial sum at most
    mag = (x.double().abs() @ wr.double().abs().t()).cpu().numpy()
    assert (np.abs(z - ref) <= 2.0 ** -24 * np.sqrt(H) * mag + 1e-30).all()
    check(T, E, k, how, bias, rb)
    _, _, again = route(T, H, E, k, how, x=x, wr=wr, bias=bias, keep_logits=False)
    for name in ("topk_ids", "topk_w", "counts", "offsets", "perm", "inv_perm"):
        assert torch.equal(getattr(rb, name), getattr(again, name)), name


@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("G, top", [(1, 1), (4, 2)])
def test_equal_scores_tie_to_the_lowest_group_and_id(score, G, top):
    T, H, E, k = 37, 128, 64, 6
    wr = torch.zeros((E, H), dtype=torch.bfloat16, device="cuda")
    how = how_of(score, G, top, B.GROUP_TOP2)
    _, _, rb = route(T, H, E, k, how, wr=wr)
    assert (rb.topk_ids.cpu().numpy() == np.arange(k)).all()
    check(T, E, k, how, None, rb)


@pytest.mark.parametrize("std", [0.5, 3.0, 20.0])
@pytest.mark.parametrize("score", [SIG, SOFT])
def test_saturated_scores(score, std):
    """Logits so far out that binary32 scores are 0 or 1 for many experts."""
    T, H, E, k = 200, 128, 64, 6
    for how in (how_of(score, 4, 2, B.GROUP_TOP2), how_of(score, renorm=False)):
        _, _, rb = route(T, H, E, k, how, std=std, seed=3)
        check(T, E, k, how, None, rb)


def test_choices_next_to_each_other():
    """Biases that differ by less than binary32's rounding of a score: the
    decision is the one in 64 bits."""
    T, H, E, k = 400, 128, 64, 6
    rng = np.random.default_rng(1)
    bias = (rng.integers(0, 3, E) * 1e-8).astype(np.float32)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.from_numpy(rng.integers(-3, 4, T).astype(np.float32)).cuda()
    wr = torch.zeros((E, H), dtype=torch.bfloat16, device="cuda")
    wr[:, 0] = torch.from_numpy(rng.integers(-1, 2, E).astype(np.float32)).cuda()
    for how in (how_of(SIG), how_of(SIG, 8, 3, B.GROUP_TOP2), how_of(SOFT, 8, 3, B.GROUP_MAX)):
        _, _, rb = route(T, H, E, k, how, x=x, wr=wr, bias=bias)
        check(T, E, k, how, bias, rb)


def test_experts_taken_out():
    T, H, E, k = 100, 128, 32, 4
    rng = np.random.default_rng(2)
    for left, G, top in ((20, 1, 1), (20, 4, 2), (2, 1, 1), (0, 1, 1), (0, 4, 2)):
        bias = np.full(E, -np.inf, np.float32)
        bias[rng.permutation(E)[:left]] = rng.normal(0, 0.1, left)
        for renorm in (True, False):
            how = how_of(SIG, G, top, B.GROUP_MAX, renorm, 2.5)
            _, _, rb = route(T, H, E, k, how, bias=bias)
            check(T, E, k, how, bias, rb)
            w = rb.topk_w.cpu().numpy()
            assert (w[np.isneginf(bias[rb.topk_ids.cpu().numpy()])] == 0).all()


def test_non_finite_logits_and_biases_are_reported():
    T, H, E, k = 200, 256, 16, 4
    x = I.make_tokens(T, H, 9).cuda()
    x[17, 3] = float("nan")
    how = how_of(SIG, 4, 2, B.GROUP_TOP2)
    x, wr, rb = route(T, H, E, k, how, x=x, status=-6)
    ids = rb.topk_ids.cpu().numpy()
    assert all(len(set(r.tolist())) == k and r.min() >= 0 and r.max() < E for r in ids)
    clean = x.clone()
    clean[17, 3] = 0.0
    _, _, ok = route(T, H, E, k, how, x=clean, wr=wr)
    good = np.arange(T) != 17
    assert np.array_equal(ids[good], ok.topk_ids.cpu().numpy()[good])
    for v in (float("nan"), float("inf")):
        bias = np.zeros(E, np.float32)
        bias[5] = v
        _, _, rb = route(T, H, E, k, how, x=clean, wr=wr, bias=bias, status=-6)
        assert all(len(set(r.tolist())) == k for r in rb.topk_ids.cpu().numpy())


def test_no_tokens():
    rt = B.Runtime(256, 64, 16, 4, 0, 8, 1, 0)
    rb = B.RouteBuffers(0, 16, 4)
    rb.counts.fill_(3)
    rb.offsets.fill_(3)
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    rt.route_scored(x, torch.zeros((16, 256), dtype=torch.bfloat16, device="cuda"), None, how_of(SIG), rb)
    torch.cuda.synchronize()
    assert (rb.counts == 0).all() and (rb.offsets == 0).all()
    rt.close()


def test_refusals():
    T, H, E, k = 8, 256, 16, 4
    rt = B.Runtime(H, 64, E, k, 0, T, 1, 0)
    try:
        x = I.make_tokens(T, H, 1).cuda()
        wr = I.randn_bf16((E, H), 0.02, 2).cuda()
        rb = B.RouteBuffers(T, E, k)
        bad = [(how_of(2), -1), (how_of(SIG, 0, 1), -1), (how_of(SIG, 3, 1), -1), (how_of(SIG, 4, 0), -1),
               (how_of(SIG, 4, 5), -1), (how_of(SIG, 8, 1), -1), (how_of(SIG, 1, 1, 2), -1),
               (how_of(SIG, scale=0.0), -1), (how_of(SIG, scale=float("nan")), -1),
               (how_of(SIG, scale=float("inf")), -1), (how_of(SIG, scale=-1.0), -1)]
        for how, code in bad:
            with pytest.raises(B.DwdpError) as ei:
                rt.route_scored(x, wr, None, how, rb)
            assert ei.value.code == code
        how = how_of(SIG)
        how.renormalize = 2
        with pytest.raises(B.DwdpError):
            rt.route_scored(x, wr, None, how, rb)
        for args in ((x.cpu().pin_memory(), wr, None), (x, wr.cpu().pin_memory(), None), (None, wr, None)):
            with pytest.raises(B.DwdpError) as ei:
                B.dwdp_route_scored(rt.ctx, args[0], T, args[1], args[2], how_of(SIG), rb.c, rt.ws, rt.ws_bytes)
            assert ei.value.code == -1
        with pytest.raises(B.DwdpError):
            B.dwdp_route_scored(rt.ctx, x, T + 1, wr, None, how_of(SIG), rb.c, rt.ws, rt.ws_bytes)
        with pytest.raises(B.DwdpError):
            B.dwdp_route_scored(rt.ctx, x, T, wr, None, how_of(SIG), rb.c, rt.ws, 16)
        torch.cuda.synchronize()
        assert rt.device_status() == 0
    finally:
        rt.close()
    big = B.Runtime(256, 64, 64, 1, 0, T, 1, 0)
    try:
        with pytest.raises(B.DwdpError) as ei:
            big.route_scored(x, torch.zeros((64, 256), dtype=torch.bfloat16, device="cuda"), None,
                             how_of(SIG, 64, 1), B.RouteBuffers(T, 64, 1))
        assert ei.value.code == -5
    finally:
        big.close()


@pytest.mark.parametrize("H, E, k", [(64, 1020, 1), (7168, 256, 8), (2048, 60, 4)])
def test_workspace_of_more_tokens_is_enough_for_fewer(H, E, k):
    rt = B.Runtime(H, 64, E, k, 0, 30000, 1, 0)
    try:
        need = [B.lib().dwdp_workspace_bytes(rt.ctx, T) for T in list(range(1, 5000, 3)) + list(range(5000, 30000, 101))]
        assert need == sorted(need)
    finally:
        rt.close()


@pytest.mark.parametrize("T, H, E", [(600, 320, 148), (300, 64, 300), (1100, 1024, 20), (65, 576, 1020)])
def test_logits_of_experts_that_are_no_whole_sectors(T, H, E):
    x = I.randn_bf16((T, H), 1.0, 41, "cuda")
    w = I.randn_bf16((E, H), I.sqrt_inv(H), 42, "cuda")
    rt, rb = B.Runtime(H, 64, E, 4, 0, T, 1, 0), B.RouteBuffers(T, E, 4, keep_logits=True)
    rb.logits.fill_(float("nan"))
    try:
        rt.route_scored(x, w, None, how_of(SIG), rb)
        torch.cuda.synchronize()
        assert rt.device_status() == 0
    finally:
        rt.close()
    want = x.double() @ w.double().t()
    # binary32 sums of H products
    assert bool(((rb.logits.double() - want).abs() <= 2.0 ** -20 * (x.double().abs() @ w.double().abs().t())).all())
    best = rb.logits.topk(4, dim=1).indices.sort(dim=1).values
    assert torch.equal(best.int(), rb.topk_ids[:T])


@pytest.mark.parametrize("E, G, top, gs", [(64, 1, 1, B.GROUP_MAX), (256, 1, 1, B.GROUP_MAX), (256, 8, 4, B.GROUP_MAX),
                                           (256, 8, 4, B.GROUP_TOP2), (300, 5, 2, B.GROUP_TOP2),
                                           (1020, 1, 1, B.GROUP_MAX), (1020, 17, 9, B.GROUP_TOP2)])
@pytest.mark.parametrize("T", [1, 37, 300])
def test_experts_taken_out_fill_up_from_the_lowest_id(T, E, G, top, gs):
    """Lanes of several experts: fewer than k others are left, or none, and
    what fills the choice up goes by id."""
    H, k = 64, 8
    rng = np.random.default_rng(E + G)
    for left in (0, 1, 3, k - 1, 2 * k):
        bias = np.full(E, -np.inf, np.float32)
        bias[rng.permutation(E)[:left]] = rng.normal(0, 0.1, left)
        for score, renorm in ((SIG, True), (SOFT, False)):
            how = how_of(score, G, top, gs, renorm, 2.5)
            _, _, rb = route(T, H, E, k, how, bias=bias, seed=left)
            check(T, E, k, how, bias, rb)


@pytest.mark.parametrize("E, G, top", [(256, 8, 4), (128, 8, 4), (992, 31, 7)])
@pytest.mark.parametrize("size", [8.0, 100.0, 1e3, 3e4])
def test_group_scores_of_biases_that_cancel(size, E, G, top):
    """One expert of each group at about +size, the others at about -size: the
    sum of the best two is a small difference of large values, whose binary32
    errors are those of the large ones."""
    T, H, k = 4099, 64, 4
    rng = np.random.default_rng(int(size) + E)
    of_group = np.float32(size) * (1 + rng.random(G)).astype(np.float32)
    bias = np.repeat(-of_group, E // G)
    bias[np.arange(G) * (E // G) + rng.integers(0, E // G, G)] = of_group
    for score in (SIG, SOFT):
        how = how_of(score, G, top, B.GROUP_TOP2, True, 2.5)
        _, _, rb = route(T, H, E, k, how, bias=bias, seed=E, std=0.5)
        check(T, E, k, how, bias, rb)


def test_group_scores_beside_experts_masked_with_large_negative_biases():
    """Finite masks: groups whose second value is -1e30 are far below the
    others and must not blur them."""
    T, H, E, G, top, k = 1003, 64, 256, 8, 4, 4
    rng = np.random.default_rng(3)
    bias = rng.normal(0, 0.1, E).astype(np.float32)
    bias[rng.permutation(E)[:100]] = -1e30
    bias[3 * 32 + 1:4 * 32] = -1e30          # a group of one expert that is left
    bias[6 * 32:7 * 32] = -1e30              # and one of none
    how = how_of(SIG, G, top, B.GROUP_TOP2, True, 2.5)
    _, _, rb = route(T, H, E, k, how, bias=bias)
    check(T, E, k, how, bias, rb)


def test_two_threads_with_different_numbers_of_experts():
    """The same kernel with other sizes of shared memory from two host
    threads, a context each: neither call is refused."""
    import threading

    H, k, failed = 64, 4, []
    made = []
    for E in (400, 500):
        rt = B.Runtime(H, 64, E, k, 0, 8, 1, 0)
        made.append((rt, I.randn_bf16((8, H), 1.0, E, "cuda"), I.randn_bf16((E, H), 0.1, E + 1, "cuda"),
                     B.RouteBuffers(8, E, k), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(rt, x, wr, rb, stream):
        try:
            for i in range(3000):
                rt.route_scored(x, wr, None, how_of(SIG), rb, stream)
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
    for m in made:
        m[0].close()
    assert not failed, failed[0]


@pytest.mark.parametrize("T", [1025, 1055, 2049, 8205])
@pytest.mark.parametrize("H, E", [(256, 256), (7168, 256), (192, 513), (64, 72)])
def test_last_rows_of_a_warp_of_the_tensor_core_router(T, H, E):
    """Token counts that end inside a warp's 32 rows: every column of the
    rows that exist, and nothing beyond them."""
    x, wr, rb = route(T, H, E, 4, how_of(SIG), seed=T)
    ref, mag = x.double() @ wr.double().t(), x.double().abs() @ wr.double().abs().t()
    assert bool(((rb.logits.double() - ref).abs() <= 2.0 ** -24 * H ** 0.5 * mag + 1e-30).all())
    check(T, E, 4, how_of(SIG), None, rb)


@pytest.mark.parametrize("T", [9, 33, 64])
@pytest.mark.parametrize("E", [40, 270, 300, 513, 1001])
def test_one_kernel_of_a_cluster_with_counts_that_end_inside_a_warp(T, E):
    x, wr, rb = route(T, 64, E, 4, how_of(SIG), seed=E)
    check(T, E, 4, how_of(SIG), None, rb)
