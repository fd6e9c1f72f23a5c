"""dwdp_balance_loss and dwdp_route_scored_grad at logits where binary32's
exponentials or their reciprocals leave its range.  Tolerances as in
test_gpu_balance, and what vanishes below 2^-126: a share, or a 1 - s, of that
size may be 0 (or 2^-126), and its terms of the gradient with it, so every
element may be off by 2^-126 times the sum of those terms' other factors:
2 |dz| lse / T_b of the z loss, |dbalance| E / (k T_b^2) times twice the largest
count of the balance loss, twice scale |dtopk_w| of the weights; and the balance
loss itself by 2^-126 E / (k T_b) times the sum of the counts."""
import pytest
import torch
from test_gpu_balance import HOWS, TINY, U, Made, near

from moe_expert_grouped_split_gb300.build import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def factors(m, counts):
    """[T, 1]: the sum of the factors above."""
    f = torch.zeros((m.T, 1), dtype=torch.float64, device="cuda")
    for i in range(m.S):
        z, n = m.z[m.seq(i)].double(), m.ends[i + 1] - m.ends[i]
        if n:
            f[m.seq(i)] += 2 * m.dz[i].double().abs() / n * torch.logsumexp(z, 1, keepdim=True).abs()
            f[m.seq(i)] += 2 * m.db[i].double().abs() * m.E / (m.k * n * n) * counts[i].max()
    return f + 2 * m.scale * m.dw.double().abs().amax(1, keepdim=True)


def check_losses(m, out):
    for b in range(m.S):
        z, ids = m.z[m.seq(b)].double(), m.ids[m.seq(b)]
        n = z.shape[0]
        counts = torch.bincount(ids.reshape(-1).long(), minlength=m.E)
        assert torch.equal(out.counts[b].long(), counts)
        p = m.shares(z).mean(0)
        rel = m.rel(z) + n * U / 2
        near(out.mean_p[b], p, rel * p + TINY)
        loss, most = m.E / (m.k * n) * (counts * p).sum(), m.E / (m.k * n) * counts.sum()
        near(out.balance[b], loss, (rel + (m.E / 32 + 16) * U) * loss + 2.0 ** -126 * most + TINY)
        lse = torch.logsumexp(z, 1)
        err = m.rel(z) + 4 * U * lse.abs()
        near(out.z[b], lse.square().mean(), (2 * lse.abs() * err + err ** 2).mean() + rel * lse.square().mean())


def check_grad(m, counts, **parts):
    want, tol = m.formula(counts, **parts)
    near(m.grad(counts=counts, **parts), want, tol + 2.0 ** -126 * factors(m, counts))


@pytest.mark.parametrize("how", HOWS, ids=str)
@pytest.mark.parametrize("E, k", [(9, 3), (24, 4), (64, 4), (256, 8), (600, 8)])
def test_logits_whose_exponentials_reciprocal_is_subnormal(how, E, k):
    """86 to 90 in steps of 0.1 beside ordinary logits, every token a sequence of
    its own, the large one chosen in every other token; then the same in every
    column at once."""
    T = 41
    m = Made(T, E, k, list(range(T + 1)), how, seed=E)
    large = 86 + 0.1 * torch.arange(T, device="cuda")
    m.z[:, 5] = large
    m.ids[::2] = torch.arange(5 - k // 2, 5 - k // 2 + k, dtype=torch.int32, device="cuda")
    m.ids[1::2] = torch.arange(E - k, E, dtype=torch.int32, device="cuda")
    for _ in range(2):
        out = m.losses()
        check_losses(m, out)
        for parts in (dict(), dict(w=False, z=False), dict(b=False, z=False), dict(b=False, w=False)):
            check_grad(m, out.counts, **parts)
        m.z[:] = large[:, None]
    m.close()


@pytest.mark.parametrize("how", HOWS, ids=str)
@pytest.mark.parametrize("E, k", [(9, 3), (24, 4), (256, 8), (600, 8)])
def test_large_logits_and_scaled_losses(how, E, k):
    """Logits around 20 to 79, under gradients of a loss times 2^24: their product
    is beyond binary32 where neither factor is."""
    T = 60
    m = Made(T, E, k, [0, 30, T], how, seed=E)
    m.z += 20 + torch.arange(T, device="cuda")[:, None]
    m.dw *= 2.0 ** 24
    m.db *= 2.0 ** 24
    m.dz *= 2.0 ** 24
    counts = m.losses().counts
    for parts in (dict(), dict(w=False, z=False), dict(b=False, z=False), dict(b=False, w=False)):
        check_grad(m, counts, **parts)
    m.close()


@pytest.mark.parametrize("how", HOWS, ids=str)
@pytest.mark.parametrize("at", [-85.0, -46.0, 33.0, 70.0])
def test_logits_far_from_zero_and_near_each_other(how, at):
    """A share's error goes with the logits' spread (0.5), not with where they
    lie: exponentials of at most 0.5 are off by 2^-22, and a sum over 64 experts
    (4 terms, 4 exchanges) with its reciprocal and one product by 10 2^-24; as
    much for 1 - s, and half an ulp of the quotient that the oracle is not off by.
    s next to 1 is off by the error of 1 - s only."""
    T, E, k = 200, 64, 4
    m = Made(T, E, k, list(range(T + 1)), how, seed=3)
    g = torch.Generator("cuda").manual_seed(4)
    m.z = at + 0.5 * torch.rand((T, E), generator=g, device="cuda")
    p = m.shares(m.z.double())
    near(m.losses().mean_p, p, (2 * 2.0 ** -22 + 11 * 2.0 ** -24) * p)
    m.close()
