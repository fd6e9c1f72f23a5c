"""Logits of -inf: experts with a share of 0 and no gradient, in both calls, every
score and part, as long as a token (and, renormalised, its choice) has a finite
one.  Against the formulas in 64 bits, which have them as they are."""
import pytest
import torch
from test_gpu_balance import HOWS, Made

from moe_expert_grouped_split_gb300.build import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


@pytest.mark.parametrize("how", HOWS, ids=str)
@pytest.mark.parametrize("shift", [0.0, -100.0, 60.0])
@pytest.mark.parametrize("E, k", [(9, 3), (64, 4), (130, 6), (600, 8)])
def test_masked_experts(how, shift, E, k):
    T = 45
    m = Made(T, E, k, [0, 20, T], how, seed=E)
    g = torch.Generator("cuda").manual_seed(7)
    m.z += shift
    masked = torch.rand((T, E), generator=g, device="cuda") < 0.4
    masked[:, 1] = False  # one is left
    masked[0] = True
    masked[0, 1] = False  # only one
    m.z[masked] = -float("inf")
    m.ids[::3] = torch.arange(1, k + 1, dtype=torch.int32, device="cuda")  # 1, and masked ones beside it
    others = torch.sort(torch.where(masked, -1e9, torch.rand((T, E), generator=g, device="cuda")).topk(k, 1)[1], 1)[0].int()
    rest = torch.arange(T, device="cuda") % 3 != 0
    m.ids[rest] = others[rest]
    assert bool(masked.gather(1, m.ids.long()).any())
    out = m.losses()
    m.check_losses(out)
    everywhere = masked[:20].all(0)
    assert (out.mean_p[0][everywhere] == 0).all()
    for parts in (dict(), dict(w=False, z=False), dict(b=False, z=False), dict(b=False, w=False)):
        dl = m.grad(counts=out.counts, **parts)
        m.check_grad(dl, out.counts, **parts)
        assert (dl[masked] == 0).all()
    m.close()  # no device error
