"""Rows in no group may be read ahead: whatever every array holds there, infinities
and NaN among it, no other row, no sum and no byte of theirs changes."""
import pytest
import torch
from test_gpu_sandwich import Grads, Made

from moe_expert_grouped_split_gb300.build import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("rows, H", [(200, 2048), (1300, 7168), (300, 8200)])  # a block a row, staying blocks, wide rows
@pytest.mark.parametrize("form", [dict(), dict(post=False), dict(pre=False)], ids=str)
def test_what_padding_holds(rows, H, x8, form):
    m = Made(rows, H, groups=[rows // 4, rows // 3, rows // 3, rows - rows // 5], **form)
    out = ~m.inside
    o = m.forward()
    g = Grads(m, x8, x8 and m.pre is not None)
    b = g.run()
    for bad in (float("nan"), float("inf"), -3e38):
        for t in (m.x, m.residual, g.x, g.h, g.dout, g.dres):
            if t is not None and t.dtype == torch.bfloat16:
                t[out] = bad
            elif t is not None:
                t.view(torch.uint8)[out] = 0x7F  # E4M3's NaN
        for t in (g.rstd, g.x_scale, g.h_scale):
            if t is not None:
                t[out] = bad
        again, back = m.forward(), g.run()
        for n in o:
            assert torch.equal(o[n].view(torch.uint8), again[n].view(torch.uint8)), n
        for n in b:
            assert torch.equal(b[n].view(torch.uint8), back[n].view(torch.uint8)), n
