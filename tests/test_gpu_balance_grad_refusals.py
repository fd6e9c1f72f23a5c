"""DecoderBlockTail.balance_grad with sequences it would misread, on the device:
refused, and nothing is written."""
import pytest
import torch
from test_gpu_block_training import Made

from moe_expert_grouped_split_gb300.build import build

pytestmark = pytest.mark.gpu


def test_sequences():
    build()
    m = Made(40)
    kept = m.block.keep(40)
    m.run(kept)
    good = torch.tensor([0, 15, 40], dtype=torch.int32, device="cuda")
    db = torch.ones(2, device="cuda")
    want = m.block.balance_grad(kept, dbalance=db, seq_offsets=good)
    for bad in (good.cpu(), good.long(), torch.tensor([0, 9, 15, 9, 40, 9], dtype=torch.int32, device="cuda")[::2], good[:1],
                good[:0], good.view(1, 3), good.float()):
        with pytest.raises(ValueError):
            m.block.balance_grad(kept, dbalance=db, seq_offsets=bad)
    again = m.block.balance_grad(kept, dbalance=db, seq_offsets=good)
    torch.cuda.synchronize()
    for n, t in want.items():
        assert t is None or torch.equal(t, again[n]), n
    assert m.rt.device_status() == 0
    m.close()
