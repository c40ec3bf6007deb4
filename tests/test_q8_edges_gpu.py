"""The 8-bit cache's kernels where their bookkeeping or arithmetic can go wrong:
rings, masks that leave a block's rows empty, units of the accumulators, rows
of zeros, the top of the format's range."""
import pytest
import torch

import q8_reference as R
from test_q8_gpu import BF16, Dev, lib  # noqa: F401 (lib: builds the library)

pytestmark = pytest.mark.gpu


def places(pr, s, pos):
    """Page and slot of positions `pos` (a tensor) of sequence s."""
    return pr.table[s].long()[pos // pr.p], pos % pr.p


@pytest.mark.parametrize("d", [64, 128, 256])
def test_chunk_scales_change_from_block_to_block(d):
    """V scales that differ by 2^6 from key to key, the other way round in the next
    block: a factor taken from another block would show at once.  Repeats bit for bit."""
    pr = R.make([300, 150, 280], [3000, 2500, 280], hq=4, hkv=4, d=d, p=16, seed=3)
    for s, b in enumerate(pr.kv_lens):
        pos = torch.arange(b)
        page, slot = places(pr, s, pos)
        up = ((pos + pos // 128) % 2 * 6).to(torch.uint8)[:, None]
        pr.v_scales[page, :, slot] += up
    dv = Dev(pr).attend()
    dv.checked(what=f"head_dim {d}")
    first = dv.out.clone(), dv.lse.clone()
    for _ in range(20):
        dv.out.fill_(77.0)
        dv.attend()
        assert torch.equal(dv.out, first[0]) and torch.equal(dv.lse, first[1])
