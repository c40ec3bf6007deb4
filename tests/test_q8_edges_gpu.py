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


def low_scores(pr, by):
    """Shifts every score of the problem down by about `by` (natural units): the first value of
    each K row becomes the largest power of two it can hold, q's first one its opposite."""
    for codes in (pr.k_codes,):
        codes[..., 0] = 0x70                       # 2^7 of the row's scale
    for s, b in enumerate(pr.kv_lens):
        if b:
            page, slot = places(pr, s, torch.arange(b))
            pr.k_scales[page, :, slot] = 121       # 2^-6: k_0 = 2
    pr.q[..., 0] = -by / (2 * pr.scale)


@pytest.mark.parametrize("by", [90.0, 100.0, 300.0, 5000.0])
@pytest.mark.parametrize("dtype,hq,q_len", [(BF16, 8, 3), (BF16, 16, 8), (BF16, 8, 16), (torch.float32, 8, 3), (torch.float32, 16, 40)])
def test_rows_without_a_key_in_a_block_and_low_scores(dtype, hq, q_len, by):
    """The causal mask hides a sequence's last block from all but its last tokens, and all scores
    are far below zero.  Many sequences, so that one CTA runs over both blocks of a group."""
    n = 120
    pr = R.make([q_len] * n, [128 + 1 + i % max(1, q_len - 1) for i in range(n)], hq=hq, hkv=8, d=64, p=16,
                dtype=dtype, seed=5)
    low_scores(pr, by)
    Dev(pr).attend().checked(what=f"scores around -{by}")
