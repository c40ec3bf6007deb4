"""The 8-bit attention on the GPU within the tight bounds of q8_bounds."""
import pytest
import torch

import q8_bounds as Q
import q8_reference as R
from test_q8_gpu import BF16, F32, G, Dev, lib, problem  # noqa: F401 (lib: builds the library)

pytestmark = pytest.mark.gpu


def test_scores_hold_fp32():
    pr, tol = Q.score_problem()
    want = R.attend(pr)[1]
    dv = Dev(pr).attend()
    assert ((dv.lse.double().cpu() - want).abs() <= tol * want.abs()).all()


@pytest.mark.parametrize("dtype,rows", [(F32, 64), (BF16, 16), (BF16, 64), (BF16, 300)])
def test_weights_hold_their_bits(dtype, rows):
    pr, out, tol, _ = Q.weight_problem(dtype, rows)
    dv = Dev(pr).attend()
    assert ((dv.out.double().cpu() - out).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", sorted(G))
def test_attend(name, dtype):
    pr = problem(name, dtype)
    Dev(pr).attend().checked(Q.attend(pr), what=name)


# size of the values beside the row of zeros; how far its score is above the others'
@pytest.mark.parametrize("size,lift", [(1.0, 8.0), (1e-4, 8.0), (1e-6, 8.0), (1e-6, -8.0), (1e-6, 0.0), (1e-3, 25.0)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype,q_len", [(BF16, 4), (BF16, 40), (BF16, 150), (F32, 4), (F32, 40)])
def test_rows_of_zeros_do_not_coarsen_the_others(dtype, q_len, d, size, lift):
    pr = Q.zero_sink(dtype, size, q_len=q_len, kv_len=333, hq=4, hkv=2, d=d, lift=lift, n=2)
    Dev(pr).attend().checked(Q.attend(pr), what=f"values of {size}")


@pytest.mark.parametrize("name", ["decode", "decode_d256", "decode_g16", "few", "one", "chunk", "chunk_d64", "chunk_d256", "cross_gqa", "fresh"])
def test_scattered_rows_of_zeros(name):
    """Rows of zeros (of both signs) and rows at scale 2^0 or the smallest one that are not zeros
    but for a late value, among small ones."""
    pr = problem(name, gain=1e-5, poison=True)
    gen = torch.Generator().manual_seed(2)
    for s, b in enumerate(pr.kv_lens):
        pos = torch.arange(b)
        page, slot = pr.table[s].long()[pos // pr.p], pos % pr.p
        kind = torch.randint(0, 8, (b,), generator=gen)
        for codes, scales in ((pr.k_codes, pr.k_scales), (pr.v_codes, pr.v_scales)):
            z = kind < 2
            codes[page[z], slot[z]] = torch.where(kind[z] == 0, 0, 0x80).to(torch.uint8)[:, None, None]
            scales[page[z], :, slot[z]] = 127
        late = kind == 2
        pr.v_codes[page[late], slot[late]] = 0
        pr.v_codes[page[late], slot[late], :, pr.d - 1 - s % pr.d] = 0x7E        # 448 of the smallest scale
        pr.v_scales[page[late], :, slot[late]] = 0
    Dev(pr).attend().checked(Q.attend(pr), what=name)
