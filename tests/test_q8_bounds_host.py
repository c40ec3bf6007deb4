"""The tight error bounds of the 8-bit attention, without a GPU: a model of the
parts that the kernels make meets them, one with fewer parts does not."""
import pytest
import torch

import q8_bounds as Q
import q8_reference as R

BF16, F32 = torch.bfloat16, torch.float32
PARTS = {BF16: (2, 4), F32: (6, 6)}


def test_parts_of_q_count():
    pr, tol = Q.score_problem()
    want = R.attend(pr)[1]
    worst = [((Q.model(pr, n, 6)[1] - want).abs() / want.abs()).max().item() for n in (6, 4)]
    assert worst[0] <= 1.01 * Q.U < tol < 0.5 * worst[1]


# rows: what the row-group kernel takes for bf16 (16), and more
@pytest.mark.parametrize("dtype,rows,few", [(F32, 64, 3), (BF16, 16, 3)])
def test_parts_of_the_weights_count(dtype, rows, few):
    pr, out, tol, w = Q.weight_problem(dtype, rows)
    got = Q.model(pr, PARTS[dtype][0], PARTS[dtype][1])[0]
    half = torch.finfo(dtype).eps / 2 * out.abs()
    assert ((got - out).abs() <= tol - half).all()
    got = Q.model(pr, PARTS[dtype][0], few)[0]
    assert ((got - out).abs() > tol).any()


def test_a_bit_of_the_fp16_weights_counts():
    """The chunk kernel's weights, fp16 at 2^5 for the largest, and with one bit fewer."""
    pr, out, tol, w = Q.weight_problem(BF16, 64)
    w = 32 * w
    h = w.to(torch.float16).double()
    step = torch.exp2(torch.floor(torch.log2(w)) - 9)           # 10 significant bits
    less = torch.round(w / step) * step
    half = torch.finfo(BF16).eps / 2 * out.abs()
    for got, ok in ((h, True), (less, False)):
        o = 256 * (75 * got - 53 * 32) / (53 * 32 + 75 * w)
        over = (o[:, None, None] - out).abs() > (tol - half if ok else tol)
        assert over.any() != ok


SHAPES = [([1, 3, 1], [200, 130, 1], 4, 2, True), ([5, 0, 2], [5, 7, 300], 3, 3, True), ([2, 9], [129, 50], 4, 1, False)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_model_is_within_the_bounds(shape, dtype):
    q, kv, hq, hkv, causal = SHAPES[shape]
    pr = R.make(q, kv, hq=hq, hkv=hkv, d=64, p=8, dtype=dtype, causal=causal, seed=shape)
    out, lse, tol_o, tol_l = Q.attend(pr)
    got = Q.model(pr, *PARTS[dtype])
    half = torch.finfo(dtype).eps / 2
    assert ((got[0] - out).abs() <= tol_o - half * out.abs()).all()
    fine = torch.isfinite(lse)
    assert torch.equal(got[1][~fine], lse[~fine]) and ((got[1] - lse).abs()[fine] <= tol_l[fine]).all()
    # and they are well below the loose ones
    loose = R.attend(pr)
    rest = out.abs() > 0
    assert (tol_o[rest] < loose[2][rest]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_zeros_do_not_widen_the_bounds(dtype):
    """A row of zeros at scale 2^0 that has most of the weight, among values of 1e-6: a model that
    measures the weights in its units is outside, one that does not is inside."""
    pr = Q.zero_sink(dtype, 1e-6)
    out, lse, tol_o, tol_l = Q.attend(pr)
    assert (tol_o <= 2.0 ** -5 * out.abs().amax(-1, keepdim=True)).all()
    for count, ok in ((False, True), (True, False)):
        over = (Q.model(pr, *PARTS[dtype], zeros_count=count)[0] - out).abs() > tol_o
        assert over.any() != ok

