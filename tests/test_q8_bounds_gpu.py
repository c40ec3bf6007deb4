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
