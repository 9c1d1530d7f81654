"""kvq_prompt_mass over keys with infinite elements: a score of -inf is a weight of 0 and leaves its row's other weights as
they are; a score of +inf, or one that is NaN, makes the row NaN, and it adds nothing. Against the plain evaluation in 64 bits."""

import math

import pytest
import torch

from test_gpu_prompt import inputs
from test_gpu_prompt_mass import call, check, reference

pytestmark = pytest.mark.gpu


# groups of 5, 3, 33 and 43 heads leave places of a query tile empty (128 rows hold whole tokens only), groups of 1, 2 and 64 none
@pytest.mark.parametrize("heads", [(20, 4), (3, 1), (33, 1), (43, 1), (64, 1), (4, 2), (3, 3)])
@pytest.mark.parametrize("rows", [1, 64, 130, 0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_scores_of_minus_infinity(heads, rows, dtype):
    lens = [150, 300, 90]
    q, k, _ = inputs(lens, *heads, dtype, seed=rows + heads[0])
    q[..., 5] = -q[..., 5].abs() - 0.25
    q[..., 9] = q[..., 9].abs() + 0.25
    k[[10, 149, 150, 150 + 260, 450], 0, 5] = math.inf
    k[[11, 450 + 70], heads[1] - 1, 9] = -math.inf
    # a row all of whose scores are -inf is NaN
    skip = [(t, h) for t in (150, 450) for h in range(heads[0] // heads[1])]
    want = reference(q, k, lens, rows, skip=skip)
    assert all(bool(torch.isfinite(m).all()) for m, _ in want)
    held = call(q, k, lens, rows)
    check(held, want, lens)
    assert float(held["mass"][0, 0, 10]) == 0.0 and float(held["mass"][1, 0, 260]) == 0.0


@pytest.mark.parametrize("rows", [64, 0])
@pytest.mark.parametrize("heads", [(20, 4), (4, 2)])
def test_scores_of_both_signs(heads, rows):
    """Rows whose score with the infinite key is +inf add nothing; the others' weights stay."""
    lens = [150, 300]
    q, k, _ = inputs(lens, *heads, torch.bfloat16, seed=3 + rows)
    q[..., 5] = torch.where(q[..., 5] < 0, q[..., 5] - 0.25, q[..., 5] + 0.25)
    k[150 + 200, 0, 5] = -math.inf
    G = heads[0] // heads[1]
    skip = [(t, h) for t in range(350, 450) for h in range(G) if float(q[t, h, 5]) < 0]
    assert 0 < len(skip) < 100 * G
    held = call(q, k, lens, rows)
    check(held, reference(q, k, lens, rows, skip=skip), lens)
    assert float(held["mass"][1, 0, 200]) == 0.0
