"""Offsets of packed prompts that go back or leave the tensors: what is skipped, and that nothing else changes."""

import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq
from test_gpu_prompt import call, check, inputs, reference

pytestmark = pytest.mark.gpu
D = 128


@pytest.mark.parametrize("T,cu,taken", [
    (600, [0, 300, 100, 500], [(0, 300)]),                              # back into the first
    (600, [0, 300, 100, 300, 600], [(0, 300), (300, 600)]),             # and on from its end
    (600, [200, 300, 0, 200, 250], [(200, 300)]),                       # before the first: the earlier one counts
    (600, [0, 5, 1000, 8, 12], [(0, 5), (8, 12)]),                      # an end that is outside hides no other
    (600, [-4, 100, 100, 40, 40, 200], [(40, 200)]),                    # empty ones and those outside take no rows
    (600, [0, 1, 0, 1, 0, 1, 0, 2], [(0, 1)]),
    (600, [100, 228, 600], [(100, 228), (228, 600)])])                  # rows before the first are nobody's
def test_offsets_that_go_back(T, cu, taken):
    q, k, v = inputs([T], 4, 2, torch.bfloat16, seed=len(cu))
    offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = call(q, k, v, None, cu=offsets, want_err=0 if cu == sorted(cu) and cu[0] >= 0 and cu[-1] <= T else kvq.DEVERR_POS)
    left = torch.ones(T, dtype=torch.bool, device="cuda")
    for s, e in taken:
        left[s:e] = False
        check(out[s:e], *reference(q[s:e], k[s:e], v[s:e], [e - s], 0, D ** -0.5))
    assert bool((out[left] == 7).all())
