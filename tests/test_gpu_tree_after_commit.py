"""A ring tree without new rows right behind the commit that writes its positions: both lengths in one buffer, side by
side, call after call without a wait."""

import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq
from test_gpu_tree import RingCase, i32, tree, words

pytestmark = pytest.mark.gpu
D = 128


@pytest.mark.parametrize("N,heads,B", [(12, (20, 4), 4), (12, (20, 4), 60), (4, (20, 4), 4), (9, (2, 1), 300)])
def test_positions_of_the_commit_before(N, heads, B):
    c = RingCase([100 + 7 * (i % 50) for i in range(B)], N, *heads, 200, seed=N + B, capacity=512)
    masks = [tree(N, c.rng) for _ in range(B)]
    c.call(masks)  # appends
    w, path = words(masks), i32([list(range(N))] * B)  # the first tokens in order: records stay where they are
    at = torch.zeros(2, B, dtype=torch.int32, device="cuda")
    at[0] = c.pos_t
    n = torch.ones(B, dtype=torch.int32, device="cuda")
    ws = kvq.alloc_tree_workspace(B, N, *heads)
    outs = [torch.full((B, N, heads[0], D), 9.0, device="cuda") for _ in range(12)]

    def steps(wait):
        at[0] = c.pos_t
        for i, o in enumerate(outs):
            kvq.kvq_tree_commit_fp8([c.ring], at[i % 2], path, n, c.err, ctx_out=at[1 - i % 2])
            kvq.kvq_tree_attn_fp8_swa(c.ring, c.q, at[1 - i % 2], w, 200, c.KS, c.VS, o, ws, c.err)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return [o.clone() for o in outs]

    want = steps(True)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(steps(False), want))
    assert c.err.item() == 0 and not torch.equal(want[0], want[1])
