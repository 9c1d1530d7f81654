"""A pool of one page: alloc, fork, compact and copy with empty lists of moves."""

import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq

pytestmark = pytest.mark.gpu


def test_pool_of_one_page():
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    refs, table, err, moves = i32([0]), i32([[-1], [-1]]), i32([0]), i32([7])
    tensors, cache = kvq.alloc_int4_cache(1, 2, table.cpu())
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    for held in (0, 1):
        if held:
            kvq.kvq_pages_alloc(refs, table, i32([1]), i32([0]), i32([64]), err)
        kvq.kvq_pages_compact(refs, table, none, none, moves, err)
        kvq.kvq_pages_copy([cache], none, none, err, count=moves)
        assert moves.item() == 0 and refs.tolist() == [held] and table.tolist() == [[-1], [0 if held else -1]]
        moves.fill_(7)
    src, dst = i32([5]), i32([5])
    kvq.kvq_pages_fork(refs, table, i32([1]), i32([0]), i32([64]), src, dst, err)
    assert refs.tolist() == [2] and table.tolist() == [[0], [0]] and src.tolist() == dst.tolist() == [-1] and err.item() == 0
