"""Lists of the commit and of the page pool that overlap are refused: a call writes some of them while it still reads the
others. Nothing is launched, so no GPU is needed."""

import ctypes

import pytest

import quantized_kv_cache_fold_gb300 as kvq

L = kvq.lib
INVALID = 1


@pytest.mark.parametrize("out", [0x1000, 0x101c, 0x2000, 0x2000 + 4 * 8 * 7, 0x2000 + 4 * 8 * 8 - 4, 0x2000 - 28, 0x3000, 0x301c, 0x3000 - 28])
def test_commit_refuses_an_output_within_its_lists(out):
    c = kvq.Int4Cache(pages=0x10000, block_table=0x50000, num_seqs=8, max_pages_per_seq=8, num_pages=64, num_kv_heads=4,
                      page_size=64, head_dim=128)
    assert L.kvq_tree_commit_int4(ctypes.byref(c), 1, 8, 8, 0x1000, 0x2000, 0x3000, out, 0x5000, None) == INVALID
    r = kvq.Fp8Ring(0x10000, 8, 4, 576, 128)
    assert L.kvq_tree_commit_fp8(ctypes.byref(r), 1, 8, 8, 0x1000, 0x2000, 0x3000, out, 0x5000, None) == INVALID


@pytest.mark.parametrize("src,dst", [(0x3000, 0x7000), (0x4004, 0x7000), (0x5000, 0x7000), (0x6000, 0x3004), (0x6000, 0x4000),
                                     (0x6000, 0x5000 - 4), (0x6000, 0x6000), (0x6000, 0x6004)])
def test_fork_refuses_lists_that_overlap(src, dst):
    assert L.kvq_pages_fork(0x1000, 10, 0x2000, 4, 8, 2, 0x3000, 0x4000, 0x5000, src, dst, 0x8000, None) == INVALID


@pytest.mark.parametrize("src,dst,moves", [(0x3000, 0x3000, 0x5000), (0x3000, 0x3010, 0x5000), (0x3000, 0x4000, 0x3010),
                                           (0x3000, 0x4000, 0x4000)])
def test_compact_refuses_lists_that_overlap(src, dst, moves):
    assert L.kvq_pages_compact(0x1000, 10, 0x2000, 4, 8, src, dst, moves, 0x8000, None) == INVALID
