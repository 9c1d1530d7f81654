"""Arguments of the session calls that overlap are refused: a call writes some of them while it still reads the
others. Nothing is launched, so no GPU is needed. Trees whose output takes the very place of their queries are right."""

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


@pytest.mark.parametrize("q,k,out,dtype,out_dtype", [
    (0x1000000, None, 0x1000000, 1, 0), (0x1000000, None, 0x1000000, 0, 1), (0x1000000, None, 0x1000010, 1, 1),
    (0x1000000, None, 0x1000000 - 16, 0, 0), (0x1000000, 0x2000000, 0x2000000, 1, 1), (0x1000000, 0x2000000, 0x2000000 + 4080, 1, 1),
    (0x1000000, 0x2000000, 0x3000000, 1, 1), (0x1000000, 0x2000000, 0x3000000 - 4096, 0, 0)])
@pytest.mark.parametrize("N", [2, 16])
def test_ring_trees_refuse_an_output_within_their_inputs(N, q, k, out, dtype, out_dtype):
    r = kvq.Fp8Ring(0x10000, 4, 4, 576, 128)
    assert L.kvq_tree_attn_fp8_swa(ctypes.byref(r), q, dtype, 2, N, 20, 0x90000, 0x91000, 513, k, k and 0x3000000, 0.01, 0.01, 0.09, out,
                                   out_dtype, 0xB0000, 1 << 30, 0xC0000, None) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("kind,N,heads,B", [("int4", 3, (6, 2), 3), ("int4", 8, (20, 4), 3), ("int4", 16, (20, 4), 3), ("ring", 3, (6, 2), 3),
                                            ("ring", 3, (6, 2), 200), ("ring", 8, (2, 2), 100), ("ring", 16, (20, 4), 3),
                                            ("ring", 16, (20, 4), 60)])
def test_trees_write_over_their_queries(kind, N, heads, B, dtype):
    import torch

    from test_gpu_session_edges import issue
    from test_gpu_tree import Int4Case, RingCase, tree, words
    dt = getattr(torch, dtype)
    lens = [(70, 1000, 5)[i % 3] for i in range(B)]
    c = Int4Case(lens, N, *heads, seed=N, dtype=dt) if kind == "int4" else RingCase(lens, N, *heads, 513, seed=N, dtype=dt)
    masks = [tree(N, c.rng) for _ in range(B)]
    want = c.call(masks, dt)
    issue(c, words(masks), c.q, kvq.alloc_tree_workspace(B, N, *heads))
    assert torch.equal(c.q, want) and c.err.item() == 0
