"""The layers of one commit or page copy are descriptors of the call's kind: others would be read as what they are not."""

import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq

CACHE = kvq.Int4Cache(pages=0x10000, block_table=0x50000, num_seqs=4, max_pages_per_seq=8, num_pages=32, num_kv_heads=4,
                      page_size=64, head_dim=128)
RING = kvq.Fp8Ring(0x10000, 4, 4, 576, 128)


@pytest.mark.parametrize("call,layers", [
    ("kvq_tree_commit_int4", [RING]), ("kvq_tree_commit_int4", [CACHE, RING]), ("kvq_tree_commit_int4", [b"x" * 48]),
    ("kvq_tree_commit_int4", [CACHE, None]), ("kvq_tree_commit_fp8", [CACHE]), ("kvq_tree_commit_fp8", [RING, CACHE]),
    ("kvq_pages_copy", [RING]), ("kvq_pages_copy", [bytearray(8)]), ("kvq_pages_copy", [CACHE, 3])])
def test_other_layers_are_refused(call, layers):
    one, many = torch.zeros(1, dtype=torch.int32), torch.zeros((1, 4), dtype=torch.int32)
    with pytest.raises(TypeError, match="layers must be"):
        if call == "kvq_pages_copy":
            kvq.kvq_pages_copy(layers, one, one, one)
        else:
            getattr(kvq, call)(layers, one, many, one, one)
