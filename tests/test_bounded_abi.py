"""Host-side refusals of the calls that hold a cache to a size: no GPU is needed, nothing is launched for a bad argument."""

import pytest

import quantized_kv_cache_fold_gb300 as kvq

L = kvq.lib
INVALID, UNSUPPORTED = 1, 2


def cache(**over):
    d = dict(pages=0x10000, block_table=0x50000, num_seqs=4, max_pages_per_seq=8, num_pages=32, num_kv_heads=4,
             page_size=64, head_dim=128)
    d.update(over)
    return kvq.Int4Cache(**d)


def prompt(**over):
    a = dict(q=0x1000000, k=0x2000000, v=0x3000000, dtype=kvq.BF16, T=100, B=2, Hq=20, Hkv=4, cu=0x9000, window=64, sinks=4,
             sm=0.09, out=0x4000000, ws=0xB0000, n=1 << 30, err=0xC0000)
    a.update(over)
    return L.kvq_prompt_attn_sinks(a["q"], a["k"], a["v"], a["dtype"], a["T"], a["B"], a["Hq"], a["Hkv"], None, a["cu"],
                                   a["window"], a["sinks"], a["sm"], a["out"], a["ws"], a["n"], a["err"], None)


@pytest.mark.parametrize("over,want", [
    (dict(sinks=-1), INVALID), (dict(q=0), INVALID), (dict(cu=0), INVALID), (dict(err=0), INVALID), (dict(T=-1), INVALID),
    (dict(Hq=21), INVALID), (dict(sm=0.0), INVALID), (dict(dtype=kvq.F32), UNSUPPORTED), (dict(out=0x1000000), INVALID),
    (dict(T=0, sinks=-1), INVALID), (dict(T=0), 0)])
def test_prompt_sinks_refuses(over, want):
    assert prompt(**over) == want
