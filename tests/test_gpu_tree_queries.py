"""Tree rows whose query is not finite, or holds elements that the fp16 products do not: such a row is NaN in every form
of the calls, a row that sees nothing is 0 all the same, and no other row changes."""

import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq
from test_gpu_tree import Int4Case, RingCase, i32, tree, words

pytestmark = pytest.mark.gpu
D = 128

# The forms by rows per KV head. int4: 9 and 12 (8-row tiles), 40 (tensor cores), 80 and 160 (page tiles, one row group and
# two); the ring: 9 and 15 (one launch), 45 and 80 (page tiles).
FORMS = [("int4", 3, (6, 2)), ("int4", 4, (6, 2)), ("int4", 8, (20, 4)), ("int4", 16, (20, 4)), ("int4", 32, (10, 2)),
         ("ring", 3, (6, 2)), ("ring", 3, (20, 4)), ("ring", 9, (20, 4)), ("ring", 16, (20, 4))]


def case(kind, N, heads, dtype, lens=(70, 3000, 5)):
    if kind == "int4":
        return Int4Case(list(lens), N, *heads, seed=N, dtype=dtype)
    return RingCase(list(lens), N, *heads, 513, seed=N, dtype=dtype)


def run(c, masks, out_dtype=torch.float32):
    out = torch.full((c.B, c.N, c.Hq, D), 9.0, dtype=out_dtype, device="cuda")
    ws = kvq.alloc_tree_workspace(c.B, c.N, c.Hq, c.Hkv)
    if isinstance(c, Int4Case):
        kvq.kvq_tree_attn_int4(c.cache, c.Mq, c.Mk, c.q, c.ctx_t, words(masks), out, ws, c.err, k_new=c.k_new, v_new=c.v_new)
    else:
        kvq.kvq_tree_attn_fp8_swa(c.ring, c.q, c.pos_t, words(masks), c.window, c.KS, c.VS, out, ws, c.err, k_new=c.k_new,
                                  v_new=c.v_new)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("kind,N,heads", FORMS)
def test_a_query_that_is_not_finite(kind, N, heads, bad, dtype, out_dtype):
    c = case(kind, N, heads, dtype)
    masks = [tree(N, c.rng) for _ in range(3)]
    want = run(c, masks, out_dtype)
    rows = [(0, 0, 1), (1, N - 1, 0), (1, 0, heads[0] - 1), (2, N // 2, 0)]
    keep = torch.ones(want.shape[:3], dtype=torch.bool, device="cuda")
    for i, r in enumerate(rows):
        c.q[r + (17 * i,)] = float(bad)
        keep[r] = False
    out = run(c, masks, out_dtype)
    assert bool(out[~keep].isnan().all())
    assert torch.equal(out[keep], want[keep])
    assert c.err.item() == (kvq.DEVERR_NONFINITE if kind == "int4" else 0)


@pytest.mark.parametrize("bad", ["inf", "-inf"])
@pytest.mark.parametrize("kind,N,heads", FORMS)
def test_scores_that_are_all_minus_infinity(kind, N, heads, bad):
    """One visible key of one sign: an infinite element gives the score +inf or -inf, and NaN either way; a row that sees
    nothing is 0 whatever its query holds."""
    c = case(kind, N, heads, torch.float32, (0, 0, 40))
    c.k_new.abs_()
    masks = [[1 << i for i in range(N)], [0] * N, tree(N, c.rng)]
    c.q[:2, :, :, 5] = float(bad)
    out = run(c, masks)
    assert bool(out[0].isnan().all()) and bool((out[1] == 0).all()) and bool(torch.isfinite(out[2]).all())


@pytest.mark.parametrize("size,finite", [(65000.0, True), (65519.0, True), (65520.0, False), (1e5, False), (3e38, False)])
@pytest.mark.parametrize("kind,N,heads", [f for f in FORMS if f[0] == "ring"])
def test_ring_queries_at_the_end_of_fp16(kind, N, heads, size, finite):
    c = case(kind, N, heads, torch.float32)
    masks = [tree(N, c.rng) for _ in range(3)]
    want = run(c, masks)
    c.q[1, N - 1, 0] = 0.0
    c.q[1, N - 1, 0, 3] = size
    out = run(c, masks)
    keep = torch.ones(out.shape[:3], dtype=torch.bool, device="cuda")
    keep[1, N - 1, 0] = False
    assert torch.equal(out[keep], want[keep]) and c.err.item() == 0
    assert bool(torch.isfinite(out[~keep]).all() if finite else out[~keep].isnan().all())


@pytest.mark.parametrize("kind,N,heads", [f for f in FORMS if f[0] == "int4"])
def test_int4_rotated_queries_past_fp16(kind, N, heads):
    """Gains that put elements of q~ past 65504."""
    c = case(kind, N, heads, torch.float32)
    masks = [tree(N, c.rng) for _ in range(3)]
    c.Mq *= 1e6
    out = run(c, masks)
    assert bool(out.isnan().all()) and c.err.item() == 0
