"""kvq_tree_attn_int4, kvq_tree_attn_fp8_swa and the commits against plain evaluations in 64 bits.

Tolerance, per output element (u = 2^-11, half a step of fp16 relative to the value): q~, the
dequantised keys and values, and the weights p are rounded to fp16 once each, so a score is off by at
most d = 2 u sum|q k| sm (and its fp32 sum, 136 half steps of 2^-24) and a weight by the factor exp(d),
above and below the division: tol = (2 d + 2 u) sum p|v| / sum p, plus the output's own rounding
(2^-8 |o| for bf16). The ring's e4m3 values are exact in fp16.
"""

import math

import numpy as np
import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq
from gpu_util import unpack_fp8, unpack_int4

pytestmark = pytest.mark.gpu
D, SM = 128, 128 ** -0.5
U = 2.0 ** -11


def chain(N):
    return [(1 << (i + 1)) - 1 for i in range(N)]


def tree(N, rng):
    m = []
    for i in range(N):
        p = int(rng.integers(-1, i)) if i else -1
        m.append((1 << i) | (m[p] if p >= 0 else 0))
    return m


def words(masks):
    return torch.tensor([[w - (1 << 64) if w >> 63 else w for w in m] for m in masks], dtype=torch.int64, device="cuda")


def bits(masks, N):
    return torch.tensor([[[(w >> j) & 1 for j in range(N)] for w in m] for m in masks], dtype=torch.bool, device="cuda")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def attend(q, k, v, seen, sm, out_dtype):
    """q [R, 128], k, v [L, 128] in fp64, seen [R, L] -> (o, tol); rows that see nothing: 0."""
    z = torch.where(seen, q @ k.T * sm, -math.inf)
    p = torch.where(seen, torch.softmax(z, 1), 0.0).nan_to_num(0)
    o = p @ v
    mag = (seen * (q.abs() @ k.abs().T)).amax(1, keepdim=True) * abs(sm)
    d = 2 * U * mag + 136 * 2.0 ** -24 * mag + 2.0 ** -21
    tol = (2 * d + 2 * U) * (p @ v.abs()) + 1e-6
    if out_dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * o.abs()
    return o, tol


class Int4Case:
    def __init__(self, ctx, N, Hq, Hkv, seed=0, dtype=torch.bfloat16, fwht=False, extra_pages=0, k_gain=1.0, v_gain=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        self.ctx, self.N, self.Hq, self.Hkv, self.B, self.fwht = ctx, N, Hq, Hkv, len(ctx), fwht
        B = self.B
        P = max(-(-(c + N) // 64) for c in ctx) + extra_pages
        table = torch.from_numpy(self.rng.permutation(B * P).astype(np.int32).reshape(B, P))
        self.tensors, self.cache = kvq.alloc_int4_cache(B * P, Hkv, table)
        R, s = kvq.kvq_build_rotation(seed + 5)
        gq, gk = (self.rng.uniform(0.5, 1.5, D).astype(np.float32) for _ in range(2))
        M = kvq.kvq_fold_qk_fwht(s, gq, gk) if fwht else kvq.kvq_fold_qk(R, gq, gk)
        self.Mq, self.Mk = (torch.from_numpy(m).cuda() for m in M)
        self.Mq64 = torch.from_numpy(R.astype(np.float64) * (gq.astype(np.float64) * gk)[None, :]).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        rows = [(b, p) for b in range(B) for p in range(ctx[b] + N)]
        T = len(rows)
        k = (torch.randn(T, Hkv, D, generator=g, device="cuda") * k_gain).to(dtype)
        v = (torch.randn(T, Hkv, D, generator=g, device="cuda") * v_gain).to(dtype)
        seq, pos = i32([r[0] for r in rows]), i32([r[1] for r in rows])
        new = torch.tensor([p >= ctx[b] for b, p in rows], device="cuda")
        self.k_new, self.v_new = (x[new].view(B, N, Hkv, D).contiguous() for x in (k, v))
        old = ~new
        if bool(old.any()):
            kvq.kvq_rotate_quant_append(self.cache, self.Mk, k[old].contiguous(), v[old].contiguous(), seq[old].contiguous(),
                                        pos[old].contiguous(), self.err, fwht=fwht)
        self.q = torch.randn(B, N, Hq, D, generator=g, device="cuda").to(dtype)
        self.ctx_t = i32(ctx)

    def append(self):
        seq = torch.arange(self.B, device="cuda", dtype=torch.int32).repeat_interleave(self.N)
        pos = (self.ctx_t[:, None] + torch.arange(self.N, device="cuda", dtype=torch.int32)).flatten()
        kvq.kvq_rotate_quant_append(self.cache, self.Mk, self.k_new.flatten(0, 1), self.v_new.flatten(0, 1), seq, pos,
                                    self.err, fwht=self.fwht)

    def call(self, masks, out_dtype=torch.float32, append=True, sm=SM, want_err=0, stream=None):
        out = torch.full((self.B, self.N, self.Hq, D), 9.0, dtype=out_dtype, device="cuda")
        ws = kvq.alloc_tree_workspace(self.B, self.N, self.Hq, self.Hkv)
        new = (self.k_new, self.v_new) if append else (None, None)
        kvq.kvq_tree_attn_int4(self.cache, self.Mq, self.Mk, self.q, self.ctx_t, words(masks), out, ws, self.err,
                               k_new=new[0], v_new=new[1], sm_scale=sm, fwht=self.fwht, stream=stream)
        torch.cuda.synchronize()
        assert self.err.item() == want_err
        return out

    def dequantised(self, b, h, L):
        c = unpack_int4(self.tensors, b, h, L)
        f = lambda a: torch.from_numpy(a.view(np.float16).astype(np.float64))[:, None]  # noqa: E731
        return ((torch.from_numpy(c["kc"].astype(np.float64)) * f(c["ks"]) + f(c["ko"])).cuda(),
                (torch.from_numpy(c["vc"].astype(np.float64)) * f(c["vs"]) + f(c["vo"])).cuda())

    def check(self, out, masks, sm=SM, hide=None):
        seen_new = bits(masks, self.N)
        x = self.q.double()
        q = (x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()) @ self.Mq64.T
        G = self.Hq // self.Hkv
        for b in range(self.B):
            L = self.ctx[b] + self.N
            seen = torch.ones(self.N, L, dtype=torch.bool, device="cuda")
            seen[:, self.ctx[b]:] = seen_new[b]
            if hide is not None:
                seen &= ~hide(b, L)[None, :]
            for h in range(self.Hkv):
                k, v = self.dequantised(b, h, L)
                for hq in range(h * G, (h + 1) * G):
                    o, tol = attend(q[b, :, hq], k, v, seen, sm, out.dtype)
                    off = (out[b, :, hq].double() - o).abs()
                    assert bool((off <= tol).all()), (b, hq, float((off / tol).max()))


@pytest.mark.parametrize("N", [1, 2, 7, 8, 16, 25, 33, 64])
@pytest.mark.parametrize("heads", [(20, 4), (8, 1), (2, 2)])
def test_int4_sizes(N, heads):
    c = Int4Case([0, 1, 63, 64, 65, 200], N, *heads, seed=N)
    masks = [tree(N, c.rng) for _ in range(c.B)]
    c.check(c.call(masks), masks)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fwht", [False, True])
def test_int4_types_and_prologues(out_dtype, dtype, fwht):
    c = Int4Case([300, 129], 12, 20, 4, seed=3, dtype=dtype, fwht=fwht)
    masks = [tree(12, c.rng), chain(12)]
    c.check(c.call(masks, out_dtype), masks)


def test_int4_long_ragged():
    c = Int4Case([9000, 3, 2500, 16, 4097], 20, 20, 4, seed=4)
    masks = [tree(20, c.rng) for _ in range(5)]
    c.check(c.call(masks), masks)


def test_int4_one_long_sequence():
    c = Int4Case([70001], 64, 5, 1, seed=14)
    masks = [tree(64, c.rng)]
    c.check(c.call(masks), masks)


def test_int4_many_sequences():
    c = Int4Case([(i * 7) % 90 for i in range(700)], 3, 4, 2, seed=15)
    masks = [tree(3, c.rng) for _ in range(c.B)]
    c.check(c.call(masks, torch.bfloat16), masks)


def test_int4_wide_groups():
    c = Int4Case([500, 77], 40, 64, 1, seed=16)  # 2560 rows of one KV head
    masks = [tree(40, c.rng) for _ in range(2)]
    c.check(c.call(masks), masks)


def test_int4_empty_rows_and_odd_masks():
    """Rows that attend to nothing give 0; tokens may skip themselves or look ahead; bits from N on count for nothing."""
    N = 10
    c = Int4Case([0, 0, 130], N, 8, 2, seed=5)
    masks = [[0] * N, [(0 if i % 2 else 1 << 9) | (~0 << N) & (2 ** 64 - 1) for i in range(N)], [1 << (N - 1 - i) for i in range(N)]]
    out = c.call(masks)
    assert bool((out[0] == 0).all()) and bool((out[1, 1::2] == 0).all())
    c.check(out, [[w & (1 << N) - 1 for w in m] for m in masks])


def test_int4_a_chain_is_the_verify_block():
    c = Int4Case([777, 1000], 8, 20, 4, seed=6)
    out = c.call([chain(8)] * 2)
    ref = torch.empty_like(out)
    ws = kvq.alloc_workspace(2, 8, 20, 4)
    kvq.kvq_decode_attn_int4(c.cache, c.Mq, c.Mk, c.q, c.ctx_t, ref, ws, c.err)
    torch.cuda.synchronize()
    assert float((out - ref).abs().max()) <= 4e-3  # both within 2e-3 of the exact values


def test_int4_appended_before_or_within():
    c = Int4Case([500, 64], 9, 20, 4, seed=7)
    masks = [tree(9, c.rng) for _ in range(2)]
    a = c.call(masks)
    before = c.tensors["pages"].clone()
    c.append()
    torch.cuda.synchronize()
    assert torch.equal(before, c.tensors["pages"])
    assert torch.equal(a, c.call(masks, append=False))


@pytest.mark.parametrize("sm", [-SM, 0.0, 1.0])
def test_int4_scales(sm):
    c = Int4Case([400, 90], 6, 10, 2, seed=8)
    masks = [tree(6, c.rng) for _ in range(2)]
    c.check(c.call(masks, sm=sm), masks, sm=sm)


@pytest.mark.parametrize("v_gain", [1e-6, 3e3, 1.1e4])
def test_int4_value_ranges(v_gain):
    c = Int4Case([300, 1], 6, 10, 2, seed=9, v_gain=v_gain)
    masks = [tree(6, c.rng) for _ in range(2)]
    out = c.call(masks)
    if v_gain >= 1:
        c.check(out, masks)
    else:  # tiny values: fp16 subnormals of the cache itself; only magnitudes
        assert bool(torch.isfinite(out).all()) and float(out.abs().max()) < 1e-4


@pytest.mark.parametrize("N,heads", [(60, (2, 1)), (16, (20, 4)), (12, (4, 2))])
@pytest.mark.parametrize("gain", [1.0 / 64, 5.0, 300.0])
def test_int4_key_scales(gain, N, heads):
    """Key scales on both sides of those that normalised keys have (M_k times a gain)."""
    c = Int4Case([0, 0], N, *heads, seed=19)
    c.Mk *= gain
    masks = [tree(N, c.rng), chain(N)]
    c.check(c.call(masks, sm=SM / gain), masks, sm=SM / gain)


def test_int4_bad_page_is_skipped():
    c = Int4Case([300, 300], 5, 8, 2, seed=10)
    masks = [tree(5, c.rng) for _ in range(2)]
    c.append()
    bt = c.tensors["block_table"]
    bt[0, 2] = 1 << 28
    out = c.call(masks, append=False, want_err=kvq.DEVERR_PAGE)
    c.tensors["block_table"][0, 2] = 0
    c.check(out, masks, hide=lambda b, L: (torch.arange(L, device="cuda") // 64 == 2) & (b == 0))


def test_int4_context_past_the_capacity_is_flagged():
    c = Int4Case([100, 50], 5, 8, 2, seed=11)
    c.append()
    c.ctx_t = i32([100, 1 << 29])
    c.call([tree(5, c.rng)] * 2, append=False, want_err=kvq.DEVERR_POS)
    c.err.zero_()
    c.ctx_t = i32([-5, 50])
    c.call([tree(5, c.rng)] * 2, append=False, want_err=kvq.DEVERR_POS)


def test_int4_repeats_bitwise_streams_and_graph():
    c = Int4Case([5000, 700, 64], 16, 20, 4, seed=12)
    masks = [tree(16, c.rng) for _ in range(3)]
    first = c.call(masks)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert torch.equal(first, c.call(masks, stream=s))
    ws = kvq.alloc_tree_workspace(3, 16, 20, 4)
    out, w = torch.zeros_like(first), words(masks)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.kvq_tree_attn_int4(c.cache, c.Mq, c.Mk, c.q, c.ctx_t, w, out, ws, c.err, k_new=c.k_new, v_new=c.v_new)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


@pytest.mark.parametrize("rows,heads", [(r, h) for r in (16, 17, 24, 25, 32, 33, 40, 41, 48, 49) for h in [(2, 2)]] +
                         [(r, (16, 1)) for r in (16, 32, 48, 64)])
def test_int4_rows_per_kv_head(rows, heads):
    c = Int4Case([3, 64, 190, 1500, 0, 127], rows // (heads[0] // heads[1]), *heads, seed=rows)
    masks = [tree(c.N, c.rng) for _ in range(c.B)]
    c.check(c.call(masks), masks)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,heads,copies", [(3, (2, 2), 1), (3, (2, 2), 200), (14, (2, 2), 1), (14, (2, 2), 300), (10, (4, 1), 150),
                                            (20, (4, 1), 1), (20, (4, 1), 150)])
def test_int4_empty_rows_of_every_size(N, heads, copies, out_dtype):
    c = Int4Case([0, 70, 0] * copies, N, *heads, seed=N + copies)
    masks = [[0 if i % 3 else 1 << i for i in range(N)], [0] * N, [0] * N] * copies
    out = c.call(masks, out_dtype)
    for b in range(0, c.B, 3):
        assert bool((out[b + 2] == 0).all()) and all(bool((out[b, i] == 0).all()) for i in range(N) if i % 3)
    c.B = min(c.B, 9)  # enough of the copies for the plain evaluation
    c.check(out, masks[:c.B])


@pytest.mark.parametrize("N,heads", [(2, (8, 2)), (8, (20, 4)), (16, (20, 4))])
def test_int4_a_far_larger_key_in_a_hidden_drafted_token(N, heads):
    """The scores of hidden drafted tokens may pass the visible ones by any amount."""
    c = Int4Case([130, 4], N, *heads, seed=77)
    c.v_new[:, N - 1] *= 100.0
    masks = [[w & ~(1 << (N - 1)) for w in chain(N)]] * 2
    a = c.call(masks, sm=1.0)
    c.check(a, masks, sm=1.0)
    c.k_new[:, N - 1] = -c.k_new[:, N - 1]
    assert torch.equal(a, c.call(masks, sm=1.0))


# ---------------------------------------------------------------- the ring

class RingCase:
    KS, VS = 6 / 448, 5 / 448

    def __init__(self, pos0, N, Hq, Hkv, window, seed=0, dtype=torch.bfloat16, capacity=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        self.pos0, self.N, self.Hq, self.Hkv, self.window, self.B = pos0, N, Hq, Hkv, window, len(pos0)
        self.cap = capacity or -(-(window + N - 1) // 64) * 64
        self.tensors, self.ring = kvq.alloc_fp8_ring(self.B, Hkv, self.cap)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        for b, p0 in enumerate(pos0):
            lo = max(0, p0 - window + 1)
            T = p0 - lo
            if T:
                k, v = (torch.randn(T, Hkv, D, generator=g, device="cuda").to(dtype) for _ in range(2))
                kvq.kvq_fp8_append(self.ring, k, v, i32([b] * T), torch.arange(lo, p0, device="cuda", dtype=torch.int32),
                                   self.KS, self.VS, self.err)
        self.k_new, self.v_new = (torch.randn(self.B, N, Hkv, D, generator=g, device="cuda").to(dtype) for _ in range(2))
        self.q = (torch.randn(self.B, N, Hq, D, generator=g, device="cuda") * 2).to(dtype)
        self.pos_t = i32(pos0)

    def call(self, masks, out_dtype=torch.float32):
        out = torch.full((self.B, self.N, self.Hq, D), 9.0, dtype=out_dtype, device="cuda")
        ws = kvq.alloc_tree_workspace(self.B, self.N, self.Hq, self.Hkv)
        kvq.kvq_tree_attn_fp8_swa(self.ring, self.q, self.pos_t, words(masks), self.window, self.KS, self.VS, out, ws,
                                  self.err, k_new=self.k_new, v_new=self.v_new)
        torch.cuda.synchronize()
        assert self.err.item() == 0
        return out

    def check(self, out, masks):
        G = self.Hq // self.Hkv
        ks, vs = (float(np.float32(x)) for x in (self.KS, self.VS))
        for b, p0 in enumerate(self.pos0):
            pos = np.arange(max(0, p0 - self.window + 1), p0 + self.N)
            at = [p0 + max(1, bin(w).count("1")) - 1 for w in masks[b]]
            seen = torch.tensor([[(p > at[i] - self.window) if p < p0 else bool((masks[b][i] >> int(p - p0)) & 1) for p in pos]
                                 for i in range(self.N)], device="cuda")
            for h in range(self.Hkv):
                kb, vb = unpack_fp8(self.tensors, b, h, pos)
                k, v = (torch.from_numpy(x.copy()).view(torch.float8_e4m3fn).double().cuda() for x in (kb, vb))
                for hq in range(h * G, (h + 1) * G):
                    o, tol = attend(self.q[b, :, hq].double(), k * ks, v * vs, seen, SM, out.dtype)
                    off = (out[b, :, hq].double() - o).abs()
                    assert bool((off <= tol).all()), (b, hq, float((off / tol).max()))


@pytest.mark.parametrize("N,window", [(1, 1), (1, 513), (8, 8), (16, 513), (33, 100), (64, 64), (64, 513), (5, 1500)])
@pytest.mark.parametrize("heads", [(20, 4), (8, 1)])
def test_ring_sizes(N, window, heads):
    c = RingCase([0, 1, 5, window, 700, 5001], N, *heads, window, seed=N + window)
    masks = [tree(N, c.rng) for _ in range(c.B)]
    c.check(c.call(masks), masks)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_ring_types(dtype, out_dtype):
    c = RingCase([600, 64], 12, 20, 4, 513, seed=2, dtype=dtype, capacity=1024)
    masks = [tree(12, c.rng), [0] * 12]
    c.check(c.call(masks, out_dtype), masks)


def test_ring_empty_rows():
    c = RingCase([0], 4, 4, 2, 64, seed=3)
    out = c.call([[0, 1, 0, 2]])
    assert bool((out[0, 0] == 0).all()) and bool((out[0, 2] == 0).all())
    c.check(out, [[0, 1, 0, 2]])


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("copies", [1, 40])
@pytest.mark.parametrize("N,heads,window", [(1, (20, 4), 513), (2, (20, 4), 100), (4, (20, 4), 513), (5, (8, 8), 5), (8, (2, 2), 513), (8, (6, 2), 8),
                                            (8, (3, 1), 4000), (3, (8, 1), 64), (8, (8, 2), 513)])
def test_ring_few_rows(N, heads, window, copies, out_dtype):
    """Few rows of one KV head, few and many sequences; trees, tokens that see nothing, tokens without themselves."""
    c = RingCase([0, 1, 5, window, 700, 5001] * copies, N, *heads, window, seed=N + window, dtype=torch.float32)
    masks = [[tree(N, c.rng), [0] * N, [(1 << 60) | (1 << (N - 1 - i)) for i in range(N)]][b % 3] for b in range(c.B)]
    keep = c.tensors["data"].clone()
    out = c.call(masks, out_dtype)
    c.B, c.pos0 = min(c.B, 18), c.pos0[:18]
    c.check(out, [[w & (1 << N) - 1 for w in m] for m in masks])
    now = c.tensors["data"].clone()
    c.tensors["data"].copy_(keep)  # the ring after the call: as after the separate append
    seq = torch.arange(len(masks), device="cuda", dtype=torch.int32).repeat_interleave(N)
    pos = (c.pos_t[:, None] + torch.arange(N, device="cuda", dtype=torch.int32)).flatten()
    kvq.kvq_fp8_append(c.ring, c.k_new.flatten(0, 1), c.v_new.flatten(0, 1), seq, pos, c.KS, c.VS, c.err)
    assert torch.equal(now, c.tensors["data"])


@pytest.mark.parametrize("N", [2, 10])
@pytest.mark.parametrize("bad", [-3, -(1 << 31), (1 << 31) - 1])
def test_ring_positions_outside_are_flagged(N, bad):
    c = RingCase([100, 700], N, 8, 2, 513, seed=6)
    masks = [tree(N, c.rng) for _ in range(2)]
    c.pos_t = i32([100, bad])
    was = c.tensors["data"].clone()
    out = torch.full((2, N, 8, D), 9.0, device="cuda")
    kvq.kvq_tree_attn_fp8_swa(c.ring, c.q, c.pos_t, words(masks), 513, c.KS, c.VS, out, kvq.alloc_tree_workspace(2, N, 8, 2), c.err,
                              k_new=c.k_new, v_new=c.v_new)
    torch.cuda.synchronize()
    assert c.err.item() == kvq.DEVERR_POS
    now = c.tensors["data"].clone()
    c.tensors["data"].copy_(was)  # new rows are written where their own positions are any
    rows = [(b, i) for b, p in enumerate([100, bad]) for i in range(N) if 0 <= p + i < 1 << 31]
    pick = lambda x: torch.stack([x[b, i] for b, i in rows])  # noqa: E731
    kvq.kvq_fp8_append(c.ring, pick(c.k_new), pick(c.v_new), i32([b for b, _ in rows]), i32([[100, bad][b] + i for b, i in rows]),
                       c.KS, c.VS, c.err)
    assert torch.equal(now, c.tensors["data"])
    c.tensors["data"].copy_(now)
    c.B, c.pos0 = 1, [100]  # the other sequence is as ever
    c.check(out, masks)


# ---------------------------------------------------------------- the commits

def logical4(c, b, L):
    return [unpack_int4(c.tensors, b, h, L) for h in range(c.Hkv)]


@pytest.mark.parametrize("N", [1, 8, 64])
def test_commit_int4_every_layer(N):
    layers = [Int4Case([0, 60, 64, 1000], N, 4, 2, seed=s) for s in (1, 2, 3)]
    for c in layers:
        c.append()
    path = np.stack([np.sort(layers[0].rng.permutation(N)) for _ in range(4)]).astype(np.int32)
    n = [0, 1, N, max(1, N // 2)]
    for b, a in enumerate(n):
        path[b, :a] = np.sort(layers[0].rng.choice(N, a, replace=False))
    before = [[logical4(c, b, c.ctx[b] + N) for b in range(4)] for c in layers]
    ctx_out = torch.zeros(4, dtype=torch.int32, device="cuda")
    err = layers[0].err
    kvq.kvq_tree_commit_int4([c.cache for c in layers], layers[0].ctx_t, i32(path), i32(n), err, ctx_out=ctx_out)
    torch.cuda.synchronize()
    assert err.item() == 0 and ctx_out.tolist() == [c + a for c, a in zip(layers[0].ctx, n)]
    for c, was in zip(layers, before):
        for b, a in enumerate(n):
            now, ctx = logical4(c, b, c.ctx[b] + N), c.ctx[b]
            for h in range(2):
                for key in ("kc", "ks", "ko", "vc", "vs", "vo"):
                    want = was[b][h][key].copy()
                    want[ctx:ctx + a] = was[b][h][key][ctx + path[b, :a]]
                    assert np.array_equal(now[h][key], want), (b, h, key)


def test_commit_any_path_reads_before_it_writes():
    c = Int4Case([50], 6, 2, 1, seed=4)
    c.append()
    was = unpack_int4(c.tensors, 0, 0, 56)
    path = [5, 5, 0, 1, 2, 3]
    kvq.kvq_tree_commit_int4([c.cache], c.ctx_t, i32([path]), i32([6]), c.err)
    now = unpack_int4(c.tensors, 0, 0, 56)
    assert c.err.item() == 0
    for key in was:
        assert np.array_equal(now[key][50:], was[key][50:][path])


def test_commit_flags_bad_paths_and_counts():
    c = Int4Case([50, 10], 4, 2, 1, seed=5)
    c.append()
    was = [unpack_int4(c.tensors, b, 0, c.ctx[b] + 4) for b in range(2)]
    out = torch.zeros(2, dtype=torch.int32, device="cuda")
    kvq.kvq_tree_commit_int4([c.cache], c.ctx_t, i32([[3, 99, -1, 2], [1, 2, 3, 3]]), i32([3, 9]), c.err, ctx_out=out)
    assert c.err.item() == kvq.DEVERR_POS and out.tolist() == [53, 14]
    now = [unpack_int4(c.tensors, b, 0, c.ctx[b] + 4) for b in range(2)]
    assert np.array_equal(now[0]["kc"][50:], was[0]["kc"][50:][[3, 1, 2, 3]])
    assert np.array_equal(now[1]["vc"][10:], was[1]["vc"][10:][[1, 2, 3, 3]])


def test_commit_fp8_around_the_ring():
    cs = [RingCase([0, 570, 1000], 10, 2, 2, 513, seed=s) for s in (1, 2)]
    for c in cs:
        c.call([tree(10, c.rng) for _ in range(3)])  # appends
    path, n = [[2, 4, 9] + [0] * 7, [1, 3, 5, 7, 9] + [0] * 5, [0, 1, 8] + [0] * 7], [3, 5, 3]
    was = [[[unpack_fp8(c.tensors, b, h, np.arange(p, p + 10)) for h in range(2)] for b, p in enumerate(c.pos0)] for c in cs]
    kvq.kvq_tree_commit_fp8([c.ring for c in cs], cs[0].pos_t, i32(path), i32(n), cs[0].err)
    torch.cuda.synchronize()
    assert cs[0].err.item() == 0
    for c, w in zip(cs, was):
        for b, p in enumerate(c.pos0):
            for h in range(2):
                now = unpack_fp8(c.tensors, b, h, np.arange(p, p + 10))
                for x, y in zip(now, w[b][h]):
                    want = y.copy()
                    want[:n[b]] = y[path[b][:n[b]]]
                    assert np.array_equal(x, want)
