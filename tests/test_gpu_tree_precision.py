"""Tile form of the trees: keys far smaller than normalised ones, a second group of few rows, and the layer stack's outputs.

Small keys: the tile holds (c s + o) 2^-9 in fp16. The value is rounded by 2^-11 of itself or by half of fp16's smallest
step, 2^-25; an offset below 2^-5 is rounded by as much before. Undoing the 2^-9 that is 2^-16 each, so beside the roundings
relative to the values (test_gpu_tree.py) a score is off by up to 2^-15 sum|q| sm.
"""

import math

import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq
from quantized_kv_cache_fold_gb300.runner import DecodeStack
from test_gpu_tree import SM, U, Int4Case, RingCase, chain, i32, tree

pytestmark = pytest.mark.gpu
D = 128


@pytest.mark.parametrize("N,heads", [(60, (2, 1)), (16, (20, 4)), (64, (8, 2))])
@pytest.mark.parametrize("gain", [2.0 ** -4, 2.0 ** -6, 2.0 ** -8, 2.0 ** -10])
def test_small_keys(gain, N, heads):
    c = Int4Case([0, 0], N, *heads, seed=23)
    c.Mk *= gain
    masks = [tree(N, c.rng), chain(N)]
    sm = SM / gain
    out = c.call(masks, sm=sm)
    x = c.q.double()
    q = (x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()) @ c.Mq64.T
    G = heads[0] // heads[1]
    for b in range(2):
        seen = torch.tensor([[bool((w >> j) & 1) for j in range(N)] for w in masks[b]], device="cuda")
        for h in range(heads[1]):
            k, v = c.dequantised(b, h, N)
            for hq in range(h * G, (h + 1) * G):
                p = torch.softmax(torch.where(seen, q[b, :, hq] @ k.T * sm, -math.inf), 1)
                mag = (seen * (q[b, :, hq].abs() @ k.abs().T)).amax(1, keepdim=True) * sm
                d = (2 * U + 136 * 2.0 ** -24) * mag + 2.0 ** -21 + 2.0 ** -15 * q[b, :, hq].abs().sum(1, keepdim=True) * sm
                tol = (torch.expm1(2 * d) + 2 * U) * (p @ v.abs()) + 1e-6
                off = (out[b, :, hq].double() - p @ v).abs()
                assert bool((off <= tol).all()), (b, hq, float((off / tol).max()))


@pytest.mark.parametrize("N,heads", [(43, (3, 1)), (26, (5, 1)), (33, (4, 1)), (35, (8, 2)), (52, (5, 1)), (64, (4, 1)), (9, (64, 1))])
def test_a_second_group_of_few_rows(N, heads):
    """129 to 140 rows of a KV head, 260, 256 and 576."""
    c = Int4Case([0, 64, 190, 1500], N, *heads, seed=N)
    masks = [tree(N, c.rng) for _ in range(c.B)]
    c.check(c.call(masks), masks)
    r = RingCase([0, 64, 1000], N, *heads, 100, seed=N)
    masks = [tree(N, r.rng) for _ in range(r.B)]
    r.check(r.call(masks, torch.bfloat16), masks)


@pytest.mark.parametrize("N", [3, 12])
def test_the_stacks_outputs_are_the_calls_outputs(N):
    """tree_step and prompt_layer against the calls over the same layers, bit for bit (those are tested against 64 bits)."""
    B, Hq, Hkv, lens = 2, 20, 4, [130, 77]
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    st = DecodeStack(B, Hq, Hkv, 1, 4, n_layers=2, full_every=2, window=64, ring_capacity=128, swa_k_scale=6 / 448, swa_v_scale=5 / 448)
    st.set_int4_params(1, 4, *(torch.rand(D, generator=torch.Generator().manual_seed(i)).add(0.5).numpy() for i in range(2)))
    T, cu = sum(lens), i32([0, lens[0], sum(lens)])
    seq, pos = i32([b for b in range(B) for _ in range(lens[b])]), i32([p for b in range(B) for p in range(lens[b])])
    late = torch.tensor([p >= lens[b] - 64 for b in range(B) for p in range(lens[b])], device="cuda")
    for l in range(2):
        q, k, v = rand(T, Hq, D), rand(T, Hkv, D), rand(T, Hkv, D)
        got, want = torch.zeros_like(q), torch.ones_like(q)
        st.prompt_layer(l, q, k, v, cu, got)
        kvq.kvq_prompt_attn(q, k, v, cu, want, kvq.alloc_prompt_workspace(T, B, Hq, Hkv), st.dev_err, window=0 if l else 64)
        assert torch.equal(got, want)
        keep = torch.ones_like(late) if l else late
        st.append_prompt(l, k[keep].contiguous(), v[keep].contiguous(), seq[keep].contiguous(), pos[keep].contiguous())
    masks = torch.tensor([chain(N)] * B, device="cuda")
    qs, ks, vs = ([rand(B, N, h, D) for _ in range(2)] for h in (Hq, Hkv, Hkv))
    got, want = ([torch.full((B, N, Hq, D), x, device="cuda") for _ in range(2)] for x in (7.0, 9.0))
    st.tree_step(qs, i32(lens), masks, got, ks, vs)
    ws, R, F = kvq.alloc_tree_workspace(B, N, Hq, Hkv), st.layers[0], st.layers[1]
    kvq.kvq_tree_attn_fp8_swa(R.ring, qs[0], i32(lens), masks, 64, R.k_scale, R.v_scale, want[0], ws, st.dev_err)
    kvq.kvq_tree_attn_int4(F.cache, F.Mq, F.Mk, qs[1], i32(lens), masks, want[1], ws, st.dev_err)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and st.read_error() == 0


@pytest.mark.parametrize("v_gain", [1e-3, 1.0, 2e3])
@pytest.mark.parametrize("N,heads", [(3, (2, 2)), (4, (4, 1)), (7, (12, 4)), (8, (20, 4)), (16, (20, 4))])
def test_rows_of_one_key_are_its_value(N, heads, v_gain):
    """No context and one bit: the output is the dequantised value. Row kernels (up to 48 rows per KV head): its weight is a
    power of two, so code and offset terms are off by fp32 roundings of the record's range; tiles: the value in fp16."""
    c = Int4Case([0, 0], N, *heads, seed=31, v_gain=v_gain)
    at = [[(5 * i + b) % N for i in range(N)] for b in range(2)]
    out = c.call([[1 << j for j in a] for a in at]).double()
    G = heads[0] // heads[1]
    few = N * G <= 48
    for b in range(2):
        for h in range(heads[1]):
            _, v = c.dequantised(b, h, N)
            want = v[at[b]][:, None]
            tol = 2.0 ** -23 * (v.amax(1) - v.amin(1) + v.abs().amax(1))[at[b]][:, None, None] + (0.0 if few else U * want.abs() + 2.0 ** -25)
            assert bool(((out[b, :, h * G:(h + 1) * G] - want).abs() <= tol).all())
