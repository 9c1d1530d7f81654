"""kvq_prompt_attn_sinks against a plain evaluation in 64 bits; the tolerance is that of test_gpu_prompt.py (the same
roundings: more keys are seen, nothing else changes)."""

import math

import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq
from test_gpu_prompt import check, inputs, offsets

pytestmark = pytest.mark.gpu
D = 128


def reference(q, k, v, lens, window, sinks, sm=D ** -0.5):
    u = torch.finfo(q.dtype).eps / 2
    Hq, Hkv = q.shape[1], k.shape[1]
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    at = 0
    for n in lens:
        s = slice(at, at + n)
        at += n
        if n == 0:
            continue
        j = torch.arange(n, device=q.device)
        seen = (j[None] <= j[:, None]) & ((j[None] > j[:, None] - window) | (j[None] < sinks))
        for h in range(Hq):
            Q, K, V = q[s, h].double(), k[s, h * Hkv // Hq].double(), v[s, h * Hkv // Hq].double()
            z = torch.where(seen, torch.nan_to_num(Q, 0, 0, 0) @ torch.nan_to_num(K, 0, 0, 0).T * sm, -math.inf)
            bad = torch.where(seen, (Q @ K.T) * sm, 0.0)
            p = torch.softmax(torch.where(torch.isfinite(bad) | ~seen, z, bad), 1)
            vz = torch.nan_to_num(V, 0, 0, 0)
            o[s, h] = p @ vz
            for c in torch.unique(torch.nonzero(~torch.isfinite(V))[:, 0]).tolist():
                rows = seen[:, c]
                o[s, h][rows] += p[rows, c:c + 1] * torch.where(torch.isfinite(V[c]), 0.0, V[c])
            mag = (seen * (Q.abs() @ K.abs().T)).nan_to_num(0, 0, 0).amax(1, keepdim=True) * sm
            d = 136 * 2.0 ** -24 * mag + 2.0 ** -21
            tol[s, h] = u * o[s, h].abs() + (u + 2 * d) * (p @ vz.abs()) + 1e-30
            if q.dtype == torch.float16:
                tol[s, h] += 2.0 ** -25  # half the smallest fp16 step
    return o, tol


def call(q, k, v, lens, window, sinks, stream=None, out=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if out is None else out
    cu = offsets(lens)
    ws = kvq.alloc_prompt_workspace(q.shape[0], len(lens), q.shape[1], k.shape[1])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    kvq.kvq_prompt_attn(q, k, v, cu, out, ws, err, window=window, sinks=sinks, stream=stream)
    torch.cuda.synchronize()
    assert err.item() == 0
    return out


# sinks around a block's end and past it, windows that meet them, overlap them, start one block or several behind them
@pytest.mark.parametrize("sinks", [1, 4, 127, 128, 129, 300, 1 << 30])
@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 257, 513, 1 << 30])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_windows_and_first_tokens(window, sinks, dtype):
    lens = [1030, 1, 129, 0, 300, 700]
    q, k, v = inputs(lens, 4, 2, dtype, seed=(window + sinks) % 97)
    check(call(q, k, v, lens, window, sinks), *reference(q, k, v, lens, window, sinks))


# odd groups take items of 256 rows of one head, whose tiles differ in their blocks
@pytest.mark.parametrize("heads", [(3, 3), (5, 1), (20, 4), (6, 2)])
@pytest.mark.parametrize("window,sinks", [(128, 4), (513, 64), (130, 200)])
def test_groups_of_heads(heads, window, sinks):
    lens = [1500, 257, 3, 385]
    q, k, v = inputs(lens, *heads, torch.bfloat16, seed=heads[0], fused=True)
    check(call(q, k, v, lens, window, sinks), *reference(q, k, v, lens, window, sinks))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_values_that_are_not_finite(dtype):
    """In a first token: in every row. Between the first tokens and a window, or behind a row: in none of it."""
    lens = [900, 140, 650]
    q, k, v = inputs(lens, 3, 1, dtype, seed=5)
    for tok, x in ((2, math.inf), (300, math.nan), (450, -math.inf), (901, math.nan), (1045, math.inf), (1400, math.nan)):
        v[tok, 0, tok % D] = x
    k[650, 0, 3] = math.nan
    out = call(q, k, v, lens, 150, 4)
    check(out, *reference(q, k, v, lens, 150, 4))
    assert torch.isfinite(out[520:600]).sum() > 0 and not torch.isfinite(out[899, :, 2]).any()


def test_large_scores_of_first_tokens():
    """First tokens that gather nearly all weight, as models with sinks have them: the base is set by the first block."""
    lens = [1200, 333]
    q, k, v = inputs(lens, 4, 2, torch.bfloat16, seed=6)
    k[0] = q[:1200, ::2].float().mean(0).to(k.dtype) * 20
    k[1200] = 0
    check(call(q, k, v, lens, 200, 4), *reference(q, k, v, lens, 200, 4))


def test_equal_to_the_window_or_causal_call():
    """No row's result depends on the form that computes it where the visible tokens are the same: compared in the type."""
    lens = [600, 77]
    q, k, v = inputs(lens, 4, 2, torch.bfloat16, seed=7)
    full = call(q, k, v, lens, 0, 0)
    assert torch.equal(call(q, k, v, lens, 0, 4), full)           # no window: the causal call
    assert torch.equal(call(q, k, v, lens, 1 << 20, 4), full)     # a window that holds everything
    assert torch.equal(call(q, k, v, lens, 5, 600), full)         # first tokens that are everything


def test_repeats_stream_and_graph():
    lens = [700, 1, 513]
    q, k, v = inputs(lens, 20, 4, torch.bfloat16, seed=8)
    want = call(q, k, v, lens, 300, 17)
    other = torch.cuda.Stream()
    assert torch.equal(call(q, k, v, lens, 300, 17, stream=other), want)
    out, cu = torch.zeros_like(want), offsets(lens)
    ws, err = kvq.alloc_prompt_workspace(q.shape[0], 3, 20, 4), torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.kvq_prompt_attn(q, k, v, cu, out, ws, err, window=300, sinks=17)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and err.item() == 0


def test_rows_behind_the_last_sequence_stay():
    q, k, v = inputs([500, 40], 4, 2, torch.bfloat16, seed=9)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    call(q, k, v, [500], 100, 4, out=out)
    assert bool((out[500:] == 7).all()) and bool((out[:500] != 7).any())
