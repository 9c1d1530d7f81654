"""kvq_window_attn_int4 against a plain evaluation in 64 bits; tolerances are those of test_gpu_tree.py (the same roundings
of q~ and of the weights)."""

import math

import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq
from test_gpu_tree import D, SM, Int4Case, attend

pytestmark = pytest.mark.gpu


def call(c, window, sinks, out_dtype=torch.float32, append=True, want_err=0, stream=None, sm=SM):
    out = torch.full((c.B, c.N, c.Hq, D), 9.0, dtype=out_dtype, device="cuda")
    ws = kvq.alloc_workspace(c.B, c.N, c.Hq, c.Hkv)
    new = (c.k_new, c.v_new) if append else (None, None)
    torch.cuda.synchronize()
    kvq.kvq_window_attn_int4(c.cache, c.Mq, c.Mk, c.q, c.ctx_t, window, sinks, out, ws, c.err, k_new=new[0], v_new=new[1],
                             sm_scale=sm, fwht=c.fwht, stream=stream)
    torch.cuda.synchronize()
    assert c.err.item() == want_err
    return out


def check(c, out, window, sinks, sm=SM, rows=None):
    x = c.q.double()
    q = (x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()) @ c.Mq64.T
    G = c.Hq // c.Hkv
    for b in range(c.B) if rows is None else rows:
        L = c.ctx[b] + c.N
        j = torch.arange(L, device="cuda")[None]
        i = c.ctx[b] + torch.arange(c.N, device="cuda")[:, None]
        seen = (j <= i) & ((j > i - window) | (j < sinks))
        for h in range(c.Hkv):
            k, v = c.dequantised(b, h, L)
            for hq in range(h * G, (h + 1) * G):
                o, tol = attend(q[b, :, hq], k, v, seen, sm, out.dtype)
                off = (out[b, :, hq].double() - o).abs()
                assert bool((off <= tol).all()), (b, hq, float((off / tol).max()))


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 130, 500, 1 << 30, 2 ** 31 - 1])
@pytest.mark.parametrize("sinks", [0, 1, 4, 63, 64, 65, 200, 2 ** 31 - 1])
@pytest.mark.parametrize("S", [1, 4])
def test_windows_and_first_tokens(window, sinks, S):
    c = Int4Case([0, 1, 62, 63, 64, 65, 200, 700], S, 10, 2, seed=(window + sinks) % 89)
    check(c, call(c, window, sinks), window, sinks)


# every tile count of the kernel: 1..6 tiles of 8 rows
@pytest.mark.parametrize("S,heads", [(1, (2, 2)), (8, (2, 2)), (2, (20, 4)), (3, (20, 4)), (5, (20, 4)), (7, (20, 4)),
                                     (8, (20, 4)), (8, (6, 1)), (1, (48, 1)), (1, (33, 1))])
@pytest.mark.parametrize("window,sinks", [(100, 4), (7, 0), (129, 70)])
def test_rows_of_a_head(S, heads, window, sinks):
    c = Int4Case([400, 5, 64, 1000], S, *heads, seed=S)
    check(c, call(c, window, sinks), window, sinks)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fwht", [False, True])
def test_types_and_prologues(out_dtype, dtype, fwht):
    c = Int4Case([300, 129], 3, 20, 4, seed=3, dtype=dtype, fwht=fwht)
    check(c, call(c, 90, 5, out_dtype), 90, 5)


def test_long_and_ragged():
    c = Int4Case([9000, 3, 2500, 16, 4097], 1, 20, 4, seed=4)
    check(c, call(c, 2000, 64), 2000, 64)
    c = Int4Case([(i * 7) % 300 for i in range(500)], 2, 4, 2, seed=15)
    check(c, call(c, 70, 3), 70, 3)


def test_everything_visible_is_the_decode_call():
    c = Int4Case([777, 1000], 8, 20, 4, seed=6)
    out = call(c, 1 << 20, 0)
    ref = torch.empty_like(out)
    ws = kvq.alloc_workspace(2, 8, 20, 4)
    kvq.kvq_decode_attn_int4(c.cache, c.Mq, c.Mk, c.q, c.ctx_t, ref, ws, c.err)
    torch.cuda.synchronize()
    assert float((out - ref).abs().max()) <= 4e-3  # both within 2e-3 of the exact values


def test_pages_between_are_not_read():
    """The block-table entries between the first tokens and the windows name no page; the records there are not finite."""
    c = Int4Case([1000, 640], 2, 10, 2, seed=7)
    c.append()
    want = call(c, 100, 70, append=False)
    bt = c.tensors["block_table"]
    for b, last in ((0, (1000 - 99) // 64), (1, (640 - 99) // 64)):
        for p in range(2, last):
            c.tensors["pages"][bt[b, p].long()] = 255
            bt[b, p] = -1 if p % 2 else 1 << 30
    torch.cuda.synchronize()
    assert torch.equal(call(c, 100, 70, append=False), want)


def test_hidden_records_that_are_not_finite():
    """Slots of visible pages outside the window, and behind the last row, hold infinite and NaN scales."""
    c = Int4Case([300, 300], 1, 10, 2, seed=8, extra_pages=1)
    c.append()
    want = call(c, 37, 3, append=False)
    page = c.tensors["block_table"].long()
    meta = c.tensors["pages"][:, :, 8192:8704].view(torch.int32)  # K words 0..63, V words 64..127
    for b in range(2):
        for pos, word in ((3, 0x7E007E00), (63, 0x7C007C00), (263, 0x7E00FC00), (301, 0x7E007E00), (319, 0x7C007C00)):
            meta[page[b, pos // 64], :, pos % 64] = word
            meta[page[b, pos // 64], :, 64 + pos % 64] = word
    c.tensors["pages"][:, :, 8192:8704] = meta.view(torch.uint8)
    torch.cuda.synchronize()
    got = call(c, 37, 3, append=False)
    assert bool(torch.isfinite(got).all()) and torch.equal(got, want)


def test_bad_pages_and_lengths():
    c = Int4Case([300, 300, 40], 1, 8, 2, seed=9)
    c.append()
    bt = c.tensors["block_table"]
    bt[0, 4] = -5            # inside row 0's window
    bt[2, 0] = 1 << 20       # all that row 2 sees
    torch.cuda.synchronize()
    out = call(c, 100, 4, append=False, want_err=kvq.DEVERR_PAGE)
    assert bool((out[2] == 0).all()) and bool(torch.isfinite(out).all())
    check(c, out, 100, 4, rows=[1])
    c = Int4Case([100, 100], 2, 8, 2, seed=10)
    c.append()
    c.ctx_t[0] = 1 << 20
    out = call(c, 50, 4, append=False, want_err=kvq.DEVERR_POS)
    check(c, out, 50, 4, rows=[1])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_queries_that_are_not_finite(bad):
    c = Int4Case([200, 90], 2, 10, 2, seed=11, dtype=torch.float32)
    c.append()
    want = call(c, 60, 4, append=False)
    c.q[1, 0, 3, 17] = bad
    got = call(c, 60, 4, append=False, want_err=kvq.DEVERR_NONFINITE)
    assert bool(torch.isnan(got[1, 0, 3]).all())
    got[1, 0, 3] = want[1, 0, 3]
    assert torch.equal(got, want)


def test_repeats_stream_and_graph():
    c = Int4Case([900, 64, 5000], 3, 20, 4, seed=12)
    c.append()
    want = call(c, 513, 17, append=False)
    assert torch.equal(call(c, 513, 17, append=False, stream=torch.cuda.Stream()), want)
    ws = kvq.alloc_workspace(3, 3, 20, 4)
    out, other = torch.zeros_like(want), torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.kvq_window_attn_int4(c.cache, c.Mq, c.Mk, c.q, c.ctx_t, 513, 17, out, ws, c.err)
        kvq.kvq_window_attn_int4(c.cache, c.Mq, c.Mk, c.q, c.ctx_t, 2000, 0, other, ws, c.err)
    for n in ([900, 64, 5000], [5, 3000, 4990]):
        c.ctx_t.copy_(torch.tensor(n, dtype=torch.int32))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert c.err.item() == 0
        assert torch.equal(out, call(c, 513, 17, append=False)) and torch.equal(other, call(c, 2000, 0, append=False))


def test_two_calls_at_once():
    cases = [Int4Case([900, 30, 2000], 4, 20, 4, seed=30 + i) for i in range(2)]
    for c in cases:
        c.append()
    want = [call(c, 300, 5, append=False) for c in cases]
    outs, ws = [torch.zeros_like(w) for w in want], [kvq.alloc_workspace(3, 4, 20, 4) for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, o, w, s in zip(cases, outs, ws, streams):
            kvq.kvq_window_attn_int4(c.cache, c.Mq, c.Mk, c.q, c.ctx_t, 300, 5, o, w, c.err, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want)) and all(c.err.item() == 0 for c in cases)


@pytest.mark.parametrize("S", [1, 4])
def test_rows_written_by_the_call_before(S):
    """A step's rows are appended by the call, the next step's window reads them: steps in a row without a wait between."""
    c = Int4Case([60, 127, 500], S, 20, 4, seed=33)
    ws = kvq.alloc_workspace(3, S, 20, 4)
    g = torch.Generator(device="cuda").manual_seed(5)
    steps = 8
    P = c.tensors["block_table"].shape[1]
    table = torch.arange(3 * (P + 2), dtype=torch.int32, device="cuda").reshape(3, P + 2)
    tensors, cache = kvq.alloc_int4_cache(3 * (P + 2), 4, table)
    for b in range(3):
        tensors["pages"][table[b, :P].long()] = c.tensors["pages"][c.tensors["block_table"][b].long()]
    new = [[torch.randn(3, S, 4, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)] for _ in range(steps)]
    ctx = [c.ctx_t + S * i for i in range(steps + 1)]
    outs = [torch.zeros(3, S, 20, D, device="cuda") for _ in range(steps)]
    start = tensors["pages"].clone()
    got = []
    for wait in (False, True):
        tensors["pages"].copy_(start)
        torch.cuda.synchronize()
        for i in range(steps):
            kvq.kvq_window_attn_int4(cache, c.Mq, c.Mk, c.q, ctx[i], 70, 3, outs[i], ws, c.err, k_new=new[i][0], v_new=new[i][1])
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        got.append([o.clone() for o in outs])
    assert all(torch.equal(a, b) for a, b in zip(*got)) and c.err.item() == 0


def test_tensors_that_do_not_fit():
    c = Int4Case([100, 20], 2, 10, 2, seed=34)
    ws, out = kvq.alloc_workspace(2, 2, 10, 2), torch.empty(2, 2, 10, D, device="cuda")
    args = dict(cache=c.cache, Mq=c.Mq, Mk=c.Mk, q=c.q, ctx_len=c.ctx_t, window=10, sinks=1, out=out, workspace=ws, dev_err=c.err)
    for bad in (dict(q=c.q[:, :, :, ::2]), dict(q=c.q.half()), dict(q=c.q.cpu()), dict(out=out[:1]), dict(out=out.half()), dict(ctx_len=c.ctx_t.long()),
                dict(ctx_len=c.ctx_t[:1]), dict(Mq=c.Mq[:64]), dict(k_new=c.k_new[:, :1], v_new=c.v_new), dict(dev_err=c.err.long()),
                dict(workspace=ws.cpu())):
        with pytest.raises(ValueError):
            kvq.kvq_window_attn_int4(**{**args, **bad})
    for bad in (dict(window=0), dict(sinks=-1), dict(workspace=ws[:256]), dict(k_new=c.k_new)):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_window_attn_int4(**{**args, **bad})
