"""kvq_prompt_attn against a plain evaluation in 64 bits.

The tolerance, per output element, from the roundings that the call makes (u: half a step of the
16-bit type relative to the value, torch.finfo(t).eps / 2): the output is rounded once (u |o|), each
weight p is rounded to the type before the product with v (u sum p|v| / sum p), and an error d of a
score changes a weight by the factor exp(d), on either side of the division: 2 d sum p|v| / sum p.
A score is a fp32 sum of 128 products (at most 136 half steps of the sum of magnitudes, with the
scale and the base subtracted) and its power of two comes from ex2.approx (2^-21 is above its error).
"""

import math

import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq

pytestmark = pytest.mark.gpu
D = 128


def reference(q, k, v, lens, window, sm):
    """(o, bound) in fp64: the outputs and the tolerance of each element."""
    u = torch.finfo(q.dtype).eps / 2
    Hq, Hkv = q.shape[1], k.shape[1]
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    at = 0
    for n in lens:
        if n == 0:
            continue
        s = slice(at, at + n)
        i = torch.arange(n, device=q.device)
        seen = i[None, :] <= i[:, None]
        if window > 0:
            seen &= i[None, :] > i[:, None] - window
        for h in range(Hq):
            Q, K, V = q[s, h].double(), k[s, h * Hkv // Hq].double(), v[s, h * Hkv // Hq].double()
            # what a masked place holds does not count
            z = torch.where(seen, torch.nan_to_num(Q, 0, 0, 0) @ torch.nan_to_num(K, 0, 0, 0).T * sm, -math.inf)
            bad = torch.where(seen, (Q @ K.T) * sm, 0.0)
            z = torch.where(torch.isfinite(bad) | ~seen, z, bad)
            p = torch.softmax(z, 1)
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
        at += n
    return o, tol


def offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def inputs(lens, Hq, Hkv, dtype, seed=0, fused=False, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens)
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda")
    x[:, :Hq + Hkv] *= gain
    x = x.to(dtype)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def call(q, k, v, lens, window=0, sm=D ** -0.5, out=None, cu=None, want_err=0, stream=None):
    cu = offsets(lens) if cu is None else cu
    B = cu.numel() - 1
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if out is None else out
    ws = kvq.alloc_prompt_workspace(q.shape[0], B, q.shape[1], k.shape[1])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.kvq_prompt_attn(q, k, v, cu, out, ws, err, window=window, sm_scale=sm, stream=stream)
    torch.cuda.synchronize()
    assert err.item() == want_err
    return out


def check(out, o, tol):
    assert torch.equal(torch.isfinite(out), torch.isfinite(o))
    fine = torch.isfinite(o)
    off = (out.double() - o).abs()[fine]
    assert bool((off <= tol[fine]).all()), f"worst {float((off / tol[fine]).max()):.2f} of the tolerance"


LENS = [[1], [2, 1, 3], [64, 65, 63], [127, 128, 129], [255, 256, 257, 1], [0, 5, 0, 300, 0], [513, 33, 1000, 700],
        [1, 1, 1, 1, 1, 1, 1, 1, 40]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("heads", [(20, 4), (3, 3), (8, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_lengths_heads_types(lens, heads, dtype):
    q, k, v = inputs(lens, *heads, dtype, seed=len(lens))
    check(call(q, k, v, lens), *reference(q, k, v, lens, 0, D ** -0.5))


@pytest.mark.parametrize("window", [1, 2, 64, 127, 128, 129, 200, 256, 513, 1 << 30])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_windows(window, dtype):
    lens = [700, 1, 129, 300, 1030]
    q, k, v = inputs(lens, 4, 2, dtype, seed=window % 97)
    check(call(q, k, v, lens, window), *reference(q, k, v, lens, window, D ** -0.5))


@pytest.mark.parametrize("lens", [[300, 7, 129], [1]])
def test_views_of_a_fused_projection(lens):
    q, k, v = inputs(lens, 20, 4, torch.bfloat16, seed=3, fused=True)
    whole = torch.full((sum(lens), 24, D), 5.0, dtype=q.dtype, device="cuda")
    out = whole[:, 2:22]
    check(call(q, k, v, lens, out=out), *reference(q, k, v, lens, 0, D ** -0.5))
    assert bool((whole[:, :2] == 5).all() and (whole[:, 22:] == 5).all())


def test_heads_outermost():
    lens = [200, 150]
    q, k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in inputs(lens, 6, 2, torch.float16, seed=4))
    out = torch.empty_like(q)
    assert out.stride(0) == D
    check(call(q, k, v, lens, out=out), *reference(q, k, v, lens, 0, D ** -0.5))


@pytest.mark.parametrize("gain", [0.0, 4.0, 12.0])
@pytest.mark.parametrize("sm", [D ** -0.5, 1e-4, 0.5])
def test_score_ranges(gain, sm):
    """From equal weights to one key taking all: the running maximum moves often and far."""
    lens = [400, 260]
    q, k, v = inputs(lens, 4, 2, torch.bfloat16, seed=5, gain=gain)
    check(call(q, k, v, lens, sm=sm), *reference(q, k, v, lens, 0, sm))


def test_climbing_and_falling_scores():
    n = 1100
    q, k, v = inputs([n], 2, 1, torch.bfloat16, seed=6)
    ramp = torch.linspace(-60, 60, n, device="cuda")[:, None, None]
    q = torch.ones_like(q)
    for r in (ramp, -ramp):
        k2 = (r * D ** -0.5 + 0.1 * k.float()).to(k.dtype)
        check(call(q, k2, v, [n]), *reference(q, k2, v, [n], 0, D ** -0.5))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", ["v", "k"])
@pytest.mark.parametrize("window", [0, 70])
def test_masked_places_do_not_count(bad, which, window):
    """Later tokens, tokens before the window and the neighbouring sequences hold non-finite values."""
    lens = [150, 300, 90]
    q, k, v = inputs(lens, 4, 2, torch.bfloat16, seed=7)
    x = {"k": k, "v": v}[which]
    x[150 + 200] = bad           # inside: rows 200.. (or the window's) see it
    x[150 + 299, 0, 5] = bad     # the last token, one element
    x[150 + 3] = bad if window else 1.0
    x[450] = bad                 # the first token of the next sequence
    out = call(q, k, v, lens, window)
    o, tol = reference(q, k, v, lens, window, D ** -0.5)
    if which == "k" and math.isinf(bad):
        # q.k with infinities of both signs: rows that see one are not compared, the others are
        at = torch.arange(540, device="cuda")
        hit = torch.zeros(540, dtype=torch.bool, device="cuda")
        for t, end in ((350, 450), (449, 450), (153, 450), (450, 540)):
            if t == 153 and not window:
                continue
            hit |= (at >= t) & (at < end) & ((at < t + window) if window else True)
        check(out[~hit], o[~hit], tol[~hit])
    else:
        check(out, o, tol)


def test_all_keys_nan_is_nan_not_a_hang():
    q, k, v = inputs([600], 2, 1, torch.bfloat16, seed=8)
    assert bool(torch.isnan(call(q, k, torch.full_like(v, math.nan), [600])).all())


def test_rows_behind_the_last_sequence_stay():
    lens = [130, 20]
    q, k, v = inputs(lens + [50], 4, 2, torch.bfloat16, seed=9)
    out = call(q, k, v, lens)
    assert bool((out[150:] == 7).all())
    o, tol = reference(q, k, v, lens, 0, D ** -0.5)
    check(out[:150], o[:150], tol[:150])


def test_bad_offsets_are_flagged_and_skipped():
    q, k, v = inputs([100, 100], 2, 1, torch.bfloat16, seed=10)
    cu = torch.tensor([0, 100, 60, 200, 260], dtype=torch.int32, device="cuda")  # back, and past the end
    out = call(q, k, v, None, cu=cu, want_err=kvq.DEVERR_POS)
    o, tol = reference(q, k, v, [60], 0, D ** -0.5)
    check(out[:60], o[:60], tol[:60])


def test_long_prompt_sampled_rows():
    n = 20001
    q, k, v = inputs([n], 5, 1, torch.bfloat16, seed=11)
    out = call(q, k, v, [n])
    rows = [0, 1, 127, 128, 255, 256, 5000, 12345, 19967, 19968, n - 1]
    u = torch.finfo(q.dtype).eps / 2
    for r in rows:
        for h in (0, 4):
            Q, K, V = q[r, h].double(), k[:r + 1, 0].double(), v[:r + 1, 0].double()
            p = torch.softmax(K @ Q * D ** -0.5, 0)
            o = p @ V
            d = 136 * 2.0 ** -24 * float((K.abs() @ Q.abs()).max()) * D ** -0.5 + 2.0 ** -21
            tol = u * o.abs() + (u + 2 * d) * (p @ V.abs())
            assert bool(((out[r, h].double() - o).abs() <= tol).all()), (r, h)


def test_many_sequences():
    lens = [1 + (i * 37) % 41 for i in range(1024)]
    q, k, v = inputs(lens, 2, 1, torch.float16, seed=12)
    check(call(q, k, v, lens), *reference(q, k, v, lens, 0, D ** -0.5))


def test_repeated_calls_are_bitwise_equal_on_other_streams_and_in_a_graph():
    lens = [333, 1, 700]
    q, k, v = inputs(lens, 20, 4, torch.bfloat16, seed=13)
    first = call(q, k, v, lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert torch.equal(first, call(q, k, v, lens, stream=s))
    cu, err = offsets(lens), torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(2)]
    ws = [kvq.alloc_prompt_workspace(sum(lens), 3, 20, 4) for _ in range(2)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.kvq_prompt_attn(q, k, v, cu, outs[0], ws[0], err)
        kvq.kvq_prompt_attn(q, k, v, cu, outs[1], ws[1], err, window=100)
    for _ in range(3):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], first)
        assert torch.equal(outs[1], call(q, k, v, lens, 100))


def test_two_streams_at_once():
    lens = [900, 40]
    ins = [inputs(lens, 8, 2, torch.bfloat16, seed=20 + i) for i in range(2)]
    want = [call(*x, lens) for x in ins]
    cu, err = offsets(lens), torch.zeros(1, dtype=torch.int32, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [kvq.alloc_prompt_workspace(940, 2, 8, 2) for _ in range(2)]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            kvq.kvq_prompt_attn(*ins[i], cu, outs[i], ws[i], err, stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want)) and err.item() == 0
