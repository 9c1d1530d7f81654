"""Attention where a few keys take nearly all weight and hold zero values, so that the output is what the many others add,
each 17 to 20 nats below: weights far under the smallest step of fp16 relative to the largest one.

Tolerance per output element, u = 2^-11 (fp16): the trees' terms are those of test_gpu_tree.py (a score off by at most
d = 2 u sum|q k| sm and its fp32 sum; a weight off by exp(d) above and below the division; one rounding of each weight and
of each value), and a term for weights below fp16's normal range: half a step of 2^-24, where the largest weight of the same
row stands at 2^6 or above (the exponents' base keeps it between 2^7 and 2^15, and the factor of a value's scale in the row
kernels, up to its power of two, takes one bit): 2^-31 of the largest weight per key, times the largest |v|. The output's
own rounding is added (fp16: half a step, at least 2^-25).
"""

import numpy as np
import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq
from gpu_util import unpack_fp8
from test_gpu_tree import Int4Case, RingCase, i32, words

pytestmark = pytest.mark.gpu
D, U = 128, 2.0 ** -11


def keys_and_values(n, Hkv, u, every, gain, g):
    """[n, Hkv, 128]: keys orthogonal to u with values of +-gain per dim; every `every`-th: the key u with the value 0."""
    k = torch.randn(n, Hkv, D, generator=g, device="cuda")
    k -= (k @ u / (u @ u))[..., None] * u
    sign = torch.randn(D, generator=g, device="cuda").sign()
    v = gain * (sign + 0.2 * torch.randn(n, Hkv, D, generator=g, device="cuda"))
    k[::every], v[::every] = u, 0.0
    return k, v


def direction(g):
    u = torch.randn(D, generator=g, device="cuda")
    return u * (D / (u @ u)).sqrt()


def expect(out, q, k, v, seen, sm, roundings):
    """out, q [R, 128], k, v [L, 128] in fp64, seen [R, L]; roundings: of a score's terms (q, k) in halves of a step."""
    z = torch.where(seen, q @ k.T * sm, -torch.inf)
    p = torch.softmax(z, 1)
    o = p @ v
    mag = (seen * (q.abs() @ k.abs().T)).amax(1, keepdim=True) * sm
    d = roundings * U * mag + 136 * 2.0 ** -24 * mag + 2.0 ** -21
    tol = (2 * d + 2 * U) * (p @ v.abs()) + 2.0 ** -31 * seen.sum(1, keepdim=True) * p.amax(1, keepdim=True) * v.abs().max()
    if out.dtype != torch.float32:
        tol = tol + torch.finfo(out.dtype).eps / 2 * o.abs() + (2.0 ** -25 if out.dtype == torch.float16 else 0.0)
    off = (out.double() - o).abs()
    assert bool((off <= tol).all()), f"worst {float((off / tol).max()):.2f} of the tolerance"


BELOW = [12.0, 17.0, 18.0, 20.0]


@pytest.mark.parametrize("gain", [1.0, 1e-3, 3e4])
@pytest.mark.parametrize("below", BELOW)
@pytest.mark.parametrize("N,heads", [(3, (2, 2)), (6, (2, 1)), (8, (20, 4)), (16, (20, 4)), (32, (5, 1))])
def test_int4(N, heads, below, gain):
    n, B = 4000, 2
    c = Int4Case([n] * B, N, *heads, seed=N)
    g = torch.Generator(device="cuda").manual_seed(N)
    R, _ = kvq.kvq_build_rotation(9)
    c.Mq = c.Mk = torch.from_numpy(R).cuda()
    u = direction(g)
    for b in range(B):
        k, v = keys_and_values(n, heads[1], u, 64, gain, g)
        kvq.kvq_rotate_quant_append(c.cache, c.Mk, k, v, i32([b] * n), torch.arange(n, device="cuda", dtype=torch.int32), c.err)
    c.k_new, c.v_new = (x.view(B, N, heads[1], D) for x in keys_and_values(B * N, heads[1], u, 1 << 30, gain, g))
    c.q = u + 0.02 * torch.randn(B, N, heads[0], D, generator=g, device="cuda")
    masks = [[1 << i for i in range(N)]] * B
    sm = below / D
    out = c.call(masks, sm=sm)
    q = c.q.double()
    q = (q / (q.square().mean(-1, keepdim=True) + 1e-6).sqrt()) @ torch.from_numpy(R.astype(np.float64)).cuda().T
    seen = torch.cat([torch.ones(N, n, dtype=torch.bool, device="cuda"), torch.eye(N, dtype=torch.bool, device="cuda")], 1)
    G = heads[0] // heads[1]
    for b in range(B):
        for h in range(heads[1]):
            k, v = c.dequantised(b, h, n + N)
            for hq in range(h * G, (h + 1) * G):
                expect(out[b, :, hq], q[b, :, hq], k, v, seen, sm, 2)


@pytest.mark.parametrize("below", BELOW)
@pytest.mark.parametrize("N,heads,window,B", [(3, (6, 2), 513, 2), (3, (6, 2), 513, 200), (8, (2, 2), 100, 2), (16, (20, 4), 513, 2),
                                              (16, (20, 4), 513, 50), (20, (5, 1), 3000, 2)])
def test_ring(N, heads, window, B, below):
    n = 3500
    c = RingCase([n] * B, N, *heads, window, seed=N, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(N)
    u = direction(g)
    lo = n - window + 1
    for b in range(B):
        k, v = keys_and_values(n - lo, heads[1], u, 32, 1.0, g)
        kvq.kvq_fp8_append(c.ring, k, v, i32([b] * (n - lo)), torch.arange(lo, n, device="cuda", dtype=torch.int32), c.KS, c.VS, c.err)
    c.k_new, c.v_new = (x.view(B, N, heads[1], D) for x in keys_and_values(B * N, heads[1], u, 1 << 30, 1.0, g))
    c.q = u + 0.02 * torch.randn(B, N, heads[0], D, generator=g, device="cuda")
    masks = [[1 << i for i in range(N)]] * B
    sm = below / D
    out = torch.full((B, N, heads[0], D), 9.0, device="cuda")
    kvq.kvq_tree_attn_fp8_swa(c.ring, c.q, c.pos_t, words(masks), window, c.KS, c.VS, out, kvq.alloc_tree_workspace(B, N, *heads),
                              c.err, k_new=c.k_new, v_new=c.v_new, sm_scale=sm)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    pos = np.arange(lo, n + N)
    seen = torch.cat([torch.ones(N, n - lo, dtype=torch.bool, device="cuda"), torch.eye(N, dtype=torch.bool, device="cuda")], 1)
    ks, vs = (float(np.float32(x)) for x in (c.KS, c.VS))
    G = heads[0] // heads[1]
    for b in sorted({0, 1, B - 1}):
        for h in range(heads[1]):
            kb, vb = unpack_fp8(c.tensors, b, h, pos)
            k, v = (torch.from_numpy(x.copy()).view(torch.float8_e4m3fn).double().cuda() for x in (kb, vb))
            for hq in range(h * G, (h + 1) * G):
                expect(out[b, :, hq], c.q[b, :, hq].double(), k * ks, v * vs, seen, sm, 1)


@pytest.mark.parametrize("below", BELOW)
@pytest.mark.parametrize("window", [0, 1500])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_prompt(dtype, window, below):
    lens, heads = [5000, 130, 1801], (3, 1)
    T = sum(lens)
    g = torch.Generator(device="cuda").manual_seed(5)
    u = direction(g)
    k, v = (x.to(dtype) for x in keys_and_values(T, heads[1], u, 64, 1024.0, g))
    q = (u + 0.02 * torch.randn(T, heads[0], D, generator=g, device="cuda")).to(dtype)
    out, err = torch.full_like(q, 9.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = i32([0, lens[0], lens[0] + lens[1], T])
    sm = below / D
    kvq.kvq_prompt_attn(q, k, v, cu, out, kvq.alloc_prompt_workspace(T, 3, *heads), err, window=window, sm_scale=sm)
    torch.cuda.synchronize()
    assert err.item() == 0
    at = 0
    for n in lens:
        i = torch.arange(n, device="cuda")
        rows = i[-200:]
        seen = (i[None, :] <= rows[:, None]) & ((i[None, :] > rows[:, None] - window) if window else True)
        for h in range(heads[0]):
            expect16(out[at:at + n, h][rows], q[at:at + n, h][rows].double(), k[at:at + n, 0].double(), v[at:at + n, 0].double(), seen, sm,
                     dtype)
        at += n


def expect16(out, q, k, v, seen, sm, dtype):
    """As expect, with exact inputs and weights of the 16-bit type (bf16 rounds by 2^-8)."""
    if dtype == torch.float16:
        expect(out, q, k, v, seen, sm, 0)
        return
    z = torch.where(seen, q @ k.T * sm, -torch.inf)
    p = torch.softmax(z, 1)
    o = p @ v
    mag = (seen * (q.abs() @ k.abs().T)).amax(1, keepdim=True) * sm
    d = 136 * 2.0 ** -24 * mag + 2.0 ** -21
    tol = (2 * d + 2.0 ** -8) * (p @ v.abs()) + 2.0 ** -8 * o.abs()
    off = (out.double() - o).abs()
    assert bool((off <= tol).all()), f"worst {float((off / tol).max()):.2f} of the tolerance"


@pytest.mark.parametrize("below", [12.0, 18.0])
@pytest.mark.parametrize("N,heads", [(3, (2, 2)), (4, (2, 1)), (12, (1, 1)), (8, (20, 4)), (16, (20, 4))])
def test_int4_beside_a_hidden_value_of_any_size(N, heads, below):
    """A drafted token that no row sees, with values and so a scale near the end of fp16, in the page of all the others: in
    slot 24, which the threads of the row kernels hold together with slot 0, where the heavy key is."""
    n, B = 24 - (N - 1), 2
    c = Int4Case([n] * B, N, *heads, seed=N)
    g = torch.Generator(device="cuda").manual_seed(N)
    R, _ = kvq.kvq_build_rotation(9)
    c.Mq = c.Mk = torch.from_numpy(R).cuda()
    u = direction(g)
    for b in range(B):
        k, v = keys_and_values(n, heads[1], u, 64, 1.0, g)
        kvq.kvq_rotate_quant_append(c.cache, c.Mk, k, v, i32([b] * n), torch.arange(n, device="cuda", dtype=torch.int32), c.err)
    c.k_new, c.v_new = (x.view(B, N, heads[1], D) for x in keys_and_values(B * N, heads[1], u, 1 << 30, 1.0, g))
    c.k_new[:, 0], c.v_new[:, 0] = c.k_new[:, 1], c.v_new[:, 1]
    c.v_new[:, N - 1] *= 4e4
    c.q = u + 0.02 * torch.randn(B, N, heads[0], D, generator=g, device="cuda")
    masks = [[1 << (i % (N - 1)) for i in range(N)]] * B
    sm = below / D
    out = c.call(masks, sm=sm)
    q = c.q.double()
    q = (q / (q.square().mean(-1, keepdim=True) + 1e-6).sqrt()) @ torch.from_numpy(R.astype(np.float64)).cuda().T
    drafted = torch.tensor([[(m >> j) & 1 for j in range(N - 1)] for m in masks[0]], dtype=torch.bool, device="cuda")
    seen = torch.cat([torch.ones(N, n, dtype=torch.bool, device="cuda"), drafted], 1)
    G = heads[0] // heads[1]
    for b in range(B):
        for h in range(heads[1]):
            k, v = (x[:n + N - 1] for x in c.dequantised(b, h, n + N))
            for hq in range(h * G, (h + 1) * G):
                expect(out[b, :, hq], q[b, :, hq], k, v, seen, sm, 2)
