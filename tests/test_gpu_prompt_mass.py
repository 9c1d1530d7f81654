"""kvq_prompt_mass against a plain evaluation in 64 bits.

A score is a fp32 sum of 128 exact products (136 half steps of 2^-24 of the sum of magnitudes, with the scale); a row's
log-sum a is rounded once and subtracted in one step (half steps of |a| and of the score, in powers of two), its sum of n
powers of two takes n half steps at most; a power of two 2^-21. So a weight is off by the factor
exp(2 d + ln 2 (|a| + |z|) 2^-23 + n 2^-24 + 2^-19), and a token's sum of R weights by R half steps more.
"""

import math

import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq
from test_gpu_prompt import inputs, offsets

pytestmark = pytest.mark.gpu
D = 128


def reference(q, k, lens, rows, sm=D ** -0.5, skip=()):
    """[(mass [Hkv, n], tolerance)] of every sequence; rows (token of the packing, head) in `skip` add nothing."""
    Hq, Hkv = q.shape[1], k.shape[1]
    res, at = [], 0
    for n in lens:
        s = slice(at, at + n)
        r = max(0, n - rows) if rows > 0 else 0
        mass = torch.zeros(Hkv, n, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(mass)
        seen = torch.arange(n, device="cuda")[None] <= torch.arange(r, n, device="cuda")[:, None]
        for h in range(Hq if n else 0):
            Q, K = q[s, h][r:].double(), k[s, h * Hkv // Hq].double()
            z = torch.where(seen, (Q @ K.T) * sm, -math.inf)
            w = torch.softmax(z, 1)
            mag = (seen * (Q.abs() @ K.abs().T)).nan_to_num(0, 0, 0).amax(1, keepdim=True) * sm
            a = torch.logsumexp(z, 1, keepdim=True).abs()
            off = 2 * 136 * 2.0 ** -24 * mag + (a + mag) * 2.0 ** -23 + n * 2.0 ** -24 + 2.0 ** -19
            for tok, head in skip:
                if head == h and at + r <= tok < at + n:
                    w[tok - at - r] = 0
                    off[tok - at - r] = 0
            mass[h * Hkv // Hq] += w.sum(0)
            tol[h * Hkv // Hq] += (w * torch.expm1(off)).sum(0)
        res.append((mass, tol + (n - r) * Hq // Hkv * 2.0 ** -24 * mass + 1e-30))
        at += n
    return res


def call(q, k, lens, rows, held=None, seq_ids=None, sm=D ** -0.5, cu=None, want_err=0, stream=None, num_seqs=None):
    cu = offsets(lens) if cu is None else cu
    B, Hkv = cu.numel() - 1, k.shape[1]
    if held is None:
        P = max(1, -(-max(lens) // 64))
        held, _ = kvq.alloc_token_mass(num_seqs or B, Hkv, P)
        held["mass"].fill_(math.nan)
        held["ids"].fill_(-7)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = kvq.alloc_prompt_mass_workspace(q.shape[0], B, q.shape[1], Hkv, rows)
    ws.fill_(255)
    torch.cuda.synchronize()
    kvq.kvq_prompt_mass(q, k, cu, rows, kvq.token_mass(held["mass"], held["ids"]), ws, err,
                        seq_ids=None if seq_ids is None else torch.tensor(seq_ids, dtype=torch.int32, device="cuda"),
                        sm_scale=sm, stream=stream)
    torch.cuda.synchronize()
    assert err.item() == want_err
    return held


def check(held, want, lens, seq_ids=None):
    for b, (n, (mass, tol)) in enumerate(zip(lens, want)):
        r = b if seq_ids is None else seq_ids[b]
        got = held["mass"][r, :, :n].double()
        off = (got - mass).abs()
        assert bool((off <= tol).all()), (b, float((off / tol).max()))
        assert bool((held["ids"][r, :, :n] == torch.arange(n, device="cuda")).all())
        assert bool(torch.isnan(held["mass"][r, :, n:]).all()) and bool((held["ids"][r, :, n:] == -7).all())


@pytest.mark.parametrize("rows", [1, 2, 24, 25, 26, 64, 130, 0, 1 << 30])
@pytest.mark.parametrize("heads", [(20, 4), (3, 3), (8, 1), (6, 2)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_heads_types(rows, heads, dtype):
    lens = [1, 127, 128, 129, 0, 300, 700, 2, 25]
    q, k, _ = inputs(lens, *heads, dtype, seed=rows % 97)
    check(call(q, k, lens, rows), reference(q, k, lens, rows), lens)


@pytest.mark.parametrize("heads", [(64, 1), (48, 1), (128, 2), (33, 1), (65, 5)])
@pytest.mark.parametrize("rows", [3, 70])
def test_wide_groups(heads, rows):
    lens = [260, 5, 64]
    q, k, _ = inputs(lens, *heads, torch.bfloat16, seed=heads[0])
    check(call(q, k, lens, rows), reference(q, k, lens, rows), lens)


@pytest.mark.parametrize("rows", [16, 64, 0])
def test_views_of_a_fused_projection(rows):
    lens = [300, 7, 129]
    q, k, _ = inputs(lens, 20, 4, torch.bfloat16, seed=3, fused=True)
    check(call(q, k, lens, rows), reference(q, k, lens, rows), lens)


def test_one_token_views():
    q, k, _ = inputs([1], 20, 4, torch.bfloat16, seed=4, fused=True)
    check(call(q, k, [1], 16), reference(q, k, [1], 16), [1])


# split keys (few query tiles, long prompts) and whole ones
@pytest.mark.parametrize("lens,rows", [([9000], 64), ([20001], 1), ([4000, 9001, 33, 6000], 40), ([5000, 100], 300), ([3000], 0)])
def test_long_prompts(lens, rows):
    q, k, _ = inputs(lens, 5, 1, torch.bfloat16, seed=len(lens))
    check(call(q, k, lens, rows), reference(q, k, lens, rows), lens)


@pytest.mark.parametrize("gain", [0.0, 4.0, 12.0])
@pytest.mark.parametrize("sm", [D ** -0.5, 1e-4, 0.5])
def test_score_ranges(gain, sm):
    lens = [400, 260]
    q, k, _ = inputs(lens, 4, 2, torch.bfloat16, seed=5, gain=gain)
    check(call(q, k, lens, 50, sm=sm), reference(q, k, lens, 50, sm=sm), lens)


def test_climbing_and_falling_scores():
    """The base moves often and far, up to 87 nats in a block."""
    n = 1100
    q, k, _ = inputs([n], 2, 1, torch.bfloat16, seed=6)
    ramp = torch.linspace(-60, 60, n, device="cuda")[:, None, None]
    q = torch.ones_like(q)
    for r in (ramp, -ramp, ramp * 4):
        k2 = (r * D ** -0.5 + 0.1 * k.float()).to(k.dtype)
        check(call(q, k2, [n], 64), reference(q, k2, [n], 64), [n])


def test_many_sequences_and_their_rows():
    lens = [1 + (i * 37) % 41 for i in range(1024)]
    q, k, _ = inputs(lens, 2, 1, torch.float16, seed=12)
    ids = [(i * 5 + 3) % 1024 for i in range(1024)]
    check(call(q, k, lens, 8, seq_ids=ids), reference(q, k, lens, 8), lens, ids)


def test_rows_that_are_not_named_stay():
    lens = [200, 64]
    q, k, _ = inputs(lens, 4, 2, torch.bfloat16, seed=13)
    held = call(q, k, lens, 20, seq_ids=[4, 1], num_seqs=6)
    check(held, reference(q, k, lens, 20), lens, [4, 1])
    for r in (0, 2, 3, 5):
        assert bool(torch.isnan(held["mass"][r]).all()) and bool((held["ids"][r] == -7).all())


def test_bad_rows_offsets_and_lengths_are_flagged_and_skipped():
    lens = [100, 60, 80]
    q, k, _ = inputs(lens, 4, 2, torch.bfloat16, seed=14)
    want = reference(q, k, lens, 20)
    for ids, good in (([2, 9, 1], (0, 2)), ([-1, 0, 1], (1, 2)), ([1, 1, 0], (0, 2))):
        held = call(q, k, lens, 20, seq_ids=ids, num_seqs=3, want_err=kvq.DEVERR_POS)
        for b in good:
            n, (mass, tol) = lens[b], want[b]
            assert bool(((held["mass"][ids[b], :, :n].double() - mass).abs() <= tol).all())
    cu = torch.tensor([0, 100, 60, 240, 260], dtype=torch.int32, device="cuda")  # back, and past the end
    held = call(q, k, lens, 20, cu=cu, want_err=kvq.DEVERR_POS)
    assert bool(((held["mass"][0, :, :100].double() - want[0][0]).abs() <= want[0][1]).all())
    assert bool(torch.isnan(held["mass"][1]).all()) and bool(torch.isnan(held["mass"][3]).all())
    # offsets that name the same tokens again and again: more in all than the call's tokens
    cu = torch.tensor([0, 240] * 40 + [0], dtype=torch.int32, device="cuda")
    held, _ = kvq.alloc_token_mass(80, 2, 4)
    held["mass"].fill_(math.nan)
    call(q, k, lens, 0, held=held, cu=cu, want_err=kvq.DEVERR_POS)
    whole = reference(q, k, [240], 0)[0]
    assert bool(((held["mass"][0, :, :240].double() - whole[0]).abs() <= whole[1]).all())
    assert bool(torch.isnan(held["mass"][1:]).all())
    # a prompt longer than its place
    held, _ = kvq.alloc_token_mass(3, 2, 1)
    held["mass"].fill_(math.nan)
    call(q, k, lens, 20, held=held, want_err=kvq.DEVERR_POS)
    assert bool(torch.isnan(held["mass"][0]).all()) and bool(torch.isnan(held["mass"][2]).all())
    assert bool(((held["mass"][1, :, :60].double() - want[1][0]).abs() <= want[1][1]).all())


@pytest.mark.parametrize("rows", [30, 64, 0])
def test_rows_that_are_not_finite_add_nothing(rows):
    lens = [150, 300, 90]
    q, k, _ = inputs(lens, 4, 2, torch.bfloat16, seed=15)
    q[445, 1, 7] = math.nan
    q[440, 3, 0] = math.inf
    q[150 + 299, 0] = math.nan
    k[450 + 80, 0, 5] = math.nan   # rows 530.. of heads 0 and 1 see it
    skip = [(445, 1), (440, 3), (449, 0)] + [(t, h) for t in range(530, 540) for h in (0, 1)]
    held = call(q, k, lens, rows)
    assert bool(torch.isfinite(held["mass"][1, :, :300]).all())
    kk = k.clone()
    kk[530, 0, 5] = 0
    qq = q.clone()
    qq[445, 1, 7] = qq[440, 3, 0] = 0
    qq[449, 0] = 0
    check(held, reference(qq, kk, lens, rows, skip=skip), lens)


def test_repeats_stream_graph_and_two_at_once():
    lens = [1333, 1, 4700]
    ins = [inputs(lens, 20, 4, torch.bfloat16, seed=16 + i) for i in range(2)]
    want = [call(q, k, lens, 64) for q, k, _ in ins]
    again = call(*ins[0][:2], lens, 64, stream=torch.cuda.Stream())
    assert all(torch.equal(want[0][x].nan_to_num(-1), again[x].nan_to_num(-1)) for x in want[0])
    cu, err = offsets(lens), torch.zeros(1, dtype=torch.int32, device="cuda")
    held = [kvq.alloc_token_mass(3, 4, -(-4700 // 64))[0] for _ in ins]
    desc = [kvq.token_mass(h["mass"], h["ids"]) for h in held]
    ws = [kvq.alloc_prompt_mass_workspace(sum(lens), 3, 20, 4, 64) for _ in ins]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):  # two calls that share a workspace, one behind the other
        for (q, k, _), d in zip(ins, desc):
            kvq.kvq_prompt_mass(q, k, cu, 64, d, ws[0], err)

    def equal():
        torch.cuda.synchronize()
        for h, w in zip(held, want):
            for b, n in enumerate(lens):
                assert torch.equal(h["mass"][b, :, :n], w["mass"][b, :, :n])
        for h in held:
            h["mass"].zero_()
        torch.cuda.synchronize()
    for _ in range(2):
        g.replay()
        equal()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for (q, k, _), d, s, w in zip(ins, desc, streams, ws):
            kvq.kvq_prompt_mass(q, k, cu, 64, d, w, err, stream=s)
    equal()
    assert err.item() == 0


def test_tensors_that_do_not_fit():
    q, k, _ = inputs([100, 20], 4, 2, torch.bfloat16, seed=20)
    held, mass = kvq.alloc_token_mass(2, 2, 2)
    err, cu = torch.zeros(1, dtype=torch.int32, device="cuda"), offsets([100, 20])
    args = dict(q=q, k=k, cu_seqlens=cu, rows=16, mass=mass, workspace=kvq.alloc_prompt_mass_workspace(120, 2, 4, 2, 16), dev_err=err)
    for bad in (dict(k=k.half()), dict(k=k[:100]), dict(cu_seqlens=cu.long()), dict(q=q.transpose(1, 2)), dict(seq_ids=cu),
                dict(seq_ids=torch.zeros(2, device="cuda"))):
        with pytest.raises(ValueError):
            kvq.kvq_prompt_mass(**{**args, **bad})
    with pytest.raises(TypeError):
        kvq.kvq_prompt_mass(**{**args, "q": q.float(), "k": k.float()})
    for bad in (dict(mass=kvq.alloc_token_mass(1, 2, 2)[1]), dict(mass=kvq.alloc_token_mass(2, 1, 2)[1]), dict(workspace=args["workspace"][:256])):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_prompt_mass(**{**args, **bad})
