"""kvq_mass_attn_int4 against a plain evaluation in 64 bits.

Outputs: the tolerance of test_gpu_tree.py. Weights: q~ is a fp32 chain of 128 products (136 half steps of 2^-24 with the
norm), enters the scores in two fp16 parts (2^-22 of it), and a score is a fp32 sum of 128 products of q~ and codes and of
the offset's part (136 half steps again), of magnitudes that add up to a = sum |q~| (s c + |o|): off by
d = sm a (272 2^-24 + 2^-22); the base and the power of two take 2^-20 at most. A weight is off by the factor exp(2 d + 2^-19)
(above and below the division), their sum and the mass by a half step of 2^-24 for every addition.
"""

import math

import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq
from test_gpu_tree import D, SM, Int4Case, attend, i32

pytestmark = pytest.mark.gpu


class MassCase(Int4Case):
    def __init__(self, ctx, Hq, Hkv, seed=0, **kw):
        super().__init__(ctx, 1, Hq, Hkv, seed=seed, **kw)
        P = self.tensors["block_table"].shape[1]
        self.held, self.mass = kvq.alloc_token_mass(self.B, Hkv, P)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.held["mass"].copy_(torch.rand(self.held["mass"].shape, generator=g, device="cuda") * 0.01)
        self.held["ids"].fill_(-7)
        self.before = self.held["mass"].clone()
        self.pos = self.ctx_t + 1000
        self.ws = kvq.alloc_mass_workspace(self.B, Hq, Hkv, 64 * P)

    def run(self, out_dtype=torch.float32, append=True, want_err=0, stream=None, sm=SM):
        out = torch.full((self.B, self.Hq, D), 9.0, dtype=out_dtype, device="cuda")
        new = (self.k_new[:, 0], self.v_new[:, 0]) if append else (None, None)
        torch.cuda.synchronize()
        kvq.kvq_mass_attn_int4(self.cache, self.mass, self.Mq, self.Mk, self.q[:, 0], self.ctx_t, self.pos, out, self.ws,
                               self.err, k_new=new[0], v_new=new[1], sm_scale=sm, fwht=self.fwht, stream=stream)
        torch.cuda.synchronize()
        assert self.err.item() == want_err
        return out

    def verify(self, out, calls=1, sm=SM, skip=(), hide=None):
        """Outputs, masses and numbers after `calls` calls; rows (b, hq) in `skip` are NaN and add nothing."""
        x = self.q[:, 0].double()
        q = (x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()) @ self.Mq64.T
        G = self.Hq // self.Hkv
        for b in range(self.B):
            n = self.ctx[b] + 1
            seen = torch.ones(1, n, dtype=torch.bool, device="cuda")
            if hide is not None:
                seen &= ~hide(b, n)
            for h in range(self.Hkv):
                k, v = self.dequantised(b, h, n)
                # |k| as the codes and the offset add up to it: the offset is the record's smallest value
                a_k = (k - k.amin(1, keepdim=True)) + k.amin(1, keepdim=True).abs() + 1e-3
                want, tol = torch.zeros(n, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
                for hq in range(h * G, (h + 1) * G):
                    if (b, hq) in skip:
                        assert bool(torch.isnan(out[b, hq]).all())
                        continue
                    o, t = attend(q[b, hq:hq + 1], k, v, seen, sm, out.dtype)
                    off = (out[b, hq].double() - o[0]).abs()
                    assert bool((off <= t[0]).all()), (b, hq, float((off / t[0]).max()))
                    z = torch.where(seen[0], k @ q[b, hq] * sm, -math.inf)
                    w = torch.softmax(z, 0) if bool(seen.any()) else torch.zeros_like(z)
                    d = abs(sm) * (a_k @ q[b, hq].abs()) * (272 * 2.0 ** -24 + 2.0 ** -22)
                    d = d.max() + d  # of the sum below the division, and of the token itself
                    want += w
                    tol += w * torch.expm1(2 * d + 2.0 ** -19)
                old = self.before[b, h, :n].double().clone()
                old[n - 1] = 0
                shown = old + want * calls
                shown[n - 1] = want[n - 1]
                if hide is not None:  # slots of a page outside the pool are left as they were
                    shown[~seen[0]] = self.before[b, h, :n].double()[~seen[0]]
                got = self.held["mass"][b, h, :n].double()
                lim = tol * calls + (G + calls) * 2.0 ** -24 * (shown.abs() + want) + 1e-30
                assert bool(((got - shown).abs() <= lim).all()), (b, h, float(((got - shown).abs() / lim).max()))
                assert torch.equal(self.held["mass"][b, h, n:], self.before[b, h, n:])
                ids = self.held["ids"][b, h]
                if hide is None or bool(seen[0, n - 1]):
                    assert int(ids[n - 1]) == int(self.pos[b])
                    ids = torch.cat([ids[:n - 1], ids[n:]])
                assert bool((ids == -7).all())


@pytest.mark.parametrize("heads", [(20, 4), (2, 2), (8, 1), (9, 1), (16, 1), (17, 1), (48, 1), (66, 2)])
def test_lengths_and_groups(heads):
    c = MassCase([0, 1, 2, 63, 64, 65, 200, 1030], *heads, seed=heads[0])
    c.verify(c.run())


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fwht", [False, True])
def test_types_and_prologues(out_dtype, dtype, fwht):
    c = MassCase([300, 129], 20, 4, seed=3, dtype=dtype, fwht=fwht)
    c.verify(c.run(out_dtype))


@pytest.mark.parametrize("gain", [0.01, 1.0, 8.0])
def test_peaked_and_even_weights(gain):
    c = MassCase([1500, 700], 10, 2, seed=4)
    c.verify(c.run(sm=SM * gain), sm=SM * gain)


def test_long_ragged_and_many():
    c = MassCase([9000, 3, 2500, 16, 4097], 20, 4, seed=5)
    c.verify(c.run())
    c = MassCase([(i * 7) % 90 for i in range(700)], 4, 2, seed=6)
    c.verify(c.run(torch.bfloat16))
    c = MassCase([70001], 5, 1, seed=7)
    c.verify(c.run())


def test_weights_of_a_row_add_up_to_one():
    c = MassCase([3000, 64], 20, 4, seed=8)
    c.held["mass"].zero_()
    c.run()
    total = c.held["mass"].double().sum(-1)
    assert float((total - 5).abs().max()) < 5 * (3001 * 2.0 ** -24 + 2.0 ** -19)


def test_steps_add_up_and_the_new_slot_is_set():
    """The same step again: every slot gathers once more but the new one, which is set. Garbage there before counts nothing."""
    c = MassCase([500, 64, 0], 20, 4, seed=9)
    c.held["mass"][:, :, [0, 64, 500]] = math.nan
    c.before = c.held["mass"].clone()
    c.before[1:, :, 0] = c.held["mass"][1:, :, 0] = 0.0
    c.before[0, :, [0, 64]] = 0.0
    c.held["mass"][0, :, [0, 64]] = 0.0
    c.before[1, :, 500:] = c.held["mass"][1, :, 500:] = 0.0
    c.before[2, :, 1:] = c.held["mass"][2, :, 1:] = 0.0
    out = [c.run() for _ in range(3)]
    assert torch.equal(out[0], out[2])
    c.verify(out[0], calls=3)


def test_rows_that_are_not_finite_add_nothing():
    c = MassCase([400, 70], 10, 2, seed=10, dtype=torch.float32)
    c.append()
    c.q[0, 0, 2, 5] = math.inf
    c.q[1, 0, 7, 0] = math.nan
    out = c.run(append=False, want_err=kvq.DEVERR_NONFINITE)
    c.verify(out, skip={(0, 2), (1, 7)})


def test_too_large_queries_add_nothing():
    c = MassCase([130], 4, 2, seed=11)
    c.Mq *= 1e5
    out = c.run()
    assert bool(torch.isnan(out).any())
    assert bool(torch.isfinite(c.held["mass"]).all())


def test_pages_outside_the_pool():
    c = MassCase([300, 64], 10, 2, seed=12)
    c.append()
    bt = c.tensors["block_table"]
    good = bt.clone()
    bt[0, 1], bt[0, 4], bt[1, 1] = -1, 1 << 20, -3
    torch.cuda.synchronize()
    out = c.run(append=False, want_err=kvq.DEVERR_PAGE)
    bad = {0: (1, 4), 1: (1,)}
    bt.copy_(good)

    def hide(b, n):
        j = torch.arange(n, device="cuda") // 64
        return torch.stack([j == p for p in bad[b]]).any(0)
    c.verify(out, hide=hide)


def test_slots_behind_the_new_one_may_hold_anything():
    c = MassCase([300, 63], 10, 2, seed=17, extra_pages=1)
    c.append()
    want = c.run(append=False)
    held = c.held["mass"].clone()
    page = c.tensors["block_table"].long()
    meta = c.tensors["pages"][:, :, 8192:8704].view(torch.int32)  # K words 0..63, V words 64..127
    for b, pos, word in ((0, 301, 0x7E007E00), (0, 319, 0x7C007C00), (1, 64, 0x7E007E00)):
        meta[page[b, pos // 64], :, pos % 64] = word
        meta[page[b, pos // 64], :, 64 + pos % 64] = word
    c.tensors["pages"][:, :, 8192:8704] = meta.view(torch.uint8)
    c.held["mass"].copy_(c.before)
    assert torch.equal(c.run(append=False), want) and torch.equal(c.held["mass"], held)


def test_lengths_outside_the_cache():
    c = MassCase([100, 100], 4, 2, seed=13)
    c.append()
    c.ctx_t[0] = -5
    c.run(append=False, want_err=kvq.DEVERR_POS)
    assert torch.equal(c.held["mass"][0, :, 1:], c.before[0, :, 1:])


def test_a_full_sequence_keeps_what_it_gathered():
    """The token that finds no slot is not appended, and the slots' masses and numbers stay."""
    c = MassCase([127, 100], 10, 2, seed=18)
    c.append()
    pages = c.tensors["pages"].clone()
    full = 64 * c.tensors["block_table"].shape[1]
    for n in (full, full + 1, 1 << 30):
        c.ctx_t[0] = n
        c.err.zero_()
        c.held["mass"].copy_(c.before)
        c.run(want_err=kvq.DEVERR_POS)
        assert torch.equal(c.held["mass"][0], c.before[0]) and bool((c.held["ids"][0] == -7).all())
        assert torch.equal(c.tensors["pages"], pages)
        assert not torch.equal(c.held["mass"][1], c.before[1])


def test_other_rows_stay():
    """A mass of more sequences and slots than the call's."""
    c = MassCase([200, 90], 10, 2, seed=14)
    big, desc = kvq.alloc_token_mass(5, 2, c.tensors["block_table"].shape[1] + 3)
    big["mass"].fill_(0.5)
    big["ids"].fill_(3)
    out = torch.empty(2, 10, D, device="cuda")
    kvq.kvq_mass_attn_int4(c.cache, desc, c.Mq, c.Mk, c.q[:, 0], c.ctx_t, c.pos, out, c.ws, c.err, k_new=c.k_new[:, 0],
                           v_new=c.v_new[:, 0])
    torch.cuda.synchronize()
    assert bool((big["mass"][2:] == 0.5).all() and (big["ids"][2:] == 3).all())
    for b, n in enumerate((201, 91)):
        assert bool((big["mass"][b, :, n:] == 0.5).all()) and bool((big["ids"][b, :, n - 1] == c.pos[b]).all())
    c.run()
    for b, n in enumerate((200, 90)):
        d = (big["mass"][b, :, :n] - 0.5) - (c.held["mass"][b, :, :n] - c.before[b, :, :n])
        assert float(d.abs().max()) < 1e-6


def test_repeats_streams_and_graph():
    """Bit for bit on another stream and replayed with other lengths; a workspace shared with another graph's call."""
    lens = [900, 64, 5000]
    c = MassCase(lens, 20, 4, seed=15)
    c.append()
    want = c.run(append=False)
    held = c.held["mass"].clone()
    c.held["mass"].copy_(c.before)
    assert torch.equal(c.run(append=False, stream=torch.cuda.Stream()), want) and torch.equal(c.held["mass"], held)
    out = torch.zeros(3, 20, D, device="cuda")
    graphs = []
    for sm in (SM, 2 * SM):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvq.kvq_mass_attn_int4(c.cache, c.mass, c.Mq, c.Mk, c.q[:, 0], c.ctx_t, c.pos, out, c.ws, c.err, sm_scale=sm)
        graphs.append(g)
    for n in (lens, [5, 3000, 4990]):
        c.ctx_t.copy_(i32(n))
        for g, sm in zip(graphs, (SM, 2 * SM)):
            c.held["mass"].copy_(c.before)
            g.replay()
            torch.cuda.synchronize()
            got, o = c.held["mass"].clone(), out.clone()
            c.held["mass"].copy_(c.before)
            assert torch.equal(c.run(append=False, sm=sm), o) and torch.equal(c.held["mass"], got)


def test_wide_tables_pass_32_bits():
    """48 rows of 64 x 800,000 scores each: places behind 2^31."""
    c = MassCase([130], 48, 1, seed=16)
    P = 800_000
    table = torch.zeros(1, P, dtype=torch.int32, device="cuda")
    table[0, :3] = c.tensors["block_table"][0, :3]
    cache = kvq.int4_cache(c.tensors["pages"], table)
    held, desc = kvq.alloc_token_mass(1, 1, P)
    ws = kvq.alloc_mass_workspace(1, 48, 1, 64 * P)
    out = torch.empty(1, 48, D, device="cuda")
    kvq.kvq_mass_attn_int4(cache, desc, c.Mq, c.Mk, c.q[:, 0], c.ctx_t, c.pos, out, ws, c.err, k_new=c.k_new[:, 0],
                           v_new=c.v_new[:, 0])
    torch.cuda.synchronize()
    c.held["mass"].zero_()
    assert torch.equal(c.run(), out) and torch.equal(c.held["mass"][0, 0, :131], held["mass"][0, 0, :131])


def test_two_calls_at_once():
    cases = [MassCase([900, 30, 2000], 20, 4, seed=40 + i) for i in range(2)]
    for c in cases:
        c.append()
    want = [(c.run(append=False), c.held["mass"].clone()) for c in cases]
    outs, streams = [torch.zeros(3, 20, D, device="cuda") for _ in cases], [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        for c in cases:
            c.held["mass"].copy_(c.before)
        torch.cuda.synchronize()
        for c, o, s in zip(cases, outs, streams):
            kvq.kvq_mass_attn_int4(c.cache, c.mass, c.Mq, c.Mk, c.q[:, 0], c.ctx_t, c.pos, o, c.ws, c.err, stream=s)
        torch.cuda.synchronize()
        for c, o, (w, m) in zip(cases, outs, want):
            assert torch.equal(o, w) and torch.equal(c.held["mass"], m) and c.err.item() == 0


def test_steps_without_a_wait_between():
    """Steps in a row, each reading what the one before appended and adding to what it left."""
    got = []
    for wait in (False, True):
        c = MassCase([60, 127, 500], 20, 4, seed=43, extra_pages=1)
        g = torch.Generator(device="cuda").manual_seed(6)
        ctx = [c.ctx_t + i for i in range(9)]
        new = [[torch.randn(3, 4, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)] for _ in range(8)]
        outs = [torch.zeros(3, 20, D, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        for i in range(8):
            kvq.kvq_mass_attn_int4(c.cache, c.mass, c.Mq, c.Mk, c.q[:, 0], ctx[i], ctx[i + 1], outs[i], c.ws, c.err, k_new=new[i][0],
                                   v_new=new[i][1])
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert c.err.item() == 0
        got.append(outs + [c.held["mass"], c.held["ids"], c.tensors["pages"]])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert all(int(got[0][-2][b, h, n + i]) == n + i + 1 for b, n in enumerate((60, 127, 500)) for h in range(4) for i in range(8))


def test_tensors_that_do_not_fit():
    c = MassCase([100, 20], 10, 2, seed=44)
    out = torch.empty(2, 10, D, device="cuda")
    args = dict(cache=c.cache, mass=c.mass, Mq=c.Mq, Mk=c.Mk, q=c.q[:, 0], ctx_len=c.ctx_t, positions=c.pos, out=out, workspace=c.ws,
                dev_err=c.err)
    for bad in (dict(q=c.q.repeat(1, 2, 1, 1)), dict(q=c.q[:, 0].half()), dict(out=out[:1]), dict(positions=c.pos.long()), dict(positions=c.pos[:1]),
                dict(k_new=c.k_new, v_new=c.v_new), dict(workspace=c.ws.cpu()), dict(Mk=c.Mk[0])):
        with pytest.raises(ValueError):
            kvq.kvq_mass_attn_int4(**{**args, **bad})
    for bad in (dict(workspace=c.ws[:256]), dict(mass=kvq.token_mass(c.held["mass"][:1], c.held["ids"][:1])),
                dict(mass=kvq.token_mass(c.held["mass"][:, :1].contiguous(), c.held["ids"][:, :1].contiguous()))):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_mass_attn_int4(**{**args, **bad})
    with pytest.raises(ValueError):
        kvq.token_mass(c.held["mass"], c.held["ids"].long())
    with pytest.raises(ValueError):
        kvq.token_mass(c.held["mass"][:, :, ::2], c.held["ids"][:, :, ::2])
