"""Caches held to a size on the page pool: what windows leave behind and what evictions free goes to other sessions while the
steps go on. A twin whose pages nobody takes has the same outputs, masses and numbers bit for bit."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq

pytestmark = pytest.mark.gpu
D, Hq, Hkv, B = 128, 20, 4, 3


def i32(x):
    return torch.tensor(np.asarray(x, np.int32).reshape(-1), device="cuda")


class Pooled:
    """Three sequences on a pool; a fourth row stands for the other sessions, which fill whatever page they get."""

    def __init__(self, num_pages, max_pages, lens, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
        table = torch.full((B + 1, max_pages), -1, dtype=torch.int32, device="cuda")
        self.tensors, self.cache = kvq.alloc_int4_cache(num_pages, Hkv, table)
        self.table = self.tensors["block_table"]
        r = np.random.default_rng(seed)
        R, _ = kvq.kvq_build_rotation(seed)
        self.Mq, self.Mk = (torch.from_numpy(m).cuda() for m in kvq.kvq_fold_qk(R, *(r.uniform(0.5, 1.5, D).astype(np.float32) for _ in range(2))))
        self.held, self.mass = kvq.alloc_token_mass(B + 1, Hkv, max_pages)
        self.ws, self.mass_ws = kvq.alloc_workspace(B, 1, Hq, Hkv), kvq.alloc_mass_workspace(B, Hq, Hkv, 64 * max_pages)
        kvq.kvq_pages_alloc(self.refs, self.table, i32(range(B)), i32([0] * B), i32(lens), self.err)
        T = sum(lens)
        k, v = (torch.randn(T, Hkv, D, generator=g, device="cuda") for _ in range(2))
        kvq.kvq_rotate_quant_append(self.cache, self.Mk, k, v, i32([b for b in range(B) for _ in range(lens[b])]),
                                    i32([p for n in lens for p in range(n)]), self.err)

    def grow(self, ctx):
        kvq.kvq_pages_alloc(self.refs, self.table, i32(range(B)), i32(ctx), i32([c + 1 for c in ctx]), self.err)

    def free(self, ids, old, new):
        kvq.kvq_pages_free(self.refs, self.table, i32(ids), i32(old), i32(new), self.err)

    def others(self, held, n):
        """Other sessions take n more pages and fill them."""
        kvq.kvq_pages_alloc(self.refs, self.table, i32([B]), i32([64 * held]), i32([64 * (held + n)]), self.err)
        got = self.table[B, held:held + n].long()
        assert bool((got >= 0).all())
        self.tensors["pages"][got] = 255

    def ok(self):
        torch.cuda.synchronize()
        assert self.err.item() == 0

    def done(self):
        self.ok()
        assert bool((self.table[:B] == -1).all()) and int(self.refs.sum()) == int((self.table[B] >= 0).sum())


def rows(seed, steps):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [[torch.randn(B, 1, h, D, generator=g, device="cuda") for h in (Hq, Hkv, Hkv)] for _ in range(steps)]


@pytest.mark.parametrize("window,sinks", [(100, 4), (130, 70), (64, 0), (1, 64), (65, 200)])
def test_pages_between_first_tokens_and_windows(window, sinks):
    lens, most, steps = [700, 300, 64], 20, 70
    p, twin = Pooled(60, most, lens, 3), Pooled(60, most, lens, 3)
    ctx, back, taken = list(lens), [sinks] * B, 0
    for q, k, v in rows(4, steps):
        # what no row from here on sees: behind the first tokens, up to the page where this step's windows begin
        upto = [64 * (max(0, c - window + 1) // 64) for c in ctx]
        p.free(range(B), upto, back)
        back = [max(x, u) for x, u in zip(back, upto)]
        free = int((p.refs == 0).sum())
        if free > 8 and taken < most - 6:
            p.others(taken, 6)
            taken += 6
        outs = []
        for s in (p, twin):
            s.grow(ctx)
            outs.append(torch.empty(B, 1, Hq, D, device="cuda"))
            kvq.kvq_window_attn_int4(s.cache, s.Mq, s.Mk, q, i32(ctx), window, sinks, outs[-1], s.ws, s.err, k_new=k, v_new=v)
            s.ok()
        assert torch.equal(*outs)
        ctx = [c + 1 for c in ctx]
    first, start = -(-sinks // 64), [max(0, c - window) // 64 for c in ctx]  # (of the last step's windows)
    for b in range(B):
        held = set(np.nonzero(p.table[b].cpu().numpy() >= 0)[0].tolist())
        assert held == set(range(min(first, -(-ctx[b] // 64)))) | set(range(max(0, start[b]), -(-ctx[b] // 64)))
    # the whole of it: the pages behind, then the first ones
    p.free(range(B), ctx, back)
    p.free(range(B), [min(sinks, c) for c in ctx], [0] * B)
    p.done()


@pytest.mark.parametrize("budget", [64, 100, 256])
def test_pages_behind_an_eviction(budget):
    lens, most, steps = [700, 300, 64], 20, 40
    p, twin = Pooled(60, most, lens, 5), Pooled(60, most, lens, 5)
    ctx, seen, taken = list(lens), list(lens), 0
    for i, (q, k, v) in enumerate(rows(6, steps)):
        if i % 13 == 5:
            new = []
            for s in (p, twin):
                new.append(i32([0] * B))
                kvq.kvq_evict_int4([s.cache], [s.mass], i32(ctx), i32(seen), budget, 4, 16, s.err, ctx_out=new[-1])
            assert torch.equal(*new)
            kvq.kvq_pages_free(p.refs, p.table, i32(range(B)), i32(ctx), new[0], p.err)
            ctx = new[0].tolist()
            p.others(taken, 3)
            taken += 3
        outs = []
        for s in (p, twin):
            if s is p or i < 5:  # (the twin goes on over the pages that it still has)
                s.grow(ctx)
            outs.append(torch.empty(B, 1, Hq, D, device="cuda"))
            kvq.kvq_mass_attn_int4(s.cache, s.mass, s.Mq, s.Mk, q, i32(ctx), i32(seen), outs[-1], s.mass_ws, s.err, k_new=k, v_new=v)
            s.ok()
        assert torch.equal(*outs)
        ctx, seen = [c + 1 for c in ctx], [c + 1 for c in seen]
    for b in range(B):
        for x in ("mass", "ids"):
            assert torch.equal(p.held[x][b, :, :ctx[b]], twin.held[x][b, :, :ctx[b]])
        assert int((p.table[b] >= 0).sum()) == -(-ctx[b] // 64)
    p.free(range(B), ctx, [0] * B)
    p.done()
