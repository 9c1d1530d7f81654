"""kvq_evict_int4 against a plain model on the host: exact, records, masses and numbers alike."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Layers with tables of their own, random bytes for records (they are only moved)."""

    def __init__(self, ctx, Hkv, layers=1, pages=0, seed=0, extra_rows=0, slack=0):
        r = self.rng = np.random.default_rng(seed)
        self.ctx, self.B, self.Hkv, self.layers = ctx, len(ctx), Hkv, layers
        P = self.P = max(pages, max(1, -(-max(ctx) // 64)))
        rows = self.B + extra_rows
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.pages, self.tables, self.caches, self.held, self.masses = [], [], [], [], []
        for _ in range(layers):
            need = sum(max(1, -(-c // 64)) for c in ctx)
            num = need + int(r.integers(0, 5))
            perm = r.permutation(num).astype(np.int32)
            table = np.full((rows, P), -1, np.int32)
            at = 0
            for b, c in enumerate(ctx):
                k = max(1, -(-c // 64))
                table[b, :k] = perm[at:at + k]
                at += k
            pages_t = torch.randint(0, 256, (num, Hkv, kvq.INT4_BLOCK_BYTES), generator=g, device="cuda", dtype=torch.uint8)
            table_t = torch.from_numpy(table).cuda()
            L = 64 * P + slack
            mass = torch.rand(rows, Hkv, L, generator=g, device="cuda").pow(4)
            ids = torch.arange(L, dtype=torch.int32, device="cuda").repeat(rows, Hkv, 1)
            self.pages.append(pages_t)
            self.tables.append(table_t)
            self.caches.append(kvq.int4_cache(pages_t, table_t))
            self.held.append({"mass": mass, "ids": ids})
        self.ctx_t, self.seen = i32(ctx), i32(ctx)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.out = i32([-9] * self.B)

    def state(self):
        return ([p.cpu().numpy() for p in self.pages], [h["mass"].cpu().numpy() for h in self.held],
                [h["ids"].cpu().numpy() for h in self.held])

    def call(self, budget, sinks=0, recent=0, want_err=0, stream=None):
        self.masses = [kvq.token_mass(h["mass"], h["ids"]) for h in self.held]
        torch.cuda.synchronize()
        kvq.kvq_evict_int4(self.caches, self.masses, self.ctx_t, self.seen, budget, sinks, recent, self.err, ctx_out=self.out,
                           stream=stream)
        torch.cuda.synchronize()
        assert self.err.item() == want_err

    def model(self, before, budget, sinks, recent, ctx=None):
        pages, mass, ids = ([x.copy() for x in part] for part in before)
        seen = self.seen.cpu().numpy()
        for l in range(self.layers):
            table = self.tables[l].cpu().numpy()
            for b, n in enumerate(self.ctx if ctx is None else ctx):
                k = min(n, budget)
                if n <= budget:
                    continue
                for h in range(self.Hkv):
                    m, d = mass[l][b, h, :n].astype(np.float64), ids[l][b, h, :n].astype(np.int64)
                    top = (d < sinks) | (d >= int(seen[b]) - recent)
                    rank = np.where(top, 2, np.where(np.isnan(m), 0, 1))  # NaN below -inf
                    m[rank != 1] = 0.0  # the first and newest: by slots alone
                    order = np.lexsort((np.arange(n), -m, -rank))
                    keep = np.zeros(n, bool)
                    keep[order[:k]] = True
                    holes, movers = np.nonzero(~keep[:k])[0], k + np.nonzero(keep[k:])[0]
                    assert len(holes) == len(movers)
                    if not len(holes):
                        continue
                    P, Q = (table[b, x // 64] for x in (movers, holes))
                    s, t = movers % 64, holes % 64
                    blk = pages[l]
                    c = np.arange(4)[None]
                    kz = lambda x: ((x >> 1) & 1) | ((x >> 2) & 2)  # noqa: E731
                    for base, swz in ((0, kz), (4096, lambda x: (x >> 1) & 3)):
                        v = blk[:, h, base:base + 4096].reshape(-1, 64, 4, 16)
                        new = v[P[:, None], s[:, None], c ^ swz(s)[:, None]].copy()
                        v[Q[:, None], t[:, None], c ^ swz(t)[:, None]] = new
                        blk[:, h, base:base + 4096] = v.reshape(-1, 4096)
                    for base in (8192, 8448):
                        v = blk[:, h, base:base + 256].reshape(-1, 64, 4)
                        v[Q, t] = v[P, s].copy()
                        blk[:, h, base:base + 256] = v.reshape(-1, 256)
                    mass[l][b, h, holes] = mass[l][b, h, movers]
                    ids[l][b, h, holes] = ids[l][b, h, movers]
        return pages, mass, ids

    def check(self, before, budget, sinks=0, recent=0, ctx=None):
        for want, got in zip(self.model(before, budget, sinks, recent, ctx), self.state()):
            for a, b in zip(want, got):
                assert a.tobytes() == b.tobytes()
        assert self.out.tolist() == [min(n, budget) for n in (self.ctx if ctx is None else ctx)]

    def both(self, budget, sinks=0, recent=0):
        before = self.state()
        self.call(budget, sinks, recent)
        self.check(before, budget, sinks, recent)


@pytest.mark.parametrize("budget", [1, 2, 63, 64, 65, 128, 200, 511, 512, 5000])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 0), (0, 30), (4, 60), (70, 70)])
def test_budgets(budget, sinks, recent):
    Case([0, 1, 2, 64, 65, 130, 512, 777], 2, seed=budget + sinks).both(budget, sinks, recent)


# one CTA a pair up to clusters of eight: by pairs, and by the table's width
@pytest.mark.parametrize("ctx,Hkv,layers,pages", [
    ([3000], 1, 1, 0), ([20001], 1, 1, 0), ([9000, 4097, 30], 2, 2, 0), ([60003], 1, 1, 0), ([500] * 40, 4, 3, 0),
    ([3000, 2999], 1, 1, 6144), ([260001], 1, 1, 0), ([100, 900], 1, 1, 900), ([5000] * 20, 8, 2, 0)])
@pytest.mark.parametrize("share", [0.05, 0.9])
def test_sizes_and_clusters(ctx, Hkv, layers, pages, share):
    c = Case(ctx, Hkv, layers, pages, seed=len(ctx))
    c.both(max(1, int(max(ctx) * share)), 4, 20)


@pytest.mark.parametrize("budget", [1, 100, 555, 899])
def test_equal_masses_keep_the_lower_slots(budget):
    c = Case([900, 640], 2, seed=3)
    c.held[0]["mass"].fill_(0.25)
    c.both(budget, 3, 10)
    c = Case([900, 640], 2, seed=4)
    c.held[0]["mass"].copy_((c.held[0]["mass"] * 4).floor())  # few values, zeros among them
    c.both(budget, 3, 10)


def test_equal_masses_over_a_cluster():
    c = Case([40000], 1, seed=5)
    c.held[0]["mass"].copy_((c.held[0]["mass"] * 3).floor())
    c.both(12345, 4, 64)
    c = Case([40000], 1, seed=6)
    c.held[0]["mass"].fill_(1.0)
    c.both(25001, 0, 64)


def test_unusual_masses():
    """Signs, zeros of both signs, subnormals, infinities and NaN in their order."""
    c = Case([700, 333], 2, seed=7)
    vals = torch.tensor([0.0, -0.0, 1e-40, -1e-40, np.inf, -np.inf, np.nan, -np.nan, 3e38, -3e38, 1.0, -1.0], device="cuda")
    pick = torch.randint(0, 12, c.held[0]["mass"].shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    c.held[0]["mass"].copy_(vals[pick])
    for budget in (10, 150, 300, 320):
        c.both(budget, 2, 5)
        assert torch.equal(c.out, i32([budget, budget]))


def test_first_and_newest_above_the_budget():
    c = Case([600, 100], 2, seed=8)
    c.both(50, 40, 300)
    c = Case([600, 100], 2, seed=9)
    c.both(50, 1 << 30, 1 << 30)


def test_numbers_after_evictions():
    """Numbers that are no longer the slots': rounds of growth and eviction, as a session has them."""
    c = Case([512, 512, 448], 2, layers=2, seed=10, slack=4)
    g = torch.Generator(device="cuda").manual_seed(3)
    lens = list(c.ctx)
    for _ in range(6):
        before = c.state()
        c.call(320, 4, 40)
        c.check(before, 320, 4, 40)
        for l in range(2):
            ids = c.held[l]["ids"]
            for b in range(3):
                assert all(len(set(ids[b, h, :320].tolist())) == 320 for h in range(2))
                kept = ids[b, :, :320]
                seen = int(c.seen[b])
                for first in range(4):
                    assert bool((kept == first).any(1).all())
                for new in range(seen - 40, seen):
                    assert bool((kept == new).any(1).all())
        # 100 new tokens behind the new lengths, and masses that moved on
        for l in range(2):
            for b in range(3):
                n = min(100, lens[b] - 320)
                c.held[l]["ids"][b, :, 320:320 + n] = c.seen[b] + torch.arange(n, dtype=torch.int32, device="cuda")
            c.held[l]["mass"].mul_(torch.rand(c.held[l]["mass"].shape, generator=g, device="cuda") + 0.5)
        c.ctx = [320 + min(100, n - 320) for n in lens]
        c.ctx_t = i32(c.ctx)
        c.seen += i32([min(100, n - 320) for n in lens])


def test_other_rows_and_slots_stay():
    c = Case([500, 300], 2, seed=11, extra_rows=3, slack=12)
    c.both(111, 4, 8)


def test_lengths_outside_the_table_and_pages_outside_the_pool():
    c = Case([640, 300], 2, seed=12)
    before = c.state()
    c.ctx_t[0] = 1 << 20  # counts as 640
    c.call(100, 4, 8, want_err=kvq.DEVERR_POS)
    c.check(before, 100, 4, 8)
    c = Case([640, 300, 90], 2, seed=13)
    c.ctx_t[1] = -4
    before = c.state()
    c.call(100, want_err=kvq.DEVERR_POS)
    c.check(before, 100, ctx=[640, 0, 90])
    c = Case([640, 300], 1, seed=14)
    before = c.state()
    c.tables[0][0, 5] = -1
    c.tables[0][0, 0] = 1 << 20
    c.call(200, want_err=kvq.DEVERR_PAGE)
    after = c.state()
    want = c.model(before, 200, 0, 0, ctx=[0, 300])
    assert np.array_equal(want[1][0][1], after[1][0][1]) and np.array_equal(want[2][0][1], after[2][0][1])
    table = c.tables[0].cpu().numpy()
    mine = [int(x) for x in table[1] if x >= 0]
    assert np.array_equal(want[0][0][mine], after[0][0][mine])
    # of the other sequence only slots of its pages in the pool have changed
    lost = torch.from_numpy(after[1][0][0, 0] != before[1][0][0, 0]).nonzero()[:, 0]
    assert len(lost) and int(lost.min()) >= 64 and int(lost.max()) < 200


def test_repeats_streams_and_graph():
    c = Case([3000, 64, 5000, 4096], 4, layers=3, seed=15)
    first = c.state()
    saved = [p.clone() for p in c.pages], [{k: v.clone() for k, v in h.items()} for h in c.held]

    def restore():
        for p, q in zip(c.pages, saved[0]):
            p.copy_(q)
        for h, q in zip(c.held, saved[1]):
            for k in h:
                h[k].copy_(q[k])
    c.call(1000, 4, 100)
    c.check(first, 1000, 4, 100)
    want = c.state()
    restore()
    c.call(1000, 4, 100, stream=torch.cuda.Stream())
    assert all(a.tobytes() == b.tobytes() for x, y in zip(want, c.state()) for a, b in zip(x, y))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.kvq_evict_int4(c.caches, c.masses, c.ctx_t, c.seen, 1000, 4, 100, c.err, ctx_out=c.out)
    for n in ([3000, 64, 5000, 4096], [1200, 0, 4999, 1000]):
        restore()
        c.ctx = n
        c.ctx_t.copy_(i32(n))
        c.seen.copy_(i32(n))
        g.replay()
        torch.cuda.synchronize()
        assert c.err.item() == 0
        c.check(first, 1000, 4, 100)


def test_two_calls_at_once():
    cases = [Case([4000, 900, 77], 4, layers=2, seed=20 + i) for i in range(2)]
    before = [c.state() for c in cases]
    for c in cases:
        c.masses = [kvq.token_mass(h["mass"], h["ids"]) for h in c.held]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for c, s in zip(cases, streams):
        kvq.kvq_evict_int4(c.caches, c.masses, c.ctx_t, c.seen, 500, 4, 32, c.err, ctx_out=c.out, stream=s)
    torch.cuda.synchronize()
    for c, x in zip(cases, before):
        assert c.err.item() == 0
        c.check(x, 500, 4, 32)


def test_many_sequences_and_layers():
    c = Case([(i * 37) % 200 for i in range(1024)], 1, seed=30)
    c.both(70, 2, 9)
    c = Case([300, 200], 1, layers=64, seed=31)
    c.both(150, 2, 9)
