"""The page pool (alloc, fork, free, compact, copy) against a plain model of lists: counts, tables and
bytes are equal, and a session's life on it (prompt, fork, tree, commit, free, compact) ends with the
same cache as one that never shared or moved a page."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq
from gpu_util import unpack_int4

pytestmark = pytest.mark.gpu
D = 128


def i32(x):
    return torch.tensor(np.asarray(x, np.int32).reshape(-1), device="cuda")


def pages_of(n):
    return -(-n // 64)


class Pool:
    """The device pool and its model, called side by side."""

    def __init__(self, num_pages, num_seqs, max_pages):
        self.refs = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
        self.table = torch.full((num_seqs, max_pages), -1, dtype=torch.int32, device="cuda")
        self.r = np.zeros(num_pages, np.int64)
        self.t = np.full((num_seqs, max_pages), -1, np.int64)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def same(self, err=0):
        torch.cuda.synchronize()
        assert np.array_equal(self.refs.cpu().numpy(), self.r)
        assert np.array_equal(self.table.cpu().numpy(), self.t)
        assert self.err.item() == err
        self.err.zero_()

    def free_page(self):
        z = np.nonzero(self.r == 0)[0]
        return int(z[0]) if len(z) else -1

    def ok(self, i, ids, *lens):
        S, M = self.t.shape
        return 0 <= ids[i] < S and ids[i] not in ids[:i] and all(0 <= x[i] <= 64 * M for x in lens)

    def alloc(self, ids, old, new, err=0):
        kvq.kvq_pages_alloc(self.refs, self.table, i32(ids), i32(old), i32(new), self.err)
        for i in range(len(ids)):
            if self.ok(i, ids, old, new):
                for p in range(pages_of(old[i]), pages_of(new[i])):
                    g = self.free_page()
                    self.t[ids[i], p] = g
                    if g >= 0:
                        self.r[g] = 1
        self.same(err)

    def free(self, ids, old, new, err=0):
        kvq.kvq_pages_free(self.refs, self.table, i32(ids), i32(old), i32(new), self.err)
        for i in range(len(ids)):
            if self.ok(i, ids, old, new):
                for p in range(pages_of(new[i]), pages_of(old[i])):
                    g = self.t[ids[i], p]
                    if 0 <= g < len(self.r):
                        self.t[ids[i], p] = -1
                        self.r[g] = max(0, self.r[g] - 1)
        self.same(err)

    def fork(self, par, ch, lens, err=0):
        src, dst = i32([5] * len(par)), i32([5] * len(par))
        kvq.kvq_pages_fork(self.refs, self.table, i32(par), i32(ch), i32(lens), src, dst, self.err)
        ws, wd = [-1] * len(par), [-1] * len(par)
        live = self.r.copy()
        for i in range(len(par)):
            if not (self.ok(i, ch, lens) and 0 <= par[i] < len(self.t) and ch[i] not in par):
                continue
            for p in range(lens[i] // 64):
                g = self.t[par[i], p]
                good = 0 <= g < len(self.r) and live[g] > 0
                self.t[ch[i], p] = g if good else -1
                if good:
                    self.r[g] += 1
            if lens[i] % 64:
                p = lens[i] // 64
                g = self.t[par[i], p]
                n = -1
                if 0 <= g < len(self.r) and live[g] > 0:
                    ws[i] = int(g)
                    n = wd[i] = self.free_page()
                    if n >= 0:
                        self.r[n] = 1
                self.t[ch[i], p] = n
        self.same(err)
        assert src.tolist() == ws and dst.tolist() == wd
        return src, dst

    def compact(self, err=0):
        n = len(self.r)
        src, dst = i32([-7] * n), i32([-7] * n)
        moves = i32([-1])
        kvq.kvq_pages_compact(self.refs, self.table, src, dst, moves, self.err)
        L = int((self.r > 0).sum())
        s = [p for p in range(L, n) if self.r[p] > 0]
        d = [p for p in range(L) if self.r[p] == 0]
        to = dict(zip(s, d))
        for a, b in to.items():
            self.r[b], self.r[a] = self.r[a], 0
        self.t = np.vectorize(lambda v: to.get(v, v))(self.t)
        self.same(err)
        assert moves.item() == len(s) and src[:len(s)].tolist() == s and dst[:len(s)].tolist() == d
        assert bool((src[len(s):] == -7).all() and (dst[len(s):] == -7).all())
        return src, dst, moves


@pytest.mark.parametrize("num_pages", [1, 7, 128, 129, 1000, 40000, 300001])
def test_random_life_of_a_pool(num_pages):
    rng = np.random.default_rng(num_pages)
    S, M = 24, max(1, min(200, num_pages // 6))
    pool = Pool(num_pages, S, M)
    lens = [0] * S
    for step in range(12):
        free = [b for b in range(S) if lens[b] == 0]
        used = [b for b in range(S) if lens[b] > 0]
        room = int((pool.r == 0).sum())
        grow, old, new = [], [], []
        for b in rng.permutation(S)[:rng.integers(1, 9)].tolist():
            n = int(min(64 * M, lens[b] + rng.integers(0, 64 * M // 2 + 1)))
            need = pages_of(n) - pages_of(lens[b])
            if need <= room:
                room -= need
                grow.append(b), old.append(lens[b]), new.append(n)
                lens[b] = n
        if grow:
            pool.alloc(grow, old, new)
        used = [b for b in range(S) if lens[b] > 0]
        free = [b for b in range(S) if lens[b] == 0]
        if used and free:
            k = min(len(free), int(rng.integers(1, 6)), int((pool.r == 0).sum()))
            par = [int(rng.choice(used)) for _ in range(k)]
            if k:
                ln = [int(rng.integers(0, lens[p] + 1)) for p in par]
                pool.fork(par, free[:k], ln)
                for c, n in zip(free[:k], ln):
                    lens[c] = n
        drop = [b for b in range(S) if lens[b] > 0 and rng.random() < 0.3]
        keep = [int(rng.integers(0, lens[b] + 1)) if rng.random() < 0.5 else 0 for b in drop]
        if drop:
            pool.free(drop, [lens[b] for b in drop], keep)
            for b, n in zip(drop, keep):
                lens[b] = n
        if step % 4 == 3:
            pool.compact()


def test_requests_at_their_most():
    pool = Pool(5000, 1024, 8)
    pool.alloc(list(range(1024)), [0] * 1024, [64 * (i % 5) + i % 3 for i in range(1024)])
    pool.free(list(range(0, 1024, 2)), [64 * (i % 5) + i % 3 for i in range(0, 1024, 2)], [0] * 512)
    pool.compact()


def test_empty_calls_change_nothing():
    pool = Pool(10, 2, 2)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    kvq.kvq_pages_alloc(pool.refs, pool.table, none, none, none, pool.err)
    kvq.kvq_pages_free(pool.refs, pool.table, none, none, none, pool.err)
    kvq.kvq_pages_fork(pool.refs, pool.table, none, none, none, none, none, pool.err)
    pool.same()
    pool.compact()


def test_bad_requests_are_flagged_and_skipped():
    pool = Pool(20, 4, 3)
    pool.alloc([0, 9, -1, 1, 1], [0, 0, 0, 0, 0], [100, 64, 64, 64, 128], err=kvq.DEVERR_POS)
    pool.alloc([2], [0], [193], err=kvq.DEVERR_POS)
    pool.alloc([2], [-1], [64], err=kvq.DEVERR_POS)
    pool.fork([0, 0, 1], [2, 2, 0], [100, 64, 64], err=kvq.DEVERR_POS)  # a child twice; a parent as a child
    pool.fork([0], [3], [150], err=kvq.DEVERR_PAGE)                     # more than the parent holds
    pool.free([0, 0], [100, 100], [0, 64], err=kvq.DEVERR_POS)
    pool.free([1], [128], [0], err=kvq.DEVERR_PAGE)                     # one page held, two named


def test_no_page_left():
    pool = Pool(5, 3, 4)
    pool.alloc([0, 1], [0, 0], [192, 256], err=kvq.DEVERR_POOL)
    assert pool.t[1].tolist() == [3, 4, -1, -1]
    pool.fork([0], [2], [100], err=kvq.DEVERR_POOL)


def test_freed_too_often():
    pool = Pool(5, 2, 2)
    pool.table[0, 0] = 3
    pool.t[0, 0] = 3
    pool.free([0], [64], [0], err=kvq.DEVERR_POOL)


def test_a_dead_entry_is_flagged_by_compact():
    pool = Pool(8, 2, 4)
    pool.alloc([0], [0], [256])
    pool.free([0], [256], [0])
    pool.refs[6] = 1
    pool.r[6] = 1
    pool.table[0, 0], pool.table[1, 0] = 6, 7
    pool.t[0, 0], pool.t[1, 0] = 6, 7
    pool.compact(err=kvq.DEVERR_PAGE)
    assert pool.t[0, 0] == 0 and pool.t[1, 0] == 7


def caches(n, pages, heads, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    data = [torch.randint(0, 256, (pages, heads, 8704), generator=g, device="cuda", dtype=torch.uint8) for _ in range(n)]
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    return data, [kvq.int4_cache(d, table) for d in data], table


@pytest.mark.parametrize("layers,heads,pages", [(1, 1, 2), (3, 4, 50), (64, 1, 6), (2, 8, 700)])
def test_copy(layers, heads, pages):
    data, cs, _t = caches(layers, pages, heads)
    rng = np.random.default_rng(pages)
    perm = rng.permutation(pages)
    k = pages // 2
    src, dst = perm[:k].copy(), perm[k:2 * k].copy()
    if k > 2:
        src[0], dst[1] = -1, -1
    want = [d.clone() for d in data]
    for w in want:
        for a, b in zip(src, dst):
            if a >= 0 and b >= 0:
                w[b] = w[a]
    err = i32([0])
    kvq.kvq_pages_copy(cs, i32(src), i32(dst), err)
    torch.cuda.synchronize()
    assert err.item() == 0 and all(torch.equal(a, b) for a, b in zip(data, want))


def test_copy_counts_and_bad_pages():
    data, cs, _t = caches(2, 10, 2)
    was = [d.clone() for d in data]
    err = i32([0])
    kvq.kvq_pages_copy(cs, i32([0, 1, 2]), i32([5, 6, 7]), err, count=i32([1]))
    kvq.kvq_pages_copy(cs, i32([0, 1]), i32([8, 9]), err, count=i32([-3]))
    assert err.item() == 0
    kvq.kvq_pages_copy(cs, i32([10, 3, -2]), i32([1, 1 << 20, 2]), err)
    kvq.kvq_pages_copy(cs, i32([3]), i32([3]), err)
    assert err.item() == kvq.DEVERR_PAGE
    for d, w in zip(data, was):
        w[5] = w[0]
        assert torch.equal(d, w)


def test_a_sessions_life_on_shared_and_moved_pages():
    """Prompt attention and append, three forks, a tree verified and committed on each, the others
    freed, the pool compacted: the branch's cache and its next attention equal those of a session that
    was appended token by token on pages of its own."""
    from test_gpu_tree import tree, words
    rng = np.random.default_rng(3)
    g = torch.Generator(device="cuda").manual_seed(3)
    Hq, Hkv, n, N, layers = 20, 4, 150, 12, 2
    pool = Pool(64, 6, 8)
    data = [torch.zeros((64, Hkv, 8704), dtype=torch.uint8, device="cuda") for _ in range(layers)]
    cs = [kvq.int4_cache(d, pool.table) for d in data]
    pool.alloc([4], [0], [300])  # another session in front
    pool.alloc([0], [0], [n + N])
    R, _ = kvq.kvq_build_rotation(1)
    Mq, Mk = (torch.from_numpy(m).cuda() for m in kvq.kvq_fold_qk(R, np.ones(D, np.float32), np.ones(D, np.float32)))
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    k, v, q = rand(n, Hkv, D), rand(n, Hkv, D), rand(n, Hq, D)
    ids = lambda b, t: torch.full((t,), b, dtype=torch.int32, device="cuda")  # noqa: E731
    pos = lambda a, e: torch.arange(a, e, dtype=torch.int32, device="cuda")  # noqa: E731
    norm = lambda x: (x.float() / (x.float().square().mean(-1, keepdim=True) + 1e-6).sqrt()).to(torch.bfloat16)  # noqa: E731
    out = torch.empty_like(q)
    kvq.kvq_prompt_attn(norm(q), norm(k), v, i32([0, n]), out, kvq.alloc_prompt_workspace(n, 1, Hq, Hkv), pool.err)
    for c in cs:
        kvq.kvq_rotate_quant_append(c, Mk, k, v, ids(0, n), pos(0, n), pool.err)
    # the prompt's last row is close to what decoding it over the 4-bit cache gives
    dec = torch.empty((1, 1, Hq, D), dtype=torch.float32, device="cuda")
    kvq.kvq_decode_attn_int4(cs[0], Mq, Mk, q[None, -1:].contiguous(), i32([n - 1]), dec, kvq.alloc_workspace(1, 1, Hq, Hkv), pool.err)
    assert float((dec[0, 0] - out[-1].float()).norm() / out[-1].float().norm()) < 0.4
    src, dst = pool.fork([0, 0, 0], [1, 2, 3], [n, n, n])
    kvq.kvq_pages_copy(cs, src, dst, pool.err)
    pool.alloc([1, 2, 3], [n] * 3, [n + N] * 3)
    # the tree of each branch
    kn, vn, qn = rand(3, N, Hkv, D), rand(3, N, Hkv, D), rand(3, N, Hq, D)
    masks = [tree(N, rng) for _ in range(3)]
    path = np.zeros((3, N), np.int32)
    acc = [3, 5, 0]
    for b in range(3):
        path[b, :acc[b]] = np.sort(rng.choice(N, acc[b], replace=False))
    rows = [kvq.int4_cache(d, pool.table[1:4]) for d in data]
    tout = torch.empty((3, N, Hq, D), dtype=torch.float32, device="cuda")
    for c in rows:
        kvq.kvq_tree_attn_int4(c, Mq, Mk, qn, i32([n] * 3), words(masks), tout, kvq.alloc_tree_workspace(3, N, Hq, Hkv),
                               pool.err, k_new=kn, v_new=vn)
    ctx = i32([0] * 3)
    kvq.kvq_tree_commit_int4(rows, i32([n] * 3), torch.from_numpy(path).cuda(), i32(acc), pool.err, ctx_out=ctx)
    assert ctx.tolist() == [n + a for a in acc]
    # the winner is branch 2; everything else goes, and the pool is compacted
    pool.free([4, 0, 1, 3], [300, n + N, n + N, n + N], [0] * 4)
    pool.free([2], [n + N], [n + 5])
    src, dst, moves = pool.compact()
    kvq.kvq_pages_copy(cs, src, dst, pool.err, count=moves)
    torch.cuda.synchronize()
    assert pool.t[2].tolist()[:3] == sorted(pool.t[2].tolist()[:3]) or moves.item() > 0
    # the same tokens on a cache of their own
    own_t, own = kvq.alloc_int4_cache(4, Hkv, torch.arange(4, dtype=torch.int32)[None])
    kk, vv = (torch.cat([a, b[1, torch.from_numpy(path[1, :5].astype(np.int64)).cuda()]]) for a, b in ((k, kn), (v, vn)))
    kvq.kvq_rotate_quant_append(own, Mk, kk, vv, ids(0, n + 5), pos(0, n + 5), pool.err)
    for d in data:
        for h in range(Hkv):
            a = unpack_int4({"pages": d, "block_table": pool.table}, 2, h, n + 5)
            b = unpack_int4(own_t, 0, h, n + 5)
            assert all(np.array_equal(a[x], b[x]) for x in a)
    qd = rand(1, 1, Hq, D)
    outs = []
    for c in (kvq.int4_cache(data[1], pool.table[2:3]), own):
        o = torch.empty((1, 1, Hq, D), dtype=torch.float32, device="cuda")
        kvq.kvq_decode_attn_int4(c, Mq, Mk, qd, i32([n + 4]), o, kvq.alloc_workspace(1, 1, Hq, Hkv), pool.err)
        outs.append(o)
    assert torch.equal(*outs) and pool.err.item() == 0


def test_pool_calls_in_a_graph():
    pool = Pool(100, 4, 8)
    data, cs, _t = caches(2, 100, 2)
    pool.alloc([0], [0], [200])
    src, dst = i32([-1]), i32([-1])
    a = [i32(x) for x in ([0], [1], [200], [0])]
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        kvq.kvq_pages_fork(pool.refs, pool.table, a[0], a[1], a[2], src, dst, pool.err)
        kvq.kvq_pages_copy(cs, src, dst, pool.err)
        kvq.kvq_pages_free(pool.refs, pool.table, a[1], a[2], a[3], pool.err)
    refs = pool.refs.clone()
    for _ in range(3):
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(refs, pool.refs) and src.tolist() == [3] and dst.tolist() == [4]
        assert all(torch.equal(d[3], d[4]) for d in data) and pool.err.item() == 0
