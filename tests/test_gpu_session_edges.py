"""Calls of the session operators that users make around the plain ones: replays with other contents, graphs
that share a workspace, calls at once, offsets past 32 bits, the most sequences."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq
from test_gpu_prompt import check, inputs, offsets, reference
from test_gpu_tree import Int4Case, RingCase, i32, tree, words

pytestmark = pytest.mark.gpu
D = 128

# int4 in the row kernels (R <= 16, 17..48) and in tile form; the ring in both of its forms
FORMS = [("int4", 3, (6, 2)), ("int4", 8, (20, 4)), ("int4", 16, (20, 4)), ("ring", 3, (6, 2)), ("ring", 16, (20, 4))]


def case(kind, N, heads, seed):
    return Int4Case([70, 1000, 5], N, *heads, seed=seed) if kind == "int4" else RingCase([70, 1000, 5], N, *heads, 513, seed=seed)


def issue(c, w, out, ws, stream=None):
    if isinstance(c, Int4Case):
        kvq.kvq_tree_attn_int4(c.cache, c.Mq, c.Mk, c.q, c.ctx_t, w, out, ws, c.err, k_new=c.k_new, v_new=c.v_new, stream=stream)
    else:
        kvq.kvq_tree_attn_fp8_swa(c.ring, c.q, c.pos_t, w, c.window, c.KS, c.VS, out, ws, c.err, k_new=c.k_new, v_new=c.v_new,
                                  stream=stream)


@pytest.mark.parametrize("kind,N,heads", FORMS)
def test_tree_replays_with_other_contents(kind, N, heads):
    """A captured call reads lengths, masks and rows anew: two graphs over one workspace, replayed in turns."""
    c = case(kind, N, heads, 30)
    masks = [[tree(N, c.rng) for _ in range(3)] for _ in range(2)]
    want = [c.call(m) for m in masks]
    w = words(masks[0])
    outs = [torch.zeros_like(want[0]) for _ in range(2)]
    ws = kvq.alloc_tree_workspace(3, N, *heads)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            issue(c, w, o, ws)
    for turn in range(4):
        w.copy_(words(masks[turn % 2]))
        graphs[turn // 2 % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[turn // 2 % 2], want[turn % 2])
    t = c.ctx_t if kind == "int4" else c.pos_t
    keep = t.clone()
    w.copy_(words(masks[0]))
    t.copy_(i32([3, 2, 5]))  # shorter contexts: the rows behind them are the drafted ones now
    graphs[0].replay()
    torch.cuda.synchronize()
    c.ctx = c.pos0 = [3, 2, 5]
    c.check(outs[0], masks[0])
    t.copy_(keep)
    assert c.err.item() == 0


@pytest.mark.parametrize("kind,N,heads", FORMS)
def test_trees_at_once(kind, N, heads):
    cs = [case(kind, N, heads, 40 + i) for i in range(2)]
    masks = [[tree(N, c.rng) for _ in range(3)] for c in cs]
    want = [c.call(m) for c, m in zip(cs, masks)]
    ws = [kvq.alloc_tree_workspace(3, N, *heads) for _ in cs]
    outs = [torch.zeros_like(x) for x in want]
    w = [words(m) for m in masks]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(6):
        for i in range(2):
            issue(cs[i], w[i], outs[i], ws[i], streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want)) and all(c.err.item() == 0 for c in cs)


@pytest.mark.parametrize("kind,N,heads", FORMS)
def test_tree_rows_beside_a_nan_query(kind, N, heads):
    """A query that is not finite is flagged (int4) or gives NaN, and no other row changes."""
    c = case(kind, N, heads, 45)
    masks = [tree(N, c.rng) for _ in range(3)]
    want = c.call(masks)
    c.q[1, N - 1, 0, 7] = float("nan")
    out, ws = torch.zeros_like(want), kvq.alloc_tree_workspace(3, N, *heads)
    ws.view(torch.float32).fill_(float("nan"))
    issue(c, words(masks), out, ws)
    torch.cuda.synchronize()
    keep = torch.ones(out.shape[:3], dtype=torch.bool, device="cuda")
    keep[1, N - 1, 0] = False
    assert torch.equal(out[keep], want[keep])
    assert c.err.item() == (kvq.DEVERR_NONFINITE if kind == "int4" else 0)


def test_tree_padded_batch():
    """Trees of 3 and 6 tokens padded to 9: padding rows of any content change nothing."""
    c = Int4Case([100, 30], 9, 20, 4, seed=50)
    masks = [tree(3, c.rng) + [0] * 6, tree(6, c.rng) + [0] * 3]
    a = c.call(masks)
    c.q[0, 3:] = 1e4
    c.k_new[0, 3:], c.v_new[1, 6:] = 1e4, -1e4
    b = c.call(masks)
    assert torch.equal(a[0, :3], b[0, :3]) and torch.equal(a[1, :6], b[1, :6])
    c.check(b, masks)


@pytest.mark.parametrize("N,heads", [(25, (2, 1)), (2, (2, 1)), (10, (2, 1))])
def test_tree_most_sequences(N, heads):
    c = Int4Case([(i * 13) % 130 for i in range(1024)], N, *heads, seed=51)
    masks = [tree(N, c.rng) for _ in range(c.B)]
    out = c.call(masks, torch.bfloat16)
    c.B = 1024
    for b in (0, 1, 500, 1023):  # some of them against the plain evaluation
        one = Int4Case.__new__(Int4Case)
        one.__dict__.update(c.__dict__)
        one.B, one.ctx, one.q = 1, [c.ctx[b]], c.q[b:b + 1]
        one.dequantised = lambda _, h, L, b=b: c.dequantised(b, h, L)
        one.check(out[b:b + 1], [masks[b]])


@pytest.mark.parametrize("N,heads", [(9, (4, 1)), (2, (4, 1))])
def test_ring_most_sequences(N, heads):
    c = RingCase([(i * 13) % 900 for i in range(1024)], N, *heads, 100, seed=52)
    masks = [tree(N, c.rng) for _ in range(c.B)]
    out = c.call(masks, torch.bfloat16)
    c.B, c.pos0 = 20, c.pos0[:20]
    c.check(out, masks[:20])


@pytest.mark.parametrize("N,heads", [(2, (8, 4)), (8, (16, 4)), (20, (16, 4))])
def test_tree_and_commit_past_4_gib_of_pool(N, heads):
    """The same contents in the first pages and in the last ones of a pool of more than 2^32 bytes."""
    low = Int4Case([200, 64], N, *heads, seed=53)
    masks = [tree(N, low.rng) for _ in range(2)]
    want = low.call(masks)
    P = low.tensors["block_table"].shape[1]
    pages = (1 << 32) // (4 * kvq.INT4_BLOCK_BYTES) + 2 * P + 1
    high = Int4Case.__new__(Int4Case)
    high.__dict__.update(low.__dict__)
    table = (pages - 1 - torch.arange(2 * P, dtype=torch.int32)).view(2, P)
    high.tensors, high.cache = kvq.alloc_int4_cache(pages, 4, table)
    lt, ht = low.tensors["block_table"].long().flatten(), table.flatten().long().cuda()
    high.tensors["pages"][ht] = low.tensors["pages"][lt]
    assert torch.equal(high.call(masks), want)
    path = np.zeros((2, N), np.int64)
    path[:, :N // 2] = [np.sort(low.rng.choice(N, N // 2, replace=False)) for _ in range(2)]
    path[0, 0] = N - 1
    for c in (low, high):
        kvq.kvq_tree_commit_int4([c.cache], c.ctx_t, i32(path), i32([N // 2] * 2), c.err)
    assert torch.equal(high.tensors["pages"][ht], low.tensors["pages"][lt])
    src, dst = i32(ht.tolist()), i32([int(x) - 2 * P for x in ht])
    kvq.kvq_pages_copy([high.cache], src, dst, high.err)
    assert torch.equal(high.tensors["pages"][ht - 2 * P], low.tensors["pages"][lt]) and high.err.item() == 0


def test_prompt_offsets_past_32_bits():
    """1,050,000 tokens x 20 heads x 128 elements: more than 2^31 elements of q and of out."""
    lens = [1200] * 875
    T = sum(lens)
    assert T * 20 * 128 > 1 << 31
    q = torch.empty(T, 20, D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.empty(T, 4, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for i, x in enumerate((q, k, v)):
        x.normal_(generator=torch.Generator(device="cuda").manual_seed(60 + i))
    out, err = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.kvq_prompt_attn(q, k, v, offsets(lens), out, kvq.alloc_prompt_workspace(T, len(lens), 20, 4), err)
    torch.cuda.synchronize()
    assert err.item() == 0
    for b in (0, 699, 874):
        s = slice(1200 * b, 1200 * (b + 1))
        check(out[s], *reference(q[s], k[s], v[s], [1200], 0, D ** -0.5))


def test_prompt_replays_with_other_sequences():
    T = 700
    q, k, v = inputs([T], 20, 4, torch.bfloat16, seed=61)
    cu, err = offsets([T, 0, 0]), torch.zeros(1, dtype=torch.int32, device="cuda")
    out, ws = torch.empty_like(q), kvq.alloc_prompt_workspace(T, 3, 20, 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.kvq_prompt_attn(q, k, v, cu, out, ws, err)
    for lens in ([700, 0, 0], [1, 300, 399], [0, 0, 0], [129, 129, 128]):
        cu.copy_(offsets(lens))
        out.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        n = sum(lens)
        check(out[:n], *(x[:n] for x in reference(q, k, v, lens, 0, D ** -0.5)))
        assert bool((out[n:] == 3).all()) and err.item() == 0


def test_commit_replays():
    """Rings and pages under one capture, with other paths and lengths at each replay."""
    cs = [Int4Case([100, 61], 6, 4, 2, seed=s) for s in (1, 2)]
    for c in cs:
        c.append()
    r = RingCase([100, 61], 6, 4, 2, 513, seed=3)
    r.call([tree(6, r.rng)] * 2)
    path, n = i32([[0] * 6] * 2), i32([0, 0])
    ctx = cs[0].ctx_t.clone()
    out = torch.zeros(2, dtype=torch.int32, device="cuda")

    def both():
        kvq.kvq_tree_commit_int4([c.cache for c in cs], ctx, path, n, cs[0].err, ctx_out=out)
        kvq.kvq_tree_commit_fp8([r.ring], ctx, path, n, r.err)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    data = [c.tensors["pages"] for c in cs] + [r.tensors["data"]]
    for p, a, at in (([[1, 3, 5, 0, 0, 0], [0, 2, 0, 0, 0, 0]], [3, 2], [100, 61]), ([[2, 0, 1, 5, 4, 3]] * 2, [6, 1], [98, 61]),
                     ([[5] * 6] * 2, [0, 6], [100, 60])):
        path.copy_(i32(p))
        n.copy_(i32(a))
        ctx.copy_(i32(at))
        before = [x.clone() for x in data]
        both()
        torch.cuda.synchronize()
        want = [x.clone() for x in data]
        for x, y in zip(data, before):
            x.copy_(y)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(data, want)) and out.tolist() == [s + t for s, t in zip(at, a)]
    assert cs[0].err.item() == 0 == r.err.item()


def test_tensors_that_do_not_fit_are_refused():
    """Nothing is launched for a tensor of another type, shape or place."""
    c = Int4Case([10], 4, 4, 2, seed=70)
    w, out, ws = words([tree(4, c.rng)]), torch.zeros(1, 4, 4, D, device="cuda"), kvq.alloc_tree_workspace(1, 4, 4, 2)

    def tree_call(**o):
        a = dict(Mq=c.Mq, Mk=c.Mk, q=c.q, ctx=c.ctx_t, w=w, out=out, ws=ws, err=c.err, fwht=False, k=c.k_new, v=c.v_new)
        a.update(o)
        kvq.kvq_tree_attn_int4(c.cache, a["Mq"], a["Mk"], a["q"], a["ctx"], a["w"], a["out"], a["ws"], a["err"], k_new=a["k"],
                               v_new=a["v"], fwht=a["fwht"])

    for bad in (dict(Mq=c.Mq[0]), dict(Mk=c.Mk[0]), dict(fwht=True), dict(Mq=c.Mq.cpu()), dict(Mq=c.Mq.double()), dict(q=c.q.half()),
                dict(q=c.q.cpu()), dict(ctx=c.ctx_t.long()), dict(ctx=c.ctx_t.cpu()), dict(w=w[:, :3]), dict(w=w.int()), dict(out=out[:, :3]),
                dict(out=out.cpu()), dict(ws=ws.cpu()), dict(err=c.err.cpu()), dict(err=c.err.float()), dict(err=c.err[:0]),
                dict(k=c.k_new.float()), dict(v=c.v_new[:, :, :1])):
        with pytest.raises(ValueError):
            tree_call(**bad)
    q, k, v = inputs([40], 4, 2, torch.bfloat16)
    pws, err = kvq.alloc_prompt_workspace(40, 1, 4, 2), c.err
    for bad in ((q.cpu(), k, v, q.clone(), pws, err), (q, k.cpu(), v, q.clone(), pws, err), (q, k, v, q.half(), pws, err),
                (q, k, v, q[:39], pws, err), (q, k, v, q.clone(), pws.cpu(), err), (q, k, v, q.clone(), pws, err.cpu())):
        with pytest.raises(ValueError):
            kvq.kvq_prompt_attn(bad[0], bad[1], bad[2], offsets([40]), bad[3], bad[4], bad[5])
    with pytest.raises(ValueError):
        kvq.kvq_tree_commit_int4([c.cache], c.ctx_t, i32([[0, 1, 2, 3]]), i32([1]), c.err.cpu())
    refs, table, one = i32([0] * 8), i32([[-1] * 4]), i32([0])
    for bad in ((refs.long(), table, one, c.err), (refs, table[:, ::2], one, c.err), (refs, table, one.cpu(), c.err), (refs, table, one, one.cpu())):
        with pytest.raises(ValueError):
            kvq.kvq_pages_alloc(bad[0], bad[1], bad[2], one, one, bad[3])
    torch.cuda.synchronize()
    assert c.err.item() == 0 and bool((out == 0).all())
