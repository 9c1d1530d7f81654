"""Host-side refusals of the prompt, tree, commit and page-pool calls: no GPU is needed, nothing is
launched for a bad argument."""

import ctypes

import pytest

import quantized_kv_cache_fold_gb300 as kvq

L = kvq.lib
INVALID, UNSUPPORTED = 1, 2


def cache(**over):
    d = dict(pages=0x10000, block_table=0x50000, num_seqs=4, max_pages_per_seq=8, num_pages=32, num_kv_heads=4,
             page_size=64, head_dim=128)
    d.update(over)
    return kvq.Int4Cache(**d)


def prompt(strides=None, **over):
    a = dict(q=0x1000000, k=0x2000000, v=0x3000000, dtype=kvq.BF16, T=100, B=2, Hq=20, Hkv=4, cu=0x9000, window=0, sm=0.09,
             out=0x4000000, ws=0xB0000, n=1 << 30, err=0xC0000)
    a.update(over)
    st = (ctypes.c_int64 * 8)(*strides) if strides else None
    return L.kvq_prompt_attn(a["q"], a["k"], a["v"], a["dtype"], a["T"], a["B"], a["Hq"], a["Hkv"], st, a["cu"],
                             a["window"], a["sm"], a["out"], a["ws"], a["n"], a["err"], None)


PACKED = [2560, 128, 512, 128, 512, 128, 2560, 128]


@pytest.mark.parametrize("over", [
    dict(q=0), dict(k=None), dict(v=0), dict(out=0), dict(cu=0), dict(ws=0), dict(err=0), dict(dtype=7), dict(dtype=-1),
    dict(T=-1), dict(B=0), dict(B=1025), dict(Hq=21), dict(Hkv=0), dict(Hq=0), dict(T=1 << 27), dict(sm=0.0), dict(sm=-1.0),
    dict(sm=float("nan")), dict(sm=float("inf")), dict(q=0x1000008), dict(out=0x4000002), dict(ws=0xB0010), dict(n=8),
    dict(out=0x1000000), dict(out=0x2000000 + 256), dict(out=0x1000000 - 2560)])
def test_prompt_refuses(over):
    assert prompt(**over) == INVALID


def test_prompt_strides_and_types():
    assert prompt(dtype=kvq.F32) == UNSUPPORTED
    for i in range(8):
        for bad in (0, -8, 4, 129, 1 << 40):
            assert prompt(PACKED[:i] + [bad] + PACKED[i + 1:]) == INVALID
    assert prompt(PACKED[:6] + [1280, 128]) == INVALID  # the output's rows overlap
    assert prompt(PACKED[:6] + [2560, 64]) == INVALID
    assert prompt(T=0, q=0, k=0, v=0, out=0, cu=0, ws=0, n=0, err=0) == 0
    assert kvq.kvq_prompt_workspace_bytes(100, 2, 20, 4) > 0
    assert kvq.kvq_prompt_workspace_bytes(100, 0, 20, 4) == 0 == kvq.kvq_prompt_workspace_bytes(-1, 2, 20, 4)
    assert kvq.kvq_prompt_workspace_bytes(100, 2, 20, 3) == 0


def tree4(c=None, fn="kvq_tree_attn_int4", **over):
    a = dict(Mq=0x60000, Mk=0x70000, q=0x80000, dtype=1, B=2, N=16, Hq=20, ctx=0x90000, mask=0x91000, k=None, v=None, sm=0.09,
             eps=1e-6, out=0xA0000, od=1, ws=0xB0000, n=1 << 30, err=0xC0000)
    a.update(over)
    return getattr(L, fn)(ctypes.byref(c or cache()), a["Mq"], a["Mk"], a["q"], a["dtype"], a["B"], a["N"], a["Hq"], a["ctx"],
                          a["mask"], a["k"], a["v"], a["sm"], a["eps"], a["out"], a["od"], a["ws"], a["n"], a["err"], None)


BAD_TREE = [(dict(B=0), INVALID), (dict(B=5), INVALID), (dict(N=0), UNSUPPORTED), (dict(N=65), UNSUPPORTED), (dict(Hq=21), UNSUPPORTED),
            (dict(Hq=0), UNSUPPORTED), (dict(Hq=260), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(od=2), INVALID), (dict(q=0), INVALID),
            (dict(q=0x80004), INVALID), (dict(ctx=0), INVALID), (dict(mask=0), INVALID), (dict(mask=0x91004), INVALID), (dict(out=0), INVALID),
            (dict(out=0xA0008), INVALID), (dict(ws=0), INVALID), (dict(ws=0xB0080), INVALID), (dict(n=100), INVALID), (dict(err=0), INVALID),
            (dict(k=0xD0000), INVALID), (dict(v=0xD0000), INVALID), (dict(k=0xD0008, v=0xE0000), INVALID), (dict(sm=float("nan")), INVALID),
            (dict(sm=float("inf")), INVALID)]


@pytest.mark.parametrize("over,want", BAD_TREE + [
    (dict(Mq=0), INVALID), (dict(Mq=0x60004), INVALID), (dict(k=0xD0000, v=0xE0000, Mk=0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID)])
@pytest.mark.parametrize("fn", ["kvq_tree_attn_int4", "kvq_tree_attn_int4_fwht"])
def test_tree_int4_refuses(over, want, fn):
    assert tree4(fn=fn, **over) == want


def test_tree_int4_refuses_bad_caches():
    assert tree4(cache(head_dim=64)) == UNSUPPORTED
    assert tree4(cache(page_size=32)) == UNSUPPORTED
    assert tree4(cache(pages=0x10008)) == INVALID
    assert tree4(cache(max_pages_per_seq=2 ** 21, num_seqs=1024), B=1024) == UNSUPPORTED
    assert kvq.kvq_tree_workspace_bytes(2, 65, 20, 4) == 0 == kvq.kvq_tree_workspace_bytes(0, 6, 20, 4)


def tree8(r=(0x10000, 4, 4, 576, 128), **over):
    a = dict(q=0x80000, dtype=1, B=2, N=16, Hq=20, ctx=0x90000, mask=0x91000, window=513, k=None, v=None, ks=0.01, vs=0.01,
             sm=0.09, out=0xA0000, od=1, ws=0xB0000, n=1 << 30, err=0xC0000)
    a.update(over)
    return L.kvq_tree_attn_fp8_swa(ctypes.byref(kvq.Fp8Ring(*r)), a["q"], a["dtype"], a["B"], a["N"], a["Hq"], a["ctx"], a["mask"],
                                   a["window"], a["k"], a["v"], a["ks"], a["vs"], a["sm"], a["out"], a["od"], a["ws"], a["n"],
                                   a["err"], None)


@pytest.mark.parametrize("over,want", BAD_TREE + [
    (dict(window=15), INVALID), (dict(window=0), INVALID), (dict(window=562), INVALID), (dict(window=2 ** 31 - 1), INVALID),
    (dict(ks=0.0), INVALID), (dict(vs=float("nan")), INVALID), (dict(vs=float("inf")), INVALID)])
def test_tree_ring_refuses(over, want):
    assert tree8(**over) == want


def test_tree_ring_refuses_bad_rings():
    assert tree8((0x10000, 4, 4, 500, 128)) == INVALID
    assert tree8((0, 4, 4, 576, 128)) == INVALID
    assert tree8((0x10000, 4, 4, 576, 64)) == UNSUPPORTED


def test_commit_refuses():
    def c4(cs=None, n=None, B=2, N=8, ctx=0x1000, path=0x2000, acc=0x3000, out=None, err=0x5000):
        cs = cs or [cache(), cache(pages=0x20000)]
        return L.kvq_tree_commit_int4((kvq.Int4Cache * len(cs))(*cs), len(cs) if n is None else n, B, N, ctx, path, acc, out, err, None)

    for over in (dict(n=0), dict(B=0), dict(B=5), dict(B=1025), dict(ctx=0), dict(path=0), dict(acc=0), dict(err=0), dict(out=0x1000),
                 dict(out=0x1004), dict(cs=[cache(), cache(num_kv_heads=2)]), dict(cs=[cache(), cache(num_seqs=1)]),
                 dict(cs=[cache(pages=0)]), dict(cs=[cache(), cache(pages=0x20000), cache()])):
        assert c4(**over) == INVALID, over
    for over in (dict(N=0), dict(N=65), dict(cs=[cache()] * 65), dict(cs=[cache(head_dim=64)])):
        assert c4(**over) == UNSUPPORTED, over
    assert L.kvq_tree_commit_int4(None, 1, 2, 8, 0x1000, 0x2000, 0x3000, None, 0x5000, None) == INVALID

    def c8(rs, **o):
        a = dict(B=2, N=8, ctx=0x1000, path=0x2000, acc=0x3000, out=None, err=0x5000)
        a.update(o)
        rs = [kvq.Fp8Ring(*r) for r in rs]
        return L.kvq_tree_commit_fp8((kvq.Fp8Ring * len(rs))(*rs), len(rs), a["B"], a["N"], a["ctx"], a["path"], a["acc"], a["out"],
                                     a["err"], None)

    ring = (0x10000, 4, 4, 576, 128)
    assert c8([ring, (0x10000, 4, 4, 640, 128)]) == INVALID
    assert c8([ring, (0x10000, 4, 2, 576, 128)]) == INVALID
    assert c8([(0x10000, 1, 4, 576, 128)]) == INVALID
    assert c8([(0x10000, 4, 4, 500, 128)]) == INVALID
    assert c8([ring], N=65) == UNSUPPORTED
    assert c8([ring, (0x20000, 4, 4, 576, 128), ring]) == INVALID
    assert L.kvq_tree_commit_fp8(None, 1, 2, 8, 0x1000, 0x2000, 0x3000, None, 0x5000, None) == INVALID


def test_pool_refuses():
    def call(fn, refs=0x1000, pages=10, table=0x2000, seqs=4, most=8, n=2, a=0x3000, b=0x4000, c=0x5000, src=0x6000, dst=0x7000, err=0x8000):
        if fn == "kvq_pages_fork":
            return L.kvq_pages_fork(refs, pages, table, seqs, most, n, a, b, c, src, dst, err, None)
        return getattr(L, fn)(refs, pages, table, seqs, most, n, a, b, c, err, None)

    for fn in ("kvq_pages_alloc", "kvq_pages_free", "kvq_pages_fork"):
        for over in (dict(refs=0), dict(pages=0), dict(table=0), dict(seqs=0), dict(most=0), dict(n=-1), dict(n=1025), dict(a=0), dict(b=0),
                     dict(c=0), dict(err=0)):
            assert call(fn, **over) == INVALID, (fn, over)
        assert call(fn, seqs=1 << 16, most=1 << 15) == UNSUPPORTED
        assert call(fn, most=(1 << 24) + 1, seqs=1) == UNSUPPORTED
        assert call(fn, n=0, a=0, b=0, c=0, src=0, dst=0) == 0
    assert call("kvq_pages_fork", src=0) == INVALID == call("kvq_pages_fork", dst=0)
    for i in (0, 2, 5, 6, 7, 8):
        a = [0x1000, 10, 0x2000, 4, 8, 0x3000, 0x4000, 0x5000, 0x6000, None]
        a[i] = 0
        assert L.kvq_pages_compact(*a) == INVALID


def test_copy_refuses():
    def call(cs, n=3, src=0x1000, dst=0x2000, err=0x3000, num=None):
        return L.kvq_pages_copy((kvq.Int4Cache * len(cs))(*cs), len(cs) if num is None else num, n, src, dst, None, err, None)

    assert call([cache()], n=-1) == INVALID == call([cache()], src=0) == call([cache()], dst=0) == call([cache()], err=0)
    assert call([cache()], num=0) == INVALID
    assert call([cache()] * 65) == UNSUPPORTED
    assert call([cache(), cache(num_kv_heads=1)]) == INVALID
    assert call([cache()], n=0, src=0, dst=0) == 0
    assert L.kvq_pages_copy(None, 1, 3, 0x1000, 0x2000, None, 0x3000, None) == INVALID


def test_status_of_the_binding_without_a_device():
    torch = pytest.importorskip("torch")
    q = torch.zeros(4, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # host tensors
        kvq.kvq_prompt_attn(q, q, q, torch.tensor([0, 4], dtype=torch.int32), q.clone(), q, q)
    with pytest.raises(ValueError):
        kvq.kvq_pages_alloc(torch.zeros(4, dtype=torch.int32), torch.zeros((1, 4), dtype=torch.int32), *[torch.zeros(1, dtype=torch.int32)] * 3, q)
