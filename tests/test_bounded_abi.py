"""Host-side refusals of the calls that hold a cache to a size: no GPU is needed, nothing is launched for a bad argument."""

import pytest

import quantized_kv_cache_fold_gb300 as kvq

L = kvq.lib
INVALID, UNSUPPORTED = 1, 2


def cache(**over):
    d = dict(pages=0x10000, block_table=0x50000, num_seqs=4, max_pages_per_seq=8, num_pages=32, num_kv_heads=4,
             page_size=64, head_dim=128)
    d.update(over)
    return kvq.Int4Cache(**d)


def prompt(**over):
    a = dict(q=0x1000000, k=0x2000000, v=0x3000000, dtype=kvq.BF16, T=100, B=2, Hq=20, Hkv=4, cu=0x9000, window=64, sinks=4,
             sm=0.09, out=0x4000000, ws=0xB0000, n=1 << 30, err=0xC0000)
    a.update(over)
    return L.kvq_prompt_attn_sinks(a["q"], a["k"], a["v"], a["dtype"], a["T"], a["B"], a["Hq"], a["Hkv"], None, a["cu"],
                                   a["window"], a["sinks"], a["sm"], a["out"], a["ws"], a["n"], a["err"], None)


@pytest.mark.parametrize("over,want", [
    (dict(sinks=-1), INVALID), (dict(q=0), INVALID), (dict(cu=0), INVALID), (dict(err=0), INVALID), (dict(T=-1), INVALID),
    (dict(Hq=21), INVALID), (dict(sm=0.0), INVALID), (dict(dtype=kvq.F32), UNSUPPORTED), (dict(out=0x1000000), INVALID),
    (dict(T=0, sinks=-1), INVALID), (dict(T=0), 0)])
def test_prompt_sinks_refuses(over, want):
    assert prompt(**over) == want


ATTN = dict(Mq=0x60000, Mk=0x70000, q=0x80000, dtype=1, B=2, Hq=20, ctx=0x90000, k=None, v=None, sm=0.09, eps=1e-6, out=0xA0000,
            od=1, ws=0xB0000, n=1 << 40, err=0xC0000)
BAD_ATTN = [(dict(B=0), INVALID), (dict(B=5), INVALID), (dict(Hq=21), UNSUPPORTED), (dict(Hq=0), UNSUPPORTED), (dict(Hq=196), UNSUPPORTED),
            (dict(dtype=2), INVALID), (dict(od=2), INVALID), (dict(q=0), INVALID), (dict(q=0x80004), INVALID), (dict(ctx=0), INVALID),
            (dict(out=0), INVALID), (dict(out=0xA0008), INVALID), (dict(ws=0), INVALID), (dict(ws=0xB0080), INVALID),
            (dict(n=100), INVALID), (dict(err=0), INVALID), (dict(k=0xD0000), INVALID), (dict(v=0xD0000), INVALID),
            (dict(k=0xD0008, v=0xE0000), INVALID), (dict(sm=float("nan")), INVALID), (dict(Mq=0), INVALID),
            (dict(Mq=0x60004), INVALID), (dict(k=0xD0000, v=0xE0000, Mk=0), INVALID), (dict(eps=-1.0), INVALID)]


def window(c=None, fn="kvq_window_attn_int4", **over):
    a = dict(ATTN, S=2, window=100, sinks=4, **{})
    a.update(over)
    return getattr(L, fn)(c or cache(), a["Mq"], a["Mk"], a["q"], a["dtype"], a["B"], a["S"], a["Hq"], a["ctx"], a["window"],
                          a["sinks"], a["k"], a["v"], a["sm"], a["eps"], a["out"], a["od"], a["ws"], a["n"], a["err"], None)


@pytest.mark.parametrize("over,want", BAD_ATTN + [
    (dict(window=0), INVALID), (dict(window=-3), INVALID), (dict(sinks=-1), INVALID), (dict(S=0), UNSUPPORTED),
    (dict(S=9), UNSUPPORTED), (dict(S=8, Hq=28), UNSUPPORTED)])
@pytest.mark.parametrize("fn", ["kvq_window_attn_int4", "kvq_window_attn_int4_fwht"])
def test_window_refuses(over, want, fn):
    assert window(fn=fn, **over) == want


def mass_of(**over):
    d = dict(mass=0x1000000, ids=0x2000000, num_seqs=4, num_kv_heads=4, max_tokens=512)
    d.update(over)
    return kvq.TokenMass(**d)


def mass(c=None, m=None, fn="kvq_mass_attn_int4", **over):
    a = dict(ATTN, pos=0x98000)
    a.update(over)
    return getattr(L, fn)(c or cache(), m or mass_of(), a["Mq"], a["Mk"], a["q"], a["dtype"], a["B"], a["Hq"], a["ctx"], a["pos"],
                          a["k"], a["v"], a["sm"], a["eps"], a["out"], a["od"], a["ws"], a["n"], a["err"], None)


@pytest.mark.parametrize("over,want", BAD_ATTN + [(dict(pos=0), INVALID)])
@pytest.mark.parametrize("fn", ["kvq_mass_attn_int4", "kvq_mass_attn_int4_fwht"])
def test_mass_refuses(over, want, fn):
    assert mass(fn=fn, **over) == want


@pytest.mark.parametrize("over", [
    dict(mass=0), dict(ids=0), dict(mass=0x1000008), dict(num_seqs=1), dict(num_kv_heads=2), dict(max_tokens=511),
    dict(max_tokens=508), dict(max_tokens=514), dict(ids=0x1000000 + 4096), dict(mass=0xA0000 - 4096), dict(ids=0x90000 - 64),
    dict(ids=0x98000)])
def test_mass_refuses_descriptors(over):
    assert mass(m=mass_of(**over)) == INVALID


def test_wide_tables_and_workspaces():
    wide = cache(max_pages_per_seq=1 << 24, num_seqs=1024)
    assert window(wide, B=1024) == UNSUPPORTED and mass(wide, mass_of(num_seqs=1024, max_tokens=1 << 30), B=1024) == UNSUPPORTED
    assert window(cache(head_dim=64)) == UNSUPPORTED and mass(cache(page_size=32)) == UNSUPPORTED
    size = kvq.kvq_mass_workspace_bytes
    assert size(2, 20, 4, 8) >= kvq.kvq_decode_workspace_bytes(2, 1, 20, 4) + 4 * 2 * 20 * 512
    assert size(1, 48, 1, 1 << 24) > 2 ** 37
    for bad in ((0, 20, 4, 8), (2, 21, 4, 8), (2, 20, 4, 0), (2, 196, 4, 8), (1, 20, 4, (1 << 24) + 1), (1024, 20, 4, 1 << 20)):
        assert size(*bad) == 0


def evict(n=2, caches=None, masses=None, **over):
    a = dict(B=2, ctx=0x90000, seen=0x98000, budget=100, sinks=4, recent=10, out=0xA0000, err=0xC0000)
    a.update(over)
    cs = caches or [cache(pages=0x10000 + 0x1000000 * i) for i in range(n)]
    ms = masses or [mass_of(mass=0x10000000 + 0x200000 * i, ids=0x10100000 + 0x200000 * i) for i in range(n)]
    return L.kvq_evict_int4(b"".join(cs), b"".join(ms), n, a["B"], a["ctx"], a["seen"], a["budget"], a["sinks"], a["recent"],
                            a["out"], a["err"], None)


@pytest.mark.parametrize("over,want", [
    (dict(B=0), INVALID), (dict(B=5), INVALID), (dict(ctx=0), INVALID), (dict(seen=0), INVALID), (dict(err=0), INVALID),
    (dict(budget=0), INVALID), (dict(sinks=-1), INVALID), (dict(recent=-1), INVALID), (dict(out=0x90000), INVALID),
    (dict(out=0x98004), INVALID), (dict(n=0), INVALID), (dict(n=65), UNSUPPORTED), (dict(ctx=0x10000000 + 64), INVALID),
    (dict(out=0x10100000), INVALID)])
def test_evict_refuses(over, want):
    assert evict(**over) == want


def test_evict_refuses_layers():
    two = [cache(), cache(pages=0x2000000)]
    assert evict(caches=[cache(), cache()]) == INVALID                       # a layer twice
    assert evict(caches=[cache(), cache(pages=0x2000000, num_kv_heads=2)]) == INVALID
    assert evict(caches=[cache(), cache(pages=0x2000000, num_seqs=1)]) == INVALID
    assert evict(caches=[cache(), cache(pages=0x2000000, head_dim=64)]) == UNSUPPORTED
    wide = [cache(), cache(pages=0x2000000, max_pages_per_seq=6145)]
    ok = mass_of()
    assert evict(caches=wide, masses=[ok, mass_of(mass=0x40000000, ids=0x50000000, max_tokens=6145 * 64)]) == UNSUPPORTED
    for bad in (dict(mass=0), dict(ids=0), dict(mass=0x1000000 + 4096), dict(ids=0x1000000), dict(ids=0x2000000), dict(mass=0x8),
                dict(ids=0x40000004), dict(num_seqs=1), dict(num_kv_heads=3), dict(max_tokens=508)):
        over = dict(mass=0x30000000, ids=0x40000000)
        over.update(bad)
        assert evict(caches=two, masses=[ok, mass_of(**over)]) == INVALID, bad


def observe(strides=None, m=None, **over):
    import ctypes
    a = dict(q=0x100000000, k=0x200000000, dtype=kvq.BF16, T=100, B=2, Hq=20, Hkv=4, cu=0x9000, rows=16, seq=0, sm=0.09, ws=0xB0000,
             n=1 << 30, err=0xC0000)
    a.update(over)
    st = (ctypes.c_int64 * 4)(*strides) if strides else None
    return L.kvq_prompt_mass(a["q"], a["k"], a["dtype"], a["T"], a["B"], a["Hq"], a["Hkv"], st, a["cu"], a["rows"], a["seq"], a["sm"],
                             m or mass_of(mass=0x300000000, ids=0x400000000), a["ws"], a["n"], a["err"], None)


@pytest.mark.parametrize("over,want", [
    (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(cu=0), INVALID), (dict(ws=0), INVALID), (dict(err=0), INVALID), (dict(dtype=7), INVALID),
    (dict(dtype=kvq.F32), UNSUPPORTED), (dict(T=-1), INVALID), (dict(B=0), INVALID), (dict(B=5), INVALID), (dict(B=1025, seq=0x8000), INVALID),
    (dict(Hq=21), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=260), UNSUPPORTED), (dict(T=1 << 27), INVALID), (dict(sm=0.0), INVALID),
    (dict(sm=float("nan")), INVALID), (dict(q=0x100000008), INVALID), (dict(ws=0xB0010), INVALID), (dict(n=8), INVALID),
    (dict(Hkv=2), INVALID), (dict(q=0x300000000 + 64), INVALID), (dict(k=0x400000000), INVALID), (dict(seq=0x300000010), INVALID),
    (dict(T=0), 0)])
def test_observe_refuses(over, want):
    assert observe(**over) == want


def test_observe_refuses_strides_and_descriptors():
    packed = [2560, 128, 512, 128]
    for i in range(4):
        for bad in (0, -8, 4, 129, 1 << 40):
            assert observe(packed[:i] + [bad] + packed[i + 1:]) == INVALID
    for bad in (dict(mass=0), dict(ids=0), dict(max_tokens=510), dict(mass=0x300000004), dict(ids=0x300000000)):
        over = dict(mass=0x300000000, ids=0x400000000)
        over.update(bad)
        assert observe(m=mass_of(**over)) == INVALID
    size = kvq.kvq_prompt_mass_workspace_bytes
    assert size(100, 2, 20, 4, 16) > 0 and size(100, 2, 20, 4, 0) > 0
    assert size(-1, 2, 20, 4, 16) == size(100, 0, 20, 4, 16) == size(100, 2, 20, 3, 16) == size(100, 2, 130, 2, 16) == 0
