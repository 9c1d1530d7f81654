"""What serving a session asks of the cache besides decoding one block: the prompt's attention, the
attention of a tree of drafted tokens, the commit of the accepted branch, and the page pool.

kinds of case
  prompt    causal attention over whole prompts packed end to end, grouped heads, with or without
            the window of the sliding-window layers
  tree      attention of the drafted tokens of a tree over the paged 4-bit cache (their keys and
            values already appended behind the context)
  treeswa   the same over the e4m3 ring of a sliding-window layer
  commit    the accepted branch of each tree moved to the positions right behind the context, in
            every layer's cache
  fork      old branches freed, new ones forked from their parents (full pages shared, the last
            one copied in every layer)
  compact   the live pages of a fragmented pool moved to its front in every layer
"""

import math
import random

import torch

own = False

D = 128          # head dim
PAGE = 64        # tokens of a page, slots of a ring block
BLOCK4 = 8704    # bytes of one (page, KV head): K codes 4096, V codes 4096, K meta 256, V meta 256
BLOCK8 = 16384   # bytes of 64 ring slots of one head: K 8192, V 8192
EPS = 1e-6
SM = D ** -0.5


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # four short chat turns arriving together: the smallest prefill, all latency
        {"name": "prompt-turns", "kind": "prompt", "B": 4, "lo": 1, "hi": 96, "spread": 1, "Hq": 20, "Hkv": 4,
         "dtype": "bf16", "window": 0, "fused": False},
        # an ordinary prefill batch: ragged prompts, q/k/v views of one projection's output
        {"name": "prompt-packed", "kind": "prompt", "B": 24, "lo": 100, "hi": 4000, "spread": 2, "Hq": 20, "Hkv": 4,
         "dtype": "bf16", "window": 0, "fused": True},
        # one long document in a full-attention layer
        {"name": "prompt-long", "kind": "prompt", "B": 1, "lo": 32768, "hi": 32768, "spread": 3, "Hq": 20, "Hkv": 4,
         "dtype": "bf16", "window": 0, "fused": False},
        # the sliding-window layers' prefill (window 513), half precision, odd lengths
        {"name": "prompt-window", "kind": "prompt", "B": 5, "lo": 1500, "hi": 9000, "spread": 4, "Hq": 20, "Hkv": 4,
         "dtype": "f16", "window": 513, "fused": False},
        # one session with a small draft tree: decode latency
        {"name": "tree-one", "kind": "tree", "B": 1, "lo": 4096, "hi": 4096, "spread": 5, "N": 8, "Hq": 20, "Hkv": 4},
        # the verify batch: 64 sessions of 16,384 tokens, 16 drafted tokens each
        {"name": "tree-batch", "kind": "tree", "B": 64, "lo": 16384, "hi": 16384, "spread": 6, "N": 16, "Hq": 20,
         "Hkv": 4},
        # few long ragged sessions with the widest trees
        {"name": "tree-wide", "kind": "tree", "B": 8, "lo": 32768, "hi": 65536, "spread": 7, "N": 64, "Hq": 20,
         "Hkv": 4},
        # a sliding-window layer of the verify batch
        {"name": "tree-window", "kind": "treeswa", "B": 64, "lo": 100, "hi": 16384, "spread": 8, "N": 16, "Hq": 20,
         "Hkv": 4, "window": 513},
        # one session's accepted branch over the ten full-attention layers
        {"name": "commit-one", "kind": "commit", "B": 1, "lo": 4096, "hi": 4096, "spread": 9, "N": 8, "Hkv": 4,
         "layers4": 10, "layers8": 0},
        # a batch's accepted branches over a whole stack of 50 layers
        {"name": "commit-stack", "kind": "commit", "B": 64, "lo": 300, "hi": 700, "spread": 10, "N": 32, "Hkv": 4,
         "layers4": 10, "layers8": 40},
        # best-of-n: losing branches dropped, winners forked, over ten layers
        {"name": "fork-beams", "kind": "fork", "parents": 4, "children": 28, "lo": 400, "hi": 3000, "spread": 11,
         "Hkv": 4, "layers": 10, "spare": 100},
        # a pool in which most sessions ended, compacted
        {"name": "compact-pool", "kind": "compact", "B": 96, "lo": 200, "hi": 4000, "spread": 12, "Hkv": 4,
         "layers": 4, "keep": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    return rng.choice([(20, 4), (20, 4), (8, 1), (16, 4), (6, 2), (4, 4)])


def draw(rng):
    kind = rng.choice(["prompt", "prompt", "prompt", "tree", "tree", "treeswa", "commit", "fork", "compact"])
    c = {"kind": kind, "spread": rng.randrange(1 << 20)}
    if kind == "prompt":
        c["Hq"], c["Hkv"] = _heads(rng)
        c["B"] = _log(rng, 1, 40)
        c["hi"] = _log(rng, 1, max(64, min(20000, 60000 // c["B"])))
        c["lo"] = max(1, _log(rng, 1, c["hi"]))
        c["dtype"] = rng.choice(["bf16", "bf16", "f16"])
        c["window"] = rng.choice([0, 0, 513, _log(rng, 1, 2000)])
        c["fused"] = rng.random() < 0.4
    elif kind == "tree":
        c["Hq"], c["Hkv"] = _heads(rng)
        c["B"] = _log(rng, 1, 80)
        c["hi"] = _log(rng, 1, max(256, min(100000, 600000 // c["B"])))
        c["lo"] = _log(rng, 1, c["hi"])
        c["N"] = _log(rng, 1, 64)
    elif kind == "treeswa":
        c["Hq"], c["Hkv"] = _heads(rng)
        c["B"] = _log(rng, 1, 128)
        c["hi"] = _log(rng, 1, 100000)
        c["lo"] = _log(rng, 1, c["hi"])
        c["N"] = _log(rng, 1, 64)
        c["window"] = rng.choice([513, _log(rng, c["N"], 2000)])
    elif kind == "commit":
        c["Hkv"] = rng.choice([4, 4, 1, 2, 8])
        c["B"] = _log(rng, 1, 100)
        c["hi"] = _log(rng, 1, 2000)
        c["lo"] = _log(rng, 1, c["hi"])
        c["N"] = _log(rng, 1, 64)
        c["layers4"] = rng.randrange(1, 11)
        c["layers8"] = rng.choice([0, rng.randrange(1, 31)])
    elif kind == "fork":
        c["Hkv"] = rng.choice([4, 4, 1, 2, 8])
        c["parents"] = _log(rng, 1, 16)
        c["children"] = _log(rng, 1, 120)
        c["hi"] = _log(rng, 1, 4000)
        c["lo"] = _log(rng, 1, c["hi"])
        c["layers"] = rng.randrange(1, 11)
        c["spare"] = rng.randrange(0, 200)
    else:
        c["Hkv"] = rng.choice([4, 4, 1, 2])
        c["B"] = _log(rng, 2, 96)
        c["hi"] = _log(rng, 64, 4000)
        c["lo"] = _log(rng, 1, c["hi"])
        c["layers"] = rng.randrange(1, 5)
        c["keep"] = round(rng.uniform(0.1, 0.9), 3)
    return c


def _lengths(c, count):
    """The case's token counts: spread over [lo, hi] by their logarithm, the longest of them hi."""
    r = random.Random(c["spread"])
    n = [min(c["hi"], max(c["lo"], _log(r, c["lo"], c["hi"]))) for _ in range(count)]
    n[r.randrange(count)] = c["hi"]
    return n


def _pages_of(n):
    return (n + PAGE - 1) // PAGE


def _accepted(c):
    """Accepted tokens of each sequence's tree: none up to all of a branch."""
    r = random.Random(c["spread"] + 1)
    return [r.randint(0 if c["B"] > 1 else 1, min(c["N"], 16)) for _ in range(c["B"])]


# ------------------------------------------------------------------------------------- inputs

def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _tree(rng, N):
    """A draft tree: each token's parent comes before it; returns the parents (-1: a root)."""
    return [-1 if i == 0 else rng.randrange(max(-1, i - 9), i) for i in range(N)]


def _tree_masks(rng, B, N):
    """int64 [B][N]: bit j of word i says that token i sees token j (itself and its ancestors)."""
    words = []
    for _ in range(B):
        m = []
        for i, p in enumerate(_tree(rng, N)):
            m.append((1 << i) | (m[p] if p >= 0 else 0))
        words.append([w - (1 << 64) if w >> 63 else w for w in m])
    return _ints(words, torch.int64)


def _table(g, B, max_pages):
    perm = torch.randperm(B * max_pages, generator=g, device="cuda")
    return perm.to(torch.int32).reshape(B, max_pages).contiguous()


def _slot_chunks(swizzle, chunks):
    """int64 [64][chunks]: the physical 16-byte chunk of each logical chunk of a slot's record."""
    t = torch.arange(PAGE, device="cuda")[:, None]
    return torch.arange(chunks, device="cuda")[None, :] ^ swizzle(t)


def _k_chunks():
    return _slot_chunks(lambda t: ((t >> 1) & 1) | ((t >> 2) & 2), 4)


def _v_chunks():
    return _slot_chunks(lambda t: (t >> 1) & 3, 4)


def _ring_chunks():
    return _slot_chunks(lambda t: t & 7, 8)


def _quantised(x):
    """Codes (uint8) and the fp16 scale and offset of rows of 128: offset rounded down, scale up."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    o = (lo - lo.abs() * 0.001).half()
    s = ((hi - o.float()) / 15 * 1.001).half()
    code = ((x - o.float()) / s.float()).round().clamp_(0, 15).to(torch.uint8)
    return code, s[..., 0].contiguous(), o[..., 0].contiguous()


def _fill4(pages, g, some=2048):
    """Blocks of [*][8704] filled with rows like those of rotated keys and of values."""
    flat = pages.view(-1, BLOCK4)
    kc, vc = _k_chunks(), _v_chunks()
    bank = []
    for values in (False, True):
        code, s, o = _quantised(_normal(g, some, PAGE, D))
        c = code.to(torch.int32)
        if values:
            q = c.view(some, PAGE, 32, 4)
            neg = (q < 8).to(torch.int32)
            e = torch.where(q < 8, 7 - q, q - 8)
            w = ((e[..., 0] << 1) | (neg[..., 0] << 15) | (e[..., 1] << 4) | (neg[..., 1] << 14)
                 | (e[..., 2] << 11) | (neg[..., 2] << 7) | (e[..., 3] << 8) | neg[..., 3])
            b = torch.stack([w & 255, w >> 8], -1).to(torch.uint8).view(some, PAGE, 4, 16)
        else:
            b = (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8).view(some, PAGE, 4, 16)
        ch = (vc if values else kc)[None, :, :, None].expand(some, PAGE, 4, 16)
        rec = torch.empty_like(b).scatter_(2, ch, b).view(some, PAGE * 64)
        meta = torch.stack([s.view(torch.int16), o.view(torch.int16)], -1).contiguous().view(torch.uint8).view(some, 256)
        bank.append((rec, meta))
    # block i takes its keys and its values from two records of the bank of its own
    for at in range(0, flat.shape[0], 1 << 17):
        part = flat[at:at + (1 << 17)]
        pick = torch.randint(some, (2, part.shape[0]), generator=g, device="cuda")
        part[:, 0:4096] = bank[0][0][pick[0]]
        part[:, 4096:8192] = bank[1][0][pick[1]]
        part[:, 8192:8448] = bank[0][1][pick[0]]
        part[:, 8448:8704] = bank[1][1][pick[1]]


def _fill8(data, g, some=1024):
    """Ring blocks of [*][16384] filled with e4m3 rows (scale 6/448)."""
    flat = data.view(-1, BLOCK8)
    x = (_normal(g, some, 2, PAGE, 8, 16) * (448 / 6)).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    bank = torch.empty_like(x).scatter_(3, _ring_chunks()[None, None, :, :, None].expand_as(x), x).view(some, BLOCK8)
    for at in range(0, flat.shape[0], 1 << 15):
        part = flat[at:at + (1 << 15)]
        part[:] = bank[torch.randint(some, (part.shape[0],), generator=g, device="cuda")]


def _folded(g, seed):
    """M_q = R diag(g_q g_k) of a layer: a signed Hadamard rotation and the QK-norm gains."""
    h = torch.ones(1, 1, device="cuda", dtype=torch.float64)
    while h.shape[0] < D:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    r = random.Random(seed)
    s = _ints([r.choice([-1, 1]) for _ in range(D)], torch.float64)
    gain = (torch.rand(D, generator=g, device="cuda", dtype=torch.float64) * 2 + 1)
    return (h * s[None, :] * gain[None, :] / math.sqrt(D)).float().contiguous()


def _packed_offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _ring_capacity(c):
    return _pages_of(c["window"] + c["N"] - 1) * PAGE


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = random.Random(seed)
    kind = c["kind"]
    st = {"c": c, "err": torch.zeros(1, dtype=torch.int32, device="cuda"), "kept": {}}
    if kind == "prompt":
        lens = _lengths(c, c["B"])
        at = _packed_offsets(lens)
        T, Hq, Hkv = at[-1], c["Hq"], c["Hkv"]
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float16
        gain = torch.rand(D, generator=g, device="cuda") + 0.75
        normed = lambda x: x / (x.square().mean(-1, keepdim=True) + EPS).sqrt()  # noqa: E731
        q = (normed(_normal(g, T, Hq, D)) * gain).to(dt)
        k = (normed(_normal(g, T, Hkv, D)) * gain).to(dt)
        v = _normal(g, T, Hkv, D).to(dt)
        if c["fused"]:
            qkv = torch.cat([q, k, v], 1).contiguous()
            q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        st.update(q=q, k=k, v=v, at=at, lens=lens, offsets=_ints(at), out=torch.empty(T, Hq, D, dtype=dt, device="cuda"))
    elif kind == "tree":
        ctx = _lengths(c, c["B"])
        P = _pages_of(max(ctx) + c["N"])
        table = _table(g, c["B"], P)
        pages = torch.empty(c["B"] * P, c["Hkv"], BLOCK4, dtype=torch.uint8, device="cuda")
        _fill4(pages, g)
        st.update(pages=pages, table=table, ctx=_ints(ctx), M=_folded(g, seed),
                  mask=_tree_masks(rng, c["B"], c["N"]),
                  q=_normal(g, c["B"], c["N"], c["Hq"], D).to(torch.bfloat16),
                  out=torch.empty(c["B"], c["N"], c["Hq"], D, dtype=torch.bfloat16, device="cuda"))
    elif kind == "treeswa":
        ring = torch.empty(c["B"], c["Hkv"], _ring_capacity(c) // PAGE, BLOCK8, dtype=torch.uint8, device="cuda")
        _fill8(ring, g)
        st.update(ring=ring, ctx=_ints(_lengths(c, c["B"])), mask=_tree_masks(rng, c["B"], c["N"]),
                  q=(_normal(g, c["B"], c["N"], c["Hq"], D) * 1.5).to(torch.bfloat16),
                  out=torch.empty(c["B"], c["N"], c["Hq"], D, dtype=torch.bfloat16, device="cuda"))
    elif kind == "commit":
        B, N, Hkv = c["B"], c["N"], c["Hkv"]
        ctx, acc = _lengths(c, B), _accepted(c)
        P = _pages_of(max(ctx) + N)
        pages = torch.empty(c["layers4"], B * P, Hkv, BLOCK4, dtype=torch.uint8, device="cuda")
        _fill4(pages, g, 256)
        rings = torch.empty(c["layers8"], B, Hkv, _pages_of(513 + N - 1), BLOCK8, dtype=torch.uint8, device="cuda")
        _fill8(rings, g, 256)
        path = [sorted(rng.sample(range(N), a)) + [0] * (N - a) for a in acc]
        st.update(pages=pages, rings=rings, table=_table(g, B, P), ctx=_ints(ctx), path=_ints(path), n=_ints(acc),
                  ctx_out=torch.zeros(B, dtype=torch.int32, device="cuda"))
    elif kind == "fork":
        np_, nc = c["parents"], c["children"]
        lens = _lengths(c, np_)
        P = _pages_of(max(lens)) + 1
        who = [rng.randrange(np_) for _ in range(nc)]
        before = [rng.randrange(np_) for _ in range(nc)]
        full = sum(_pages_of(n) for n in lens)
        num = full + 2 * nc + c["spare"]
        order = list(range(num))
        rng.shuffle(order)
        table = [[-1] * P for _ in range(np_ + nc)]
        refs = [0] * num
        for b, n in enumerate(lens):
            for p in range(_pages_of(n)):
                table[b][p] = order.pop()
                refs[table[b][p]] = 1
        for i, b in enumerate(before):  # the branches of the step before, dropped by this pass
            for p in range(_pages_of(lens[b])):
                own_page = p == lens[b] // PAGE
                table[np_ + i][p] = order.pop() if own_page else table[b][p]
                refs[table[np_ + i][p]] += 1
        pages = torch.empty(c["layers"], num, c["Hkv"], BLOCK4, dtype=torch.uint8, device="cuda")
        _fill4(pages, g, 256)
        st.update(pages=pages, table=_ints(table), refs=_ints(refs), parent=_ints(who),
                  child=_ints([np_ + i for i in range(nc)]), was=_ints([lens[b] for b in before]),
                  next=_ints([lens[b] for b in who]), zero=_ints([0] * nc),
                  src=_ints([-1] * nc), dst=_ints([-1] * nc),
                  tails=_ints([i for i, b in enumerate(who) if lens[b] % PAGE], torch.int64))
        # after the first pass the branches dropped are those that it forked
        st["lens_now"] = [st["was"], st["next"]]
    else:
        B = c["B"]
        lens = _lengths(c, B)
        P = _pages_of(max(lens))
        num = sum(_pages_of(n) for n in lens)
        order = list(range(num))
        rng.shuffle(order)
        alive = set(random.Random(c["spread"] + 2).sample(range(B), max(1, int(round(c["keep"] * B)))))
        table, refs = [[-1] * P for _ in range(B)], [0] * num
        for b, n in enumerate(lens):
            for p in range(_pages_of(n)):
                page = order.pop()
                if b in alive:
                    table[b][p] = page
                    refs[page] = 1
        pages = torch.empty(c["layers"], num, c["Hkv"], BLOCK4, dtype=torch.uint8, device="cuda")
        _fill4(pages, g, 256)
        st.update(pages=pages, table0=_ints(table), refs0=_ints(refs), table=_ints(table), refs=_ints(refs),
                  src=torch.full((num,), -1, dtype=torch.int32, device="cuda"),
                  dst=torch.full((num,), -1, dtype=torch.int32, device="cuda"),
                  moves=torch.zeros(1, dtype=torch.int32, device="cuda"))
    return st


# ------------------------------------------------------------------------------------- one pass

def _framework(st, name, make):
    """A descriptor or workspace that a user's program makes once and keeps."""
    if name not in st["kept"]:
        st["kept"][name] = make()
    return st["kept"][name]


def _run_own(st):
    import quantized_kv_cache_fold_gb300 as kv
    c, kind = st["c"], st["c"]["kind"]
    if kind == "prompt":
        ws = _framework(st, "ws", lambda: kv.alloc_prompt_workspace(st["at"][-1], c["B"], c["Hq"], c["Hkv"]))
        kv.kvq_prompt_attn(st["q"], st["k"], st["v"], st["offsets"], st["out"], ws, st["err"], window=c["window"],
                           sm_scale=SM)
        return st["out"]
    if kind == "tree":
        cache = _framework(st, "cache", lambda: kv.int4_cache(st["pages"], st["table"]))
        ws = _framework(st, "ws", lambda: kv.alloc_tree_workspace(c["B"], c["N"], c["Hq"], c["Hkv"]))
        kv.kvq_tree_attn_int4(cache, st["M"], None, st["q"], st["ctx"], st["mask"], st["out"], ws, st["err"],
                              sm_scale=SM, eps=EPS)
        return st["out"]
    if kind == "treeswa":
        ring = _framework(st, "ring", lambda: kv.fp8_ring(st["ring"]))
        ws = _framework(st, "ws", lambda: kv.alloc_tree_workspace(c["B"], c["N"], c["Hq"], c["Hkv"]))
        kv.kvq_tree_attn_fp8_swa(ring, st["q"], st["ctx"], st["mask"], c["window"], 6 / 448, 6 / 448, st["out"], ws,
                                 st["err"], sm_scale=SM)
        return st["out"]
    if kind == "commit":
        caches = _framework(st, "caches", lambda: [kv.int4_cache(p, st["table"]) for p in st["pages"]])
        rings = _framework(st, "rings", lambda: [kv.fp8_ring(r) for r in st["rings"]])
        if caches:
            kv.kvq_tree_commit_int4(caches, st["ctx"], st["path"], st["n"], st["err"], ctx_out=st["ctx_out"])
        if rings:
            kv.kvq_tree_commit_fp8(rings, st["ctx"], st["path"], st["n"], st["err"])
        return {"pages": st["pages"], "rings": st["rings"], "ctx": st["ctx_out"]}
    caches = _framework(st, "caches", lambda: [kv.int4_cache(p, st["table"]) for p in st["pages"]])
    if kind == "fork":
        was, st["lens_now"] = st["lens_now"][0], [st["next"], st["next"]]
        kv.kvq_pages_free(st["refs"], st["table"], st["child"], was, st["zero"], st["err"])
        kv.kvq_pages_fork(st["refs"], st["table"], st["parent"], st["child"], st["next"], st["src"], st["dst"],
                          st["err"])
        kv.kvq_pages_copy(caches, st["src"], st["dst"], st["err"])
    else:
        st["refs"].copy_(st["refs0"])  # the fragmented pool again (the copies moved leave their sources as they were)
        st["table"].copy_(st["table0"])
        kv.kvq_pages_compact(st["refs"], st["table"], st["src"], st["dst"], st["moves"], st["err"])
        kv.kvq_pages_copy(caches, st["src"], st["dst"], st["err"], count=st["moves"])
        return {"pages": st["pages"], "table": st["table"], "refs": st["refs"], "moves": st["moves"]}
    return {"pages": st["pages"], "table": st["table"], "refs": st["refs"], "src": st["src"], "dst": st["dst"]}


def _plain_prompt(st):
    """softmax(q k' / sqrt(128)) v of each prompt, a part of its query rows at a time."""
    c = st["c"]
    Hq, Hkv, W = c["Hq"], c["Hkv"], c["window"]
    out = st["out"]
    for lo, hi in zip(st["at"], st["at"][1:]):
        q = st["q"][lo:hi].float().view(hi - lo, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3)  # [Hkv, G, n, D]
        k, v = st["k"][lo:hi].float().transpose(0, 1), st["v"][lo:hi].float().transpose(0, 1)
        for r0 in range(0, hi - lo, 2048):
            r1 = min(hi - lo, r0 + 2048)
            j0 = max(0, r0 - W + 1) if W else 0
            s = torch.matmul(q[:, :, r0:r1], k[:, None, j0:r1].transpose(-1, -2)) * SM
            i = torch.arange(r0, r1, device="cuda")[:, None]
            j = torch.arange(j0, r1, device="cuda")[None, :]
            seen = (j <= i) & (j > i - W) if W else j <= i
            s = torch.where(seen, s, -math.inf)
            p = torch.exp(s - s.amax(-1, keepdim=True))
            o = torch.matmul(p, v[:, None, j0:r1]) / p.sum(-1, keepdim=True)
            out[lo + r0:lo + r1] = o.permute(2, 0, 1, 3).reshape(r1 - r0, Hq, D).to(out.dtype)
    return out


def _decoded4(blocks):
    """Blocks [..., 8704] -> keys and values [..., 64, 128] as fp32."""
    lead = blocks.shape[:-1]
    both = []
    for first, chunks in ((0, _k_chunks()), (4096, _v_chunks())):
        b = blocks[..., first:first + 4096].reshape(*lead, PAGE, 4, 16)
        b = torch.gather(b, -2, chunks[:, :, None].expand(*lead, PAGE, 4, 16)).reshape(*lead, PAGE, 64)
        meta = blocks[..., 8192 + first // 16:8448 + first // 16].contiguous().view(torch.float16).view(*lead, PAGE, 2).float()
        if first == 0:
            code = torch.stack([b & 15, b >> 4], -1).reshape(*lead, PAGE, D).float()
        else:
            lo, hi = b[..., 0::2], b[..., 1::2]  # low and high byte of the 16-bit elements
            e = torch.stack([(lo >> 1) & 7, (lo >> 4) & 7, (hi >> 3) & 7, hi & 7], -1)
            neg = torch.stack([hi >> 7, (hi >> 6) & 1, (lo >> 7) & 1, lo & 1], -1) > 0
            code = torch.where(neg, 7 - e, e + 8).reshape(*lead, PAGE, D).float()
        both.append(code * meta[..., :1] + meta[..., 1:])
    return both


def _bits(mask, N):
    return ((mask[:, :, None] >> torch.arange(N, device="cuda")) & 1) > 0  # [B, N, N]


def _attend(q, k, v, seen, B, N, Hq, Hkv):
    """q [B, N, Hq, D], k and v [B, Hkv, L, D], seen [B, N, L]; rows that see nothing give 0."""
    q = q.view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    s = torch.matmul(q, k.transpose(-1, -2)).view(B, Hkv, Hq // Hkv, N, -1) * SM
    s = torch.where(seen[:, None, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, -1, p.shape[-1]), v).view(B, Hkv, Hq // Hkv, N, D) / torch.where(l == 0, 1.0, l)
    return o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)


def _plain_tree(st):
    c = st["c"]
    B, N, Hq, Hkv = c["B"], c["N"], c["Hq"], c["Hkv"]
    x = st["q"].float()
    q = torch.matmul(x / (x.square().mean(-1, keepdim=True) + EPS).sqrt(), st["M"].t())
    L = st["table"].shape[1] * PAGE
    k, v = _decoded4(st["pages"][st["table"].long()].transpose(1, 2))
    j = torch.arange(L, device="cuda")[None, :] - st["ctx"][:, None]  # position behind the context
    drafted = torch.gather(_bits(st["mask"], N), 2, j.clamp(0, N - 1)[:, None].expand(B, N, L))
    seen = (j < 0)[:, None] | (drafted & (j >= 0)[:, None] & (j < N)[:, None])
    o = _attend(q, k.reshape(B, Hkv, L, D), v.reshape(B, Hkv, L, D), seen, B, N, Hq, Hkv)
    st["out"].copy_(o.to(torch.bfloat16))
    return st["out"]


def _plain_treeswa(st):
    c = st["c"]
    B, N, Hq, Hkv, W = c["B"], c["N"], c["Hq"], c["Hkv"], c["window"]
    L = W + N - 1  # positions ctx - W + 1 .. ctx + N - 1
    j = torch.arange(L, device="cuda")[None, :] - W + 1 + torch.zeros_like(st["ctx"])[:, None]
    pos = st["ctx"][:, None] + j
    slot = pos.remainder(_ring_capacity(c))
    ring = st["ring"].view(B, Hkv, -1, 2, PAGE, 8, 16)
    b = torch.arange(B, device="cuda")[:, None]
    rec = ring[b, :, slot // PAGE, :, slot % PAGE]  # [B, L, Hkv, 2, 8, 16]
    ch = _ring_chunks()[slot % PAGE][:, :, None, None, :, None].expand_as(rec)
    x = torch.gather(rec, 4, ch).reshape(B, L, Hkv, 2, D).view(torch.float8_e4m3fn).float() * torch.tensor(6 / 448, dtype=torch.float32, device="cuda")
    bits = _bits(st["mask"], N)
    at = st["ctx"][:, None] + bits.sum(-1).clamp(min=1) - 1  # the drafted tokens' own positions
    drafted = torch.gather(bits, 2, j.clamp(0, N - 1)[:, None].expand(B, N, L))
    past = (pos >= 0)[:, None] & (j < 0)[:, None] & (pos[:, None] > at[:, :, None] - W)
    seen = past | (drafted & (j >= 0)[:, None])
    o = _attend(st["q"].float(), x[:, :, :, 0].transpose(1, 2), x[:, :, :, 1].transpose(1, 2), seen, B, N, Hq, Hkv)
    st["out"].copy_(o.to(torch.bfloat16))
    return st["out"]


def _plain_commit(st):
    c = st["c"]
    B, N, Hkv = c["B"], c["N"], c["Hkv"]
    i = torch.arange(N, device="cuda")[None, :]
    live = i < st["n"][:, None]
    source = torch.where(live, st["path"], i) + st["ctx"][:, None]  # positions; what is not accepted stays
    target = (i + st["ctx"][:, None])
    b = torch.arange(B, device="cuda")[:, None]
    pages = st["pages"]
    ps, pt = (st["table"][b, x // PAGE].long() for x in (source, target))
    s, t = source % PAGE, target % PAGE
    for first, chunks in ((0, _k_chunks()), (4096, _v_chunks())):
        rec = pages[..., first:first + 4096].view(*pages.shape[:3], PAGE, 4, 16)  # [layers, pages, Hkv, 64, 4, 16]
        moved = rec[:, ps[..., None], :, s[..., None], chunks[s]]                 # [B, N, 4, layers, Hkv, 16]
        rec[:, pt[..., None], :, t[..., None], chunks[t]] = moved
        meta = pages[..., 8192 + first // 16:8448 + first // 16].view(*pages.shape[:3], PAGE, 4)
        meta[:, pt, :, t] = meta[:, ps, :, s]
    if c["layers8"]:
        rings = st["rings"]
        cap = rings.shape[3] * PAGE
        rec = rings.view(c["layers8"], B, Hkv, cap // PAGE, 2, PAGE, 8, 16)
        s, t, chunks = source % cap, target % cap, _ring_chunks()
        at = lambda x: (b[..., None], (x // PAGE)[..., None], (x % PAGE)[..., None], chunks[x % PAGE])  # noqa: E731
        (bb, blk, sl, ch), (_, blk2, sl2, ch2) = at(s), at(t)
        moved = rec[:, bb, :, blk, :, sl, ch]
        rec[:, bb, :, blk2, :, sl2, ch2] = moved
    st["ctx_out"].copy_(st["ctx"] + st["n"])
    return {"pages": st["pages"], "rings": st["rings"], "ctx": st["ctx_out"]}


def _copy_pages(pages, src, dst):
    pages[:, dst.long()] = pages[:, src.long()]


def _plain_fork(st):
    refs, table = st["refs"], st["table"]
    was, st["lens_now"] = st["lens_now"][0], [st["next"], st["next"]]
    p = torch.arange(table.shape[1], device="cuda")[None, :]
    rows = table[st["child"].long()]
    held = (p < ((was + PAGE - 1) // PAGE)[:, None]) & (rows >= 0)
    refs.index_add_(0, torch.where(held, rows, 0).flatten().long(), -held.flatten().to(torch.int32))
    rows = torch.where(held, -1, rows)
    # the lowest free pages, in order, for the branches that end inside a page
    n = st["next"]
    full, used = n // PAGE, (n + PAGE - 1) // PAGE
    tail = full < used
    free = refs == 0
    rank = torch.cumsum(free, 0) - 1
    lowest = torch.zeros(refs.numel() + 1, dtype=torch.int64, device="cuda")
    lowest.scatter_(0, torch.where(free, rank, refs.numel()), torch.arange(refs.numel(), device="cuda"))
    page = torch.where(tail, lowest[(torch.cumsum(tail, 0) - 1).clamp(min=0)], -1).to(torch.int32)
    up = table[st["parent"].long()]
    share = p < full[:, None]
    rows = torch.where(share, up, torch.where((p == full[:, None]) & tail[:, None], page[:, None], rows))
    refs.index_add_(0, torch.where(share, up, 0).flatten().long(), share.flatten().to(torch.int32))
    refs.index_add_(0, page.clamp(min=0).long(), tail.to(torch.int32))
    table[st["child"].long()] = rows
    last = torch.gather(up, 1, full[:, None].long().clamp(max=table.shape[1] - 1))[:, 0]
    st["src"].copy_(torch.where(tail, last, -1))
    st["dst"].copy_(page)
    _copy_pages(st["pages"], st["src"][st["tails"]], st["dst"][st["tails"]])
    return {"pages": st["pages"], "table": table, "refs": refs, "src": st["src"], "dst": st["dst"]}


def _plain_compact(st):
    refs, table = st["refs"], st["table"]
    refs.copy_(st["refs0"])
    table.copy_(st["table0"])
    live = refs > 0
    front = torch.arange(refs.numel(), device="cuda") < live.sum()
    src, dst = (live & ~front).nonzero()[:, 0], (~live & front).nonzero()[:, 0]
    to = torch.arange(refs.numel(), dtype=torch.int32, device="cuda")
    to[src] = dst.to(torch.int32)
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table))
    refs[dst] = refs[src]
    refs[src] = 0
    _copy_pages(st["pages"], src, dst)
    st["moves"].fill_(src.numel())
    return {"pages": st["pages"], "table": table, "refs": refs, "moves": st["moves"]}


def run(state):
    if own:
        return _run_own(state)
    return {"prompt": _plain_prompt, "tree": _plain_tree, "treeswa": _plain_treeswa, "commit": _plain_commit,
            "fork": _plain_fork, "compact": _plain_compact}[state["c"]["kind"]](state)


# ------------------------------------------------------------------------------------- what a pass needs

def _pairs(n, W):
    """Sum over the rows i of a prompt of the keys that row i sees."""
    if not W or n <= W:
        return n * (n + 1) // 2
    return W * (W + 1) // 2 + (n - W) * W


def work(case):
    c, kind = case, case["kind"]
    if kind == "prompt":
        lens = _lengths(c, c["B"])
        T = sum(lens)
        return {"bytes": 2 * D * T * (2 * c["Hq"] + 2 * c["Hkv"]),
                "flops": 4 * D * c["Hq"] * sum(_pairs(n, c["window"]) for n in lens)}
    if kind == "tree":
        keys = sum(n + c["N"] for n in _lengths(c, c["B"]))
        return {"bytes": keys * c["Hkv"] * 136 + 2 * 2 * D * c["B"] * c["N"] * c["Hq"],
                "flops": 4 * D * c["Hq"] * c["N"] * keys + 2 * D * D * c["B"] * c["N"] * c["Hq"]}
    if kind == "treeswa":
        keys = sum(min(n, c["window"] - 1) + c["N"] for n in _lengths(c, c["B"]))
        return {"bytes": keys * c["Hkv"] * 256 + 2 * 2 * D * c["B"] * c["N"] * c["Hq"],
                "flops": 4 * D * c["Hq"] * c["N"] * keys}
    if kind == "commit":
        acc = sum(_accepted(c))
        return {"bytes": 2 * acc * c["Hkv"] * (136 * c["layers4"] + 256 * c["layers8"]) + 4 * acc + 12 * c["B"], "flops": 0}
    if kind == "fork":
        lens = _lengths(c, c["parents"])
        tails = c["children"] * sum(n % PAGE > 0 for n in lens) / len(lens)
        shared = c["children"] * sum(_pages_of(n) for n in lens) / len(lens)
        return {"bytes": 2 * tails * c["layers"] * c["Hkv"] * BLOCK4 + 24 * shared, "flops": 0}
    lens = _lengths(c, c["B"])
    num = sum(_pages_of(n) for n in lens)
    alive = random.Random(c["spread"] + 2).sample(range(c["B"]), max(1, int(round(c["keep"] * c["B"]))))
    live = sum(_pages_of(lens[b]) for b in alive)
    moved = live * (num - live) / num  # of live pages at random places, those behind the front
    return {"bytes": 2 * moved * c["layers"] * c["Hkv"] * BLOCK4 + 8 * num, "flops": 0}


# ------------------------------------------------------------------------------------- in 64 bits

def _exact_prompt(c, st):
    if c["Hq"] * sum(_pairs(n, c["window"]) for n in st["lens"]) > 3e10:
        return None
    G, W, outs = c["Hq"] // c["Hkv"], c["window"], []
    for b, n in enumerate(st["lens"]):
        lo = st["at"][b]
        Q, K, V = (st[x][lo:lo + n].to(torch.float64) for x in "qkv")
        rows = []
        for r in range(0, n, 1024):
            first = max(0, r + 1 - W) if W else 0
            last = min(n, r + 1024)
            at = torch.arange(r, last, device="cuda").view(-1, 1) - torch.arange(first, last, device="cuda").view(1, -1)
            hide = (at < 0) | (at >= W) if W else at < 0
            heads = []
            for h in range(c["Hq"]):
                z = Q[r:last, h] @ K[first:last, h // G].T / math.sqrt(D)
                z.masked_fill_(hide, -math.inf)
                heads.append(torch.softmax(z, 1) @ V[first:last, h // G])
            rows.append(torch.stack(heads, 1))
        outs.append(torch.cat(rows, 0))
    return torch.cat(outs, 0)


def _exact_tree(c, st):
    """Sequence by sequence, head by head, from the records' bit fields."""
    B, N, G = c["B"], c["N"], c["Hq"] // c["Hkv"]
    if c["Hq"] * N * sum(_lengths(c, B)) > 2e10:
        return None
    M = st["M"].double()
    slot = torch.arange(PAGE, device="cuda")
    byte = torch.arange(64, device="cuda")
    kpos = ((byte[None] // 16) ^ (((slot >> 1) & 1) | ((slot >> 2) & 2))[:, None]) * 16 + byte[None] % 16 + slot[:, None] * 64
    vpos = 4096 + ((byte[None] // 16) ^ ((slot >> 1) & 3)[:, None]) * 16 + byte[None] % 16 + slot[:, None] * 64
    out = torch.empty(B, N, c["Hq"], D, dtype=torch.float64, device="cuda")
    words = st["mask"].tolist()
    for b, ctx in enumerate(_lengths(c, B)):
        n = ctx + N
        blocks = st["pages"][st["table"][b, :_pages_of(n)].long()]
        hide = torch.zeros(N, n, dtype=torch.bool, device="cuda")
        hide[:, ctx:] = torch.tensor([[not (w >> j) & 1 for j in range(N)] for w in words[b]], device="cuda")
        x = st["q"][b].double()
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS)
        qt = torch.einsum("nhi,ji->nhj", x, M)
        for h in range(c["Hkv"]):
            blk = blocks[:, h].to(torch.int32)
            kb = blk[:, kpos.flatten()].view(-1, 64)[:n]
            key = torch.stack([kb % 16, kb // 16], 2).view(n, D).double()
            vb = blk[:, vpos.flatten()].view(-1, 32, 2)[:n]
            w = vb[:, :, 0] + 256 * vb[:, :, 1]
            val = []
            for e, s in ((1, 15), (4, 14), (11, 7), (8, 0)):
                mag = ((w >> e) & 7).double() + 0.5
                val.append(7.5 + torch.where((w >> s) & 1 == 1, -mag, mag))
            val = torch.stack(val, 2).view(n, D)
            meta = blocks[:, h, 8192:].contiguous().view(torch.float16).double().view(-1, 2, PAGE, 2)
            ks, vs = (meta[:, i].reshape(-1, 2)[:n] for i in (0, 1))
            key = key * ks[:, :1] + ks[:, 1:]
            val = val * vs[:, :1] + vs[:, 1:]
            for hq in range(h * G, h * G + G):
                z = (qt[:, hq] @ key.T / math.sqrt(D)).masked_fill(hide, -math.inf)
                out[b, :, hq] = torch.softmax(z, 1) @ val
    return out


def _exact_treeswa(c, st):
    B, N, G, W, cap = c["B"], c["N"], c["Hq"] // c["Hkv"], c["window"], _ring_capacity(c)
    out = torch.empty(B, N, c["Hq"], D, dtype=torch.float64, device="cuda")
    scale = float(torch.tensor(6 / 448, dtype=torch.float32))
    byte = torch.arange(D, device="cuda")
    words = st["mask"].tolist()
    for b, ctx in enumerate(_lengths(c, B)):
        first = max(0, ctx - W + 1)
        pos = list(range(first, ctx + N))
        at = _ints([p % cap for p in pos], torch.int64)
        where = (at % PAGE)[:, None] * D + ((byte[None] // 16) ^ (at % 8)[:, None]) * 16 + byte[None] % 16
        hide = torch.tensor([[not (p > ctx + max(1, bin(w & (1 << 64) - 1).count("1")) - 1 - W if p < ctx else (w >> (p - ctx)) & 1)
                              for p in pos] for w in words[b]], device="cuda")
        for h in range(c["Hkv"]):
            blk = st["ring"][b, h][at // PAGE]
            key, val = (torch.gather(blk[:, o:o + 8192], 1, where).view(torch.float8_e4m3fn).double() * scale for o in (0, 8192))
            for hq in range(h * G, h * G + G):
                z = (st["q"][b, :, hq].double() @ key.T / math.sqrt(D)).masked_fill(hide, -math.inf)
                out[b, :, hq] = torch.softmax(z, 1) @ val
    return out


def exact(case, seed):
    kind = case["kind"]
    if kind not in ("prompt", "tree", "treeswa"):
        return None  # bytes and page numbers are moved, nothing is computed
    st = prepare(case, seed)
    return {"prompt": _exact_prompt, "tree": _exact_tree, "treeswa": _exact_treeswa}[kind](case, st)
