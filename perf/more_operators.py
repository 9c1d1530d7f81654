"""What a session asks of a cache that is held to a size: a window of the newest tokens beside a few first ones that stay
visible, the attention weight that every cached token has gathered, and the eviction of the tokens that gathered least.

kinds of case
  prompt    causal attention over whole prompts packed end to end, each row seeing the first `sinks` tokens and the
            last `window` ones
  window    attention of a block of S new tokens over the paged 4-bit cache under the same rule
  mass      attention of one new token per sequence over the whole paged 4-bit cache, its weights added to what every
            cached token has gathered per KV head
  observe   the weights that the last `rows` rows of each prompt put on its tokens, summed per KV head
  evict     in every layer, per sequence and KV head, the `budget` tokens that gathered most stay (with the first and
            the newest ones), moved to the front of the cache
"""

import math
import random

import torch

own = False

D = 128          # head dim
PAGE = 64        # tokens of a page
BLOCK4 = 8704    # bytes of one (page, KV head): K codes 4096, V codes 4096, K meta 256, V meta 256
EPS = 1e-6
SM = D ** -0.5


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # four short chat turns arriving together, windows barely longer than the longest: the smallest prefill
        {"name": "sinks-turns", "kind": "prompt", "B": 4, "lo": 1, "hi": 300, "spread": 1, "Hq": 20, "Hkv": 4,
         "dtype": "bf16", "window": 128, "sinks": 4, "fused": False},
        # an ordinary prefill batch: ragged prompts, q/k/v views of one projection's output, the stack's window
        {"name": "sinks-packed", "kind": "prompt", "B": 24, "lo": 100, "hi": 4000, "spread": 2, "Hq": 20, "Hkv": 4,
         "dtype": "bf16", "window": 513, "sinks": 64, "fused": True},
        # one long document, a wide window, half precision
        {"name": "sinks-long", "kind": "prompt", "B": 1, "lo": 32768, "hi": 32768, "spread": 3, "Hq": 20, "Hkv": 4,
         "dtype": "f16", "window": 4096, "sinks": 4, "fused": False},
        # one long session's decode step: latency
        {"name": "window-one", "kind": "window", "B": 1, "lo": 65536, "hi": 65536, "spread": 4, "S": 1, "Hq": 20,
         "Hkv": 4, "window": 1023, "sinks": 4},
        # the decode batch, every sequence past its window
        {"name": "window-batch", "kind": "window", "B": 64, "lo": 5000, "hi": 16384, "spread": 5, "S": 1, "Hq": 20,
         "Hkv": 4, "window": 4096, "sinks": 64},
        # verify blocks of a small batch, some sequences shorter than the window
        {"name": "window-verify", "kind": "window", "B": 16, "lo": 100, "hi": 8192, "spread": 6, "S": 4, "Hq": 20,
         "Hkv": 4, "window": 2000, "sinks": 5},
        # one session's decode step with its weights kept
        {"name": "mass-one", "kind": "mass", "B": 1, "lo": 4096, "hi": 4096, "spread": 7, "Hq": 20, "Hkv": 4},
        # the decode batch of caches that are about to be evicted from
        {"name": "mass-batch", "kind": "mass", "B": 64, "lo": 4096, "hi": 16384, "spread": 8, "Hq": 20, "Hkv": 4},
        # what the last rows of a few chat turns looked at
        {"name": "observe-turns", "kind": "observe", "B": 4, "lo": 1, "hi": 700, "spread": 9, "Hq": 20, "Hkv": 4,
         "dtype": "bf16", "rows": 16, "fused": False},
        # long documents, observed by their last 64 tokens before the cache is cut to a budget
        {"name": "observe-long", "kind": "observe", "B": 8, "lo": 2000, "hi": 32768, "spread": 10, "Hq": 20, "Hkv": 4,
         "dtype": "bf16", "rows": 64, "fused": True},
        # a decode batch that has grown by a page since its last eviction, all ten full-attention layers
        {"name": "evict-step", "kind": "evict", "B": 64, "lo": 2112, "hi": 2112, "spread": 11, "Hkv": 4, "layers": 10,
         "budget": 2048, "sinks": 4, "recent": 128},
        # long prompts cut to their budget after the prefill
        {"name": "evict-prompt", "kind": "evict", "B": 4, "lo": 20000, "hi": 32768, "spread": 12, "Hkv": 4,
         "layers": 10, "budget": 2048, "sinks": 4, "recent": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    return rng.choice([(20, 4), (20, 4), (8, 1), (16, 4), (6, 2), (4, 4)])


def draw(rng):
    kind = rng.choice(["prompt", "window", "mass", "observe", "evict"])
    c = {"kind": kind, "spread": rng.randrange(1 << 20)}
    if kind == "prompt":
        c["Hq"], c["Hkv"] = _heads(rng)
        c["B"] = _log(rng, 1, 40)
        c["hi"] = _log(rng, 1, max(64, min(20000, 60000 // c["B"])))
        c["lo"] = _log(rng, 1, c["hi"])
        c["dtype"] = rng.choice(["bf16", "bf16", "f16"])
        c["window"] = rng.choice([513, _log(rng, 1, 4000), _log(rng, 1, 4000)])
        c["sinks"] = rng.choice([4, 1, _log(rng, 1, 600)])
        c["fused"] = rng.random() < 0.4
    elif kind == "window":
        c["Hq"], c["Hkv"] = _heads(rng)
        c["S"] = rng.choice([1, 1, rng.randint(1, 8), rng.randint(1, 5)])
        c["window"] = _log(rng, 1, 8000)
        c["sinks"] = rng.choice([0, 4, _log(rng, 1, 300)])
        c["B"] = _log(rng, 1, 80)
        c["hi"] = _log(rng, 1, max(256, min(100000, 600000 // c["B"])))
        c["lo"] = _log(rng, 1, c["hi"])
    elif kind == "mass":
        c["Hq"], c["Hkv"] = _heads(rng)
        c["B"] = _log(rng, 1, 80)
        c["hi"] = _log(rng, 1, max(256, min(60000, 600000 // c["B"])))
        c["lo"] = _log(rng, 1, c["hi"])
    elif kind == "observe":
        c["Hq"], c["Hkv"] = _heads(rng)
        c["B"] = _log(rng, 1, 40)
        c["hi"] = _log(rng, 1, max(64, min(20000, 60000 // c["B"])))
        c["lo"] = _log(rng, 1, c["hi"])
        c["dtype"] = rng.choice(["bf16", "bf16", "f16"])
        c["rows"] = rng.choice([16, 64, _log(rng, 1, 300)])
        c["fused"] = rng.random() < 0.4
    else:
        c["Hkv"] = rng.choice([4, 4, 1, 2, 8])
        c["layers"] = rng.randrange(1, 11)
        c["B"] = _log(rng, 1, 64)
        c["hi"] = _log(rng, 1, max(64, min(60000, 4000000 // (c["B"] * c["Hkv"] * c["layers"]))))
        c["lo"] = _log(rng, 1, c["hi"])
        c["budget"] = _log(rng, 1, c["hi"] + 1)
        c["sinks"] = rng.choice([0, 4, 1])
        c["recent"] = rng.randint(0, max(0, min(256, c["budget"] - c["sinks"])))
    return c


def _lengths(c, count):
    """The case's token counts: spread over [lo, hi] by their logarithm, the longest of them hi."""
    r = random.Random(c["spread"])
    n = [min(c["hi"], max(c["lo"], _log(r, c["lo"], c["hi"]))) for _ in range(count)]
    n[r.randrange(count)] = c["hi"]
    return n


def _pages_of(n):
    return (n + PAGE - 1) // PAGE


# ------------------------------------------------------------------------------------- inputs

def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


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


def _sixteen(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float16


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind, B, Hkv = c["kind"], c["B"], c["Hkv"]
    lens = _lengths(c, B)
    st = {"c": c, "lens": lens, "err": torch.zeros(1, dtype=torch.int32, device="cuda"), "kept": {}}
    if kind in ("prompt", "observe"):
        at = _packed_offsets(lens)
        T, Hq, dt = at[-1], c["Hq"], _sixteen(c)
        gain = torch.rand(D, generator=g, device="cuda") + 0.75
        normed = lambda x: x / (x.square().mean(-1, keepdim=True) + EPS).sqrt()  # noqa: E731
        q = (normed(_normal(g, T, Hq, D)) * gain).to(dt)
        k = (normed(_normal(g, T, Hkv, D)) * gain).to(dt)
        v = _normal(g, T, Hkv, D).to(dt)
        if c["fused"]:
            qkv = torch.cat([q, k, v], 1).contiguous()
            q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        st.update(q=q, k=k, v=v, at=at, offsets=_ints(at))
        if kind == "prompt":
            st["out"] = torch.empty(T, Hq, D, dtype=dt, device="cuda")
        else:
            L = _pages_of(max(lens)) * PAGE
            st["mass"] = torch.zeros(B, Hkv, L, device="cuda")
            st["ids"] = torch.zeros(B, Hkv, L, dtype=torch.int32, device="cuda")
        return st
    S = c["S"] if kind == "window" else 1 if kind == "mass" else 0
    P = _pages_of(max(lens) + S)
    table = _table(g, B, P)
    layers = c.get("layers", 1)
    pages = torch.empty(layers, B * P, Hkv, BLOCK4, dtype=torch.uint8, device="cuda")
    _fill4(pages, g, 256 if kind == "evict" else 2048)
    st.update(pages=pages, table=table, ctx=_ints(lens))
    if kind == "evict":
        # one tensor of masses and one of token numbers, as they are before the eviction and as it leaves them
        before = torch.empty(2, layers, B, Hkv, P * PAGE, dtype=torch.int32, device="cuda")
        before[0] = torch.rand(layers, B, Hkv, P * PAGE, generator=g, device="cuda").pow_(6).mul_(4).view(torch.int32)
        # the sequences had 500 tokens more than are left: later tokens in the later slots, none twice
        gone = torch.rand(layers, B, Hkv, P * PAGE, generator=g, device="cuda")
        slot = torch.arange(P * PAGE, device="cuda")
        n = st["ctx"][None, :, None, None]
        early = (slot >= c["sinks"]) & (slot < n - c["recent"])
        skip = torch.cumsum(torch.where(early, gone, 0.0), -1)
        skip = skip / skip[..., -1:].clamp(min=1e-9) * 499
        before[1] = slot + torch.where(slot >= n - c["recent"], 500, torch.where(slot < c["sinks"], 0, skip.long()))
        st.update(before=before, now=before.clone(), seen=st["ctx"] + 500, new=torch.zeros_like(st["ctx"]))
        return st
    st.update(M=_folded(g, seed), q=_normal(g, B, S, c["Hq"], D).to(torch.bfloat16),
              out=torch.empty(B, S, c["Hq"], D, dtype=torch.bfloat16, device="cuda"))
    if kind == "mass":
        # what a few steps before this one may have left: four weights of 1/n from every head on average
        few = torch.rand(B, Hkv, P * PAGE, generator=g, device="cuda").pow_(8) * (36 * c["Hq"] / Hkv)
        st.update(mass=few / st["ctx"].clamp(min=1)[:, None, None],
                  ids=torch.arange(P * PAGE, dtype=torch.int32, device="cuda").repeat(B, Hkv, 1), seen=st["ctx"] + 7)
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
                           sinks=c["sinks"], sm_scale=SM)
        return st["out"]
    if kind == "observe":
        ws = _framework(st, "ws", lambda: kv.alloc_prompt_mass_workspace(st["at"][-1], c["B"], c["Hq"], c["Hkv"],
                                                                         c["rows"]))
        mass = _framework(st, "mass", lambda: kv.token_mass(st["mass"], st["ids"]))
        kv.kvq_prompt_mass(st["q"], st["k"], st["offsets"], c["rows"], mass, ws, st["err"], sm_scale=SM)
        return {"mass": st["mass"], "ids": st["ids"]}
    if kind == "evict":
        caches = _framework(st, "caches", lambda: [kv.int4_cache(p, st["table"]) for p in st["pages"]])
        mass = _framework(st, "mass", lambda: [kv.token_mass(m, i) for m, i in zip(st["now"][0].view(torch.float32),
                                                                                   st["now"][1])])
        st["now"].copy_(st["before"])  # the masses before the eviction again
        kv.kvq_evict_int4(caches, mass, st["ctx"], st["seen"], c["budget"], c["sinks"], c["recent"], st["err"],
                          ctx_out=st["new"])
        return {"pages": st["pages"], "mass": st["now"][0].view(torch.float32), "ids": st["now"][1], "ctx": st["new"]}
    cache = _framework(st, "cache", lambda: kv.int4_cache(st["pages"][0], st["table"]))
    if kind == "window":
        ws = _framework(st, "ws", lambda: kv.alloc_workspace(c["B"], c["S"], c["Hq"], c["Hkv"]))
        kv.kvq_window_attn_int4(cache, st["M"], None, st["q"], st["ctx"], c["window"], c["sinks"], st["out"], ws,
                                st["err"], sm_scale=SM, eps=EPS)
        return st["out"]
    ws = _framework(st, "ws", lambda: kv.alloc_mass_workspace(c["B"], c["Hq"], c["Hkv"], st["mass"].shape[2]))
    mass = _framework(st, "mass", lambda: kv.token_mass(st["mass"], st["ids"]))
    kv.kvq_mass_attn_int4(cache, mass, st["M"], None, st["q"], st["ctx"], st["seen"], st["out"], ws, st["err"],
                          sm_scale=SM, eps=EPS)
    return {"out": st["out"], "mass": st["mass"], "ids": st["ids"]}


def _plain_prompt(st):
    """softmax(q k' / sqrt(128)) v of each prompt, a part of its query rows at a time."""
    c = st["c"]
    Hq, Hkv, W, F = c["Hq"], c["Hkv"], c["window"], c["sinks"]
    out = st["out"]
    for lo, hi in zip(st["at"], st["at"][1:]):
        n = hi - lo
        q = st["q"][lo:hi].float().view(n, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3)  # [Hkv, G, n, D]
        k, v = st["k"][lo:hi].float().transpose(0, 1), st["v"][lo:hi].float().transpose(0, 1)
        for r0 in range(0, n, 2048):
            r1 = min(n, r0 + 2048)
            w0 = max(0, r0 - W + 1)  # the first token of a window, and behind the first ones
            j = torch.cat([torch.arange(min(F, w0), device="cuda"), torch.arange(w0, r1, device="cuda")])
            i = torch.arange(r0, r1, device="cuda")[:, None]
            s = torch.matmul(q[:, :, r0:r1], k[:, None, j].transpose(-1, -2)) * SM
            s = torch.where((j <= i) & ((j > i - W) | (j < F)), s, -math.inf)
            p = torch.exp(s - s.amax(-1, keepdim=True))
            o = torch.matmul(p, v[:, None, j]) / p.sum(-1, keepdim=True)
            out[lo + r0:lo + r1] = o.permute(2, 0, 1, 3).reshape(r1 - r0, Hq, D).to(out.dtype)
    return out


def _plain_observe(st):
    """Column sums of the softmax of each prompt's last rows, a part of them at a time."""
    c = st["c"]
    Hq, Hkv = c["Hq"], c["Hkv"]
    for b, (lo, hi) in enumerate(zip(st["at"], st["at"][1:])):
        n = hi - lo
        k = st["k"][lo:hi].float().transpose(0, 1)
        total = torch.zeros(Hkv, n, device="cuda")
        for r0 in range(max(0, n - c["rows"]), n, 64):
            r1 = min(n, r0 + 64)
            q = st["q"][lo + r0:lo + r1].float().view(r1 - r0, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3)
            s = torch.matmul(q, k[:, None].transpose(-1, -2)) * SM
            s = torch.where(torch.arange(n, device="cuda") <= torch.arange(r0, r1, device="cuda")[:, None], s, -math.inf)
            p = torch.exp(s - s.amax(-1, keepdim=True))
            total += (p / p.sum(-1, keepdim=True)).sum((1, 2))
        st["mass"][b, :, :n] = total
        st["ids"][b, :, :n] = torch.arange(n, dtype=torch.int32, device="cuda")
    return {"mass": st["mass"], "ids": st["ids"]}


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


def _rotated(st):
    x = st["q"].float()
    return torch.matmul(x / (x.square().mean(-1, keepdim=True) + EPS).sqrt(), st["M"].t())


def _weights(q, k, seen):
    """q [B, S, Hq, D], k [B, Hkv, L, D], seen [B, S, L]: softmax weights [B, Hkv, G, S, L]."""
    B, S, Hq, _ = q.shape
    Hkv = k.shape[1]
    q = q.view(B, S, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    s = torch.matmul(q, k.transpose(-1, -2)).view(B, Hkv, Hq // Hkv, S, -1) * SM
    s = torch.where(seen[:, None, None], s, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _outputs(p, v):
    """Weights [B, Hkv, G, S, L] and values [B, Hkv, L, D]: outputs [B, S, Hq, D]."""
    B, Hkv, G, S, L = p.shape
    o = torch.matmul(p.view(B, Hkv, G * S, L), v).view(B, Hkv, G, S, D)
    return o.permute(0, 3, 1, 2, 4).reshape(B, S, Hkv * G, D)


def _plain_window(st):
    """The pages of the first tokens and of the windows, gathered and decoded."""
    c = st["c"]
    B, S, W, F = c["B"], c["S"], c["window"], c["sinks"]
    P = st["table"].shape[1]
    first = min(P, _pages_of(F))
    count = min(P, _pages_of(W + S - 1) + 1)
    start = ((st["ctx"] - W + 1).clamp(min=0) // PAGE).clamp(max=P - count)
    p = torch.cat([torch.arange(first, device="cuda").expand(B, first),
                   start[:, None] + torch.arange(count, device="cuda")], 1)
    k, v = _decoded4(st["pages"][0][torch.gather(st["table"], 1, p).long()].transpose(1, 2))
    j = (p[:, :, None] * PAGE + torch.arange(PAGE, device="cuda")).view(B, 1, -1)
    once = torch.ones_like(j, dtype=torch.bool)
    once[:, :, first * PAGE:] = j[:, :, first * PAGE:] >= first * PAGE  # pages of both kinds count as first ones
    i = st["ctx"][:, None, None] + torch.arange(S, device="cuda")[:, None]
    seen = once & (j <= i) & ((j > i - W) | (j < F))
    L = j.shape[2]
    w = _weights(_rotated(st), k.reshape(B, c["Hkv"], L, D), seen)
    st["out"].copy_(_outputs(w, v.reshape(B, c["Hkv"], L, D)).to(torch.bfloat16))
    return st["out"]


def _plain_mass(st):
    c = st["c"]
    B, Hkv, L = c["B"], c["Hkv"], st["mass"].shape[2]
    k, v = _decoded4(st["pages"][0][st["table"].long()].transpose(1, 2))
    j = torch.arange(L, device="cuda")
    ctx = st["ctx"][:, None]
    w = _weights(_rotated(st), k.reshape(B, Hkv, L, D), (j <= ctx)[:, None])
    st["out"].copy_(_outputs(w, v.reshape(B, Hkv, L, D)).to(torch.bfloat16))
    w = w.sum((2, 3))
    old = st["mass"]
    at = (j == ctx)[:, None]
    old.copy_(torch.where((j < ctx)[:, None], old + w, torch.where(at, w, old)))
    st["ids"].copy_(torch.where(at, st["seen"][:, None, None], st["ids"]))
    return {"out": st["out"], "mass": st["mass"], "ids": st["ids"]}


def _plain_evict(st):
    c = st["c"]
    st["now"].copy_(st["before"])
    mass, ids = st["now"][0].view(torch.float32), st["now"][1]
    K, B, Hkv, L = mass.shape
    slot = torch.arange(L, device="cuda")
    n = st["ctx"][None, :, None, None]
    kept = torch.minimum(n, torch.full_like(n, c["budget"]))
    stays = (ids < c["sinks"]) | (ids >= st["seen"][None, :, None, None] - c["recent"])
    key = torch.where(slot < n, torch.where(stays, math.inf, mass), -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand_as(order))
    keep = (rank < kept) & (slot < n)
    hole, mover = (slot < kept) & ~keep, (slot >= kept) & keep
    # the i-th mover of a row goes to its i-th hole
    to, frm = hole.nonzero(), mover.nonzero()
    l, b, h, s, t = frm[:, 0], frm[:, 1], frm[:, 2], frm[:, 3], to[:, 3]
    ps, pt = (st["table"][b, x // PAGE].long() for x in (s, t))
    pages = st["pages"]
    cs, ct = s % PAGE, t % PAGE
    for first, chunks in ((0, _k_chunks()), (4096, _v_chunks())):
        rec = pages[..., first:first + 4096].view(*pages.shape[:3], PAGE, 4, 16)
        rec[l[:, None], pt[:, None], h[:, None], ct[:, None], chunks[ct]] = \
            rec[l[:, None], ps[:, None], h[:, None], cs[:, None], chunks[cs]]
        meta = pages[..., 8192 + first // 16:8448 + first // 16].view(*pages.shape[:3], PAGE, 4)
        meta[l, pt, h, ct] = meta[l, ps, h, cs]
    mass[l, b, h, t] = mass[l, b, h, s]
    ids[l, b, h, t] = ids[l, b, h, s]
    st["new"].copy_(kept.flatten())
    return {"pages": pages, "mass": mass, "ids": ids, "ctx": st["new"]}


def run(state):
    if own:
        return _run_own(state)
    return {"prompt": _plain_prompt, "window": _plain_window, "mass": _plain_mass, "observe": _plain_observe,
            "evict": _plain_evict}[state["c"]["kind"]](state)


# ------------------------------------------------------------------------------------- what a pass needs

def _seen_by(i, W, F):
    """Tokens that row i of a prompt sees."""
    return min(i + 1, W + min(F, max(0, i + 1 - W)))


def work(case):
    c, kind = case, case["kind"]
    lens = _lengths(c, c["B"])
    if kind == "prompt":
        T = sum(lens)
        return {"bytes": 2 * D * T * (2 * c["Hq"] + 2 * c["Hkv"]),
                "flops": 4 * D * c["Hq"] * sum(_seen_by(i, c["window"], c["sinks"]) for n in lens for i in range(n))}
    if kind == "observe":
        T, rows = sum(lens), [min(n, c["rows"]) for n in lens]
        pairs = sum(r * n - r * (r - 1) // 2 for n, r in zip(lens, rows))
        return {"bytes": 2 * D * (T * c["Hkv"] + sum(rows) * c["Hq"]) + 8 * T * c["Hkv"],
                "flops": 2 * D * c["Hq"] * pairs}
    if kind == "window":
        S = c["S"]
        keys = sum(n + S if n < c["window"] else c["window"] + S - 1 + min(c["sinks"], n - c["window"] + 1) for n in lens)
        rows = c["B"] * S * c["Hq"]
        return {"bytes": keys * c["Hkv"] * 136 + 4 * D * rows,
                "flops": 4 * D * c["Hq"] * sum(_seen_by(n + r, c["window"], c["sinks"]) for n in lens for r in range(S))
                + 2 * D * D * rows}
    if kind == "mass":
        keys = sum(n + 1 for n in lens)
        return {"bytes": keys * c["Hkv"] * (136 + 8) + 4 * D * c["B"] * c["Hq"],
                "flops": 4 * D * c["Hq"] * keys + 2 * D * D * c["B"] * c["Hq"]}
    # masses and token numbers read, and the kept tokens behind the budget moved: of those that may go, as many in
    # proportion as stay (the newest ones all lie behind it)
    total = 0
    for n in lens:
        k = min(n, c["budget"])
        may, room = max(0, n - c["sinks"] - c["recent"]), max(0, k - c["sinks"] - c["recent"])
        behind = max(0, n - c["recent"] - k)
        total += 8 * n + (272 + 16) * (0 if n == k else min(n - k, c["recent"]) + (behind * room / may if may else 0))
    return {"bytes": total * c["Hkv"] * c["layers"], "flops": 0}


# ------------------------------------------------------------------------------------- in 64 bits

def _exact_prompt(c, st):
    W, F, G = c["window"], c["sinks"], c["Hq"] // c["Hkv"]
    outs = []
    for b, n in enumerate(st["lens"]):
        lo = st["at"][b]
        Q, K, V = (st[x][lo:lo + n].to(torch.float64) for x in "qkv")
        rows = []
        for r in range(0, n, 1024):
            last = min(n, r + 1024)
            first = max(0, r + 1 - W)
            cols = list(range(min(F, first))) + list(range(first, last))
            jj = _ints(cols, torch.int64)
            back = torch.arange(r, last, device="cuda").view(-1, 1) - jj.view(1, -1)
            hide = (back < 0) | ((back >= W) & (jj >= F).view(1, -1))
            heads = []
            for h in range(c["Hq"]):
                z = Q[r:last, h] @ K[jj, h // G].T / math.sqrt(D)
                heads.append(torch.softmax(z.masked_fill_(hide, -math.inf), 1) @ V[jj, h // G])
            rows.append(torch.stack(heads, 1))
        outs.append(torch.cat(rows, 0))
    return torch.cat(outs, 0)


def _exact_observe(c, st):
    G = c["Hq"] // c["Hkv"]
    mass = torch.zeros(st["mass"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lens"]):
        lo, r = st["at"][b], max(0, n - c["rows"])
        hide = torch.arange(n, device="cuda").view(1, -1) > torch.arange(r, n, device="cuda").view(-1, 1)
        for h in range(c["Hq"]):
            z = st["q"][lo + r:lo + n, h].double() @ st["k"][lo:lo + n, h // G].double().T / math.sqrt(D)
            mass[b, h // G, :n] += torch.softmax(z.masked_fill_(hide, -math.inf), 1).sum(0)
    return {"mass": mass, "ids": None}


def _records(st, b, h, n):
    """Keys and values of the first n slots of a sequence's KV head, from the records' bit fields."""
    slot = torch.arange(PAGE, device="cuda")
    byte = torch.arange(64, device="cuda")
    kpos = ((byte[None] // 16) ^ (((slot >> 1) & 1) | ((slot >> 2) & 2))[:, None]) * 16 + byte[None] % 16 + slot[:, None] * 64
    vpos = 4096 + ((byte[None] // 16) ^ ((slot >> 1) & 3)[:, None]) * 16 + byte[None] % 16 + slot[:, None] * 64
    blk = st["pages"][0][st["table"][b, :_pages_of(n)].long(), h].to(torch.int32)
    kb = blk[:, kpos.flatten()].view(-1, 64)[:n]
    key = torch.stack([kb % 16, kb // 16], 2).view(n, D).double()
    vb = blk[:, vpos.flatten()].view(-1, 32, 2)[:n]
    w = vb[:, :, 0] + 256 * vb[:, :, 1]
    val = []
    for e, s in ((1, 15), (4, 14), (11, 7), (8, 0)):
        mag = ((w >> e) & 7).double() + 0.5
        val.append(7.5 + torch.where((w >> s) & 1 == 1, -mag, mag))
    val = torch.stack(val, 2).view(n, D)
    meta = blk[:, 8192:].to(torch.uint8).contiguous().view(torch.float16).double().view(-1, 2, PAGE, 2)
    ks, vs = (meta[:, i].reshape(-1, 2)[:n] for i in (0, 1))
    return key * ks[:, :1] + ks[:, 1:], val * vs[:, :1] + vs[:, 1:]


def _exact_cached(c, st):
    """Sequence by sequence, head by head."""
    B, S, G = c["B"], st["q"].shape[1], c["Hq"] // c["Hkv"]
    M = st["M"].double()
    out = torch.empty(B, S, c["Hq"], D, dtype=torch.float64, device="cuda")
    mass = st["mass"].double() if c["kind"] == "mass" else None
    for b, ctx in enumerate(st["lens"]):
        n = ctx + S
        j, i = torch.arange(n, device="cuda").view(1, -1), torch.arange(ctx, n, device="cuda").view(-1, 1)
        hide = j > i
        if c["kind"] == "window":
            hide = hide | ((i - j >= c["window"]) & (j >= c["sinks"]))
        x = st["q"][b].double()
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS)
        qt = torch.einsum("nhi,ji->nhj", x, M)
        for h in range(c["Hkv"]):
            key, val = _records(st, b, h, n)
            if mass is not None:
                mass[b, h, ctx] = 0
            for hq in range(h * G, h * G + G):
                w = torch.softmax((qt[:, hq] @ key.T / math.sqrt(D)).masked_fill(hide, -math.inf), 1)
                out[b, :, hq] = w @ val
                if mass is not None:
                    mass[b, h, :n] += w[0]
    return out if mass is None else {"out": out, "mass": mass, "ids": None}


def exact(case, seed):
    kind = case["kind"]
    if kind == "evict":
        return None  # records are compared and moved, nothing is computed
    st = prepare(case, seed)
    return {"prompt": _exact_prompt, "observe": _exact_observe, "window": _exact_cached, "mass": _exact_cached}[kind](case, st)
