"""Caches held to a size through the layer stack: prompts whose last rows are observed, eviction, decode steps that go on
gathering, eviction again, beside a layer with a window and first tokens and the rings. A twin stack that evicts nothing has
every token's record at the token's own position: what the stack holds under a number has to be that record bit for bit, and
its outputs are those of plain attention over the records it holds."""

import numpy as np
import pytest
import torch

from gpu_util import unpack_int4
from quantized_kv_cache_fold_gb300 import runner
from quantized_kv_cache_fold_gb300.runner import DecodeStack
from test_gpu_tree import attend

pytestmark = pytest.mark.gpu
D, SM = 128, 128 ** -0.5


def records(tensors, b, h, n):
    c = unpack_int4(tensors, b, h, n)
    return np.concatenate([c["kc"], c["vc"]] + [c[x].astype(np.int64)[:, None] for x in ("ks", "ko", "vs", "vo")], 1), c


def values(c):
    f = lambda a: torch.from_numpy(a.view(np.float16).astype(np.float64))[:, None]  # noqa: E731
    return ((torch.from_numpy(c["kc"].astype(np.float64)) * f(c["ks"]) + f(c["ko"])).cuda(),
            (torch.from_numpy(c["vc"].astype(np.float64)) * f(c["vs"]) + f(c["vo"])).cuda())


def test_prompt_observe_evict_decode_evict():
    B, Hq, Hkv, n_layers, G = 2, 20, 4, 6, 5
    lens, budget, sinks, recent = [330, 270], 200, 4, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    gains, M = {}, {}

    def stack():
        st = DecodeStack(B, Hq, Hkv, 1, 6, n_layers=n_layers, full_every=2, window=64, ring_capacity=128, swa_k_scale=6 / 448,
                         swa_v_scale=6 / 448)
        for l in st.int4_layers():
            r = np.random.default_rng(l)
            gains[l] = [r.uniform(0.5, 1.5, D).astype(np.float32) for _ in range(2)]
            st.set_int4_params(l, l + 3, *gains[l])
            M[l] = torch.from_numpy(st.layers[l].R.astype(np.float64) * (gains[l][0].astype(np.float64) * gains[l][1])[None]).cuda()
        st.set_int4_window(3, 100, 7)
        return st

    st, twin = stack(), stack()
    st.keep_mass()
    assert st.mass_layers() == [1, 5]
    T = sum(lens)
    cu = i32([0, lens[0], T])
    seq = i32([b for b in range(B) for _ in range(lens[b])])
    pos = i32([p for b in range(B) for p in range(lens[b])])
    late = torch.tensor([p >= lens[b] - 100 for b in range(B) for p in range(lens[b])], device="cuda")
    for l in range(n_layers):
        q, k, v = rand(T, Hq, D), rand(T, Hkv, D), rand(T, Hkv, D)
        out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        st.prompt_layer(l, q, k, v, cu, out)
        assert bool(torch.isfinite(out).all())
        if l in st.mass_layers():
            st.observe_prompt(l, q, k, cu, 32)
        keep = late if l in st.swa_layers() else torch.ones_like(late)
        for x in (st, twin):
            x.append_prompt(l, k[keep].contiguous(), v[keep].contiguous(), seq[keep].contiguous(), pos[keep].contiguous())

    def evict(ctx, seen):
        before = {l: {k: v.clone() for k, v in st.layers[l].held.items()} for l in st.mass_layers()}
        st.evict(i32(ctx), i32(seen), budget, sinks, recent, new := i32([0] * B))
        assert new.tolist() == [min(budget, c) for c in ctx]
        for l in st.mass_layers():
            for b in range(B):
                for h in range(Hkv):
                    ids, mass = (before[l][x][b, h, :ctx[b]].cpu().numpy() for x in ("ids", "mass"))
                    first = (ids < sinks) | (ids >= seen[b] - recent)
                    order = np.lexsort((np.arange(ctx[b]), -np.where(first, np.inf, mass)))
                    assert set(st.layers[l].held["ids"][b, h, :budget].tolist()) == set(ids[order[:budget]].tolist())
        same(new.tolist())
        return new.tolist()

    def same(ctx):
        """Every slot holds the record of its token."""
        for l in st.mass_layers():
            for b in range(B):
                for h in range(Hkv):
                    ids = st.layers[l].held["ids"][b, h, :ctx[b]].cpu().numpy()
                    assert len(set(ids.tolist())) == ctx[b]
                    mine, _ = records(st.layers[l].tensors, b, h, ctx[b])
                    all_, _ = records(twin.layers[l].tensors, b, h, int(ids.max()) + 1)
                    assert np.array_equal(mine, all_[ids])

    ctx, seen = evict(lens, list(lens)), list(lens)
    for step in range(20):
        qs = [rand(B, 1, Hq, D) for _ in range(n_layers)]
        new = [(rand(B, 1, Hkv, D), rand(B, 1, Hkv, D)) for _ in range(n_layers)]
        outs = [[torch.empty(B, 1, Hq, D, dtype=torch.float32, device="cuda") for _ in range(n_layers)] for _ in range(2)]
        st.decode_step(qs, i32(ctx), outs[0], [x[0] for x in new], [x[1] for x in new], positions=i32(seen))
        twin.decode_step(qs, i32(seen), outs[1], [x[0] for x in new], [x[1] for x in new])
        torch.cuda.synchronize()
        for l in range(n_layers):
            if l not in st.mass_layers():
                assert torch.equal(outs[0][l], outs[1][l])
        ctx, seen = [c + 1 for c in ctx], [c + 1 for c in seen]
        if step % 7 == 0:
            for l in st.mass_layers():
                x = qs[l][:, 0].double()
                qt = (x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()) @ M[l].T
                for b in range(B):
                    for h in range(Hkv):
                        k, v = values(records(st.layers[l].tensors, b, h, ctx[b])[1])
                        o, tol = attend(qt[b, h * G:h * G + G], k, v, torch.ones(G, ctx[b], dtype=torch.bool, device="cuda"), SM, torch.float32)
                        assert bool(((outs[0][l][b, 0, h * G:h * G + G].double() - o).abs() <= tol).all())
    same(ctx)
    total = [float(st.layers[l].held["mass"][b, h, :ctx[b]].double().sum()) for l in st.mass_layers() for b in range(B) for h in range(Hkv)]
    assert min(total) > 20 * G * 0.99  # 20 steps of G rows were gathered by the tokens that stay, and by the prompt's
    ctx = evict(ctx, seen)
    assert ctx == [budget] * B
    assert st.read_error() == 0 and twin.read_error() == 0


def test_layers_of_a_kind():
    st = DecodeStack(1, 4, 2, 1, 2, n_layers=4, full_every=2, window=64, ring_capacity=64)
    for bad in ((0, 64, 4), (1, -1, 0), (1, 5, -2)):
        with pytest.raises(ValueError):
            st.set_int4_window(*bad)
    st.set_int4_window(1, 64, 4)
    for bad in ([0], [1], [3, 1]):
        with pytest.raises(ValueError):
            st.keep_mass(bad)
    st.keep_mass()
    assert st.mass_layers() == [3]
    with pytest.raises(ValueError):
        st.set_int4_window(3, 64)
    for l in (1, 3):
        with pytest.raises(ValueError):
            st.tree_layer(l, None, None, None, None, None)
        with pytest.raises(ValueError):
            st.decode_layer(l, None, None, None, q_rot_out=1)


def test_stacks_that_keep_no_mass_and_masses_kept_twice():
    st = DecodeStack(1, 4, 2, 1, 2, n_layers=4, full_every=2, window=64, ring_capacity=64)
    with pytest.raises(ValueError):
        st.evict(None, None, 10, 1, 2, None)
    st.keep_mass([1])
    for l in (0, 3):
        with pytest.raises(ValueError):
            st.observe_prompt(l, None, None, None, 4)
    held = st.layers[1].held["mass"]
    held.fill_(2.0)
    st.keep_mass()
    assert st.mass_layers() == [1, 3] and st.layers[1].held["mass"] is held and bool((held == 2.0).all())


def test_more_layers_than_a_call_takes(monkeypatch):
    calls = []
    monkeypatch.setattr(runner, "kvq_evict_int4", lambda caches, masses, *a, ctx_out, stream: calls.append((list(caches), list(masses), ctx_out, stream)))
    st = DecodeStack(1, 2, 2, 1, 1, n_layers=150, full_every=2, ring_capacity=64, window=64)
    st.keep_mass()
    st.evict("ctx", "seen", 10, 1, 2, "out", stream=5)
    assert [len(c) for c, _, _, _ in calls] == [64, 11] and [o for _, _, o, _ in calls] == ["out", None]
    got = [(id(c), id(m)) for cs, ms, _, s in calls for c, m in zip(cs, ms) if s == 5]
    assert got == [(id(st.layers[l].cache), id(st.layers[l].mass)) for l in st.mass_layers()]
