"""Masses that the layer stack keeps, over a session's calls."""

import numpy as np
import pytest
import torch

from quantized_kv_cache_fold_gb300.runner import DecodeStack
from test_gpu_prompt_mass import reference
from test_gpu_stack_bounded import records, values

pytestmark = pytest.mark.gpu
D, SM = 128, 128 ** -0.5


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Session:
    """A stack of int4 layers and rings, its int4 layers with rotations and gains of their own."""

    def __init__(self, B, pages, n_layers=2, full_every=2, Hq=20, Hkv=4, seed=1):
        self.B, self.Hq, self.Hkv, self.n = B, Hq, Hkv, n_layers
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.st = DecodeStack(B, Hq, Hkv, 1, pages, n_layers=n_layers, full_every=full_every, window=64, ring_capacity=128,
                              swa_k_scale=6 / 448, swa_v_scale=6 / 448)
        self.M = {}
        for l in self.st.int4_layers():
            r = np.random.default_rng(seed + l)
            gq, gk = (r.uniform(0.5, 1.5, D).astype(np.float32) for _ in range(2))
            self.st.set_int4_params(l, l + 3, gq, gk)
            self.M[l] = torch.from_numpy(self.st.layers[l].R.astype(np.float64) * (gq.astype(np.float64) * gk)[None]).cuda()

    def rand(self, *s):
        return torch.randn(*s, generator=self.g, device="cuda").to(torch.bfloat16)

    def step_inputs(self):
        qs = [self.rand(self.B, 1, self.Hq, D) for _ in range(self.n)]
        new = [[self.rand(self.B, 1, self.Hkv, D) for _ in range(self.n)] for _ in range(2)]
        outs = [torch.full((self.B, 1, self.Hq, D), 9.0, device="cuda") for _ in range(self.n)]
        return qs, outs, *new


@pytest.mark.parametrize("seed", [1, 2])
def test_keep_mass_between_a_capture_and_its_replay(seed):
    """Captured steps go on with the memory they were captured with: tensors made after a second keep_mass stay as they are."""
    B, T = 2, 700
    s = Session(B, 12, n_layers=4, seed=seed)
    st = s.st
    st.keep_mass([1])
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    for l in range(4):
        for b in range(B):
            keep = slice(0 if l in st.int4_layers() else T - 100, T)
            st.append_prompt(l, s.rand(T, s.Hkv, D)[keep], s.rand(T, s.Hkv, D)[keep], torch.full_like(pos[keep], b), pos[keep])
    ctx = i32([T] * B)
    qs, outs, ks, vs = s.step_inputs()
    start = {x: st.layers[1].held[x].clone() for x in ("mass", "ids")}
    st.decode_step(qs, ctx, outs, ks, vs)
    torch.cuda.synchronize()
    want, masses = [o.clone() for o in outs], st.layers[1].held["mass"].clone()
    assert float(masses.sum()) > 0.9 * B * s.Hq
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.decode_step(qs, ctx, outs, ks, vs)
    size = st.mass_workspace.numel()
    st.keep_mass()
    assert st.mass_layers() == [1, 3]
    junk = [torch.full((size // 4,), 7.0, device="cuda") for _ in range(8)]
    for _ in range(3):
        for x in start:
            st.layers[1].held[x].copy_(start[x])
        for o in outs:
            o.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)) and torch.equal(st.layers[1].held["mass"], masses)
    assert all(bool((j == 7.0).all()) for j in junk) and st.read_error() == 0


@pytest.mark.parametrize("raw", [False, True])
def test_masses_on_another_stream(raw):
    """Masses laid out, gathered and read on a stream that waits while the current one fills the memory that it can get."""
    s = Session(2, 20, seed=3)
    T = 1200
    kv = [s.rand(T, s.Hkv, D) for _ in range(4)]
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    seq = [torch.full_like(pos, b) for b in range(2)]
    ctx, (qs, outs, ks, vs) = i32([T, T]), s.step_inputs()

    def session(st, stream):
        st.keep_mass(stream=stream)
        for b in range(2):
            st.append_prompt(1, kv[2 * b], kv[2 * b + 1], seq[b], pos, stream=stream)
        for _ in range(2):
            st.decode_layer(1, qs[1], ctx, outs[1], ks[1], vs[1], stream=stream)

    session(s.st, None)
    torch.cuda.synchronize()
    want = s.st.layers[1].held["mass"].clone()
    other = Session(2, 20, seed=3).st
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)  # some ten milliseconds
    session(other, stream.cuda_stream if raw else stream)
    junk = [torch.full((want.numel(),), float("nan"), device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    assert len(junk) == 16 and other.read_error() == 0
    assert torch.equal(other.layers[1].held["mass"], want) and torch.equal(other.layers[1].held["ids"], s.st.layers[1].held["ids"])


class Ledger:
    """What every token of a layer has gathered, [(mass, tolerance, additions)] by number, summed in 64 bits: prompts by
    test_gpu_prompt_mass.py's tolerance, steps by test_gpu_mass.py's."""

    def __init__(self, s, l):
        self.s, self.l, self.of = s, l, {}

    def start(self, b, numbers, mass=None, tol=None, additions=0):
        for h in range(self.s.Hkv):
            d = self.of.setdefault((b, h), {})
            for i, p in enumerate(numbers):
                d[p] = [0.0, 0.0, 0] if mass is None else [float(mass[h, i]), float(tol[h, i]), additions]

    def step(self, b, q, ctx, number):
        """A step of queries q [Hq, 128] over the records of slots 0..ctx, the new token's at ctx."""
        s, L = self.s, self.s.st.layers[self.l]
        G = s.Hq // s.Hkv
        x = q.double()
        qt = (x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()) @ s.M[self.l].T
        self.start(b, [number])
        for h in range(s.Hkv):
            k, _ = values(records(L.tensors, b, h, ctx + 1)[1])
            low = k.amin(1, keepdim=True)
            a_k = (k - low) + low.abs() + 1e-3
            want, tol = torch.zeros(ctx + 1, dtype=torch.float64, device="cuda"), torch.zeros(ctx + 1, dtype=torch.float64, device="cuda")
            for g in range(h * G, (h + 1) * G):
                w = torch.softmax(k @ qt[g] * SM, 0)
                d = SM * (a_k @ qt[g].abs()) * (272 * 2.0 ** -24 + 2.0 ** -22)
                want += w
                tol += w * torch.expm1(2 * (d.max() + d) + 2.0 ** -19)
            ids = L.held["ids"][b, h, :ctx + 1].tolist()
            assert ids[ctx] == number
            for p, w, t in zip(ids, want.tolist(), tol.tolist()):
                e = self.of[b, h][p]
                e[0], e[1], e[2] = e[0] + w, e[1] + t, e[2] + G + 1

    def check(self, b, ctx):
        L = self.s.st.layers[self.l]
        for h in range(self.s.Hkv):
            ids, mass = L.held["ids"][b, h, :ctx].tolist(), L.held["mass"][b, h, :ctx].double().tolist()
            assert len(set(ids)) == ctx
            for p, m in zip(ids, mass):
                want, tol, n = self.of[b, h][p]
                assert abs(m - want) <= tol + n * 2.0 ** -24 * want + 1e-30, (b, h, p, m, want, tol)

    def keep(self, b, ctx):
        """The tokens that are left: those of the slots below ctx."""
        for h in range(self.s.Hkv):
            ids = set(self.s.st.layers[self.l].held["ids"][b, h, :ctx].tolist())
            self.of[b, h] = {p: e for p, e in self.of[b, h].items() if p in ids}


@pytest.mark.parametrize("observed_first", [True, False])
@pytest.mark.parametrize("fwht", [False, True])
def test_masses_of_a_session_slot_by_slot(observed_first, fwht):
    """Prompts observed, evicted from, a second turn's prompt behind what is left, steps, eviction again, and a new session in
    a row that has been used. A twin that evicts nothing has every token's record at its own position."""
    B, lens, budget, sinks, recent = 2, [330, 200], 120, 4, 16
    s = Session(B, 8, seed=5)
    st, twin = s.st, Session(B, 8, seed=5).st
    if fwht:
        for x in (st, twin):
            r = np.random.default_rng(9)
            gq, gk = (r.uniform(0.5, 1.5, D).astype(np.float32) for _ in range(2))
            x.set_int4_params(1, 4, gq, gk, prologue="fwht")
        s.M[1] = torch.from_numpy(st.layers[1].R.astype(np.float64) * (gq.astype(np.float64) * gk)[None]).cuda()
    st.keep_mass()
    L, led = st.layers[1], Ledger(s, 1)
    ctx, seen = [0, 0], [0, 0]

    def tell(of, first):
        return i32([first[b] + i for b in range(B) for i in range(of[b])])

    def append(n, **kw):
        """n[b] new tokens in every row."""
        T = sum(n)
        k, v = s.rand(T, s.Hkv, D), s.rand(T, s.Hkv, D)
        row = i32([b for b in range(B) for _ in range(n[b])])
        slots = tell(n, ctx) if ctx != seen else None
        st.append_prompt(1, k, v, row, tell(n, seen), slots=slots, **kw)
        twin.append_prompt(1, k, v, row, tell(n, seen))
        return k

    def evict():
        nonlocal ctx
        before = {x: L.held[x].cpu().numpy() for x in ("ids", "mass")}
        st.evict(i32(ctx), i32(seen), budget, sinks, recent, out := i32([0] * B))
        for b in range(B):
            for h in range(s.Hkv):
                ids, mass = before["ids"][b, h, :ctx[b]], before["mass"][b, h, :ctx[b]]
                top = (ids < sinks) | (ids >= seen[b] - recent)
                order = np.lexsort((np.arange(ctx[b]), -np.where(top, np.inf, mass)))
                left = set(L.held["ids"][b, h, :out.tolist()[b]].tolist())
                assert left == set(ids[order[:budget]].tolist()) and left >= set(range(seen[b] - recent, seen[b])) | set(range(sinks))
        ctx = out.tolist()
        assert ctx == [budget] * B
        for b in range(B):
            led.keep(b, ctx[b])

    def same():
        for b in range(B):
            led.check(b, ctx[b])
            for h in range(s.Hkv):
                ids = L.held["ids"][b, h, :ctx[b]].cpu().numpy()
                mine, _ = records(L.tensors, b, h, ctx[b])
                all_, _ = records(twin.layers[1].tensors, b, h, int(ids.max()) + 1)
                assert np.array_equal(mine, all_[ids])

    def steps(n):
        nonlocal ctx, seen
        for _ in range(n):
            qs, outs, ks, vs = s.step_inputs()
            st.decode_layer(1, qs[1], i32(ctx), outs[1], ks[1], vs[1], positions=i32(seen))
            twin.decode_layer(1, qs[1], i32(seen), outs[0], ks[1], vs[1])
            torch.cuda.synchronize()
            for b in range(B):
                led.step(b, qs[1][b, 0], ctx[b], seen[b])
            ctx, seen = [c + 1 for c in ctx], [c + 1 for c in seen]

    # the prompts, and what their last rows looked at
    q, k = s.rand(sum(lens), s.Hq, D), s.rand(sum(lens), s.Hkv, D)
    cu = i32([0, lens[0], sum(lens)])
    if observed_first:
        st.observe_prompt(1, q, k, cu, 32)
        append(lens)
    else:
        append(lens)
        st.observe_prompt(1, q, k, cu, 32)
    for b, (mass, tol) in enumerate(reference(q, k, lens, 32)):
        led.start(b, range(lens[b]), mass, tol)
    ctx, seen = list(lens), list(lens)
    same()
    evict()
    steps(4)
    total = [sum(e[0] for e in led.of[b, h].values()) for b in range(B) for h in range(s.Hkv)]
    assert min(total) > 0
    same()
    # a second turn: its tokens have gathered nothing yet
    more = [50, 33]
    append(more)
    for b in range(B):
        led.start(b, range(seen[b], seen[b] + more[b]))
    ctx, seen = [c + m for c, m in zip(ctx, more)], [c + m for c, m in zip(seen, more)]
    same()
    steps(5)
    same()
    evict()
    steps(3)
    same()
    # new sessions in both rows, observed by nothing
    ctx, seen = [0, 0], [0, 0]
    led.of.clear()
    n = [150, 130]
    append(n, fresh=True)
    for b in range(B):
        led.start(b, range(n[b]))
    ctx, seen = list(n), list(n)
    same()
    steps(3)
    evict()
    same()
    assert st.read_error() == 0 and twin.read_error() == 0


def test_a_captured_append_starts_masses():
    s = Session(2, 3, seed=6)
    st = s.st
    st.keep_mass()
    held = st.layers[1].held
    k, v = s.rand(40, s.Hkv, D), s.rand(40, s.Hkv, D)
    row, pos, slot = i32([1] * 40), i32(list(range(500, 540))), i32(list(range(70, 110)))
    st.append_prompt(1, k, v, row, pos, slots=slot)  # once eagerly
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.append_prompt(1, k, v, row, pos, slots=slot)
    for turn in range(2):
        held["mass"].fill_(3.0)
        held["ids"].fill_(-5)
        pos.add_(1)
        g.replay()
        torch.cuda.synchronize()
        mass, ids = held["mass"].clone(), held["ids"].clone()
        assert bool((mass[1, :, 70:110] == 0).all()) and torch.equal(ids[1, 2, 70:110], pos)
        mass[1, :, 70:110], ids[1, :, 70:110] = 3.0, -5
        assert bool((mass == 3.0).all()) and bool((ids == -5).all())
    assert st.read_error() == 0


@pytest.mark.parametrize("Hq,Hkv", [(20, 4), (2, 2)])
def test_every_step_gathers_a_row_of_weights_a_query_head(Hq, Hkv):
    """decode_step over all layers, after an eviction of observed prompts: what the heads of a group put out adds up to their
    number, step by step, beside what the prompts' rows had left."""
    B, lens, G = 2, [300, 260], Hq // Hkv
    s = Session(B, 6, n_layers=6, Hq=Hq, Hkv=Hkv, seed=7)
    st = s.st
    st.set_int4_window(3, 100, 7)
    st.keep_mass()
    T = sum(lens)
    row, pos = i32([b for b in range(B) for _ in range(lens[b])]), i32([p for b in range(B) for p in range(lens[b])])
    for l in range(6):
        q, k, v = s.rand(T, Hq, D), s.rand(T, Hkv, D), s.rand(T, Hkv, D)
        keep = torch.ones_like(pos, dtype=torch.bool) if l in st.int4_layers() else pos >= i32(lens)[row.long()] - 100
        if l in st.mass_layers():
            st.observe_prompt(l, q, k, i32([0, lens[0], T]), 32)
        st.append_prompt(l, k[keep].contiguous(), v[keep].contiguous(), row[keep].contiguous(), pos[keep].contiguous())
    st.evict(i32(lens), i32(lens), 200, 4, 16, out := i32([0] * B))
    ctx, seen = out.tolist(), list(lens)

    def sums():
        return torch.stack([torch.stack([st.layers[l].held["mass"][b, :, :ctx[b]].double().sum(-1) for b in range(B)]) for l in st.mass_layers()])

    at = sums()
    assert float(at.min()) > G  # the prompts' rows
    for _ in range(10):
        qs, outs, ks, vs = s.step_inputs()
        st.decode_step(qs, i32(ctx), outs, ks, vs, positions=i32(seen))
        ctx, seen = [c + 1 for c in ctx], [c + 1 for c in seen]
        was, at = at, sums()
        # a row's weights add up to 1 but for the powers of two and the division (2^-19), the stored scores (half a step of
        # values below 32, times ln 2: 2^-20) and the sum below the division (300 half steps); a mass's addition takes half a
        # step of it, and all masses of a head are 32 G + 10 G at most
        assert float((at - was - G).abs().max()) < G * (2.0 ** -19 + 2.0 ** -20 + 300 * 2.0 ** -24) + 42 * G * 2.0 ** -24
    assert st.read_error() == 0
