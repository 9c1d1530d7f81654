"""Masses that the layer stack keeps, over a session's calls."""

import numpy as np
import pytest
import torch

from quantized_kv_cache_fold_gb300.runner import DecodeStack

pytestmark = pytest.mark.gpu
D = 128


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
