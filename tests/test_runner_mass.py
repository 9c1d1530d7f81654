"""What DecodeStack does on the host for layers that keep mass: memory taken once and in the order of the steps' stream, calls
refused that would part the records from their masses, and the masses of tokens that are appended."""

import contextlib

import pytest
import torch

from quantized_kv_cache_fold_gb300 import runner


@pytest.fixture
def fake(monkeypatch):
    """Allocations on the CPU: (stream, what, tensor) of each; and the streams that work was put on."""
    current, made = [None], []

    @contextlib.contextmanager
    def on(s):
        was, current[0] = current[0], s
        yield
        current[0] = was

    def token_mass(B, Hkv, pages, device):
        held = {"mass": torch.zeros(B, Hkv, 64 * pages), "ids": torch.arange(64 * pages, dtype=torch.int32).repeat(B, Hkv, 1)}
        made.append((current[0], "masses", held["mass"]))
        return held, object()

    def workspace(B, Hq, Hkv, tokens, device):
        made.append((current[0], "workspace", torch.empty(16)))
        return made[-1][2]

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("external", handle))
    monkeypatch.setattr(runner, "alloc_token_mass", token_mass)
    monkeypatch.setattr(runner, "alloc_mass_workspace", workspace)
    return made


def stack(B=3, Hkv=2, pages=2, n_layers=4, full_every=2):
    return runner.DecodeStack(B, 4, Hkv, 1, pages, n_layers=n_layers, full_every=full_every, ring_capacity=64, window=64, device="cpu")


@pytest.mark.parametrize("stream", [None, "a stream", 77])
def test_memory_is_taken_once_and_in_the_order_of_the_stream(fake, stream):
    st = stack(n_layers=6)
    st.keep_mass([1], stream=stream)
    first = st.mass_workspace
    st.keep_mass([1, 5], stream=stream)
    st.keep_mass(stream=stream)
    st.keep_mass()
    assert st.mass_workspace is first  # a step in flight, or a captured one, still writes there
    own = ("external", 77) if stream == 77 else stream
    assert [(s, what) for s, what, _ in fake] == [(own, "workspace"), (own, "masses"), (own, "masses"), (own, "masses")]
    assert st.mass_layers() == [1, 3, 5]


def appended(st, monkeypatch, seq, pos, slots=None, fresh=None, call="append_prompt"):
    """What the layer's slots hold after an append, and the slots that its records went to."""
    to = []
    monkeypatch.setattr(runner, "kvq_rotate_quant_append", lambda c, M, k, v, s, p, err, stream, fwht: to.append((s.tolist(), p.tolist(), stream)))
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32)  # noqa: E731
    k = torch.zeros(len(seq), 2, 128)
    getattr(st, call)(1, k, k, i32(seq), i32(pos), slots=i32(slots), fresh=fresh)
    assert to == [(seq, pos if slots is None else slots, None)]
    return st.layers[1].held


@pytest.mark.parametrize("call", ["append_prompt", "append_int4"])
@pytest.mark.parametrize("slots,fresh,observed", [
    ([100, 101, 5], None, False), ([100, 101, 5], None, True), ([100, 101, 5], True, True), ([100, 101, 5], False, False),
    (None, None, False), (None, None, True), (None, True, True), (None, False, False)])
def test_masses_of_appended_tokens(fake, monkeypatch, call, slots, fresh, observed):
    """Rows that another session has used: numbers in another order, and masses, at every slot."""
    st = stack()
    st.keep_mass([1])
    L = st.layers[1]
    held = L.held
    g = torch.Generator().manual_seed(1)
    held["mass"].copy_(torch.rand(held["mass"].shape, generator=g) + 1)
    held["ids"].copy_(torch.randint(1000, held["ids"].shape, generator=g, dtype=torch.int32))
    seq, pos = [0, 0, 2], [120, 121, 122]
    held["ids"][0, :, 121] = 121  # one slot holds its token's number already (as a call that observes the prompt leaves it)
    held["ids"][2, 1, 5] = 122
    L.observed = observed
    mass, ids = held["mass"].clone(), held["ids"].clone()
    appended(st, monkeypatch, seq, pos, slots, fresh, call)
    for b, p, s in zip(seq, pos, slots or pos):
        for h in range(2):
            if not (not observed if fresh is None else fresh) and ids[b, h, s] == p:
                continue
            mass[b, h, s], ids[b, h, s] = 0.0, p
    assert torch.equal(held["mass"], mass) and torch.equal(held["ids"], ids)


def test_tokens_without_a_place(fake, monkeypatch):
    """The append flags them; no slot's mass changes for them."""
    st = stack()
    st.keep_mass([1])
    held = st.layers[1].held
    held["mass"].fill_(2.0)
    mass, ids = held["mass"].clone(), held["ids"].clone()
    appended(st, monkeypatch, [-1, 3, 0, 1], [5, 5, -2, 128])
    assert torch.equal(held["mass"], mass) and torch.equal(held["ids"], ids)
    appended(st, monkeypatch, [7, 1, 2, 0], [500, 6, 1 << 30, 9], [3, 6, 128, -1])
    mass[1, :, 6] = 0.0
    ids[1, :, 6] = 6
    assert torch.equal(held["mass"], mass) and torch.equal(held["ids"], ids)
    appended(st, monkeypatch, [], [])
    assert torch.equal(held["mass"], mass)


def test_layers_without_mass_append_at_the_positions(monkeypatch):
    st = stack()
    to = []
    monkeypatch.setattr(runner, "kvq_rotate_quant_append", lambda c, M, k, v, s, p, err, stream, fwht: to.append(p))
    monkeypatch.setattr(runner, "kvq_fp8_append", lambda r, k, v, s, p, *a, stream: to.append(p))
    k = torch.zeros(1, 2, 128)
    for l in range(2):
        st.append_prompt(l, k, k, "seq", "positions", slots="slots", fresh=True)
    assert to == ["positions"] * 2


def test_commit_is_refused_where_a_layer_keeps_mass(fake, monkeypatch):
    """Records would move without their masses, and by lengths that are not the layer's after an eviction."""
    calls = []
    for name in ("kvq_tree_commit_int4", "kvq_tree_commit_fp8"):
        monkeypatch.setattr(runner, name, lambda *a, **k: calls.append(a))
    st = stack()
    st.set_int4_window(1, 64, 4)
    st.keep_mass([3])
    with pytest.raises(ValueError):
        st.commit_tree(None, None, None, None)
    assert not calls
    windows = stack()  # (verify blocks go through windows, and their records lie at their positions)
    windows.set_int4_window(1, 64, 4)
    windows.commit_tree("ctx", "path", "n", "out")
    assert len(calls) == 2
