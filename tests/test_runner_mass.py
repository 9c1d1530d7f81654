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


@pytest.mark.parametrize("call", ["append_prompt", "append_int4"])
@pytest.mark.parametrize("stream", [None, 77])
@pytest.mark.parametrize("slots", [None, [100, 101, 5]])
@pytest.mark.parametrize("fresh,observed,want", [(None, False, True), (None, True, False), (True, True, True), (False, False, False)])
def test_masses_of_appended_tokens(fake, monkeypatch, call, stream, slots, fresh, observed, want):
    """Behind the records, on their stream, at their slots, with the tokens' numbers."""
    calls = []
    monkeypatch.setattr(runner, "kvq_rotate_quant_append", lambda c, M, k, v, seq, pos, err, stream, fwht: calls.append((seq, pos, stream)))
    monkeypatch.setattr(runner, "kvq_mass_start", lambda m, seq, slot, num, err, fresh, stream: calls.append((m, seq, slot, num, err, fresh, stream)))
    st = stack()
    st.keep_mass([1])
    st.layers[1].observed = observed
    seq, pos = (torch.tensor(x, dtype=torch.int32) for x in ([0, 0, 2, 1], [120, 121, 122, 123]))
    at = pos if slots is None else torch.tensor(slots + [6], dtype=torch.int32)
    k = torch.zeros(3, 2, 128)  # (lists may be longer than the tokens)
    getattr(st, call)(1, k, k, seq, pos, stream=stream, slots=None if slots is None else at, fresh=fresh)
    (seq1, to, on), (mass, seq2, slot, num, err, how, on2) = calls
    assert seq1 is seq and to is at and on == on2 == stream and mass is st.layers[1].mass and err is st.dev_err and how is want
    assert [x.tolist() for x in (seq2, slot, num)] == [x[:3].tolist() for x in (seq, at, pos)]


def test_prompts_that_are_observed(fake, monkeypatch):
    monkeypatch.setattr(runner, "kvq_prompt_mass", lambda *a, **k: None)
    monkeypatch.setattr(runner, "alloc_prompt_mass_workspace", lambda *a: None)
    st = stack()
    st.keep_mass()
    q = torch.zeros(3, 4, 128)
    st.observe_prompt(1, q, q[:, :2], torch.zeros(2, dtype=torch.int32), 4)
    assert [st.layers[l].observed for l in st.int4_layers()] == [True, False]


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
