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
