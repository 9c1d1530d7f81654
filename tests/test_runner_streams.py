"""The layer stack's own workspaces belong to the stream that the calls run on."""

import contextlib

import pytest
import torch

from quantized_kv_cache_fold_gb300 import runner


@pytest.mark.parametrize("stream", [None, "a stream", 77])
def test_workspaces_are_allocated_in_the_order_of_the_calls_stream(monkeypatch, stream):
    current, seen = [None], []

    @contextlib.contextmanager
    def on(s):
        was, current[0] = current[0], s
        yield
        current[0] = was

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("external", handle))
    for name in ("alloc_tree_workspace", "alloc_prompt_workspace"):
        monkeypatch.setattr(runner, name, lambda *a: seen.append(current[0]) or torch.empty(1))
    for name in ("kvq_tree_attn_int4", "kvq_tree_attn_fp8_swa", "kvq_prompt_attn"):
        monkeypatch.setattr(runner, name, lambda *a, **k: seen.append(k["stream"]))
    st = runner.DecodeStack(1, 2, 2, 1, 2, n_layers=2, full_every=2, device="cpu")
    q = torch.empty(1, 3, 2, 128)
    st.tree_step([q, q], None, None, [q, q], stream=stream)
    st.prompt_layer(0, q[0], q[0], q[0], torch.zeros(2, dtype=torch.int32), q[0], stream=stream)
    own = ("external", 77) if stream == 77 else stream
    assert seen == [own, stream, stream, own, stream]


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
def test_tree_step_on_another_stream_beside_other_work(raw):
    """Memory that the current stream takes and fills while the steps wait on theirs is not the workspace of any."""
    B, N, Hq, Hkv = 2, 16, 20, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    st = runner.DecodeStack(B, Hq, Hkv, 1, 40, n_layers=2, full_every=2, window=64, ring_capacity=128, swa_k_scale=6 / 448,
                            swa_v_scale=6 / 448)
    ones = torch.ones(128).numpy()
    st.set_int4_params(1, 4, ones, ones)
    T = 2000
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    for b in range(B):
        st.append_prompt(1, rand(T, Hkv, 128), rand(T, Hkv, 128), torch.full_like(pos, b), pos)
        st.append_prompt(0, rand(100, Hkv, 128), rand(100, Hkv, 128), torch.full_like(pos[:100], b), pos[T - 100:])
    ctx = torch.full((B,), T, dtype=torch.int32, device="cuda")
    mask = torch.tensor([[(1 << (i + 1)) - 1 for i in range(N)]] * B, device="cuda")
    qs, ks, vs = ([rand(B, N, h, 128) for _ in range(2)] for h in (Hq, Hkv, Hkv))

    def outs():
        return [torch.full((B, N, Hq, 128), 9.0, device="cuda") for _ in range(2)]

    want, steps = outs(), [outs() for _ in range(4)]
    st.tree_step(qs, ctx, mask, want, ks, vs)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # some ten milliseconds
    for o in steps:
        st.tree_step(qs, ctx, mask, o, ks, vs, stream=s.cuda_stream if raw else s)
    size = runner.alloc_tree_workspace(B, N, Hq, Hkv).numel()
    junk = [torch.full((size // 4,), float("nan"), device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert st.read_error() == 0 and len(junk) == 8
    for o in steps:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
