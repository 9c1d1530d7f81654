"""DecodeStack.commit_tree over more layers of a kind than one commit takes."""

import pytest
import torch

from quantized_kv_cache_fold_gb300 import MAX_CACHES, runner


@pytest.mark.parametrize("n_layers,full_every", [(130, 2), (70, 1), (70, 100), (10, 5)])
def test_every_layer_once_and_the_lengths_once(monkeypatch, n_layers, full_every):
    calls = []
    for name in ("kvq_tree_commit_int4", "kvq_tree_commit_fp8"):
        monkeypatch.setattr(runner, name, lambda layers, *a, ctx_out, stream: calls.append((list(layers), ctx_out, stream)))
    st = runner.DecodeStack(1, 2, 2, 1, 1, n_layers=n_layers, full_every=full_every, ring_capacity=64, window=64, device="cpu")
    st.commit_tree("ctx", "path", "n", "out", stream=5)
    got = [id(x) for layers, _, _ in calls for x in layers]
    want = [id(st.layers[l].cache) for l in st.int4_layers()] + [id(st.layers[l].ring) for l in st.swa_layers()]
    assert got == want and all(len(layers) <= MAX_CACHES and s == 5 for layers, _, s in calls)
    assert [o for _, o, _ in calls] == ["out"] + [None] * (len(calls) - 1)


@pytest.mark.gpu
def test_commit_over_many_layers():
    """70 rings and 70 caches: every layer's records move as one layer's do."""
    st = runner.DecodeStack(2, 2, 1, 1, 3, n_layers=140, full_every=2, ring_capacity=128, window=64)
    g = torch.Generator(device="cuda").manual_seed(1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for L in st.layers:
        data = L.tensors["pages"] if isinstance(L, runner.Int4Layer) else L.tensors["data"]
        data.copy_(torch.randint(0, 256, data.shape, generator=g, device="cuda", dtype=torch.uint8))
    ctx, path, n = i32([60, 100]), i32([[1, 3, 4, 0, 0, 0], [0, 2, 5, 0, 0, 0]]), i32([3, 2])
    before = [{k: v.clone() for k, v in L.tensors.items()} for L in st.layers]
    out = i32([0, 0])
    st.commit_tree(ctx, path, n, out)
    assert out.tolist() == [63, 102] and st.read_error() == 0
    for L, was in zip(st.layers, before):
        kind = isinstance(L, runner.Int4Layer)
        key = "pages" if kind else "data"
        now = L.tensors[key].clone()
        L.tensors[key].copy_(was[key])
        if kind:
            runner.kvq_tree_commit_int4([L.cache], ctx, path, n, st.dev_err)
        else:
            runner.kvq_tree_commit_fp8([L.ring], ctx, path, n, st.dev_err)
        assert torch.equal(now, L.tensors[key]) and not torch.equal(now, was[key])
