"""Prompt, tree and commit through the layer stack: a stack that verified a draft tree and kept one branch
decodes the next token bit for bit as one to which the same tokens were appended in order."""

import numpy as np
import pytest
import torch

from quantized_kv_cache_fold_gb300.runner import DecodeStack

pytestmark = pytest.mark.gpu
D = 128


def test_stack_prompt_tree_commit_decode():
    B, Hq, Hkv, N, n_layers = 2, 20, 4, 12, 4
    lens = [130, 77]
    rng = np.random.default_rng(1)
    g = torch.Generator(device="cuda").manual_seed(1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731

    def stack():
        st = DecodeStack(B, Hq, Hkv, 1, 4, n_layers=n_layers, full_every=2, window=64, ring_capacity=128,
                         swa_k_scale=6 / 448, swa_v_scale=6 / 448)
        for l in st.int4_layers():
            r = np.random.default_rng(l)
            st.set_int4_params(l, l + 3, *(r.uniform(0.5, 1.5, D).astype(np.float32) for _ in range(2)))
        return st

    trees, plain = stack(), stack()
    T = sum(lens)
    cu = i32([0, lens[0], T])
    seq = i32([b for b in range(B) for _ in range(lens[b])])
    pos = i32([p for b in range(B) for p in range(lens[b])])
    late = torch.tensor([p >= lens[b] - 100 for b in range(B) for p in range(lens[b])], device="cuda")
    kv = [(rand(T, Hkv, D), rand(T, Hkv, D)) for _ in range(n_layers)]
    for l in range(n_layers):
        k, v = kv[l]
        q, out = rand(T, Hq, D), torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        trees.prompt_layer(l, q, k, v, cu, out)
        assert bool(torch.isfinite(out).all())
        keep = torch.ones_like(late) if l in trees.int4_layers() else late
        for st in (trees, plain):
            st.append_prompt(l, k[keep].contiguous(), v[keep].contiguous(), seq[keep].contiguous(), pos[keep].contiguous())
    masks = []
    for _ in range(B):
        m = []
        for i in range(N):
            p = int(rng.integers(-1, i)) if i else -1
            m.append((1 << i) | (m[p] if p >= 0 else 0))
        masks.append(m)
    new = [(rand(B, N, Hkv, D), rand(B, N, Hkv, D)) for _ in range(n_layers)]
    outs = [torch.empty(B, N, Hq, D, dtype=torch.float32, device="cuda") for _ in range(n_layers)]
    trees.tree_step([rand(B, N, Hq, D) for _ in range(n_layers)], i32(lens), torch.tensor(masks, device="cuda"), outs,
                    [x[0] for x in new], [x[1] for x in new])
    assert all(bool(torch.isfinite(o).all()) for o in outs)
    acc = [4, 6]
    path = [sorted(rng.choice(N, a, replace=False).tolist()) + [0] * (N - a) for a in acc]
    ctx = i32([0] * B)
    trees.commit_tree(i32(lens), i32(path), i32(acc), ctx)
    assert ctx.tolist() == [n + a for n, a in zip(lens, acc)]
    for l in range(n_layers):
        for b in range(B):
            pick = torch.tensor(path[b][:acc[b]], device="cuda")
            plain.append_prompt(l, new[l][0][b, pick].contiguous(), new[l][1][b, pick].contiguous(), i32([b] * acc[b]),
                                i32(list(range(lens[b], lens[b] + acc[b]))))
    qs, nk = [rand(B, 1, Hq, D) for _ in range(n_layers)], [(rand(B, 1, Hkv, D), rand(B, 1, Hkv, D)) for _ in range(n_layers)]
    got = []
    for st in (trees, plain):
        o = [torch.empty(B, 1, Hq, D, dtype=torch.float32, device="cuda") for _ in range(n_layers)]
        st.decode_step(qs, ctx, o, [x[0] for x in nk], [x[1] for x in nk])
        torch.cuda.synchronize()
        assert st.read_error() == 0
        got.append(o)
    assert all(torch.equal(a, b) for a, b in zip(*got))
