"""kvq_mass_start against a plain model: exact."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_fold_gb300 as kvq

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x, np.int32).reshape(-1), device="cuda")


def case(T, B, Hkv, N, seed, spread=False):
    """Used rows, and T tokens at slots of their own (a third of them with the number that their slot has already)."""
    r = np.random.default_rng(seed)
    held = {"mass": torch.from_numpy(r.uniform(1, 2, (B, Hkv, N)).astype(np.float32)).cuda(),
            "ids": torch.from_numpy(r.integers(0, 5000, (B, Hkv, N)).astype(np.int32)).cuda()}
    at = r.choice(B * N, T, replace=False) if spread else np.arange(B * N)[max(0, B * N - T - 3):][:T]
    seq, slot = (at // N).astype(np.int32), (at % N).astype(np.int32)
    num = r.integers(0, 5000, T).astype(np.int32)
    same = r.uniform(size=T) < 0.33
    ids = held["ids"].cpu().numpy()
    num[same] = ids[seq, 0, slot][same]
    return held, seq, slot, num


def model(held, seq, slot, num, fresh):
    mass, ids = held["mass"].cpu().numpy().copy(), held["ids"].cpu().numpy().copy()
    B, Hkv, N = mass.shape
    for q, j, n in zip(seq, slot, num):
        if 0 <= q < B and 0 <= j < N:
            for h in range(Hkv):
                if fresh or ids[q, h, j] != n:
                    mass[q, h, j], ids[q, h, j] = 0.0, n
    return mass, ids


def call(held, seq, slot, num, fresh, want_err=0, stream=None):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    kvq.kvq_mass_start(kvq.token_mass(held["mass"], held["ids"]), i32(seq), i32(slot), i32(num), err, fresh=fresh, stream=stream)
    torch.cuda.synchronize()
    assert err.item() == want_err


def same(held, want):
    assert np.array_equal(held["mass"].cpu().numpy(), want[0]) and np.array_equal(held["ids"].cpu().numpy(), want[1])


@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("T,B,Hkv,N", [(0, 2, 2, 64), (1, 1, 1, 64), (63, 3, 4, 64), (255, 2, 1, 192), (256, 5, 8, 192), (257, 2, 3, 196),
                                       (5000, 40, 2, 320)])
def test_sizes(T, B, Hkv, N, spread, fresh):
    held, seq, slot, num = case(T, B, Hkv, N, T + fresh, spread)
    want = model(held, seq, slot, num, fresh)
    call(held, seq, slot, num, fresh)
    same(held, want)


@pytest.mark.parametrize("fresh", [False, True])
def test_tokens_without_a_place(fresh):
    held, seq, slot, num = case(60, 3, 2, 64, 5, True)
    seq[[3, 9]], slot[[20, 21, 22]] = (-1, 3), (-1, 64, 1 << 30)
    seq[40], slot[41] = -2 ** 31, -2 ** 31
    want = model(held, seq, slot, num, fresh)
    call(held, seq, slot, num, fresh, want_err=kvq.DEVERR_POS)
    same(held, want)


def test_masses_that_are_not_finite():
    held, seq, slot, num = case(50, 2, 2, 64, 6, True)
    held["mass"].fill_(float("nan"))
    call(held, seq, slot, num, True)
    mass = held["mass"].cpu().numpy()
    assert (mass[seq, :, slot] == 0).all() and np.isnan(mass).sum() == mass.size - 100


def test_places_past_32_bits():
    """Masses of 2^31 slots and more."""
    B, Hkv, N = 3, 4, 1 << 28
    held = {"mass": torch.ones(B, Hkv, N, device="cuda"), "ids": torch.zeros(B, Hkv, N, dtype=torch.int32, device="cuda")}
    seq, slot = [0, 1, 2, 2, 2], [0, N - 1, 7, N // 2, N - 1]
    call(held, seq, slot, [11, 12, 13, 14, 15], False)
    assert int((held["mass"] == 0).sum()) == 20 and int((held["ids"] != 0).sum()) == 20
    for q, j, n in zip(seq, slot, range(11, 16)):
        assert bool((held["mass"][q, :, j] == 0).all()) and bool((held["ids"][q, :, j] == n).all())


def test_two_streams_and_what_follows():
    """The masses that a step adds to are those that the call behind it leaves, without a wait between."""
    from test_gpu_mass import MassCase
    got = []
    for wait in (True, False):
        c = MassCase([100, 20, 300], 20, 4, seed=7)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        row = i32([0] * 50 + [1] * 20 + [2] * 100)
        slot = i32(list(range(50, 100)) + list(range(20)) + list(range(200, 300)))
        outs = [torch.zeros(3, 20, 128, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        for o in outs:
            kvq.kvq_mass_attn_int4(c.cache, c.mass, c.Mq, c.Mk, c.q[:, 0], c.ctx_t, c.pos, o, c.ws, c.err, k_new=c.k_new[:, 0], v_new=c.v_new[:, 0])
            if wait:
                torch.cuda.synchronize()
            kvq.kvq_mass_start(c.mass, row, slot, slot, err, fresh=True)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert err.item() == 0 and c.err.item() == 0
        got.append(outs + [c.held["mass"], c.held["ids"]])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    held, seq, slot, num = case(4000, 30, 4, 320, 8, True)
    twin = {k: v.clone() for k, v in held.items()}
    want = model(held, seq, slot, num, False)
    streams = [torch.cuda.Stream() for _ in range(2)]
    err, lists = torch.zeros(1, dtype=torch.int32, device="cuda"), [i32(x) for x in (seq, slot, num)]
    torch.cuda.synchronize()
    for h, s in zip((held, twin), streams):
        kvq.kvq_mass_start(kvq.token_mass(h["mass"], h["ids"]), *lists, err, stream=s)
    torch.cuda.synchronize()
    same(held, want)
    same(twin, want)
    assert err.item() == 0


def test_tensors_that_do_not_fit():
    held, mass = kvq.alloc_token_mass(2, 2, 1)
    err, x = torch.zeros(1, dtype=torch.int32, device="cuda"), i32([0, 1, 1])
    for bad in ((x.long(), x, x), (x, x[:2], x), (x, x, x.cpu()), (x, x, x.float()), (i32([0] * 6)[::2], x, x), (x.cpu(), x, x)):
        with pytest.raises(ValueError):
            kvq.kvq_mass_start(mass, *bad, err)
    with pytest.raises(ValueError):
        kvq.kvq_mass_start(mass, x, x, x, err.float())
