"""Host-side refusals of kvq_mass_start: no GPU is needed, nothing is launched for a bad argument."""

import ctypes

import pytest

import quantized_kv_cache_fold_gb300 as kvq

INVALID = 1


def start(m=None, **over):
    d = dict(mass=0x1000000, ids=0x2000000, num_seqs=4, num_kv_heads=4, max_tokens=512)
    d.update(m or {})
    a = dict(T=100, seq=0x90000, slots=0x98000, num=0xA0000, fresh=0, err=0xC0000)
    a.update(over)
    return kvq.lib.kvq_mass_start(ctypes.byref(kvq.TokenMass(**d)), a["T"], a["seq"], a["slots"], a["num"], a["fresh"], a["err"], None)


@pytest.mark.parametrize("over", [
    dict(T=-1), dict(T=(1 << 28) + 1), dict(seq=0), dict(slots=0), dict(num=0), dict(err=0), dict(seq=0x1000000 - 396), dict(slots=0x1000000 + 32764),
    dict(num=0x2000000), dict(seq=0x2000000 + 32764)])
def test_refusals(over):
    assert start(**over) == INVALID


@pytest.mark.parametrize("m", [
    dict(mass=0), dict(ids=0), dict(mass=0x1000008), dict(ids=0x2000002), dict(num_seqs=0), dict(num_kv_heads=0), dict(max_tokens=0),
    dict(max_tokens=511), dict(ids=0x1000000 + 4096)])
@pytest.mark.parametrize("T", [0, 100])
def test_descriptors(m, T):
    if "ids" in m and m["ids"] == 0x1000000 + 4096 and T == 0:
        return  # nothing is written
    assert start(m, T=T) == INVALID


def test_nothing_to_do():
    assert start(T=0) == 0 and start(T=0, seq=0, slots=0, num=0, err=0) == 0
    assert kvq.lib.kvq_mass_start(None, 1, 1, 1, 1, 0, 1, None) == INVALID
