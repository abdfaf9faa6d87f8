"""Argument checks of eviction that its arguments reach one by one: every pointer has an address of its own, and the call
that each check breaks is one that passes all of them (CPU: nothing is launched, the addresses are never read)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def mla():
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where nothing can be launched")
    from mla_absorbed_decode_gb300 import build_lib
    build_lib.build()
    import mla_absorbed_decode_gb300 as m
    m.lib()
    return m


FAR = 1 << 40
NAMES = ("kv", "num_blocks", "table", "max_blocks", "seqlens", "B", "weights", "w_stride", "arrival", "a_stride", "budget",
         "sink", "recent", "new_seqlens", "kept", "weights_out", "arrival_out", "width", "stream")
POINTERS = ("kv", "table", "seqlens", "weights", "arrival", "new_seqlens", "kept", "weights_out", "arrival_out")
PASSED = 4    # MLA_ERR_CUDA: past every check, and no GPU to go on with


def _args(**more):
    ok = dict(num_blocks=4, max_blocks=2, B=3, w_stride=128, a_stride=128, budget=100, sink=4, recent=16, width=100,
              stream=None)
    ok.update({name: (i + 1) * FAR for i, name in enumerate(POINTERS)})
    ok.update(more)
    return [ok[n] for n in NAMES]


def _call(mla, fp8):
    return mla.lib().mla_evict_fp8 if fp8 else mla.lib().mla_evict


@pytest.mark.parametrize("fp8", [False, True])
def test_evict_a_valid_call_passes_every_check(mla, fp8):
    call = _call(mla, fp8)
    ok = dict(zip(NAMES, _args()))
    assert call(*_args()) == PASSED
    for more in (dict(arrival=None, a_stride=0), dict(arrival_out=None), dict(new_seqlens=ok["seqlens"]), dict(width=128),
                 dict(budget=20), dict(sink=84), dict(kept=ok["weights"] + 4 * 384), dict(weights_out=ok["kept"] + 1200),
                 dict(new_seqlens=ok["seqlens"] + 12), dict(new_seqlens=ok["table"] - 12)):
        assert call(*_args(**more)) == PASSED, more


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name,values", [
    ("kv", (None, FAR + 8)), ("num_blocks", (0, -1)), ("table", (None, 2 * FAR + 2)), ("max_blocks", (0,)),
    ("seqlens", (None, 3 * FAR + 2)), ("B", (0,)), ("weights", (None, 4 * FAR + 2)), ("w_stride", (0,)),
    ("arrival", (5 * FAR + 2,)), ("a_stride", (0,)), ("budget", (0, -1, 19)), ("sink", (-1, 85)),
    ("recent", (-1, 97, 2 ** 31 - 1)), ("new_seqlens", (None, 6 * FAR + 2)), ("kept", (None, 7 * FAR + 2)),
    ("weights_out", (None, 8 * FAR + 2)), ("arrival_out", (9 * FAR + 2,)), ("width", (99, 0))])
def test_evict_each_argument_by_itself(mla, fp8, name, values):
    for v in values:
        assert _call(mla, fp8)(*_args(**{name: v})) == 1, v


@pytest.mark.parametrize("fp8", [False, True])
def test_evict_each_overlap_by_itself(mla, fp8):
    call = _call(mla, fp8)
    at = {n: (i + 1) * FAR for i, n in enumerate(POINTERS)}
    sizes = dict(table=24, seqlens=12, weights=1536, arrival=1536, new_seqlens=12, kept=1200, weights_out=1200,
                 arrival_out=1200)
    outs = ("new_seqlens", "kept", "weights_out", "arrival_out")
    for out in outs:
        for other in sizes:
            if other == out:
                continue
            first, last = at[other] - sizes[out] + 4, at[other] + sizes[other] - 4     # one element over either end
            for where in (first, last):
                assert call(*_args(**{out: where})) == 1, (out, other, hex(where))
            for where in (first - 4, last + 4):                                          # right beside it
                assert call(*_args(**{out: where})) == PASSED, (out, other, hex(where))


@pytest.mark.parametrize("fp8", [False, True])
def test_evict_arrival_rows_narrower_than_the_weights_rows(mla, fp8):
    """Rows of arrival that are shorter than the pages' slots and the weights' rows bound the lengths; what lies right
    behind the last of them is none of the call's inputs."""
    call = _call(mla, fp8)
    narrow = dict(B=2, w_stride=256, max_blocks=4, a_stride=64, budget=64, sink=0, recent=0, width=256)
    end = dict(zip(NAMES, _args()))["arrival"] + 2 * 64 * 4
    for out in ("new_seqlens", "kept", "weights_out", "arrival_out"):
        assert call(*_args(**narrow, **{out: end})) == PASSED, out
        assert call(*_args(**narrow, **{out: end - 4})) == 1, out


@pytest.mark.parametrize("fp8", [False, True])
def test_evict_limits(mla, fp8):
    call = _call(mla, fp8)
    for more in (dict(num_blocks=1 << 25), dict(B=16385),
                 dict(max_blocks=4097, w_stride=262208, arrival=None, a_stride=0, budget=100, width=100)):
        assert call(*_args(**more)) == 2, more
    assert call(*_args(max_blocks=4096, w_stride=262208, arrival=None, a_stride=0)) == PASSED


def test_the_other_calls_pass_their_checks(mla):
    """The calls that test_cache_abi_cpu.py breaks argument by argument are valid ones."""
    L, A, sec = mla.lib(), 0x10000, (ctypes.c_int * 3)(16, 8, 8)
    one = (ctypes.c_int * 1)(32)
    assert L.mla_rope_axes(A, 128, 64, 2 * A, 128, 64, A, 4, sec, 3, 0, 10000.0, 0, 4, 2, None) == PASSED
    for fp8 in (False, True):
        scale = [1.0] if fp8 else []
        append = [A, 576, A + 1024, 576, 2 * A] + scale + [4, A, 2, A, None, 6, 3, A, 6, one, 1, 0, 10000.0, None]
        weights = [A, A, A] + scale + [4, A, 2, A, 3, 1, 16, 0.1, 0, A, 128, None]
        assert (L.mla_cache_append_fp8 if fp8 else L.mla_cache_append)(*append) == PASSED
        assert (L.mla_attn_weights_fp8 if fp8 else L.mla_attn_weights)(*weights) == PASSED
