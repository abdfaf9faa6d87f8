"""Argument checks of eviction that its arguments reach one by one: every pointer has an address of its own, and the call
that each check breaks is one that passes all of them (CPU: nothing is launched, the addresses are never read)."""
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
def test_evict_arrival_rows_narrower_than_the_weights_rows(mla, fp8):
    """Rows of arrival that are shorter than the pages' slots and the weights' rows bound the lengths; what lies right
    behind the last of them is none of the call's inputs."""
    call = _call(mla, fp8)
    narrow = dict(B=2, w_stride=256, max_blocks=4, a_stride=64, budget=64, sink=0, recent=0, width=256)
    end = dict(zip(NAMES, _args()))["arrival"] + 2 * 64 * 4
    for out in ("new_seqlens", "kept", "weights_out", "arrival_out"):
        assert call(*_args(**narrow, **{out: end})) == PASSED, out
        assert call(*_args(**narrow, **{out: end - 4})) == 1, out
