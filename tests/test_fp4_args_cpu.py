"""Argument checks of the 4-bit cache's calls, one by one: every pointer has an address of its own, and the call that each
check breaks is one that passes all of them (CPU: nothing is launched, the addresses are never read)."""
import math

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
PASSED = 4    # MLA_ERR_CUDA: past every check, and no GPU to go on with
DECODE = ("q", "kv", "kv_scale", "num_blocks", "table", "max_blocks", "seqlens", "indices", "index_stride", "topk_lens", "B",
          "s_q", "H", "softmax_scale", "causal", "metadata", "parts", "workspace", "workspace_bytes", "out", "lse", "stream")
LISTS = ("indices", "index_stride", "topk_lens")
APPEND = ("c", "c_stride", "k_pe", "pe_stride", "kv", "kv_scale", "num_blocks", "table", "max_blocks", "seqlens", "new_offsets",
          "N", "B", "positions", "pos_stride", "sections", "axes", "interleaved", "theta", "norm", "eps", "stream")
HUGE, TINY, NAN, INF = 2.0 ** 116, 2.0 ** -117, math.nan, math.inf


def _decode(mla, sparse, **more):
    ok = dict(kv_scale=2.0 ** -6, num_blocks=4, max_blocks=2, index_stride=100, B=3, s_q=2, H=16, softmax_scale=0.07, causal=1,
              parts=8, stream=None)
    for i, name in enumerate(("q", "kv", "table", "seqlens", "indices", "topk_lens", "metadata", "workspace", "out", "lse")):
        ok[name] = (i + 1) * FAR
    ok.update(more)
    if "workspace_bytes" not in ok:
        sizes = [ok[n] for n in ("B", "s_q", "H", "parts")]
        ok["workspace_bytes"] = mla.lib().mla_decode_workspace_size(*sizes) if min(sizes) > 0 else 1 << 30
    call = mla.lib().mla_decode_sparse_fp4 if sparse else mla.lib().mla_decode_fp4
    return call(*[ok[n] for n in DECODE if sparse or n not in LISTS])


def _append(mla, **more):
    ok = dict(c_stride=576, pe_stride=64, kv_scale=0.013, num_blocks=4, max_blocks=2, N=6, B=3, pos_stride=6, sections=None, axes=0,
              interleaved=0, theta=10000.0, eps=1e-6, stream=None, positions=None, new_offsets=None)
    for i, name in enumerate(("c", "k_pe", "kv", "table", "seqlens", "norm")):
        ok[name] = (i + 1) * FAR
    ok.update(more)
    return mla.lib().mla_cache_append_fp4(*[ok[n] for n in APPEND])


@pytest.mark.parametrize("sparse", [False, True])
def test_decode_valid_calls_pass_every_check(mla, sparse):
    for more in ({}, dict(kv=FAR + 32), dict(B=16384, s_q=1, H=1, parts=1), dict(s_q=1, H=512), dict(s_q=4, H=128),
                 dict(kv_scale=2.0 ** 115), dict(kv_scale=2.0 ** -116, softmax_scale=1.0), dict(num_blocks=2 ** 25 - 1),
                 dict(index_stride=2 ** 40), dict(max_blocks=2 ** 31 - 1), dict(softmax_scale=3e38)):
        assert _decode(mla, sparse, **more) == PASSED, more


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("name,values,error", [
    ("q", (None, FAR + 8), 1), ("kv", (None, 2 * FAR + 8, 2 * FAR + 16), 1), ("kv_scale", (0.0, -1.0, NAN, INF, HUGE, TINY), 1),
    ("num_blocks", (0, -1), 1), ("num_blocks", (2 ** 25, 2 ** 40, 2 ** 62), 2), ("table", (None, 3 * FAR + 2), 1),
    ("max_blocks", (0, -1), 1), ("seqlens", (None, 4 * FAR + 2), 1), ("B", (0, -1), 1), ("B", (16385,), 2), ("s_q", (0, -1), 1),
    ("s_q", (65,), 2), ("H", (0, -1), 1), ("H", (257, 513), 2), ("softmax_scale", (0.0, -0.1, NAN, INF, 1e-44), 1),
    ("metadata", (None, 7 * FAR + 2), 1), ("parts", (0, -1), 1), ("workspace", (None,), 3), ("workspace", (8 * FAR + 128,), 1),
    ("workspace_bytes", (0, 1 << 10), 3), ("out", (None, 9 * FAR + 8), 1), ("lse", (None, 10 * FAR + 2), 1)])
def test_decode_each_argument_by_itself(mla, sparse, name, values, error):
    for v in values:
        assert _decode(mla, sparse, **{name: v}) == error, v


@pytest.mark.parametrize("sparse", [False, True])
def test_decode_rows_a_cluster_has_no_room_for(mla, sparse):
    """512 query rows of a request at most."""
    for s_q, H in ((1, 1024), (8, 128), (1, 513), (513, 1), (2 ** 30, 2 ** 30)):
        assert _decode(mla, sparse, s_q=s_q, H=H, workspace_bytes=1 << 40) == 2, (s_q, H)


@pytest.mark.parametrize("name,values", [("indices", (None, 5 * FAR + 2)), ("index_stride", (0, -1)),
                                         ("topk_lens", (None, 6 * FAR + 2))])
def test_decode_lists_by_themselves(mla, name, values):
    for v in values:
        assert _decode(mla, True, **{name: v}) == 1, v


@pytest.mark.parametrize("sparse", [False, True])
def test_decode_score_factors_have_to_be_normal(mla, sparse):
    """softmax_scale * kv_scale * log2(e) below 2^-126, or past the largest float32."""
    assert _decode(mla, sparse, kv_scale=2.0 ** -100, softmax_scale=2.0 ** -27) == 1
    assert _decode(mla, sparse, kv_scale=2.0 ** -100, softmax_scale=2.0 ** -26) == PASSED
    assert _decode(mla, sparse, kv_scale=2.0 ** 100, softmax_scale=2.0 ** 28) == 1
    assert _decode(mla, sparse, kv_scale=2.0 ** 100, softmax_scale=2.0 ** 27) == PASSED


def test_append_valid_calls_pass_every_check(mla):
    for more in ({}, dict(norm=None, eps=NAN), dict(eps=0.0), dict(N=5, new_offsets=7 * FAR), dict(c_stride=512),
                 dict(kv_scale=2.0 ** 115), dict(kv_scale=2.0 ** -116)):
        assert _append(mla, **more) == PASSED, more


@pytest.mark.parametrize("name,values,error", [
    ("c", (None, FAR + 8), 1), ("c_stride", (504, 513, -576), 1), ("k_pe", (None, 2 * FAR + 8), 1), ("pe_stride", (56, 65), 1),
    ("kv", (None, 3 * FAR + 8), 1), ("kv_scale", (0.0, -1.0, NAN, INF, HUGE, TINY), 1), ("num_blocks", (0,), 1),
    ("num_blocks", (2 ** 26,), 2), ("table", (None, 4 * FAR + 2), 1), ("max_blocks", (0,), 1), ("seqlens", (None, 5 * FAR + 2), 1),
    ("new_offsets", (7 * FAR + 2,), 1), ("N", (0, 5), 1), ("B", (0,), 1), ("B", (16385,), 1), ("positions", (7 * FAR + 2,), 1),
    ("positions", (7 * FAR,), 1),     # (no sections to turn by)
    ("norm", (6 * FAR + 8,), 1), ("eps", (-1e-6, NAN, INF), 1)])
def test_append_each_argument_by_itself(mla, name, values, error):
    for v in values:
        assert _append(mla, **{name: v}) == error, v


def test_decode_step_takes_4_bits_with_a_scale_only(mla):
    n = torch.ones(2, dtype=torch.int32)
    for bits, scale in ((4, None), (8, None), (3, 0.5), (16, 0.5)):
        with pytest.raises(ValueError, match="kv_bits"):
            mla.DecodeStep(2, 1, 16, n, False, 0.1, kv_scale=scale, kv_bits=bits)
