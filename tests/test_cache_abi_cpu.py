"""Argument checks of the latent-cache operators: on the host, before any launch (CPU)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def mla():
    from mla_absorbed_decode_gb300 import build_lib
    build_lib.build()
    import mla_absorbed_decode_gb300 as m
    m.lib()
    return m


A = 0x10000   # 16-byte aligned, never dereferenced: every case returns before any launch


def _sections(*v):
    return (ctypes.c_int * len(v))(*v)


def _broken(call, ok, status, **by_index):
    for i, values in by_index.items():
        for v in values:
            bad = list(ok)
            bad[int(i[1:])] = v
            assert call(*bad) == status, (i, v)


def test_rope_axes_checks(mla):
    L = mla.lib()
    # (x, x_row, x_head, out, out_row, out_head, positions, pos_stride, sections, axes, interleaved, theta, inverse,
    #  N, H, stream)
    ok = [A, 128, 64, 2 * A, 128, 64, A, 4, _sections(16, 8, 8), 3, 0, 10000.0, 0, 4, 2, None]
    _broken(L.mla_rope_axes, ok, 1, _0=(None, A + 8), _3=(None, A + 2), _6=(None, A + 1), _7=(3,), _8=(None,),
            _9=(0, 5, 2), _11=(1.0, 0.0, float("nan"), float("inf")), _13=(0, -1), _14=(0,))
    _broken(L.mla_rope_axes, ok, 1, _1=(132, -128), _2=(60, -64), _4=(100, 64), _5=(32, 0, 63))   # overlapping rows of out
    _broken(L.mla_rope_axes, ok, 1, _8=(_sections(16, 8, 9), _sections(33, -1, 0), _sections(0, 0, 0)))


@pytest.mark.parametrize("fp8", [False, True])
def test_cache_append_checks(mla, fp8):
    L = mla.lib()
    call = L.mla_cache_append_fp8 if fp8 else L.mla_cache_append
    # (c, c_row, k_pe, pe_row, kv, [scale], num_blocks, table, max_blocks, seqlens, offsets, N, B, positions, pos_stride,
    #  sections, axes, interleaved, theta, stream)
    ok = [A, 576, A + 1024, 576, 2 * A] + ([1.0] if fp8 else []) + \
        [4, A, 2, A, None, 6, 3, A, 6, _sections(32), 1, 0, 10000.0, None]
    s = 1 if fp8 else 0
    _broken(call, ok, 1, _0=(None, A + 8), _1=(504, 580), _2=(None, A + 4), _3=(56, 70), _4=(None, A + 8))
    _broken(call, ok, 1, **{f"_{5 + s}": (0,), f"_{6 + s}": (None, A + 2), f"_{7 + s}": (0,), f"_{8 + s}": (None, A + 1),
                            f"_{9 + s}": (A + 2,), f"_{10 + s}": (0, 7), f"_{11 + s}": (0, 4), f"_{12 + s}": (A + 2,),
                            f"_{13 + s}": (5,), f"_{14 + s}": (None, _sections(31)), f"_{15 + s}": (0, 5),
                            f"_{17 + s}": (1.0, float("nan"))})
    _broken(call, ok, 2, **{f"_{5 + s}": (1 << 25,)})
    if fp8:
        _broken(call, ok, 1, _5=(0.0, -1.0, float("nan"), float("inf")))


@pytest.mark.parametrize("fp8", [False, True])
def test_attn_weights_checks(mla, fp8):
    L = mla.lib()
    call = L.mla_attn_weights_fp8 if fp8 else L.mla_attn_weights
    # (q, lse, kv, [scale], num_blocks, table, max_blocks, seqlens, B, s_q, H, softmax_scale, causal, weights, stride,
    #  stream)
    ok = [A, A, A] + ([1.0] if fp8 else []) + [4, A, 2, A, 3, 1, 16, 0.1, 0, A, 128, None]
    s = 1 if fp8 else 0
    _broken(call, ok, 1, _0=(None, A + 8), _1=(None, A + 2), _2=(None, A + 8))
    _broken(call, ok, 1, **{f"_{3 + s}": (0,), f"_{4 + s}": (None, A + 1), f"_{5 + s}": (0,), f"_{6 + s}": (None, A + 2),
                            f"_{7 + s}": (0,), f"_{8 + s}": (0,), f"_{9 + s}": (0,),
                            f"_{10 + s}": (0.0, -1.0, float("nan"), float("inf")), f"_{12 + s}": (None, A + 2),
                            f"_{13 + s}": (0,)})
    _broken(call, ok, 2, **{f"_{9 + s}": (513,), f"_{7 + s}": (16385,), f"_{3 + s}": (1 << 25,)})
    if fp8:
        _broken(call, ok, 1, _3=(0.0, -1.0, float("nan"), float("inf")))


@pytest.mark.parametrize("fp8", [False, True])
def test_evict_checks(mla, fp8):
    L = mla.lib()
    call = L.mla_evict_fp8 if fp8 else L.mla_evict
    # (kv, num_blocks, table, max_blocks, seqlens, B, weights, w_stride, arrival, a_stride, budget, sink, recent,
    #  new_seqlens, kept, weights_out, arrival_out, width, stream)
    ok = [A, 4, A, 2, A, 3, A, 128, 2 * A, 128, 100, 4, 16, A, 1 << 42, 1 << 40, 1 << 41, 100, None]
    _broken(call, ok, 1, _0=(None, A + 8), _1=(0,), _2=(None, A + 2), _3=(0,), _4=(None, A + 2), _5=(0,), _6=(None, A + 2),
            _7=(0,), _8=(2 * A + 2,), _9=(0,), _10=(0, -1, 19), _11=(-1, 85), _12=(-1, 97, 2 ** 31 - 1),
            _13=(None, A + 2), _14=(None, A + 2), _15=(None, A + 2), _16=(A + 2,), _17=(99, 0))
    _broken(call, ok, 1, _14=(A, 1 << 40, (1 << 41) + 1196), _15=(A, A + 4, A - 4 * 299, 2 * A + 4, (1 << 42) - 4),
            _16=(A, 2 * A, 2 * A + 4 * 383))   # over the inputs or one another
    wide = list(ok)
    wide[3], wide[7], wide[8], wide[9], wide[16] = 8193, 524352, None, 0, None
    assert call(*wide) == 2
    _broken(call, ok, 2, _1=(1 << 25,), _5=(16385,))


def test_tensors_that_are_not_on_a_gpu_are_refused(mla):
    bf, i32 = torch.bfloat16, torch.int32
    kv, table, lens = torch.zeros(2, 64, 576, dtype=bf), torch.zeros(1, 2, dtype=i32), torch.zeros(1, dtype=i32)
    with pytest.raises(ValueError):
        mla.rope_axes(torch.zeros(2, 1, 64, dtype=bf), torch.zeros(1, 2, dtype=i32))
    with pytest.raises(ValueError):
        mla.cache_append(torch.zeros(1, 512, dtype=bf), torch.zeros(1, 64, dtype=bf), kv, table, lens)
    with pytest.raises(ValueError):
        mla.attn_weights(torch.zeros(1, 1, 2, 576, dtype=bf), torch.zeros(1, 1, 2), kv, table, lens, 0.1, False,
                         torch.zeros(1, 128))
    with pytest.raises(ValueError):
        mla.evict(kv, table, lens, torch.zeros(1, 128), 4)


def test_scales_that_leave_the_normal_numbers_are_refused(mla):
    L = mla.lib()
    # softmax_scale * kv_scale * log2(e) against [2^-126 = 1.18e-38, 3.4e38]
    for scale, kv_scale in ((1e-39, 1.0), (3e38, 1.0), (1.0, 1e-39), (1e30, 1e30)):
        assert L.mla_attn_weights_fp8(A, A, A, kv_scale, 4, A, 2, A, 3, 1, 16, scale, 0, A, 128, None) == 1, scale


def test_more_rows_than_row_numbers_count_are_refused(mla):
    L = mla.lib()
    far = 1 << 44
    n = (1 << 30) + 1
    assert L.mla_rope_axes(A, 128, 64, far, 128, 64, 2 * far, n, _sections(32), 1, 0, 10000.0, 0, n, 2, None) == 2
    assert L.mla_cache_append(A, 576, 2 * far, 576, far, 4, 3 * far, 2, 4 * far, 5 * far, n, 3, 6 * far, n,
                              _sections(32), 1, 0, 10000.0, None) == 2


def test_evict_s_lengths_overlap_nothing_but_the_lengths_they_replace(mla):
    L = mla.lib()
    far = 1 << 40   # apart from one another
    table, lens, weights, arrival, new, kept, w_out, a_out = ((i + 1) * far for i in range(8))
    base = [A, 4, table, 2, lens, 3, weights, 128, arrival, 128, 100, 4, 16, new, kept, w_out, a_out, 100, None]
    for fp8 in (False, True):
        call = L.mla_evict_fp8 if fp8 else L.mla_evict
        for at in (lens + 4, lens - 8, table, table + 20, weights + 4 * 383, arrival, kept, kept - 8, w_out + 1196, a_out):
            bad = list(base)
            bad[13] = at
            assert call(*bad) == 1, hex(at)
        for i in (14, 15, 16):      # an output over the lengths or the table
            for at in (lens, table - 1196):
                bad = list(base)
                bad[i] = at
                assert call(*bad) == 1, (i, hex(at))
