"""Pins of the oracle's latent-cache operators (CPU)."""
import math

import numpy as np
import pytest

import oracle


def test_axis_of_pairs():
    assert oracle.axis_of_pairs((16, 8, 8)) == [0] * 16 + [1] * 8 + [2] * 8
    assert oracle.axis_of_pairs((16, 8, 8), True) == [0, 1, 2] * 8 + [0] * 8
    assert oracle.axis_of_pairs((0, 32), True) == [1] * 32
    assert oracle.axis_of_pairs((30, 0, 2), True) == [0, 2, 0, 2] + [0] * 28


def test_rope_axes_is_the_single_axis_rope_on_equal_positions():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((7, 3, 64))
    pos = rng.integers(0, 5000, 7)
    want = np.swapaxes(oracle.rope_interleaved(np.swapaxes(x, 0, 1), pos), 0, 1)
    for sections in ((32,), (16, 8, 8), (1, 2, 29, 0)):
        got = oracle.rope_axes(x, [pos] * len(sections), sections)
        assert np.allclose(got, want, atol=1e-12, rtol=0)


def test_rope_axes_by_hand_and_its_inverse():
    x = np.zeros((1, 1, 64))
    x[0, 0, 0], x[0, 0, 32], x[0, 0, 63] = 1.0, 2.0, 3.0      # pairs 0, 16 and 31
    pos = np.array([[1], [10], [100]])
    y = oracle.rope_axes(x, pos, (16, 8, 8))
    assert np.isclose(y[0, 0, 0], math.cos(1.0)) and np.isclose(y[0, 0, 1], math.sin(1.0))
    assert np.isclose(y[0, 0, 32], 2 * math.cos(10 * 1e4 ** -0.5))
    a = 100 * 1e4 ** (-62 / 64)
    assert np.isclose(y[0, 0, 62], -3 * math.sin(a)) and np.isclose(y[0, 0, 63], 3 * math.cos(a))
    rng = np.random.default_rng(1)
    x, g = rng.standard_normal((5, 2, 64)), rng.standard_normal((5, 2, 64))
    pos = rng.integers(0, 1000, (2, 5))
    kw = dict(interleaved=True)
    assert np.allclose(oracle.rope_axes(oracle.rope_axes(x, pos, (20, 12), **kw), pos, (20, 12), inverse=True, **kw), x)
    # the gradient of <g, rope(x)> along any direction, against a difference (the map is linear)
    d = rng.standard_normal(x.shape)
    lhs = (g * oracle.rope_axes(x + d, pos, (20, 12), **kw)).sum() - (g * oracle.rope_axes(x, pos, (20, 12), **kw)).sum()
    assert np.isclose(lhs, (oracle.rope_axes(g, pos, (20, 12), inverse=True, **kw) * d).sum())


def test_append_slots():
    table = np.array([[5, 9], [7, -1]])
    got = oracle.append_slots(table, [65, 3], [0, 2, 3])
    assert got == [(0, 5, 63), (1, 9, 0), (2, 7, 2)]


def test_append_rows_copies_without_positions():
    c, pe = np.ones((2, 512)), np.arange(128.0).reshape(2, 64)
    assert np.array_equal(oracle.append_rows(c, pe)[:, 512:], pe)
    assert np.allclose(oracle.append_rows(c, pe, positions=np.zeros((1, 2), int))[:, 512:], pe)


@pytest.mark.parametrize("causal", [False, True])
def test_attn_weights_sum_to_the_rows_that_see_a_token(causal):
    rng = np.random.default_rng(2)
    B, s_q, H = 2, 3, 4
    kv = rng.standard_normal((4, 64, 576))
    table = np.array([[2, 0], [3, 1]])
    seqlens = np.array([100, 2])          # request 1: its first query position sees nothing when causal
    q = rng.standard_normal((B, s_q, H, 576))
    out, lse = oracle.decode_absorbed(q, kv, table, seqlens, 0.05, causal=causal)
    w, _ = oracle.attn_weights(q, lse, kv, table, seqlens, 0.05, causal=causal)
    assert np.isclose(w[0].sum(), s_q * H)
    assert np.isclose(w[1].sum(), (2 if causal else 3) * H)
    # the weights are the softmax that the output is made of: sum over rows of out = sum_t weight_t v_t
    v = oracle.gather_request(kv, table[0], 100)[:, :512]
    assert np.allclose(w[0] @ v, out[0].sum(axis=(0, 1)))


def test_attn_weights_uniform():
    q, kv = np.zeros((1, 1, 2, 576)), np.zeros((1, 64, 576))
    w, _ = oracle.attn_weights(q, np.full((1, 1, 2), math.log(5)), kv, np.array([[0]]), [5], 1.0)
    assert np.allclose(w[0], 2 / 5)


def test_evict_by_hand():
    w = [0.5, 3.0, 0.0, 3.0, 1.0, 9.0, 0.1]
    # budget 4, nothing guarded: slots 5, 1, 3 and 4; 0 and 2 fall free and take 4 and 5
    m, kept, wo, ao = oracle.evict(7, w, None, 4, 0, 0, 6)
    assert m == 4 and kept.tolist() == [4, 1, 5, 3, -1, -1]
    assert wo.tolist() == [1.0, 3.0, 9.0, 3.0, 0.0, 0.0] and ao.tolist() == [4, 1, 5, 3, 7, 8]
    # the first and the last two are guarded; one of the two equal weights goes, the lower slot stays
    m, kept, wo, ao = oracle.evict(7, w, None, 4, 1, 2, 4)
    assert kept.tolist() == [0, 1, 5, 6]
    # arrival numbers decide what is guarded
    m, kept, wo, ao = oracle.evict(3, [1.0, 2.0, 3.0], [8, 0, 4], 2, 1, 1, 3)
    assert kept.tolist() == [0, 1, -1] and ao.tolist() == [8, 0, 9]
    # below the budget nothing changes; a request without tokens
    m, kept, wo, ao = oracle.evict(2, [1.0, math.nan], None, 5, 0, 0, 5)
    assert m == 2 and kept.tolist() == [0, 1, -1, -1, -1] and ao.tolist() == [0, 1, 2, 3, 4]
    assert oracle.evict(0, [], None, 5, 0, 0, 2)[3].tolist() == [0, 1]
    # NaN goes first, then minus infinity
    assert oracle.evict(3, [math.nan, -math.inf, 0.0], None, 2, 0, 0, 2)[1].tolist() == [2, 1]


def test_planted_mistakes_are_seen():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 2, 64))
    pos = rng.integers(1, 1000, (3, 4))
    good = oracle.rope_axes(x, pos, (16, 8, 8))
    assert not np.allclose(good, oracle.rope_axes(x, pos[::-1], (16, 8, 8)))
    assert not np.allclose(good, oracle.rope_axes(x, pos, (16, 8, 8), interleaved=True))
    assert not np.allclose(good, oracle.rope_axes(x, pos, (16, 8, 8), inverse=True))
    assert oracle.append_slots(np.array([[1, 2]]), [64], [0, 1]) != oracle.append_slots(np.array([[1, 2]]), [65], [0, 1])
