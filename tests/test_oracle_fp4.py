"""Pins of the 4-bit cache's oracle: its numbers against the format's definition and a search over all of them, its bytes
against hand-made rows, its rounding against the nearest value."""
import math

import numpy as np
import pytest

import oracle


def test_e2m1_numbers():
    assert oracle.E2M1_VALUES[:8].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert oracle.E2M1_VALUES[8:].tolist() == [-v for v in [0, 0.5, 1, 1.5, 2, 3, 4, 6]]


def test_e2m1_rounding_is_the_nearest_number_and_halves_go_to_the_even_code():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.normal(0, 3, 4000), oracle.E2M1_VALUES, oracle.E2M1_MIDDLES, -oracle.E2M1_MIDDLES])
    code = oracle.e2m1_round(v)
    for x, c in zip(v, code):
        off = np.abs(oracle.E2M1_VALUES - x)
        assert off[c] == off.min() or abs(x) > 6
        assert (c & 8 != 0) == (math.copysign(1, x) < 0)
    assert oracle.e2m1_round(oracle.E2M1_MIDDLES).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert oracle.e2m1_round(np.array([7.0, -1e9, np.inf, -np.inf, np.nan, -0.0])).tolist() == [7, 15, 7, 15, 0, 8]


def test_a_row_by_hand():
    row = np.zeros(576)
    row[0], row[1], row[15] = 6.0, -1.0, 0.5      # group 0: largest 6, scale 1 / kv_scale
    row[16] = 0.25                                # group 1
    row[512], row[575] = 2.0, -3.0
    data = oracle.pack_fp4(row, 0.5)
    assert data.shape == (352,)
    assert data[0] == 7 | (8 + 2) << 4 and data[7] == 1 << 4 and data[1] == 0
    assert data[256] == 0x40                       # E4M3 of 6 / (6 * 0.5) = 2
    assert data[257] == oracle.e4m3_round(np.array(0.25 / 3.0)) and data[258] == 0
    assert data[288] == 0x48 and data[351] == 0x80 | 0x4C    # 2 / 0.5 = 4, -3 / 0.5 = -6
    back = oracle.unpack_fp4(data, 0.5)
    assert back[0] == 6.0 and back[1] == -1.0 and back[15] == 0.5 and back[512] == 2.0 and back[575] == -3.0


@pytest.mark.parametrize("kv_scale", [1 / 64, 0.013, 2.0 ** -20])
def test_what_a_row_loses_is_half_a_step(kv_scale):
    rng = np.random.default_rng(3)
    x = rng.normal(0, 1, (40, 576)) * rng.choice([1e-4, 0.1, 1.0, 8.0], (40, 1))
    back = oracle.unpack_fp4(oracle.pack_fp4(x, kv_scale), kv_scale)
    unit = float(np.float32(kv_scale))
    g, b = x[:, :512].reshape(-1, 32, 16), back[:, :512].reshape(-1, 32, 16)
    top = np.abs(g).max(axis=2, keepdims=True)
    scale = oracle.unpack_fp4(oracle.pack_fp4(x, kv_scale), kv_scale)
    assert scale.shape == x.shape
    # a step of a group's numbers is at most 2 of its scale (4 to 6), its scale at most the wanted one plus half an
    # E4M3 step (2^-4, or 2^-10 kv_scale below the normal ones), and what saturates lost that half step of 6
    room = np.maximum(top / 6 * (1 + 2 ** -4), top / 6 + 2 ** -10 * unit)
    ok = top / 6 / unit <= 448
    assert np.all((np.abs(g - b) <= 1.0 * room + 6 * (2 ** -4 * top / 6 + 2 ** -10 * unit)) | ~ok)


def test_groups_of_zero_of_nan_and_beyond_the_range():
    x = np.zeros((4, 576))
    x[1, 3] = np.nan
    x[2, 0], x[2, 5] = np.inf, -np.inf
    x[3, 0] = 1e9
    data = oracle.pack_fp4(x, 1 / 64)
    assert np.all(data[0] == 0)
    assert data[1, 256] == 0x7F and np.all(data[1, :8] == 0) and np.isnan(oracle.unpack_fp4(data[1], 1 / 64)[:16]).all()
    assert data[2, 256] == 0x7E and data[2, 0] & 15 == 7 and data[2, 2] >> 4 == 15
    assert data[3, 256] == 0x7E and data[3, 0] & 15 == 7
    assert np.isfinite(oracle.unpack_fp4(data[1], 1 / 64)[16:]).all()


def test_norm():
    c = np.arange(512.0)[None] - 200
    y = oracle.normed_latent(c, np.full(512, 2.0), 0.5)
    assert np.allclose((y / 2) ** 2 * (np.mean(c ** 2) + 0.5), c ** 2)
