"""Plain float64 restatement of the latent-cache operators (test infrastructure only): rotation with
several position axes, the write of new rows, the attention weight of cached tokens, and eviction by it.

Definitions: the rotation of [MLA-paths]' tiny example (adjacent pairs; see mla.py) with a position per
pair; the cache layout and visibility of ``mla.py``; the rest as the public header states it.
"""
from __future__ import annotations

import math

import numpy as np

from .mla import D_LATENT, D_QK, D_ROPE, PAGE, gather_request, visible_tokens


def axis_of_pairs(sections, interleaved=False) -> list[int]:
    """The position axis of each of the 32 pairs: the sections one after the other, or one pair to each
    axis in turn for as long as the axis has pairs left."""
    assert sum(sections) == D_ROPE // 2
    if not interleaved:
        return [a for a, k in enumerate(sections) for _ in range(k)]
    out = []
    for turn in range(max(sections)):
        out += [a for a, k in enumerate(sections) if turn < k]
    return out


def rope_axes(x, positions, sections, base=10000.0, interleaved=False, inverse=False) -> np.ndarray:
    """x [N, H, 64]: pair j of token n, as a complex number, times e^(+-i positions[axis_j, n] base^(-2j/64))."""
    x = np.asarray(x, dtype=np.float64)
    axis = axis_of_pairs(sections, interleaved)
    out = np.empty_like(x)
    for j in range(D_ROPE // 2):
        angle = np.asarray(positions[axis[j]], dtype=np.float64) * float(base) ** (-2.0 * j / D_ROPE)
        z = (x[..., 2 * j] + 1j * x[..., 2 * j + 1]) * np.exp((-1j if inverse else 1j) * angle)[:, None]
        out[..., 2 * j], out[..., 2 * j + 1] = z.real, z.imag
    return out


def append_slots(block_table, seqlens, new_offsets) -> list[tuple[int, int, int]]:
    """(row, page, slot in the page) of every new row that belongs to a request."""
    out = []
    for b in range(len(seqlens)):
        r0, r1 = int(new_offsets[b]), int(new_offsets[b + 1])
        for r in range(r0, r1):
            t = int(seqlens[b]) - (r1 - r)
            out.append((r, int(block_table[b][t // PAGE]), t % PAGE))
    return out


def append_rows(c, k_pe, positions=None, sections=(32,), base=10000.0, interleaved=False) -> np.ndarray:
    """The new cached rows [N, 576]: c next to k_pe, rotated where positions are given."""
    pe = np.asarray(k_pe, dtype=np.float64)
    if positions is not None:
        pe = rope_axes(pe[:, None, :], positions, sections, base, interleaved)[:, 0]
    row = np.concatenate([np.asarray(c, dtype=np.float64), pe], axis=1)
    assert row.shape[1] == D_QK and np.asarray(c).shape[1] == D_LATENT
    return row


def attn_weights(q, lse, kv_cache, block_table, seqlens, softmax_scale, causal=False, kv_scale=None):
    """([B][n_b] weight of every cached token in this step, [B][n_b] sum over its rows of p |score terms|):
    weight_t = sum over (i, h) that see t of exp(scale <q, kv_t> - lse).  The second sums, with the same
    p, scale * sum_d |q_d kv_td|: what the rounding of a score can scale with (test tolerances)."""
    q = np.asarray(q, dtype=np.float64)
    B, s_q, H, _ = q.shape
    weight, spread = [], []
    for b in range(B):
        n = int(seqlens[b])
        kv = gather_request(kv_cache, block_table[b], n, kv_scale) if n > 0 else np.zeros((0, D_QK))
        w, a = np.zeros(n), np.zeros(n)
        for i in range(s_q):
            v = visible_tokens(n, s_q, i, causal)
            for h in range(H):
                if v <= 0 or lse[b, i, h] == -math.inf:
                    continue
                p = np.exp(softmax_scale * (kv[:v] @ q[b, i, h]) - float(lse[b, i, h]))
                w[:v] += p
                a[:v] += p * softmax_scale * (np.abs(kv[:v]) @ np.abs(q[b, i, h]))
        weight.append(w)
        spread.append(a)
    return weight, spread


def evict(n, weights, arrival, budget, sink, recent, width):
    """One request: (new length, kept [width], weights [width], arrival [width]); see the public header."""
    n = int(n)
    weights = [float(v) for v in weights[:n]]
    arrival = list(range(n)) if arrival is None else [int(v) for v in arrival[:n]]
    e = 1 + max(arrival, default=-1)

    def matters(t):   # ascending: first what stays longest
        guarded = arrival[t] < sink or arrival[t] >= e - recent
        nan = math.isnan(weights[t])
        return (0, 0, 0.0, t) if guarded else (1, int(nan), 0.0 if nan else -weights[t], t)

    m = min(n, int(budget))
    stay = set(sorted(range(n), key=matters)[:m])
    sources = iter(sorted(t for t in stay if t >= m))
    kept = [t if t in stay else next(sources) for t in range(m)]
    assert sorted(kept) == sorted(stay)
    return (m, np.array(kept + [-1] * (width - m), dtype=np.int64),
            np.array([weights[t] for t in kept] + [0.0] * (width - m)),
            np.array([arrival[t] for t in kept] + [e + j for j in range(width - m)], dtype=np.int64))
