"""The calls on a 4-bit latent cache at the ends of what their arguments allow, against the float64 oracle: large and small
queries, scales and rows, infinities, positions far out, NaN where a query position does not look.

Tolerances are those of test_gpu_fp4 where nothing else is said: they are relative to sum |q_d k_d| and to the values, so
powers of two on q, on the cache and on the scales leave them as they are.
"""
import numpy as np
import pytest
import torch

import oracle
import test_gpu_fp4 as base
from test_gpu_fp4 import SCALE, _case, _compare, _ref, _run

from _harness import to_np

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_absorbed_decode_gb300 import build_lib
    build_lib.build()
    yield


@pytest.fixture
def softmax_scale(monkeypatch):
    """Sets the softmax scale of test_gpu_fp4's calls, oracle and tolerances."""
    return lambda scale: monkeypatch.setattr(base, "SCALE", scale)


# -------------------------------------------------------------------------------------- queries --
@pytest.mark.parametrize("factor", [2.0 ** 13, 2.0 ** 15, 2.0 ** 40, 2.0 ** 100, 2.0 ** -40, 2.0 ** -110])
@pytest.mark.parametrize("s_q,H,topk", [(1, 128, None), (2, 24, None), (1, 128, [300, 129]), (2, 24, [300, 129])])
def test_queries_of_any_size(s_q, H, topk, factor, softmax_scale):
    """Rows of q far from size one, with a softmax scale that brings their scores back to it; every third head stays as it is."""
    inp = _case([333, 190], s_q=s_q, H=H, topk=topk, seed=71, kv_scale=2.0 ** -6)
    scaled = torch.arange(H) % 3 != 1
    inp["q"][:, :, scaled] *= factor
    if factor > 1:
        assert float(inp["q"].float().abs().max()) >= 2.0 ** 15
    else:                   # (the others' scores would pass float32's range)
        inp["q"][:, :, ~scaled] *= factor
    softmax_scale(SCALE / factor)
    for parts in (1, 5):
        _compare(inp, _run(inp, parts), _ref(inp), f"factor={factor} parts={parts}")


@pytest.mark.parametrize("topk", [None, [300, 64]])
def test_scores_past_float32_are_not_empty_rows(topk, softmax_scale):
    """Scores of some 1e39: NaN, as from an fp32 softmax, and not the 0 and -inf of a row that sees nothing.  Rows of zeros
    (scores of 0) keep their result."""
    inp = _case([400, 64], H=32, topk=topk, seed=72)
    inp["q"][:, :, 3] = 0.0
    softmax_scale(1e38)
    want = _ref(dict(inp, q=inp["q"][:, :, 3:4].contiguous()))
    for parts in (1, 4):
        out, lse = _run(inp, parts)
        rest = [h for h in range(32) if h != 3]
        assert torch.all(out[:, :, rest].isnan()), parts
        assert torch.all(lse[:, :, rest].isnan() | lse[:, :, rest].isposinf()), parts
        _compare(dict(inp, q=inp["q"][:, :, 3:4]), (out[:, :, 3:4], lse[:, :, 3:4]), want, f"parts={parts}")


# --------------------------------------------------------------------------------------- scales --
@pytest.mark.parametrize("topk", [None, [300, 64]])
def test_a_softmax_scale_whose_log2_units_pass_float32(topk, softmax_scale):
    """3e38 * log2(e) is past float32's range, its product with kv_scale is not: with rows of q of size 2^-116 and values of
    size 2^-9 the scores come to some hundreds."""
    inp = _case([400, 64], H=32, topk=topk, seed=73, values=lambda rng, pool: rng.normal(0, 2.0 ** -9, (pool, 64, 576)))
    inp["q"] *= 2.0 ** -116
    softmax_scale(3e38)
    ref = _ref(inp)
    assert np.all(np.abs(ref[2]) < 1000)
    for parts in (1, 4):
        _compare(inp, _run(inp, parts), ref, f"parts={parts}")


@pytest.mark.parametrize("kv_scale", [2.0 ** -116, 2.0 ** 115])
@pytest.mark.parametrize("topk", [None, [32768]])
def test_the_ends_of_kv_scale(topk, kv_scale, softmax_scale):
    """A long context whose first tile sets references that the rest exceeds by almost what is allowed (7.9 of 8 in log2 units), so
    that a row's sum of exponentials comes to 2^29, with the smallest and the largest scale of the cache."""
    n, rope = 32768, 7.9 / (64 * SCALE * np.log2(np.e))

    def values(rng, pool):
        x = np.concatenate((1 + 0.1 * rng.normal(0, 1, (pool, 64, 512)), np.full((pool, 64, 64), rope)), axis=2)
        return x
    inp = _case([n], H=16, topk=topk, seed=74, values=values)
    inp["q"][...] = 0.0
    inp["q"][..., 512:] = 1.0
    kv, table = inp["kv"].numpy(), inp["table"].numpy()[0]
    for page in table[:2]:
        kv[page, :, 288:] = 0                          # the first 128 tokens score 0
    inp["kv_scale"] = kv_scale                          # (the bytes are those of 2^-6)
    softmax_scale(SCALE * 2.0 ** -6 / kv_scale)
    ref = _ref(inp)
    for parts in (1, 5):
        _compare(inp, _run(inp, parts), ref, f"parts={parts}")


# -------------------------------------------------------------------------------------- appends --
def _append(rows, kv_scale, **more):
    """The bytes [N, 352] that new rows of one request become."""
    import mla_absorbed_decode_gb300 as mla
    N = rows.shape[0]
    blocks = (N + 63) // 64
    kv = torch.full((blocks, 64, 352), 0x55, dtype=torch.uint8, device="cuda")
    table = torch.arange(blocks, dtype=torch.int32, device="cuda").view(1, blocks)
    d = rows.cuda()
    mla.cache_append_fp4(d[:, :512], d[:, 512:], kv, kv_scale, table, torch.tensor([N], dtype=torch.int32, device="cuda"),
                         **{k: v.cuda() if torch.is_tensor(v) else v for k, v in more.items()})
    assert mla.get_device_status() == 0
    return kv.view(-1, 352)[:N].cpu().numpy()


@pytest.mark.parametrize("norm", [False, True])
def test_infinities_of_k_pe_saturate_when_they_turn(norm):
    """An infinite element, and pairs whose turned values pass float32's range, become +-448: never NaN but where an infinity is
    taken from another."""
    g = torch.Generator().manual_seed(75)
    N, most = 64, float(torch.finfo(BF).max)
    rows = torch.randn((N, 576), generator=g).to(BF)
    pos = torch.randint(1, 131072, (N,), generator=g, dtype=torch.int32)
    inf = float("inf")
    odd = {0: (inf, None), 3: (None, -inf), 8: (-inf, None), 11: (inf, 0.0), 17: (most, most), 19: (most, -most), 24: (inf, most),
           31: (-inf, inf)}
    for j, pair in odd.items():
        for i, v in enumerate(pair):
            if v is not None:
                rows[:, 512 + 2 * j + i] = v
    got = _append(rows, 2.0 ** -6, positions=pos, norm_weight=torch.ones(512, dtype=BF) if norm else None)[:, 288:]
    x = to_np(rows)[:, 512:]
    for j in odd:
        a = pos.numpy() * 10000.0 ** (-2.0 * j / 64)
        with np.errstate(invalid="ignore"):
            y0 = x[:, 2 * j] * np.cos(a) - x[:, 2 * j + 1] * np.sin(a)
            y1 = x[:, 2 * j] * np.sin(a) + x[:, 2 * j + 1] * np.cos(a)
        for i, y in enumerate((y0, y1)):
            want = oracle.e4m3_round(y * 2.0 ** 6)
            code = got[:, 2 * j + i]
            none = np.isnan(y)
            assert np.all((code[none] & 0x7F) == 0x7F), (j, i)
            assert np.array_equal(code[~none], want[~none]), (j, i)
    rest = np.setdiff1d(np.arange(64), [2 * j + i for j in odd for i in (0, 1)])
    assert np.all((got[:, rest] & 0x7F) != 0x7F)


@pytest.mark.parametrize("eps,sizes", [(0.0, (-120, -100, -70, -64, -40, 0, 58, 63, 100, 120)), (1e-6, (0, 20, 59, 63, 100, 120)),
                                        (1e-30, (-60, -50, -40, 0, 63, 120)), (1e30, (40, 50, 63, 100))])
def test_norms_of_rows_of_any_size(eps, sizes):
    """Rows whose squares, or their sum, float32 has no room for: the codes of 64 bits, as for rows of size one (those of a value
    that lies within 2^-40 of itself of a halfway point might differ: expected 1e-6 of them)."""
    g = torch.Generator().manual_seed(76)
    rows = torch.randn((8 * len(sizes), 576), generator=g)
    rows[:, :512] *= torch.tensor([2.0 ** s for s in sizes]).repeat_interleave(8)[:, None]
    rows[::8, 5:300] = 0.0
    rows[1::8, 7] *= 16.0
    rows = rows.to(BF)
    w = (1 + 0.3 * torch.randn(512, generator=g)).to(BF)
    for kv_scale in (2.0 ** -6, 0.013):
        got = _append(rows, kv_scale, norm_weight=w, norm_eps=eps)
        x = to_np(rows)
        x = np.concatenate((oracle.normed_latent(x[:, :512], to_np(w), float(np.float32(eps))), x[:, 512:]), axis=1)
        want = oracle.pack_fp4(x, kv_scale)
        bad = np.nonzero((got != want).any(axis=1))[0]
        assert bad.size == 0, [sizes[r // 8] for r in bad]


def test_norms_of_rows_that_have_none():
    """A row of zeros stays one of zeros, or becomes NaN where eps is 0 too (0 times infinity); a NaN makes its row NaN, an infinity
    its group, and the rest of its row 0."""
    rows = torch.randn((5, 576), generator=torch.Generator().manual_seed(77)).to(BF)
    rows[0, :512] = 0.0
    rows[1, 100] = float("nan")
    rows[2, 200] = float("-inf")
    rows[3, 0], rows[3, 511] = float("inf"), float("nan")
    w = torch.ones(512, dtype=BF)
    for eps, zeros_are in ((1e-6, 0), (1e-45, 0), (0.0, 0x7F)):
        got = _append(rows, 2.0 ** -6, norm_weight=w, norm_eps=eps)
        assert np.all(got[0, :256] == 0) and np.all(got[0, 256:288] == zeros_are)
        assert np.all(got[1, 256:288] == 0x7F) and np.all(got[3, 256:288] == 0x7F)
        scales = got[2, 256:288]
        assert scales[200 // 16] == 0x7F and np.all(np.delete(scales, 200 // 16) == 0)      # finite / infinite is 0
        assert np.all((got[4, 256:288] & 0x7F) != 0x7F)


def _quarter_turns(top):
    """Positions at which pair 0, which turns by one radian a position, is nearest to a quarter turn: denominators of fractions close
    to 2 / pi, and their neighbours."""
    p = np.arange(1, top, dtype=np.float64)
    off = np.abs(p * (2 / np.pi) - np.rint(p * (2 / np.pi)))
    return p[np.argsort(off)[:400]].astype(np.int64)


@pytest.mark.parametrize("theta", [10000.0, 500000.0])
@pytest.mark.parametrize("low,top,bits", [(0, 2 ** 17, 25), (2 ** 17, 2 ** 24, 21)])
@pytest.mark.parametrize("kv_scale", [2.0 ** -6, 0.013])
def test_rope_codes_of_turned_pairs(low, top, bits, theta, kv_scale):
    """Codes of values off by at most 2^-bits of their pair's norm: each lies between the codes of the 64-bit value less and plus that.
    (A sine off by 2^-21 would put some 2^-21 / 2^-5 of 2.1 million values, a hundred, past the first bound.)"""
    g = torch.Generator().manual_seed(78)
    N = 32768
    rows = torch.randn((N, 576), generator=g).to(BF)
    pos = torch.randint(low, top, (N,), generator=g, dtype=torch.int32)
    pos[::3] *= -1
    if low == 0:
        pos[:400] = torch.from_numpy(_quarter_turns(top)).int()
        pos[400:410] = torch.tensor([0, 1, -1, 2, 11, 355, -355, 710, top - 1, 1 - top])
    else:
        pos[:4000] = torch.arange(top - 4000, top)
        pos[4000:8000] = torch.arange(-(top - 1), -(top - 1) + 4000)
    got = _append(rows, kv_scale, positions=pos, rope_theta=theta)[:, 288:]
    x = to_np(rows)[:, 512:]
    y = oracle.rope_axes(x[:, None], pos.numpy()[None], (32,), base=theta)[:, 0]
    room = 2.0 ** -bits * np.repeat(np.hypot(x[:, 0::2], x[:, 1::2]), 2, axis=1)
    unit = float(np.float32(kv_scale))
    value = lambda code: oracle.dequantize_e4m3(code, 1.0)
    code = value(got)
    low_end, high_end = value(oracle.e4m3_round((y - room) / unit)), value(oracle.e4m3_round((y + room) / unit))
    bad = (code < low_end) | (code > high_end)
    assert not bad.any(), (int(bad.sum()), pos.numpy()[np.nonzero(bad)[0][:5]].tolist())


def _next_to_halfway(pos, pair, theta, unit, room):
    """(positions, first elements in [1, 2), their second is 0) for which the first or the second turned value lies between room and
    8 room from halfway between two codes, relative to the pair's norm."""
    x0 = 1 + np.arange(128) / 128
    p, x = [], []
    for part in np.array_split(pos, max(1, pos.size >> 16)):
        a = part * theta ** (-2.0 * pair / 64)
        for turned in (np.cos(a), np.sin(a)):
            v = np.abs(turned[:, None] * x0) / unit
            step = 2.0 ** (np.floor(np.log2(v)) - 3)
            off = np.abs(v / step - np.floor(v / step) - 0.5) * step * unit / x0
            i, k = np.nonzero((v > 2.0 ** -5) & (v < 440) & (off > room) & (off < 8 * room))
            p.append(part[i])
            x.append(x0[k])
    return np.concatenate(p), np.concatenate(x)


@pytest.mark.parametrize("low,top,bits", [(1, 2 ** 17, 25), (2 ** 24 - 2 ** 18, 2 ** 24, 21)])
@pytest.mark.parametrize("pair,theta", [(0, 10000.0), (1, 500000.0), (5, 10000.0), (30, 10000.0)])
def test_rope_codes_next_to_halfway(pair, theta, low, top, bits):
    """Turned values that lie just further than the stated error from halfway between two codes: none may get the wrong one."""
    kv_scale = 2.0 ** -6
    p, x = _next_to_halfway(np.arange(low, top), pair, theta, kv_scale, 2.0 ** -bits)
    keep = np.random.default_rng(79).permutation(p.size)[:65536]
    p, x = p[keep], x[keep]
    assert p.size > 50
    rows = torch.zeros((p.size, 576))
    rows[:, 512 + 2 * pair] = torch.from_numpy(x).float()
    got = _append(rows.to(BF), kv_scale, positions=torch.from_numpy(p).int(), rope_theta=theta)
    y = oracle.rope_axes(to_np(rows)[:, None, 512:], p[None], (32,), base=theta)[:, 0, 2 * pair:2 * pair + 2]
    # The one of the two values that the row was picked for lies further than the error from halfway: one code is allowed.  The other may
    # lie nearer (of 33181 rows two do: at 16775432 and 16701101, by 2^-27 and 2^-28.5 of the norm), and has two.
    low_end, high_end = (oracle.dequantize_e4m3(oracle.e4m3_round((y + d * 2.0 ** -bits * x[:, None]) / kv_scale), 1.0) for d in (-1, 1))
    assert np.all((low_end == high_end).any(axis=1))
    code = oracle.dequantize_e4m3(got[:, 288 + 2 * pair:290 + 2 * pair], 1.0)
    bad = np.nonzero(((code < low_end) | (code > high_end)).any(axis=1))[0]
    assert bad.size == 0, (bad.size, p.size, p[bad[:5]].tolist())


# ----------------------------------------------------------------------------------------- masks --
@pytest.mark.parametrize("s_q,H", [(2, 128), (3, 16), (4, 128)])
@pytest.mark.parametrize("code", [0x7F, 0xFF])
def test_a_nan_that_a_query_position_does_not_see(s_q, H, code):
    """The newest tokens of a request with NaN in a scale or in the RoPE key: the query positions before them are what they were, the
    others are NaN; dense and over lists."""
    n = [300, 65, 513]
    for topk in (None, [300, 40, 257]):
        inp = _case(n, s_q=s_q, H=H, topk=topk, seed=80)
        if topk:
            for b in range(3):      # the newest tokens are on the lists
                inp["indices"][b, :s_q] = torch.arange(n[b] - s_q, n[b])
        dirty = dict(inp, kv=inp["kv"].clone())
        for b, byte in enumerate((256 + 3, 288 + 20, 256 + 31)):
            t = n[b] - 1
            dirty["kv"][int(inp["table"][b, t // 64]), t % 64, byte] = code
        for parts in (1, 4):
            clean, got = _run(inp, parts), _run(dirty, parts)
            assert torch.equal(got[0][:, : s_q - 1], clean[0][:, : s_q - 1]) and torch.equal(got[1][:, : s_q - 1], clean[1][:, : s_q - 1])
            assert torch.all(got[0][:, -1].isnan()) and torch.all(got[1][:, -1].isnan())
