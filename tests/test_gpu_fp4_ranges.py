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
