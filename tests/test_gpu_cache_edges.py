"""GPU tests of the latent-cache operators where their arithmetic and their dispatch have edges.  Bounds are derived at
each test; the rest is as in test_gpu_cache.py, whose inputs these tests share.
"""
import numpy as np
import pytest
import torch

from mla_absorbed_decode_gb300 import workloads as W

from test_gpu_cache import BF, _run_weights, _weights_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_absorbed_decode_gb300 import build_lib
    build_lib.build()
    yield


# ---------------------------------------------------------------------- weights: infinite scores --
LOG2E = 1.4426950408889634
SCALES = (192 ** -0.5, 0.1, 0.05, 0.11, 0.125, 0.3)


def test_the_scales_have_residues_of_either_sign():
    residues = [float(np.float32(s)) * LOG2E - float(np.float32(float(np.float32(s)) * LOG2E)) for s in SCALES]
    assert min(residues) < 0 < max(residues)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("H", [1, 128])
def test_attn_weights_a_score_of_minus_infinity_adds_nothing(scale, H):
    """exp(-inf - lse) = 0, whether the cache holds an infinity or the products overflow; the tokens beside it keep
    their bits (a column of S depends on its own token alone)."""
    w = W.Workload("weights_inf", B=2, s_q=1, H=H, fixed_seqlens=(200, 70))
    inp = _weights_inputs(w, seed=31)
    inp["softmax_scale"] = float(np.float32(scale))
    inp["q"][..., 512:] = inp["q"][..., 512:].abs() + 1.0
    inp["lse"] = torch.full_like(inp["lse"], 3.0)
    good = _run_weights(inp)
    assert torch.isfinite(good).all()
    page, kv = inp["block_table"], inp["kv_cache"]
    where = [(0, 3), (0, 63), (0, 64), (0, 199), (1, 0), (1, 69)]
    for b, t in where[:4]:
        kv[page[b, t // 64].long(), t % 64, 520] = -float("inf")
    for b, t in where[4:]:                                   # 64 products of at least 3e38: the sum is beyond fp32
        kv[page[b, t // 64].long(), t % 64, 512:] = -3e38
    got = _run_weights(inp)
    want = good.clone()
    for b, t in where:
        want[b, t] = inp["before"][b, t]
    assert torch.equal(got, want)


def test_attn_weights_rows_whose_lse_is_huge_or_infinite_add_nothing():
    """exp(s - lse) = 0 for an lse whose product with log2(e) is beyond fp32, as for an infinite one."""
    w = W.Workload("weights_lse", B=1, s_q=1, H=16, fixed_seqlens=(150,))
    inp = _weights_inputs(w, seed=32)
    some = inp["lse"].clone()
    some[0, 0, 1::2] = -float("inf")                         # rows that are left out
    good = _run_weights(dict(inp, lse=some))
    for v in (3e38, float("inf")):
        some[0, 0, 1::2] = v
        assert torch.equal(_run_weights(dict(inp, lse=some)), good)


# ---------------------------------------------------------- weights: scores of one product, exactly --
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,H", [(130, 1), (130, 16), (64, 128)])
def test_attn_weights_scores_of_one_product(fp8, n, H):
    """A head's q has one element that is not 0, so its scores are single products, exact in fp32: what is left is the
    exponent y = log2(e) (scale s - lse), |y| <= Y, formed from float pairs in three operations (3u Y), its
    exp2 (2^-22), and the sum over H rows (H u): p moves by (3 ln 2 u |y| + 2^-22 + H u) p.  Scores reach 80, so a scale
    that is off by 2^-22 shows."""
    g = torch.Generator().manual_seed(n + H)
    w = W.Workload("weights_one", B=1, s_q=1, H=H, fixed_seqlens=(n,), kv_fp8=fp8)
    inp = W.make_inputs(w, seed=3)
    inp["q"].zero_()
    dim = torch.randint(0, 576, (H,), generator=g)
    inp["q"][0, 0, torch.arange(H), dim] = (32 + 6 * torch.rand(H, generator=g)).to(BF)
    k = torch.tensor([28.0, 30.0, 32.0, 36.0, 40.0, -40.0])[torch.randint(0, 6, (n, 576), generator=g)]
    kv, scale = inp["kv_cache"], 1.0 / 16
    if fp8:
        inp["kv_scale"] = 1.0
    codes = k.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else k.to(BF)
    for t in range(n):
        kv[inp["block_table"][0, t // 64].long(), t % 64] = codes[t]
    inp["softmax_scale"] = scale
    s = scale * torch.einsum("hd,td->ht", inp["q"][0, 0].double(), k.double()).numpy()
    assert 80 <= s.max() < 96                                # 32 * 40 / 16 and 38 * 40 / 16
    lse = (torch.from_numpy(s).logsumexp(dim=1)).float()
    inp["lse"] = lse.view(1, 1, H)
    inp["before"] = torch.zeros((1, inp["block_table"].shape[1] * 64))
    got = _run_weights(inp)[0, :n].double().numpy()
    arg = s - lse.double().numpy()[:, None]
    p = np.exp(arg)
    u = 2.0 ** -24
    room = (p * (3 * u * np.abs(arg) + 2.0 ** -22 + H * u)).sum(axis=0)
    assert np.all(np.abs(got - p.sum(axis=0)) <= room + 2.0 ** -126 * H), float((np.abs(got - p.sum(axis=0)) / p.sum(axis=0)).max())
