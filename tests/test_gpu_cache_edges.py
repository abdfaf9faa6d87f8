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


# ------------------------------------------------------------- weights: a CTA leaves nothing behind --
def _call(inp, dev, out):
    import mla_absorbed_decode_gb300 as mla
    args = (dev["block_table"], dev["seqlens"], inp["softmax_scale"], inp["causal"], out)
    if "kv_scale" in inp:
        mla.attn_weights_fp8(dev["q"], dev["lse"], dev["kv_cache"], inp["kv_scale"], *args)
    else:
        mla.attn_weights(dev["q"], dev["lse"], dev["kv_cache"], *args)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("s_q", [1, 2, 3, 4])
def test_attn_weights_calls_of_every_cluster_size_back_to_back(fp8, s_q):
    """Short calls one straight after the other, beside calls of another kernel that starts in the shared memory they
    have just left: an arrival that comes after its CTA has gone would be one that the next CTA's barriers count."""
    import mla_absorbed_decode_gb300 as mla
    w = W.Workload("weights_back", B=40, s_q=s_q, H=128, ragged_max=200, causal=True, kv_fp8=fp8)
    g = torch.Generator().manual_seed(s_q)
    inp = _weights_inputs(w, seed=33, seqlens=torch.randint(0, 200, (40,), generator=g, dtype=torch.int32))
    good = _run_weights(inp)
    dev = {k: v.cuda() for k, v in inp.items() if torch.is_tensor(v)}
    parts = mla.num_sm_parts(s_q, 128)
    meta = mla.decode_metadata(dev["seqlens"], s_q, 128, True, parts)
    pool = (dev["q"], dev["kv_cache"]) + ((inp["kv_scale"],) if fp8 else ())
    decode = lambda: (mla.decode_fp8 if fp8 else mla.decode)(*pool, dev["block_table"], dev["seqlens"],
                                                              inp["softmax_scale"], True, meta, parts)
    first = decode()
    outs = [dev["before"].clone() for _ in range(60)]
    for i, out in enumerate(outs):
        _call(inp, dev, out)
        if i % 3 == 2:
            last = decode()
    assert mla.get_device_status() == 0
    for out in outs:
        assert torch.equal(out.cpu(), good)
    assert torch.equal(last[0], first[0]) and torch.equal(last[1], first[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("s_q", [1, 2, 3, 4])
def test_attn_weights_gives_up_when_a_page_never_arrives(fp8, s_q):
    """The test hook withholds every CTA's first page: the waits on it run out of time, the call reports it and ends,
    and the calls after it are right."""
    import mla_absorbed_decode_gb300 as mla
    w = W.Workload("weights_timeout", B=3, s_q=s_q, H=128, fixed_seqlens=(300, 2000, 64), kv_fp8=fp8)
    inp = _weights_inputs(w, seed=34)
    good = _run_weights(inp)
    dev = {k: v.cuda() for k, v in inp.items() if torch.is_tensor(v)}
    out = dev["before"].clone()
    mla.debug_withhold_first_load(True)
    _call(inp, dev, out)
    assert mla.get_device_status() == 5          # MLA_ERR_TIMEOUT
    assert mla.get_device_status() == 0
    for b, n in enumerate((300, 2000, 64)):
        assert torch.equal(out[b, n:], dev["before"][b, n:])
    for _ in range(3):
        assert torch.equal(_run_weights(inp), good)
