"""GPU tests of the latent-cache operators where their arithmetic and their dispatch have edges.  Bounds are derived at
each test; the rest is as in test_gpu_cache.py, whose inputs these tests share.
"""
import numpy as np
import pytest
import torch

import oracle
from mla_absorbed_decode_gb300 import workloads as W

from _harness import to_np
from test_gpu_cache import BF, _check_evict, _evict_inputs, _positions, _rope_room, _run_weights, _weights_inputs

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


# ------------------------------------------------------------------------ every variant of a kernel --
@pytest.mark.parametrize("N,H", [(700, 40), (611, 128), (350, 130), (305, 200), (640, 33)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_axes_several_rounds_of_heads_a_block(N, H, inverse):
    """Many tokens of more than 32 heads: a block turns up to 128 heads of a token, the last round in part."""
    import mla_absorbed_decode_gb300 as mla
    g = torch.Generator().manual_seed(N + H)
    x = torch.randn((N, H, 64), generator=g).to(BF)
    pos = _positions(3, N, g)
    q = torch.full((N, H, 576), 5.0, dtype=BF, device="cuda")
    got = mla.rope_axes(x.cuda(), pos.cuda(), (10, 12, 10), out=q[..., 512:], interleaved=True, inverse=inverse)
    ref = oracle.rope_axes(to_np(x), pos.numpy(), (10, 12, 10), interleaved=True, inverse=inverse)
    assert np.all(np.abs(to_np(got) - ref) <= 2.0 ** -8 * np.abs(ref) + _rope_room(to_np(x)))
    assert torch.all(q[..., :512] == 5.0)
    flat = mla.rope_axes(x[:40].cuda(), pos[:, :40].contiguous().cuda(), (10, 12, 10), interleaved=True, inverse=inverse)
    assert torch.equal(flat, got[:40])           # a block's rounds change no bit


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("slots,lens", [(5056, [5056, 4097, 100]), (12032, [12000, 0, 8193, 4096]),
                                        (16384, [16384, 16383]), (40000, [39999, 777])])
def test_evict_equal_weights_over_the_ctas_of_a_cluster(fp8, slots, lens):
    """Requests of 2, 4 and 8 CTAs whose weights have five values: the cut lies among equals that every CTA holds."""
    for arrival in (True, False):
        s = _evict_inputs(lens, slots, fp8, seed=slots, ties=True, arrival=arrival)
        for budget in (slots // 3, slots - 700):
            _check_evict(s, budget, 3, 40, budget + 9)
    s["w"][:] = 1.5                              # nothing but equals
    _check_evict(s, slots // 2 + 1, 0, 0, slots)


@pytest.mark.parametrize("slots,lens", [(451, [451, 450, 3]), (5057, [5057, 4099]), (9001, [9001, 8193])])
@pytest.mark.parametrize("ties", [False, True])
def test_evict_rows_that_are_not_aligned(slots, lens, ties):
    """Rows of an odd number of elements, with arrival numbers: slot by slot where 16-byte loads are not possible."""
    s = _evict_inputs(lens, slots, False, seed=slots + ties, ties=ties)
    _check_evict(s, slots // 2, 2, 30, slots // 2 + 65)


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_evict_rows_that_start_anywhere(shift):
    """Weights and arrival as parts of wider buffers, of which one row or the other is aligned."""
    import mla_absorbed_decode_gb300 as mla
    s = _evict_inputs([700, 90, 640], 704, False, seed=35)
    want = _check_evict(s, 256, 4, 64, 320)
    wide_w, wide_a = torch.full((3, 709), 9.0, device="cuda"), torch.full((3, 712), 7, dtype=torch.int32, device="cuda")
    for ws, as_ in ((shift, 0), (0, shift), (shift, shift)):
        wide_w[:, ws:ws + 704], wide_a[:, as_:as_ + 704] = s["w"].cuda(), s["a"].cuda()
        kv = s["kv"].cuda()
        got = mla.evict(kv, s["table"].cuda(), s["lens"].cuda(), wide_w[:, ws:ws + 704], 256, sink=4, recent=64,
                        arrival=wide_a[:, as_:as_ + 704], width=320)
        assert mla.get_device_status() == 0
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_evict_narrow_arrival_rows_bound_the_lengths():
    import mla_absorbed_decode_gb300 as mla
    s = _evict_inputs([60, 64], 256, False, seed=36)
    a = s["a"][:, :64].contiguous()
    want = _check_evict(s, 40, 2, 8, 256)
    kv = s["kv"].cuda()
    lens = torch.tensor([60, 64], dtype=torch.int32, device="cuda")
    buf = torch.empty(2 * 64 + 2 * 256, dtype=torch.int32, device="cuda")       # kept right behind arrival
    arrival, kept = buf[:128].view(2, 64), buf[128:].view(2, 256)
    arrival.copy_(a)
    got = mla.evict(kv, s["table"].cuda(), lens, s["w"].cuda(), 40, sink=2, recent=8, arrival=arrival, kept=kept)
    assert mla.get_device_status() == 0
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert torch.equal(arrival.cpu(), a)


# ------------------------------------------------------------ weights: large channels, the decode's lse --
@pytest.mark.parametrize("factor", [30.0, 300.0, 3000.0])
@pytest.mark.parametrize("causal", [False, True])
def test_attn_weights_fp8_a_large_channel_of_q(factor, causal):
    """One channel of q is `factor` times the others.  q travels as two E4M3 terms of q 2^k, its largest element in
    (224, 448]: what they leave of another element is at most half a step of the subnormal codes, 2^-10, so at most 2^-10 / 224
    < 2^-17 of the largest; a score moves by at most that times scale sum |k_d|, a term p by e^that - 1.  The rest as
    in test_gpu_cache.py."""
    w = W.Workload("weights_channel", B=2, s_q=2, H=16, fixed_seqlens=(300, 65), causal=causal, kv_fp8=True)
    inp = W.make_inputs(w, seed=37)
    inp["q"][..., 77] *= factor
    kv = inp["kv_cache"].numpy()
    q = to_np(inp["q"])
    B, s_q, H, _ = q.shape
    rows = [oracle.gather_request(kv, inp["block_table"][b].numpy(), int(inp["seqlens"][b]), inp["kv_scale"]) for b in range(B)]
    lse = np.full((B, s_q, H), -np.inf)
    for b in range(B):
        for i in range(s_q):
            v = oracle.mla.visible_tokens(int(inp["seqlens"][b]), s_q, i, causal)
            s = inp["softmax_scale"] * q[b, i] @ rows[b][:v].T
            lse[b, i] = s.max(axis=1) + np.log(np.exp(s - s.max(axis=1, keepdims=True)).sum(axis=1))
    inp["lse"] = torch.from_numpy(lse).float()
    inp["before"] = torch.zeros((B, inp["block_table"].shape[1] * 64))
    got = _run_weights(inp).double().numpy()
    for b in range(B):
        n = int(inp["seqlens"][b])
        want, room = np.zeros(n), np.full(n, 2.0 ** -126 * s_q * H)
        for i in range(s_q):
            v = oracle.mla.visible_tokens(n, s_q, i, causal)
            for h in range(H):
                s = inp["softmax_scale"] * rows[b][:v] @ q[b, i, h]
                arg = s - float(inp["lse"][b, i, h])
                p = np.exp(arg)
                mag = inp["softmax_scale"] * np.abs(rows[b][:v])
                off = 40 * 2.0 ** -23 * (mag @ np.abs(q[b, i, h])) + 2.0 ** -17 * np.abs(q[b, i, h]).max() * mag.sum(axis=1)
                off += 3 * 2.0 ** -24 * np.abs(arg)
                want[:v] += p
                room[:v] += p * (np.expm1(off) + 2.0 ** -22 + s_q * H * 2.0 ** -24)
        assert np.all(np.abs(got[b, :n] - want) <= room), (b, float((np.abs(got[b, :n] - want) / room).max()))
        assert np.all(got[b, n:] == 0)


@pytest.mark.parametrize("fp8", [False, True])
def test_attn_weights_a_query_row_that_is_not_finite(fp8):
    """It gives NaN to the tokens that it sees, no other request and no slot past the length; without weight, nothing."""
    w = W.Workload("weights_q_inf", B=3, s_q=1, H=32, fixed_seqlens=(100, 130, 70), kv_fp8=fp8)
    inp = _weights_inputs(w, seed=38)
    good = _run_weights(inp)
    for v in (float("nan"), float("inf")):
        bad = dict(inp, q=inp["q"].clone(), lse=inp["lse"].clone())
        bad["q"][1, 0, 5, 3] = v
        bad["lse"][1, 0, 5] = float("nan")       # what the decode gives for such a row
        got = _run_weights(bad)
        assert torch.isnan(got[1, :130]).all() and torch.equal(got[1, 130:], good[1, 130:])
        assert torch.equal(got[0], good[0]) and torch.equal(got[2], good[2])
        bad["lse"][1, 0, 5] = -float("inf")
        left = dict(inp, lse=inp["lse"].clone())
        left["lse"][1, 0, 5] = -float("inf")
        assert torch.equal(_run_weights(bad), _run_weights(left))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("peak", [1.0, 6.0])
def test_attn_weights_rows_sum_to_the_heads_with_the_decode_s_lse(fp8, peak):
    """A row's weights sum to 1 with the lse that the library's own decode gives, for flat rows and for peaked ones: both
    form a score to within 40 * 2^-23 of scale sum |q_d k_d| = A, so the sum is off by at most e^(2 A') - 1 for the largest such
    A', and the lse is an fp32 number of a few fp32 roundings (2^-20 of the largest |score|)."""
    import mla_absorbed_decode_gb300 as mla
    w = W.Workload("weights_sum", B=3, s_q=1, H=64, fixed_seqlens=(900, 64, 333), kv_fp8=fp8)
    inp = W.make_inputs(w, seed=39)
    inp["q"] *= peak
    dev = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in inp.items()}
    parts = mla.num_sm_parts(1, 64)
    meta = mla.decode_metadata(dev["seqlens"], 1, 64, False, parts)
    pool = (dev["q"], dev["kv_cache"]) + ((inp["kv_scale"],) if fp8 else ())
    _, lse = (mla.decode_fp8 if fp8 else mla.decode)(*pool, dev["block_table"], dev["seqlens"], inp["softmax_scale"],
                                                     False, meta, parts)
    inp["lse"], inp["before"] = lse.cpu(), torch.zeros((3, inp["block_table"].shape[1] * 64))
    got = _run_weights(inp).double().sum(dim=1).numpy()
    kv = inp["kv_cache"].numpy() if fp8 else inp["kv_cache"].float().numpy()
    q = to_np(inp["q"])
    for b in range(3):
        rows = oracle.gather_request(kv, inp["block_table"][b].numpy(), int(inp["seqlens"][b]), inp.get("kv_scale"))
        mag = inp["softmax_scale"] * np.abs(rows) @ np.abs(q[b, 0]).T
        off = 2 * 40 * 2.0 ** -23 * mag.max()
        if fp8:
            off += 2 * 2.0 ** -17 * np.abs(q[b]).max() * inp["softmax_scale"] * np.abs(rows).sum(axis=1).max()
        off += 2.0 ** -20 * mag.max()
        assert abs(got[b] - 64) <= 64 * (np.expm1(off) + 2.0 ** -14), (b, got[b], off)


def test_a_step_s_sections_need_positions():
    """Refused before anything is launched: the query buffer stays as it was."""
    import mla_absorbed_decode_gb300 as mla
    B, H = 2, 4
    step = mla.DecodeStep(B, 1, H, torch.tensor([3, 4], dtype=torch.int32, device="cuda"), False, 0.1)
    z = lambda *s: torch.zeros(s, dtype=BF, device="cuda")
    step.q.fill_(3.0)
    kv, table = z(2, 64, 576), torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    ops = (z(B, H, 128), z(B, H, 64), z(H, 128, 512))
    for call, args in ((step.absorb, ops), (step.absorb_and_plan, ops), (step.run, (*ops, z(H, 512, 128), kv, table)),
                       (step.capture, (*ops, z(H, 512, 128), kv, table))):
        with pytest.raises(ValueError, match="positions"):
            call(*args, sections=(16, 8, 8))
    torch.cuda.synchronize()
    assert torch.all(step.q == 3.0) and mla.get_device_status() == 0


def test_append_to_a_batch_padded_with_empty_requests():
    """new_offsets give an empty request no row: nothing is reported, the others' rows are written."""
    import mla_absorbed_decode_gb300 as mla
    g = torch.Generator().manual_seed(40)
    lens = torch.tensor([5, 0, 64, 0, 65, 0], dtype=torch.int32)
    offsets = torch.tensor([0, 1, 1, 2, 2, 3, 3], dtype=torch.int32)
    table = torch.tensor([[0, -1], [-1, -1], [1, -1], [-1, -1], [2, 3], [-1, -1]], dtype=torch.int32)
    rows, kv = torch.randn((3, 576), generator=g).to(BF), torch.randn((4, 64, 576), generator=g).to(BF)
    got = mla.cache_append(rows[:, :512].cuda(), rows[:, 512:].cuda(), kv.cuda(), table.cuda(), lens.cuda(),
                           new_offsets=offsets.cuda())
    assert mla.get_device_status() == 0
    want = kv.clone()
    want[0, 4], want[1, 63], want[3, 0] = rows[0], rows[1], rows[2]
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("plan", [False, True])
def test_a_captured_step_with_sections(plan):
    """capture(sections=...) and replay give what the calls one by one give, with positions changed in place."""
    import mla_absorbed_decode_gb300 as mla
    w = W.small_variant(W.V3, B=2, seqlen=200, H=16)
    inp = W.make_inputs(w, seed=41)
    dev = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in inp.items()}
    ops = [dev[k] for k in ("q_nope", "q_pe", "w_uk", "w_uv", "kv_cache", "block_table")]
    pos = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    step = mla.DecodeStep(2, 1, 16, dev["seqlens"], False, w.softmax_scale)
    step.plan()
    step.capture(*ops, plan=plan, positions=pos, sections=(16, 8, 8), interleaved=True)
    pos.copy_(torch.tensor([[200, 199], [3, 40], [17, 0]], dtype=torch.int32))
    o, q = step.replay().clone(), step.q.clone()
    turned = mla.rope_axes(dev["q_pe"], pos, (16, 8, 8), interleaved=True)
    assert torch.equal(q.view(2, 16, 576)[..., 512:], turned)
    step.run(dev["q_nope"], turned, *ops[2:])
    assert torch.equal(step.o, o) and torch.equal(step.q, q)
    assert mla.get_device_status() == 0


# ------------------------------------------------------------------- replayed calls, addresses past 32 bits --
@pytest.mark.parametrize("slots,lens", [(704, [700, 90, 640]), (40000, [39000, 40000])])
def test_evict_recorded_and_replayed_with_lengths_in_place(slots, lens):
    """A graph of the call with new_seqlens = seqlens, for requests of one CTA and of eight: every replay from the same
    cache and lengths gives what the call gives."""
    import mla_absorbed_decode_gb300 as mla
    s = _evict_inputs(lens, slots, True, seed=42)
    budget, width = slots // 3, slots // 3 + 64
    want = _check_evict(s, budget, 4, 64, width)
    dev = {k: v.cuda() for k, v in s.items()}
    kv, n = dev["kv"].clone(), dev["lens"].clone()
    outs = [torch.empty_like(t) for t in want[1:]]
    call = lambda: mla.evict_fp8(kv, dev["table"], n, dev["w"], budget, sink=4, recent=64, arrival=dev["a"], width=width,
                                 new_seqlens=n, kept=outs[0], weights_out=outs[1], arrival_out=outs[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    after = None
    for _ in range(3):
        kv.copy_(dev["kv"])
        n.copy_(dev["lens"])
        graph.replay()
        assert torch.equal(n, want[0])
        for x, y in zip(outs, want[1:]):
            assert torch.equal(x, y)
        after = kv.clone() if after is None else after
        assert torch.equal(kv, after)
    assert mla.get_device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_a_cache_of_more_than_4_gib(fp8):
    """Append, attention weights and eviction on pages whose addresses and element numbers pass 32 bits give the bits that
    they give in a small pool."""
    import mla_absorbed_decode_gb300 as mla
    far = 117000 if fp8 else 59000                       # pages: 4.3 GB, and more than 2^31 elements
    w = W.Workload("weights_far", B=2, s_q=1, H=32, fixed_seqlens=(300, 129), kv_fp8=fp8)
    inp = _weights_inputs(w, seed=43)
    g = torch.Generator().manual_seed(44)
    rows = torch.randn((2, 576), generator=g).to(BF).cuda()
    small, table = inp["kv_cache"].cuda(), inp["block_table"].cuda()
    big = torch.zeros((far + small.shape[0], 64, 576), dtype=small.dtype, device="cuda")
    assert big.numel() > 2 ** 31 and big.numel() * big.element_size() > 2 ** 32
    big[far:] = small
    seqlens = inp["seqlens"].cuda()
    scale = (inp["kv_scale"],) if fp8 else ()
    got = []
    for kv, bt in ((small, table), (big, torch.where(table >= 0, table + far, table))):
        (mla.cache_append_fp8 if fp8 else mla.cache_append)(rows[:, :512], rows[:, 512:], kv, *scale, bt, seqlens)
        weights = inp["before"].cuda()
        (mla.attn_weights_fp8 if fp8 else mla.attn_weights)(inp["q"].cuda(), inp["lse"].cuda(), kv, *scale, bt, seqlens,
                                                            inp["softmax_scale"], False, weights)
        left = (mla.evict_fp8 if fp8 else mla.evict)(kv, bt, seqlens, weights, 100, sink=2, recent=20)
        assert mla.get_device_status() == 0
        got.append((weights, *left))
    for x, y in zip(*got):
        assert torch.equal(x, y)
    bits = lambda t: t if fp8 else t.view(torch.int16)
    assert torch.equal(bits(big[far:]), bits(small))
    assert not bits(big[:far]).any()


def test_rope_axes_into_a_query_of_more_than_2_31_elements():
    import mla_absorbed_decode_gb300 as mla
    g = torch.Generator().manual_seed(45)
    N, H = 30000, 128
    x, pos = torch.randn((1, H, 64), generator=g).to(BF).cuda(), _positions(3, N, g).cuda()
    q = torch.zeros((N, H, 576), dtype=BF, device="cuda")
    assert q.numel() > 2 ** 31
    mla.rope_axes(x.expand(N, H, 64), pos, (16, 8, 8), out=q[..., 512:])
    for n in (0, 1, 14563, 14564, 29127, N - 1):
        assert torch.equal(q[n, :, 512:], mla.rope_axes(x, pos[:, n:n + 1].contiguous(), (16, 8, 8))[0])
    assert not q[-300:, :, :512].any() and not q[:300, :, :512].any()
    assert mla.get_device_status() == 0
