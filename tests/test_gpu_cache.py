"""GPU parity of the latent-cache operators against the float64 oracle: rotation with several position
axes, the write of new rows, the attention weight of cached tokens, eviction by it, and a run of them
together.

Tolerances, derived from the arithmetic (u = 2^-24, the half step of fp32; a bf16 result is off by at
most 2^-8 of its value, an E4M3 one by 2^-4 of it, or 2^-10 where it is subnormal):
* rotation: a cosine or sine is within 2^-21 (hardware sine) + 2^-22 + 2^-23 (an argument of up to pi,
  rounded, and its ~1e-7 rad) < 2^-20 of the exact one, and two products and a sum add 3u: an
  element moves by at most (2^-20 + 3u) (|x0| + |x1|) < 2^-19 (|x0| + |x1|) before the final rounding;
* attention weight: a score's products are exact in fp32 and are summed in at most 40 additions at the
  level of the MMA (576 / 16) or of the warp, each off by at most 2^-23 of sum |q_d k_d|, so a term p moves by at
  most 40 * 2^-23 * scale * sum |q_d k_d| of itself; over an FP8 cache q travels as two E4M3 terms whose sum
  is off by at most 2^-18 max |q| an element, so it moves by 2^-18 max |q| scale sum |k_d| more;
  exp2, its argument (|x| <= 128) and the sum over <= 512 rows add (2^-22 + 2 * 128 * 2^-24 + 512 * 2^-24) < 2^-14;
* copied values, whole numbers and moved rows: equal.
"""
import numpy as np
import pytest
import torch

import oracle
from mla_absorbed_decode_gb300 import workloads as W

from _harness import compare, oracle_decode, to_np

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_absorbed_decode_gb300 import build_lib
    build_lib.build()
    yield


def _positions(axes, N, g, top=131072):
    return torch.randint(0, top, (axes, N), generator=g, dtype=torch.int32)


def _rope_room(x):
    a = np.abs(x)
    return 2.0 ** -19 * np.repeat(a[..., 0::2] + a[..., 1::2], 2, axis=-1)


# ------------------------------------------------------------------------------------- rope --
@pytest.mark.parametrize("N,H,sections,interleaved", [(1, 1, (32,), False), (5, 16, (16, 8, 8), False),
                                                      (64, 128, (16, 8, 8), True), (130, 3, (0, 31, 1), True),
                                                      (33, 40, (5, 9, 11, 7), False)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_axes(N, H, sections, interleaved, inverse):
    import mla_absorbed_decode_gb300 as mla
    g = torch.Generator().manual_seed(N * 131 + H)
    x = torch.randn((N, H, 64), generator=g).to(BF)
    pos = _positions(len(sections), N, g)
    pos[:, 0] = (1 << 24) - 1
    pos[-1, 0] = -((1 << 24) - 1)
    got = mla.rope_axes(x.cuda(), pos.cuda(), sections, interleaved=interleaved, inverse=inverse)
    ref = oracle.rope_axes(to_np(x), pos.numpy(), sections, interleaved=interleaved, inverse=inverse)
    assert np.all(np.abs(to_np(got) - ref) <= 2.0 ** -8 * np.abs(ref) + _rope_room(to_np(x)))


def test_rope_axes_strides_views_and_in_place():
    import mla_absorbed_decode_gb300 as mla
    g = torch.Generator().manual_seed(3)
    N, H, sections = 37, 12, (16, 8, 8)
    pos = _positions(3, N, g).cuda()
    wide = torch.randn((N, H, 192), generator=g).to(BF).cuda()       # q_nope and q_pe of a head side by side
    x = wide[..., 128:]
    want = mla.rope_axes(x.contiguous(), pos, sections)
    q = torch.full((N, H, 576), 7.0, dtype=BF, device="cuda")
    got = mla.rope_axes(x, pos, sections, out=q[..., 512:])
    assert got.data_ptr() == q[..., 512:].data_ptr()
    assert torch.equal(q[..., 512:], want) and torch.all(q[..., :512] == 7.0)
    heads_first = torch.empty((H, N, 64), dtype=BF, device="cuda").transpose(0, 1)
    assert torch.equal(mla.rope_axes(x, pos, sections, out=heads_first), want)
    one = x[:, :1].contiguous()                                      # a row that all heads read
    assert torch.equal(mla.rope_axes(one.expand(N, H, 64), pos, sections),
                       mla.rope_axes(one, pos, sections).expand(N, H, 64))
    odd = torch.empty((3, N + 5), dtype=torch.int32, device="cuda")  # positions that are part of a longer buffer
    odd[:, :N] = pos
    assert torch.equal(mla.rope_axes(x, odd[:, :N], sections), want)
    mla.rope_axes(x, pos, sections, out=x)
    assert torch.equal(x, want)
    assert mla.rope_axes(x[:0], pos[:, :0], sections).shape == (0, H, 64)


def test_rope_axes_one_axis_is_the_absorption_s_rope():
    import mla_absorbed_decode_gb300 as mla
    g = torch.Generator().manual_seed(4)
    N, H = 65, 8
    q_nope, q_pe = torch.randn((N, H, 128), generator=g).to(BF).cuda(), torch.randn((N, H, 64), generator=g).to(BF).cuda()
    w_uk = torch.randn((H, 128, 512), generator=g).to(BF).cuda()
    pos = torch.randint(0, 1 << 24, (N,), generator=g, dtype=torch.int32).cuda()
    q1, q2 = (torch.empty((N, H, 576), dtype=BF, device="cuda") for _ in range(2))
    mla.absorb_q(q_nope, w_uk, q1, q_pe=q_pe, positions=pos)
    mla.absorb_q(q_nope, w_uk, q2)
    mla.rope_axes(q_pe, pos, out=q2[..., 512:])
    assert torch.equal(q1, q2)


def test_rope_axes_gradient_against_differences():
    """out is linear in x: <g, out(x + d) - out(x)> = <inverse(g), d>, up to the roundings of the four calls."""
    import mla_absorbed_decode_gb300 as mla
    g = torch.Generator().manual_seed(5)
    x, d, grad = (torch.randn((9, 4, 64), generator=g).to(BF).cuda() for _ in range(3))
    xd = (x.double() + d.double()).to(BF)
    d = xd.double() - x.double()
    pos = _positions(3, 9, g).cuda()
    kw = dict(sections=(10, 12, 10), interleaved=True)
    diff = mla.rope_axes(xd, pos, **kw).double() - mla.rope_axes(x, pos, **kw).double()
    back = mla.rope_axes(grad, pos, inverse=True, **kw).double()
    lhs, rhs = (grad.double() * diff).sum(), (back * d).sum()
    size = lambda a: torch.repeat_interleave(a.double().abs()[..., 0::2] + a.double().abs()[..., 1::2], 2, dim=-1)
    room = (2.0 ** -8 + 2.0 ** -19) * ((grad.double().abs() * (size(xd) + size(x))).sum() + (size(grad) * d.abs()).sum())
    assert abs(lhs - rhs) <= room


def test_rope_axes_refusals():
    import mla_absorbed_decode_gb300 as mla
    x = torch.zeros((4, 2, 64), dtype=BF, device="cuda")
    pos = torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    for bad in (dict(sections=(16, 8)), dict(sections=(16, 8, 9)), dict(sections=(40, -4, -4)),
                dict(out=torch.zeros((4, 2, 64), device="cuda")), dict(out=torch.zeros((4, 3, 64), dtype=BF, device="cuda")),
                dict(out=torch.zeros((4, 1, 64), dtype=BF, device="cuda").expand(4, 2, 64)),
                dict(rope_theta=1.0), dict(rope_theta=float("nan"))):
        with pytest.raises((ValueError, TypeError, mla.MLAError)):
            mla.rope_axes(x, pos, **{"sections": (16, 8, 8), **bad})
    with pytest.raises((ValueError, TypeError)):
        mla.rope_axes(x, pos.long(), (16, 8, 8))
    with pytest.raises((ValueError, TypeError)):
        mla.rope_axes(x, pos.cpu(), (16, 8, 8))
    with pytest.raises((ValueError, TypeError)):
        mla.rope_axes(x.float(), pos, (16, 8, 8))
    with pytest.raises(mla.MLAError):
        mla.rope_axes(torch.zeros(4 * 2 * 64 + 1, dtype=BF, device="cuda")[1:].view(4, 2, 64), pos, (16, 8, 8))


# ----------------------------------------------------------------------------------- append --
def _append_case(lens, new, fp8, seed, pad=0, axes=3):
    """Inputs of one append: seqlens `lens` of which `new` rows each are new, `pad` rows that belong to nobody."""
    g = torch.Generator().manual_seed(seed)
    pages = [(n + 63) // 64 for n in lens]
    pool = sum(pages) + 3
    perm = torch.randperm(pool, generator=g).int()
    table = torch.full((len(lens), max(pages + [1])), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = perm[at:at + k]
        at += k
    offsets = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
    N = int(offsets[-1]) + pad
    rows = torch.randn((N, 576), generator=g).to(BF)
    kv = torch.randint(0, 255, (pool, 64, 576), generator=g, dtype=torch.uint8) if fp8 else \
        torch.randn((pool, 64, 576), generator=g).to(BF)
    return dict(lens=torch.tensor(lens, dtype=torch.int32), table=table, offsets=offsets, rows=rows, kv=kv,
                pos=_positions(axes, N, g))


def _check_append(s, kv, fp8, kv_scale, rotated, sections, interleaved=False):
    x = to_np(s["rows"])
    want = oracle.append_rows(x[:, :512], x[:, 512:], s["pos"].numpy() if rotated else None, sections,
                              interleaved=interleaved)
    room = np.zeros_like(x)
    if rotated:
        room[:, 512:] = _rope_room(x[:, 512:])
    touched = torch.zeros(kv.shape[:2], dtype=torch.bool)
    for r, page, slot in oracle.append_slots(s["table"].numpy(), s["lens"].numpy(), s["offsets"].numpy()):
        touched[page, slot] = True
        if not fp8:
            got = to_np(kv[page, slot])
            assert np.array_equal(got[:512], x[r, :512])
            if rotated:
                assert np.all(np.abs(got - want[r])[512:] <= (2.0 ** -8 * np.abs(want[r]) + room[r])[512:])
            else:
                assert np.array_equal(got, x[r])
        else:
            code = kv[page, slot].numpy()
            plain = oracle.dequantize_e4m3(oracle.e4m3_round(x[r].astype(np.float32) / np.float32(kv_scale)), 1.0)
            got = oracle.dequantize_e4m3(code, 1.0)
            exact = slice(0, 512) if rotated else slice(0, 576)
            assert np.array_equal(got[exact], plain[exact])
            y = np.clip(want[r] / kv_scale, -448, 448)
            assert np.all(np.abs(got - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10) + room[r] / kv_scale * 1.07)
    assert torch.equal(kv[~touched], s["kv"][~touched])     # nothing else was written


@pytest.mark.parametrize("lens,new,pad", [([1], [1], 0), ([64, 65, 1], [1, 1, 1], 0), ([200, 64, 63, 5], [70, 64, 1, 0], 0),
                                          ([0, 130, 0, 7], [0, 130, 0, 3], 5), ([1000, 3], [999, 2], 1)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rotated", [False, True])
def test_cache_append(lens, new, pad, fp8, rotated):
    import mla_absorbed_decode_gb300 as mla
    s = _append_case(lens, new, fp8, seed=sum(lens) + pad, pad=pad)
    kv, rows = s["kv"].cuda(), s["rows"].cuda()
    more = dict(new_offsets=s["offsets"].cuda())
    if rotated:
        more.update(positions=s["pos"].cuda(), sections=(16, 8, 8))
    if fp8:
        mla.cache_append_fp8(rows[:, :512], rows[:, 512:], kv, 2.0 ** -6, s["table"].cuda(), s["lens"].cuda(), **more)
    else:
        mla.cache_append(rows[:, :512], rows[:, 512:], kv, s["table"].cuda(), s["lens"].cuda(), **more)
    assert mla.get_device_status() == 0
    _check_append(s, kv.cpu(), fp8, 2.0 ** -6, rotated, (16, 8, 8))


def test_cache_append_even_rows_many_requests_and_a_scale_that_is_no_power_of_two():
    import mla_absorbed_decode_gb300 as mla
    B = 1100                                    # more requests than one search step of a warp covers
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(2, 150, (B,), generator=g).tolist()
    s = _append_case(lens, [2] * B, True, seed=9)
    c, pe = s["rows"][:, :512].contiguous().cuda(), s["rows"][:, 512:].contiguous().cuda()
    for offsets in (None, s["offsets"].cuda()):
        kv = s["kv"].cuda()
        mla.cache_append_fp8(c, pe, kv, 0.0123, s["table"].cuda(), s["lens"].cuda(), new_offsets=offsets,
                             positions=s["pos"].cuda(), sections=(8, 12, 12), interleaved=True)
        assert mla.get_device_status() == 0
        _check_append(s, kv.cpu(), True, float(np.float32(0.0123)), True, (8, 12, 12), interleaved=True)


def test_cache_append_fp8_special_values():
    import mla_absorbed_decode_gb300 as mla
    s = _append_case([3], [1], True, seed=2)
    row = torch.zeros(576)
    row[:8] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e30, -1e30, 2.0 ** -20, -0.0, 448.0])
    s["rows"][0] = row.to(BF)
    kv = s["kv"].cuda()
    mla.cache_append_fp8(s["rows"][:, :512].cuda(), s["rows"][:, 512:].cuda(), kv, 1.0, s["table"].cuda(), s["lens"].cuda())
    got = kv.cpu()[int(s["table"][0, 0]), 2, :8].tolist()
    assert got[0] & 0x7F == 0x7F and got[1:] == [0x7E, 0xFE, 0x7E, 0xFE, 0x00, 0x80, 0x7E]


def test_cache_append_bad_pages_and_lengths_are_reported_and_skipped():
    import mla_absorbed_decode_gb300 as mla
    s = _append_case([70, 5, 2, 300], [2, 2, 3, 1], False, seed=3)      # request 2 is shorter than its new rows
    s["table"][1, 0] = s["kv"].shape[0]                                 # and request 1's page does not exist
    s["table"][0, 1], page = -5, int(s["table"][0, 1])                  # nor do those of request 0's new rows
    kv = s["kv"].cuda()
    mla.cache_append(s["rows"][:, :512].cuda(), s["rows"][:, 512:].cuda(), kv, s["table"].cuda(), s["lens"].cuda(),
                     new_offsets=s["offsets"].cuda())
    assert mla.get_device_status() == 6                                 # MLA_ERR_DEVICE_BOUNDS
    want = s["kv"].clone()
    r = s["rows"]
    want[s["table"][2, 0].long(), 0], want[s["table"][2, 0].long(), 1] = r[5], r[6]   # its rows 1 and 2 fit
    want[s["table"][3, 4].long(), 300 - 1 - 256] = r[7]
    assert torch.equal(kv.cpu(), want)


def test_cache_refusals():
    import mla_absorbed_decode_gb300 as mla
    dev = "cuda"
    kv = torch.zeros((4, 64, 576), dtype=BF, device=dev)
    table, lens = torch.zeros((2, 2), dtype=torch.int32, device=dev), torch.ones(2, dtype=torch.int32, device=dev)
    c, pe = torch.zeros((2, 512), dtype=BF, device=dev), torch.zeros((2, 64), dtype=BF, device=dev)
    refused = (ValueError, TypeError, mla.MLAError)
    for args in ((c.float(), pe, kv, table, lens), (c, pe.float(), kv, table, lens), (c, pe, kv.view(torch.int16), table, lens),
                 (c, pe, kv[:, :, :512], table, lens), (c, pe, kv, table.long(), lens), (c, pe, kv, table[:1], lens),
                 (c, pe, kv, table, lens.cpu()), (c[:1], pe, kv, table, lens), (c[:, ::2], pe, kv, table, lens),
                 (c.repeat(2, 1)[:3], pe.repeat(2, 1)[:3], kv, table, lens)):
        with pytest.raises(refused):
            mla.cache_append(*args)
    with pytest.raises(refused):
        mla.cache_append(c, pe, kv, table, lens, new_offsets=torch.zeros(2, dtype=torch.int32, device=dev))
    with pytest.raises(refused):
        mla.cache_append(c, pe, kv, table, lens, positions=torch.zeros((2, 2), dtype=torch.int32, device=dev))
    with pytest.raises(refused):
        mla.cache_append_fp8(c, pe, kv, 1.0, table, lens)
    q, lse = torch.zeros((2, 1, 16, 576), dtype=BF, device=dev), torch.zeros((2, 1, 16), device=dev)
    w = torch.zeros((2, 128), device=dev)
    for args in ((q.float(), lse, kv, table, lens, 0.1, False, w), (q, lse.double(), kv, table, lens, 0.1, False, w),
                 (q, lse[:, :, :8], kv, table, lens, 0.1, False, w), (q, lse, kv, table, lens, 0.1, False, w.double()),
                 (q, lse, kv, table, lens, 0.0, False, w), (q, lse, kv, table, lens, 0.1, False, w[:, ::2]),
                 (q, lse, kv, table, lens, 0.1, False, w[:, :64]), (q.transpose(1, 2), lse, kv, table, lens, 0.1, False, w),
                 (torch.zeros((2, 5, 128, 576), dtype=BF, device=dev), torch.zeros((2, 5, 128), device=dev), kv, table, lens,
                  0.1, False, w)):
        with pytest.raises(refused):
            mla.attn_weights(*args)
    with pytest.raises(refused):
        mla.attn_weights_fp8(q, lse, kv, 1.0, table, lens, 0.1, False, w)
    for more in (dict(budget=0), dict(budget=8, sink=4, recent=5), dict(budget=8, sink=-1), dict(budget=100, width=99),
                 dict(budget=8, weights_out=w), dict(budget=8, kept=torch.zeros((2, 128), device=dev)),
                 dict(budget=8, arrival=torch.zeros((2, 128), device=dev)),
                 dict(budget=8, new_seqlens=torch.zeros(3, dtype=torch.int32, device=dev))):
        with pytest.raises(refused):
            mla.evict(kv, table, lens, w, **more)
    assert mla.get_device_status() == 0


# ---------------------------------------------------------------------------------- weights --
def _weights_inputs(w, seed=0, seqlens=None, slots=None):
    inp = W.make_inputs(w, seed=seed, seqlens=seqlens)      # unused pages and slots hold NaN
    _, lse, _ = oracle_decode(inp)
    g = torch.Generator().manual_seed(seed + 1)
    inp["lse"] = torch.from_numpy(lse).float()
    inp["before"] = torch.rand((inp["q"].shape[0], slots or inp["block_table"].shape[1] * 64), generator=g)
    return inp


def _run_weights(inp, before=None):
    import mla_absorbed_decode_gb300 as mla
    got = (inp["before"] if before is None else before).cuda()
    args = (inp["block_table"].cuda(), inp["seqlens"].cuda(), inp["softmax_scale"], inp["causal"], got)
    if "kv_scale" in inp:
        mla.attn_weights_fp8(inp["q"].cuda(), inp["lse"].cuda(), inp["kv_cache"].cuda(), inp["kv_scale"], *args)
    else:
        mla.attn_weights(inp["q"].cuda(), inp["lse"].cuda(), inp["kv_cache"].cuda(), *args)
    assert mla.get_device_status() == 0
    return got.cpu()


def _check_weights(inp, got, only=None):
    kv = inp["kv_cache"].numpy() if "kv_scale" in inp else inp["kv_cache"].float().numpy()
    sel = list(range(len(inp["seqlens"]))) if only is None else only
    q = to_np(inp["q"][sel])
    ref, spread = oracle.attn_weights(q, to_np(inp["lse"][sel]), kv, inp["block_table"][sel].numpy(),
                                      inp["seqlens"][sel].numpy(), inp["softmax_scale"], inp["causal"], inp.get("kv_scale"))
    for i, b in enumerate(sel):
        n = int(inp["seqlens"][b])
        before = inp["before"][b].double().numpy()
        want = before[:n] + ref[i]
        room = 40 * 2.0 ** -23 * spread[i] + 2.0 ** -14 * ref[i] + 2.0 ** -24 * want
        if "kv_scale" in inp and n:
            rows = oracle.gather_request(kv, inp["block_table"][b].numpy(), n, inp["kv_scale"])
            room += 2.0 ** -18 * np.abs(q[i]).max() * inp["softmax_scale"] * np.abs(rows).sum(axis=1) * ref[i]
        d = np.abs(got[b, :n].double().numpy() - want)
        assert np.all(d <= room), (b, float((d - room).max()))
        if n:      # the errors of a token's rows are of either sign: over the tokens they stay far below the bound
            assert np.linalg.norm(d) <= 1e-5 * np.linalg.norm(want)
        assert torch.equal(got[b, n:], inp["before"][b, n:])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,s_q,H,causal,lens", [
    (1, 1, 1, False, (1,)),
    (2, 1, 16, False, (256, 300)),
    (4, 1, 128, False, (64, 0, 65, 1000)),
    (3, 1, 77, False, (63, 128, 129)),
    (2, 2, 128, True, (130, 700)),
    (3, 3, 100, True, (1, 2, 200)),          # the first query positions of a short request see nothing
    (2, 4, 128, True, (70, 333)),
    (2, 4, 128, False, (70, 333)),
    (3, 5, 37, True, (500, 7, 0)),
])
def test_attn_weights(fp8, B, s_q, H, causal, lens):
    w = W.Workload("weights", B=B, s_q=s_q, H=H, fixed_seqlens=lens, causal=causal, kv_fp8=fp8)
    inp = _weights_inputs(w, seed=B * 7 + H)
    _check_weights(inp, _run_weights(inp))


def test_attn_weights_many_short_requests():
    w = W.Workload("weights_many", B=700, s_q=1, H=16, ragged_max=90)
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 90, (700,), generator=g, dtype=torch.int32)
    inp = _weights_inputs(w, seed=3, seqlens=lens)
    _check_weights(inp, _run_weights(inp))


def test_attn_weights_long_with_outliers():
    w = W.Workload("weights_long", B=2, s_q=1, H=128, fixed_seqlens=(20000, 777), outlier_p=0.01, outlier_scale=8.0)
    inp = _weights_inputs(w, seed=8)
    _check_weights(inp, _run_weights(inp))


@pytest.mark.parametrize("fp8", [False, True])
def test_attn_weights_same_bits_every_time_and_on_another_stream(fp8):
    w = W.Workload("weights_bits", B=5, s_q=2, H=128, fixed_seqlens=(1000, 64, 3, 513, 2000), causal=True, kv_fp8=fp8)
    inp = _weights_inputs(w, seed=4)
    first = _run_weights(inp)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = _run_weights(inp)
    assert torch.equal(first, second)
    # alone or in the batch: a request's weights do not depend on the others
    one = dict(inp, q=inp["q"][3:4], lse=inp["lse"][3:4], block_table=inp["block_table"][3:4], seqlens=inp["seqlens"][3:4])
    assert torch.equal(_run_weights(one, before=inp["before"][3:4])[0], first[3])


def test_attn_weights_row_without_weight_and_row_strides():
    """Rows whose lse is -inf add nothing, whatever their scores; rows of weights may be part of a wider buffer."""
    import mla_absorbed_decode_gb300 as mla
    w = W.Workload("weights_rows", B=2, s_q=1, H=64, fixed_seqlens=(150, 90))
    inp = _weights_inputs(w, seed=6, slots=192)
    inp["lse"][0, 0, ::2] = -float("inf")
    inp["q"][0, 0, 0] = float("nan")
    inp["lse"][1, 0, 5] = float("inf")
    wide = torch.full((2, 500), 3.0, device="cuda")
    wide[:, 100:292] = inp["before"].cuda()
    mla.attn_weights(inp["q"].cuda(), inp["lse"].cuda(), inp["kv_cache"].cuda(), inp["block_table"].cuda(),
                     inp["seqlens"].cuda(), inp["softmax_scale"], False, wide[:, 100:292])
    assert mla.get_device_status() == 0
    assert torch.all(wide[:, :100] == 3.0) and torch.all(wide[:, 292:] == 3.0)
    inp["q"][0, 0, 0] = 0.0
    _check_weights(inp, wide[:, 100:292].cpu())


def test_attn_weights_bad_lengths_and_pages_are_reported():
    import mla_absorbed_decode_gb300 as mla
    w = W.Workload("weights_bad", B=4, s_q=1, H=16, fixed_seqlens=(100, 130, 70, 64))
    inp = _weights_inputs(w, seed=7)
    lens = inp["seqlens"].clone()
    lens[0], lens[2] = 193, -3                     # longer than the table's three pages; negative
    table = inp["block_table"].clone()
    table[1, 1] = inp["kv_cache"].shape[0]
    got = inp["before"].cuda()
    mla.attn_weights(inp["q"].cuda(), inp["lse"].cuda(), inp["kv_cache"].cuda(), table.cuda(), lens.cuda(),
                     inp["softmax_scale"], False, got)
    assert mla.get_device_status() == 6
    got = got.cpu()
    good = _run_weights(inp)
    assert torch.equal(got[0], inp["before"][0]) and torch.equal(got[2], inp["before"][2])
    assert torch.equal(got[3], good[3])
    assert torch.equal(got[1, :64], good[1, :64]) and torch.equal(got[1, 64:128], inp["before"][1, 64:128])
    assert torch.equal(got[1, 128:], good[1, 128:])


@pytest.mark.parametrize("fp8", [False, True])
def test_attn_weights_full_benchmark_shape(fp8):
    """The benchmark's shape, four of its requests against the oracle (lse from the decode), the rest through the sum:
    a row's weights sum to 1, so a request's to H."""
    import mla_absorbed_decode_gb300 as mla
    w = W.Workload("weights_v3", B=64, s_q=1, H=128, seqlen=4096, kv_fp8=fp8)
    inp = W.make_inputs(w)
    dev = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in inp.items()}
    parts = mla.num_sm_parts(1, 128)
    meta = mla.decode_metadata(dev["seqlens"], 1, 128, False, parts)
    pool = (dev["q"], dev["kv_cache"]) + ((inp["kv_scale"],) if fp8 else ())
    _, lse = (mla.decode_fp8 if fp8 else mla.decode)(*pool, dev["block_table"], dev["seqlens"], inp["softmax_scale"],
                                                     False, meta, parts)
    assert mla.get_device_status() == 0
    inp["lse"], inp["before"] = lse.cpu(), torch.zeros((64, 4096))
    got = _run_weights(inp)
    _check_weights(inp, got, only=[0, 21, 40, 63])
    # lse is within 1e-3 of the exact one (the decode's bound), so a row's sum is within about as much of 1
    assert torch.all((got.double().sum(dim=1) - 128).abs() <= 128 * 2e-3)


# ------------------------------------------------------------------------------------ evict --
def _evict_inputs(lens, slots, fp8, seed, ties=False, arrival=True, pool_extra=2):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pages = [(n + 63) // 64 for n in lens]
    pool = sum(pages) + pool_extra
    perm = torch.randperm(pool, generator=g).int()
    table = torch.full((B, (slots + 63) // 64), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = perm[at:at + k]
        at += k
    kv = torch.randint(0, 256, (pool, 64, 576), generator=g, dtype=torch.uint8) if fp8 else \
        torch.randint(-32768, 32768, (pool, 64, 576), generator=g, dtype=torch.int16).view(BF)
    w = torch.exp(2 * torch.randn((B, slots), generator=g))
    if ties:
        w = torch.randint(0, 5, (B, slots), generator=g).float() * 0.25
    a = torch.full((B, slots), 123456789, dtype=torch.int32)
    for b, n in enumerate(lens):
        a[b, :n] = (torch.randperm(n, generator=g) * 2 + b).int()
        w[b, n:] = float("nan")                       # slots past the length hold anything
    return dict(lens=torch.tensor(lens, dtype=torch.int32), table=table, kv=kv, w=w, a=a if arrival else None)


def _bits(t):
    return t.view(torch.int16) if t.dtype == BF else t


def _check_evict(s, budget, sink=0, recent=0, width=None, **more):
    import mla_absorbed_decode_gb300 as mla
    kv = s["kv"].cuda()
    fp8 = kv.dtype == torch.uint8
    call = mla.evict_fp8 if fp8 else mla.evict
    left, kept, wo, ao = call(kv, s["table"].cuda(), s["lens"].cuda(), s["w"].cuda(), budget, sink=sink, recent=recent,
                              arrival=None if s["a"] is None else s["a"].cuda(), width=width, **more)
    assert mla.get_device_status() == 0
    width = s["w"].shape[1] if width is None else width
    want_kv = _bits(s["kv"]).clone()
    for b, n in enumerate(s["lens"].tolist()):
        m, k, w, a = oracle.evict(n, s["w"][b].tolist(), None if s["a"] is None else s["a"][b].tolist(), budget, sink,
                                  recent, width)
        assert int(left[b]) == m
        assert np.array_equal(kept[b].cpu().numpy(), k), b
        assert np.array_equal(wo[b].cpu().numpy(), w.astype(np.float32), equal_nan=True)
        assert np.array_equal(ao[b].cpu().numpy(), a)
        for j in np.nonzero(k[:m] != np.arange(m))[0]:
            t = int(k[j])
            want_kv[s["table"][b, j // 64].long(), j % 64] = _bits(s["kv"])[s["table"][b, t // 64].long(), t % 64]
    assert torch.equal(_bits(kv.cpu()), want_kv)
    return left, kept, wo, ao


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,slots,budget,sink,recent,width", [
    ([1], 1, 1, 0, 0, None),
    ([2], 64, 1, 0, 1, None),
    ([300, 0, 40, 1], 320, 64, 4, 16, 128),
    ([100, 65, 64, 63], 128, 64, 0, 0, 64),
    ([1000, 999, 33], 1024, 777, 10, 300, 777 + 64),
    ([5000, 64, 4097], 5056, 2048, 0, 2048, 2048),      # only the newest stay
    ([5000], 5056, 2048, 2048, 0, 2100),
    ([70, 20], 128, 500, 3, 5, 200),                    # nothing to evict: the outputs carry everything over
])
def test_evict(fp8, lens, slots, budget, sink, recent, width):
    s = _evict_inputs(lens, slots, fp8, seed=slots + budget)
    _check_evict(s, budget, sink, recent, width)


@pytest.mark.parametrize("arrival", [False, True])
def test_evict_ties_go_to_the_lowest_slot(arrival):
    s = _evict_inputs([3000, 700, 64], 3008, False, seed=5, ties=True, arrival=arrival)
    _check_evict(s, 512, 4, 32, 600)
    s["w"][:] = 0.0
    _check_evict(s, 512, 4, 32, 600)
    s["w"][0, ::2] = -0.0           # equal to +0
    _check_evict(s, 511, 0, 0, 600)


def test_evict_special_weights():
    s = _evict_inputs([900, 513], 960, True, seed=6)
    g = torch.Generator().manual_seed(1)
    for v in (float("nan"), float("inf"), -float("inf"), -1.0, 1e-44, 3e38, 0.0):
        s["w"][torch.rand(s["w"].shape, generator=g) < 0.12] = v
    _check_evict(s, 300, 2, 20, 400)
    s["w"][:] = float("nan")
    _check_evict(s, 300, 2, 20, 400)


def test_evict_long_request_beside_short_ones():
    s = _evict_inputs([131072, 5, 60000], 131072, True, seed=7)
    _check_evict(s, 16384, 64, 4096, 16384 + 64)
    s = _evict_inputs([100000], 131072, True, seed=8, arrival=False)
    _check_evict(s, 99999, 0, 0, 100032)


def test_evict_in_place_lengths_given_outputs_and_equal_bits():
    import mla_absorbed_decode_gb300 as mla
    s = _evict_inputs([700, 90, 640], 704, False, seed=9)
    first = _check_evict(s, 256, 4, 64, 320)
    outs = [torch.empty_like(t) for t in first]
    lens = s["lens"].cuda()
    outs[0] = lens
    kv = s["kv"].cuda()
    got = mla.evict(kv, s["table"].cuda(), lens, s["w"].cuda(), 256, sink=4, recent=64, arrival=s["a"].cuda(), width=320,
                    new_seqlens=lens, kept=outs[1], weights_out=outs[2], arrival_out=outs[3])
    assert mla.get_device_status() == 0
    for x, y in zip(got, first):
        assert torch.equal(x, y)
    assert got[1].data_ptr() == outs[1].data_ptr()


def test_evict_bad_lengths_and_pages_are_reported():
    import mla_absorbed_decode_gb300 as mla
    s = _evict_inputs([300, 200, 250], 320, False, seed=10)
    s["lens"][0] = 321
    table = s["table"].clone()
    table[1, 0] = s["kv"].shape[0]                    # the page that most of request 1's free slots lie in
    kv = s["kv"].cuda()
    left, kept, wo, ao = mla.evict(kv, table.cuda(), s["lens"].cuda(), s["w"].cuda(), 64, arrival=s["a"].cuda())
    assert mla.get_device_status() == 6
    assert left.tolist() == [0, 64, 64]
    want = _bits(s["kv"]).clone()
    m, k, _, _ = oracle.evict(250, s["w"][2].tolist(), s["a"][2].tolist(), 64, 0, 0, 320)
    for j in np.nonzero(k[:m] != np.arange(m))[0]:
        want[table[2, 0].long(), j] = _bits(s["kv"])[table[2, int(k[j]) // 64].long(), int(k[j]) % 64]
    assert torch.equal(_bits(kv.cpu()), want)


# ----------------------------------------------------------------------------- all together --
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("graph", [False, True])
def test_a_layer_s_steps_with_eviction(fp8, graph):
    """Decode steps over a cache that is kept within a budget: append (rotated by three axes), the step, its weights,
    eviction now and then.  Every step's output against the expanded definition over the cache's rows, whose tokens the
    oracle's own eviction (from the library's weights, which are checked beside it) keeps count of."""
    import mla_absorbed_decode_gb300 as mla
    g = torch.Generator().manual_seed(11)
    B, H, budget, sections, kv_scale = 3, 16, 128, (16, 8, 8), 2.0 ** -6
    capacity = 192
    dev = torch.device("cuda")
    lens = torch.tensor([120, 128, 7], dtype=torch.int32)
    table = torch.randperm(B * 3 + 2, generator=g).int()[:B * 3].view(B, 3)
    base = torch.randn((B * 3 + 2, 64, 576), generator=g)
    kv = ((base / kv_scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else base.to(BF)).to(dev)
    w_uk, w_uv = (torch.randn(s, generator=g) / 512 ** 0.5 for s in ((H, 128, 512), (H, 512, 128)))
    w_uk, w_uv = w_uk.to(BF), w_uv.to(BF)
    seqlens = lens.to(dev)
    step = mla.DecodeStep(B, 1, H, seqlens, False, 192 ** -0.5, device=dev, kv_scale=kv_scale if fp8 else None)
    tbl = table.to(dev)
    weights = torch.zeros((B, capacity), device=dev)
    arrival = torch.arange(capacity, dtype=torch.int32, device=dev).repeat(B, 1)
    held = [list(range(int(n))) for n in lens]                 # the oracle's cache: arrival numbers in slot order
    total = lens.tolist()
    bufs = dict(c=torch.empty((B, 512), dtype=BF, device=dev), k_pe=torch.empty((B, 64), dtype=BF, device=dev),
                q_nope=torch.empty((B, H, 128), dtype=BF, device=dev), q_pe=torch.empty((B, H, 64), dtype=BF, device=dev),
                pos=torch.zeros((3, B), dtype=torch.int32, device=dev))
    values = lambda: oracle.dequantize_e4m3(kv.cpu().numpy(), kv_scale) if fp8 else to_np(kv)

    def whole_step():
        step.append(bufs["c"], bufs["k_pe"], kv, tbl, positions=bufs["pos"], sections=sections)
        step.absorb_and_plan(bufs["q_nope"], bufs["q_pe"], wk, positions=bufs["pos"],
                             sections=sections)
        step._decode(kv, tbl)
        mla.unabsorb_o(step.out.view(B, H, 512), wv, o=step.o)
        step.accumulate_weights(kv, tbl, weights)

    wk, wv = w_uk.to(dev), w_uv.to(dev)
    recorded = None
    for i in range(24):
        c, pe = torch.randn((B, 512), generator=g).to(BF), torch.randn((B, 64), generator=g).to(BF)
        qn, qp = torch.randn((B, H, 128), generator=g).to(BF), torch.randn((B, H, 64), generator=g).to(BF)
        pos = torch.randint(0, 4096, (3, B), generator=g, dtype=torch.int32)
        for k, v in (("c", c), ("k_pe", pe), ("q_nope", qn), ("q_pe", qp), ("pos", pos)):
            bufs[k].copy_(v)
        seqlens += 1
        before_w = weights.cpu()
        if graph and recorded is None and i == 1:
            recorded = torch.cuda.CUDAGraph()
            with torch.cuda.graph(recorded):
                whole_step()
        recorded.replay() if recorded is not None else whole_step()
        assert mla.get_device_status() == 0
        for b in range(B):
            held[b].append(total[b])
            total[b] += 1
        now = values()
        n = np.array([len(h) for h in held])
        assert seqlens.tolist() == n.tolist()
        want_row = oracle.append_rows(to_np(c), to_np(pe), pos.numpy(), sections)
        got_row = np.stack([now[int(table[b, (n[b] - 1) // 64]), (n[b] - 1) % 64] for b in range(B)])
        step_of = (2.0 ** -4 * np.abs(want_row) + 2.0 ** -10 * kv_scale) if fp8 else 2.0 ** -8 * np.abs(want_row)
        assert np.all(np.abs(got_row - want_row) <= step_of * 1.01 + 2.0 ** -18 * 8)
        q_rot = oracle.rope_axes(to_np(qp), pos.numpy(), sections)
        ref, _ = oracle.decode_expanded(to_np(qn)[:, None], q_rot[:, None], to_np(w_uk), to_np(w_uv), now, table.numpy(), n,
                                        192 ** -0.5)
        assert np.abs(to_np(step.o)[:, None] - ref).max() <= 2e-2
        w_ref, _ = oracle.attn_weights(to_np(step.q), to_np(step.lse), now, table.numpy(), n, 192 ** -0.5)
        for b in range(B):
            assert np.allclose(weights[b, :n[b]].cpu().numpy(), before_w[b, :n[b]].numpy() + w_ref[b],
                               rtol=1e-3 if fp8 else 3e-4, atol=1e-6)
            assert np.array_equal(arrival[b, :n[b]].cpu().numpy(), held[b])
        if i % 8 == 7:
            rows = [[now[int(table[b, t // 64]), t % 64].copy() for t in range(n[b])] for b in range(B)]
            wh, ah = weights.cpu(), arrival.cpu()
            kept, weights2, arrival2 = step.evict(kv, tbl, weights, budget, sink=2, recent=16, arrival=arrival)
            assert mla.get_device_status() == 0
            now = values()
            for b in range(B):
                m, k, wo, ao = oracle.evict(n[b], wh[b].tolist(), ah[b].tolist(), budget, 2, 16, capacity)
                assert np.array_equal(kept[b].cpu().numpy(), k)
                held[b] = [int(v) for v in ao[:m]]
                for j in range(m):
                    assert np.array_equal(now[int(table[b, j // 64]), j % 64], rows[b][int(k[j])], equal_nan=True)
            weights.copy_(weights2)
            arrival.copy_(arrival2)
    assert n.tolist()[0] > budget - 8 and max(len(h) for h in held) <= budget


def test_evicted_cache_decodes_like_the_kept_tokens():
    """The decode over an evicted cache is the decode over the tokens that stayed (order does not matter)."""
    import mla_absorbed_decode_gb300 as mla
    w = W.Workload("evicted", B=2, s_q=1, H=128, fixed_seqlens=(1500, 800))
    inp = W.make_inputs(w, seed=12)
    dev = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in inp.items()}
    g = torch.Generator().manual_seed(2)
    weights = torch.rand((2, 1536), generator=g)
    left, kept, _, _ = mla.evict(dev["kv_cache"], dev["block_table"], dev["seqlens"], weights.cuda(), 512, sink=4, recent=64)
    parts = mla.num_sm_parts(1, 128)
    meta = mla.decode_metadata(left, 1, 128, False, parts)
    out, lse = mla.decode(dev["q"], dev["kv_cache"], dev["block_table"], left, inp["softmax_scale"], False, meta, parts)
    assert mla.get_device_status() == 0
    kv = inp["kv_cache"].float().numpy()
    idx = np.sort(np.where(kept[:, :512].cpu().numpy() < 0, 1 << 30, kept[:, :512].cpu().numpy()), axis=1)
    ref_out, ref_lse = oracle.decode_sparse(to_np(inp["q"]), kv, inp["block_table"].numpy(), inp["seqlens"].numpy(), idx,
                                            left.cpu().numpy(), inp["softmax_scale"])[:2]
    compare(out.cpu(), lse.cpu(), ref_out, ref_lse, what="after eviction")


def test_calls_on_two_streams_at_once():
    """The operators keep nothing between calls: two layers' calls on two streams give what each gives alone."""
    import mla_absorbed_decode_gb300 as mla
    cases = []
    for seed in (21, 22):
        inp = _weights_inputs(W.Workload("two", B=3, s_q=1, H=64, fixed_seqlens=(900, 64, 500)), seed=seed)
        e = _evict_inputs([900, 64, 500], 960, False, seed=seed)
        cases.append((inp, e, _run_weights(inp), _check_evict(e, 300, 2, 32, 320)))
    moved = [({k: (v.cuda() if torch.is_tensor(v) else v) for k, v in inp.items()},
              {k: v.cuda() for k, v in e.items()}) for inp, e, _, _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for (inp, e), stream in zip(moved, streams):
        with torch.cuda.stream(stream):
            for _ in range(4):     # the last one's inputs are as the first one's
                w = inp["before"].clone()
                mla.attn_weights(inp["q"], inp["lse"], inp["kv_cache"], inp["block_table"], inp["seqlens"],
                                 inp["softmax_scale"], False, w)
                ev = mla.evict(e["kv"].clone(), e["table"], e["lens"], e["w"], 300, sink=2, recent=32, arrival=e["a"],
                               width=320)
            got.append((w, ev))
    torch.cuda.synchronize()
    assert mla.get_device_status() == 0
    for (w, ev), (_, _, want_w, want_ev) in zip(got, cases):
        assert torch.equal(w.cpu(), want_w)
        for x, y in zip(ev, want_ev):
            assert torch.equal(x, y)


def test_outputs_made_for_a_given_stream_are_that_stream_s_memory():
    """`stream=` without an output: the output is free for other work only when that stream has passed."""
    import mla_absorbed_decode_gb300 as mla
    side = torch.cuda.Stream()
    x = torch.randn(33, 2, 64, generator=torch.Generator().manual_seed(31)).to(torch.bfloat16).cuda()
    pos = torch.arange(33, dtype=torch.int32).repeat(1, 1).cuda()
    want = mla.rope_axes(x, pos)
    e = {k: v.cuda() for k, v in _evict_inputs([70, 9], 128, False, seed=32).items()}
    torch.cuda.synchronize()
    out = mla.rope_axes(x, pos, stream=side)
    left = mla.evict(e["kv"], e["table"], e["lens"], e["w"], 64, arrival=e["a"], stream=side)
    before = [t.data_ptr() for t in (out, *left)]
    del left
    on_main = torch.empty_like(out)
    assert on_main.data_ptr() not in before      # the side stream's pool is not the current stream's
    side.synchronize()
    assert torch.equal(out, want)
    assert mla.get_device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,s_q,longest", [(300, 2, 90), (150, 4, 200), (220, 3, 90)])
def test_attn_weights_many_short_requests_of_several_row_blocks(fp8, B, s_q, longest):
    """Requests of a page or two, one after the other on every cluster of two, three and four CTAs."""
    w = W.Workload("weights_blocks", B=B, s_q=s_q, H=128, ragged_max=longest, causal=True, kv_fp8=fp8)
    g = torch.Generator().manual_seed(B)
    inp = _weights_inputs(w, seed=9, seqlens=torch.randint(0, longest, (B,), generator=g, dtype=torch.int32))
    _check_weights(inp, _run_weights(inp))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("s_q", [2, 3, 4])
def test_attn_weights_of_several_row_blocks_bad_pages_and_a_replayed_call(fp8, s_q):
    import mla_absorbed_decode_gb300 as mla
    w = W.Workload("weights_blocks_bad", B=4, s_q=s_q, H=128, fixed_seqlens=(100, 130, 70, 64), kv_fp8=fp8)
    inp = _weights_inputs(w, seed=17)
    good = _run_weights(inp)
    lens, table = inp["seqlens"].clone(), inp["block_table"].clone()
    lens[0], lens[2] = 193, -3
    table[1, 1] = -1
    dev = {k: inp[k].cuda() for k in ("q", "lse", "kv_cache")}
    scale = (inp["kv_scale"],) if fp8 else ()
    call = mla.attn_weights_fp8 if fp8 else mla.attn_weights
    got = inp["before"].cuda()
    call(dev["q"], dev["lse"], dev["kv_cache"], *scale, table.cuda(), lens.cuda(), inp["softmax_scale"], False, got)
    assert mla.get_device_status() == 6
    got = got.cpu()
    for b in (0, 2):
        assert torch.equal(got[b], inp["before"][b])
    assert torch.equal(got[3], good[3])
    assert torch.equal(got[1, :64], good[1, :64]) and torch.equal(got[1, 64:128], inp["before"][1, 64:128])
    assert torch.equal(got[1, 128:], good[1, 128:])
    # recorded once, replayed from the same weights
    lens, table, out = inp["seqlens"].cuda(), inp["block_table"].cuda(), inp["before"].cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(dev["q"], dev["lse"], dev["kv_cache"], *scale, table, lens, inp["softmax_scale"], False, out)
    for _ in range(3):
        out.copy_(inp["before"])
        graph.replay()
        assert torch.equal(out.cpu(), good)
    assert mla.get_device_status() == 0
