"""GPU parity of the calls on a 4-bit latent cache against the float64 oracle: the write of new rows, the dense and the
sparse decode, and a run of them together.

Tolerances, derived from the arithmetic (u = 2^-24, the half step of fp32):
* append: what is stored are whole numbers, and the float32 quotients they come from are off by less than 2^-19 of
  themselves (the norm's sum of 512 squares in 21 additions, halved by the root, rsqrt within 2^-22, four products and the
  division): a code or scale equals the oracle's unless the exact quotient lies that near to a number halfway between two.
  The rotation moves a value by at most 2^-19 (|x0| + |x1|), as for the other caches;
* decode: q (a row times a power of two in fp16; elements below 2^-28 of its largest are rounded to within 2^-39 of it) times
  the exact cached values is added up in at most 44 steps, each off by at most 2^-23 of sum |q_d k_d|: a score is off by
  r = 45 * 2^-23 * scale * sum |q_d k_d|, plus 2^-20 for the exponential.  A probability, rounded to fp16 (2^-11; 2^-31 absolute
  for those below the normal range, the offset of 2^6 included), moves by 2 r + 2^-11 of itself, and the products with the values
  are added up in n / 16 + 44 steps of 2^-23.  With A = sum p |v|:
      |out - ref| <= 2^-8 |ref| + A (2 r + 2^-11 + (n / 16 + 44) 2^-23 + 2^-18) + n 2^-31 max |v|
      |lse - ref| <= r + n u + 2^-20 + 2^-21 |ref|
"""
import numpy as np
import pytest
import torch

import oracle
from mla_absorbed_decode_gb300 import workloads as W

from _harness import make, to_np

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
SCALE = 1.0 / np.sqrt(192.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_absorbed_decode_gb300 import build_lib
    build_lib.build()
    yield


# ------------------------------------------------------------------------------------- cases --
def _poison(kv, table, lens):
    """Bytes that no request holds become codes of NaN scales and NaN rope codes."""
    used = np.zeros(kv.shape[:2], dtype=bool)
    for row, n in zip(table, lens):
        for t in range(int(n)):
            used[row[t // 64], t % 64] = True
    kv[~used] = 0x7F


def _case(seqlens, s_q=1, H=16, causal=None, seed=0, kv_scale=2.0 ** -6, outliers=0.0, topk=None, extra_blocks=0,
          values=None):
    """CPU tensors and the cache's values."""
    rng = np.random.default_rng(seed)
    B = len(seqlens)
    nb = [(n + 63) // 64 for n in seqlens]
    pool = sum(nb) + 2
    perm = rng.permutation(pool)
    table = np.full((B, max(max(nb), 1) + extra_blocks), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, : nb[b]] = perm[at:at + nb[b]]
        at += nb[b]
    x = rng.normal(0, 1, (pool, 64, 576)) if values is None else values(rng, pool)
    if outliers:
        x[rng.random((pool, 64)) < outliers] *= 8.0
    kv = oracle.pack_fp4(x, kv_scale)
    _poison(kv, table, seqlens)
    q = torch.from_numpy(rng.normal(0, 1, (B, s_q, H, 576))).to(BF)
    inp = dict(q=q, kv=torch.from_numpy(kv), kv_scale=kv_scale, table=torch.from_numpy(table),
               seqlens=torch.tensor(seqlens, dtype=torch.int32), causal=s_q > 1 if causal is None else causal)
    if topk is not None:   # a number of entries a request
        most = max(max(topk), 1)
        idx = np.full((B, most), -1, dtype=np.int32)
        for b, k in enumerate(topk):
            idx[b, :k] = np.sort(rng.choice(seqlens[b], size=k, replace=k > seqlens[b]))
        inp.update(indices=torch.from_numpy(idx), topk_lens=torch.tensor(topk, dtype=torch.int32))
    return inp


def _run(inp, parts=None, **more):
    import mla_absorbed_decode_gb300 as mla
    q, kv, table, n = (inp[k].cuda() for k in ("q", "kv", "table", "seqlens"))
    _, s_q, H, _ = q.shape
    P = mla.num_sm_parts(s_q, H) if parts is None else parts
    if "indices" in inp:
        idx, k = inp["indices"].cuda(), inp["topk_lens"].cuda()
        meta = mla.decode_metadata(k, s_q, H, inp["causal"], P)
        out, lse = mla.decode_sparse_fp4(q, kv, inp["kv_scale"], table, n, idx, k, SCALE, inp["causal"], meta, P, **more)
    else:
        meta = mla.decode_metadata(n, s_q, H, inp["causal"], P)
        out, lse = mla.decode_fp4(q, kv, inp["kv_scale"], table, n, SCALE, inp["causal"], meta, P, **more)
    assert mla.get_device_status() == 0
    return out.cpu(), lse.cpu()


def _ref(inp):
    q, kv = to_np(inp["q"]), oracle.unpack_fp4(inp["kv"].numpy(), inp["kv_scale"])
    table, n = inp["table"].numpy(), inp["seqlens"].numpy()
    if "indices" in inp:
        return (kv, *oracle.decode_sparse(q, kv, table, n, inp["indices"].numpy(), inp["topk_lens"].numpy(), SCALE,
                                          causal=inp["causal"], with_abs=True))
    return (kv, *oracle.decode_absorbed(q, kv, table, n, SCALE, causal=inp["causal"], with_abs=True))


def _compare(inp, got, ref, what=""):
    out, lse = to_np(got[0]), to_np(got[1])
    kv, r_out, r_lse, r_abs = ref
    q = np.abs(to_np(inp["q"]))
    for b, n in enumerate(inp["seqlens"].tolist()):
        t = inp["indices"].numpy()[b, : int(inp["topk_lens"][b])] if "indices" in inp else np.arange(n)
        if len(t) == 0:
            assert np.all(out[b] == 0) and np.all(np.isneginf(lse[b])), what
            continue
        k = np.abs(kv[inp["table"].numpy()[b, t // 64], t % 64])
        r = 45 * 2.0 ** -23 * SCALE * np.max(q[b] @ k.T, axis=-1) + 2.0 ** -20      # [s_q, H]
        m = len(t)
        room = 2.0 ** -8 * np.abs(r_out[b]) + r_abs[b] * (2 * r[..., None] + 2.0 ** -11 + (m / 16 + 44) * 2.0 ** -23 +
                                                          2.0 ** -18) + m * 2.0 ** -31 * k[:, :512].max()
        none = np.isneginf(r_lse[b])
        assert np.array_equal(none, np.isneginf(lse[b])), what
        d = np.abs(out[b] - r_out[b])
        assert np.all(d <= room), (what, b, d.max(), np.max(d / np.maximum(room, 1e-30)))
        with np.errstate(invalid="ignore"):
            dl = np.where(none, 0.0, np.abs(lse[b] - r_lse[b]))
        l_room = r + m * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -21 * np.where(none, 0.0, np.abs(r_lse[b]))
        assert np.all(dl <= l_room), (what, b, dl.max(), np.max(dl / l_room))


# -------------------------------------------------------------------------------------- dense --
@pytest.mark.parametrize("H", [1, 16, 128])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129])
def test_lengths_around_a_page_and_a_tile(H, n):
    inp = _case([n], H=H, seed=n)
    _compare(inp, _run(inp), _ref(inp), f"H={H} n={n}")


@pytest.mark.parametrize("H,seqlens", [(16, [63, 64, 65]), (128, [64 * 5 + 7, 1000]), (64, [130, 2, 511]), (96, [700, 1]),
                                        (128, [4096]), (17, [300, 0, 77]), (127, [513, 640])])
def test_unsplit_and_split(H, seqlens):
    inp = _case(seqlens, H=H, seed=H + len(seqlens))
    ref = _ref(inp)
    for parts in (None, 1, 2, 3, 5, 13):
        _compare(inp, _run(inp, parts), ref, f"H={H} parts={parts}")


@pytest.mark.parametrize("s_q,H", [(2, 128), (2, 16), (3, 128), (4, 128), (3, 40), (2, 20), (3, 127), (4, 1), (2, 65)])
@pytest.mark.parametrize("causal", [True, False])
def test_query_positions(s_q, H, causal):
    inp = _case([1, 2, 65, 300, 1025], s_q=s_q, H=H, causal=causal, seed=s_q * 100 + H)
    ref = _ref(inp)
    for parts in (None, 3):
        _compare(inp, _run(inp, parts), ref, f"s_q={s_q} H={H} parts={parts}")


def test_rows_that_see_nothing():
    inp = _case([0, 1, 3, 0, 66], s_q=4, H=24, seed=3)
    ref = _ref(inp)
    for parts in (1, 2, None):
        got = _run(inp, parts)
        _compare(inp, got, ref, f"parts={parts}")
        assert torch.all(got[0][1, :3] == 0) and torch.all(torch.isneginf(got[1][1, :3]))
    none = _case([0, 0], H=16)
    out, lse = _run(none)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


@pytest.mark.parametrize("kv_scale", [0.0123, 0.5, 2.0 ** -20, 2.0 ** 20])
def test_scales(kv_scale):
    # cached values of unit size whatever the scale: group scales over E4M3's whole range, or rounded to its ends
    inp = _case([300, 777], H=128, seed=2, kv_scale=kv_scale)
    _compare(inp, _run(inp, 3), _ref(inp), f"kv_scale={kv_scale}")


def test_every_code_and_scale():
    """Every pair of a scale and a code there is, in tokens and dims that go through both halves of the kernel."""
    def values(rng, pool):
        return np.zeros((pool, 64, 576))
    inp = _case([256], H=32, seed=4, values=values)
    kv = inp["kv"].numpy()
    row = kv.reshape(-1, 352)
    rng = np.random.default_rng(0)
    row[:, :256] = rng.integers(0, 256, row[:, :256].shape)
    row[:, 256:288] = rng.integers(0, 0x7F, row[:, 256:288].shape) | rng.choice([0, 0x80], row[:, 256:288].shape)
    row[:, 288:] = rng.integers(0, 0x7F, row[:, 288:].shape) | rng.choice([0, 0x80], row[:, 288:].shape)
    inp["kv_scale"] = 2.0 ** -9
    _compare(inp, _run(inp), _ref(inp), "all codes")


@pytest.mark.parametrize("parts", [None, 1, 6])
def test_outlier_rows_and_rescaling(parts):
    inp = _case([3000, 5000], H=128, outliers=0.02, seed=5)
    _compare(inp, _run(inp, parts), _ref(inp), "outliers")


def test_a_maximum_that_grows_with_every_page():
    """Scores that rise by more than any rebase threshold from tile to tile, and one-hot softmaxes."""
    inp = _case([1024], H=128, seed=6)
    kv, table = inp["kv"].numpy(), inp["table"].numpy()[0]
    for t in range(1024):
        kv[table[t // 64], t % 64, 256:288] = min(0x7E, 0x08 + 8 * (t // 64))    # the scales double from page to page
    _compare(inp, _run(inp, 1), _ref(inp), "growing")
    inp["table"] = inp["table"].flip(1).contiguous()
    _compare(inp, _run(inp, 1), _ref(inp), "falling")


@pytest.mark.parametrize("factor", [2.0 ** -60, 2.0 ** 12])
def test_heads_of_different_sizes(factor):
    """Rows of q whose sizes are far apart share a tile, and every one keeps its precision."""
    inp = _case([333, 90], H=128, seed=7)
    inp["q"][:, :, 1::3] *= factor
    inp["q"][:, :, 5] = 0.0
    inp["q"][:, :, 7, 100:] *= 2.0 ** -20
    _compare(inp, _run(inp), _ref(inp), f"factor={factor}")


def test_nan_in_q_and_in_the_cache_stays_in_its_rows():
    inp = _case([200, 130], H=40, seed=8)
    clean = _run(inp)
    inp["q"][0, 0, 3, 17] = float("nan")
    inp["q"][1, 0, 9, 570] = float("inf")
    out, lse = _run(inp)
    bad = torch.zeros((2, 1, 40), dtype=torch.bool)
    bad[0, 0, 3] = bad[1, 0, 9] = True
    assert torch.all(out[bad].isnan()) and torch.all(lse[bad].isnan())
    assert torch.equal(out[~bad], clean[0][~bad]) and torch.equal(lse[~bad], clean[1][~bad])
    again = _case([200, 130], H=40, seed=8)
    again["kv"][int(again["table"][1, 0]), 5, 256 + 3] = 0x7F         # one group of one token of request 1
    out, lse = _run(again)
    assert torch.equal(out[0], clean[0][0]) and torch.all(lse[1].isnan()) and torch.all(out[1].isnan())


def test_poison_never_reaches_the_result():
    seqlens = [100, 129, 64, 1]
    inp = _case(seqlens, H=128, seed=11, extra_blocks=4)
    clean = _case(seqlens, H=128, seed=11)
    clean["kv"][clean["kv"] == 0x7F] = 0x11
    inp["kv"] = clean["kv"].clone()
    _poison(inp["kv"].numpy(), inp["table"].numpy(), seqlens)
    assert int((inp["kv"] == 0x7F).sum()) > 0
    a, b = _run(inp, 4), _run(clean, 4)
    _compare(clean, b, _ref(clean))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_equal_inputs_give_equal_bits():
    inp = _case([700, 3000], H=128, seed=9)
    a = _run(inp, 5)
    for _ in range(3):
        b = _run(inp, 5)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------------------------- sparse --
@pytest.mark.parametrize("s_q,H", [(1, 128), (2, 128), (1, 16), (3, 50), (4, 128)])
def test_sparse(s_q, H):
    inp = _case([900, 64, 1, 300, 70], s_q=s_q, H=H, topk=[500, 64, 1, 129, 0], seed=H + s_q)
    ref = _ref(inp)
    for parts in (None, 1, 3):
        _compare(inp, _run(inp, parts), ref, f"s_q={s_q} H={H} parts={parts}")


def test_sparse_duplicates_and_unsorted_lists():
    inp = _case([500, 40], H=64, topk=[200, 100], seed=21)       # 100 entries of 40 tokens
    g = torch.Generator().manual_seed(0)
    for b, k in enumerate(inp["topk_lens"].tolist()):
        inp["indices"][b, :k] = inp["indices"][b, :k][torch.randperm(k, generator=g)]
    _compare(inp, _run(inp), _ref(inp))


def test_sparse_lists_of_all_tokens_equal_the_dense_decode():
    inp = _case([257, 640], H=128, topk=[257, 640], seed=22)
    dense = {k: v for k, v in inp.items() if k not in ("indices", "topk_lens")}
    a, b = _run(inp, 3), _run(dense, 3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_sparse_rows_of_a_wider_index_tensor():
    inp = _case([300, 200], H=32, topk=[100, 64], seed=23)
    want = _run(inp)
    wide = torch.full((2, 333), -7, dtype=torch.int32).cuda()
    wide[:, :100] = inp["indices"].cuda()
    inp["indices"] = wide[:, :100]
    got = _run(inp)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_sparse_causal_lists_whose_rows_see_nothing():
    inp = _case([200], s_q=3, H=16, topk=[4], seed=24)
    inp["indices"][0, :4] = torch.tensor([198, 199, 199, 198])
    got = _run(inp)
    _compare(inp, got, _ref(inp))
    assert torch.all(torch.isneginf(got[1][0, 0])) and torch.all(torch.isfinite(got[1][0, 1:]))


# ------------------------------------------------------------------------------------ reports --
def test_bad_pages_and_entries_are_reported():
    import mla_absorbed_decode_gb300 as mla
    inp = _case([300, 100], H=16, seed=31)
    good = _run(inp)
    for value in (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        bad = dict(inp, table=inp["table"].clone())
        bad["table"][0, 2] = value
        q, kv, table, n = (bad[k].cuda() for k in ("q", "kv", "table", "seqlens"))
        P = mla.num_sm_parts(1, 16)
        out, lse = mla.decode_fp4(q, kv, bad["kv_scale"], table, n, SCALE, False, mla.decode_metadata(n, 1, 16, False, P), P)
        assert mla.get_device_status() == 6
        assert torch.equal(out[1].cpu(), good[0][1]) and torch.equal(lse[1].cpu(), good[1][1])
        assert mla.get_device_status() == 0
    inp = _case([300, 100], H=16, topk=[50, 20], seed=32)
    good = _run(inp)
    for value in (-1, 300, 2 ** 31 - 1, -2 ** 31):
        idx = inp["indices"].clone()
        idx[0, 7] = value
        q, kv, table, n, k = (inp[k].cuda() for k in ("q", "kv", "table", "seqlens", "topk_lens"))
        P = mla.num_sm_parts(1, 16)
        out, lse = mla.decode_sparse_fp4(q, kv, inp["kv_scale"], table, n, idx.cuda(), k, SCALE, False,
                                         mla.decode_metadata(k, 1, 16, False, P), P)
        assert mla.get_device_status() == 6
        assert torch.equal(out[1].cpu(), good[0][1]) and torch.equal(lse[1].cpu(), good[1][1])
    # a list that its row of indices has no room for
    q, kv, table, n = (inp[k].cuda() for k in ("q", "kv", "table", "seqlens"))
    k = torch.tensor([80, 20], dtype=torch.int32, device="cuda")
    out, lse = mla.decode_sparse_fp4(q, kv, inp["kv_scale"], table, n, inp["indices"].cuda(), k, SCALE, False,
                                     mla.decode_metadata(k, 1, 16, False, P), P)
    assert mla.get_device_status() == 6
    # a length beyond the table
    inp = _case([300, 100], H=16, seed=33)
    q, kv, table = (inp[k].cuda() for k in ("q", "kv", "table"))
    n = torch.tensor([100, 400], dtype=torch.int32, device="cuda")
    mla.decode_fp4(q, kv, inp["kv_scale"], table, n, SCALE, False, mla.decode_metadata(n, 1, 16, False, P), P)
    assert mla.get_device_status() == 6


# ------------------------------------------------------------------------------------- append --
def _append_case(new, past, seed, axes=3, norm=True, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    B, N = len(new), sum(new)
    lens = [p + k for p, k in zip(past, new)]
    pages = [(n + 63) // 64 for n in lens]
    perm = torch.randperm(sum(pages) + 1, generator=g).to(torch.int32)
    table = torch.full((B, max(max(pages), 1)), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, : pages[b]] = perm[at:at + pages[b]]
        at += pages[b]
    rows = (torch.randn((N, 576), generator=g) * spread).to(BF)
    return dict(rows=rows, table=table, lens=torch.tensor(lens, dtype=torch.int32),
                offsets=torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32),
                kv=torch.randint(0, 256, (sum(pages) + 1, 64, 352), generator=g, dtype=torch.uint8),
                positions=torch.randint(0, 131072, (axes, N), generator=g, dtype=torch.int32),
                norm=(1 + 0.3 * torch.randn((512,), generator=g)).to(BF) if norm else None)


def _near(v, table, room):
    """Which values lie within `room` of themselves of a number halfway between two of a sorted table."""
    mid = (table[:-1] + table[1:]) / 2
    a = np.abs(v)[..., None]
    return np.any(np.abs(a - mid) <= room * a, axis=-1)


def _check_rows(got, y, pe, pe_room, kv_scale, exact):
    """The written bytes [N, 352] against the values that they come from."""
    want = oracle.pack_fp4(np.concatenate((y, pe), axis=1), kv_scale)
    unit = float(np.float32(kv_scale))
    room = 0.0 if exact else 2.0 ** -19
    e4m3 = np.array([oracle.e4m3_value(c) for c in range(127)])
    g = y.reshape(-1, 32, 16)
    scale, w_scale = got[:, 256:288], want[:, 256:288]
    if kv_scale == 2.0 ** -6 and exact:    # every quotient's halves are exact: nothing may differ
        assert np.array_equal(scale, w_scale) and np.array_equal(got[:, :256], want[:, :256])
    ok = (scale == w_scale) | _near(np.abs(g).max(axis=2) / 6 / unit, e4m3, max(room, 2.0 ** -22))
    assert np.all(ok)
    code = np.stack((got[:, :256] & 15, got[:, :256] >> 4), axis=-1).reshape(-1, 32, 16)
    w_code = np.stack((want[:, :256] & 15, want[:, :256] >> 4), axis=-1).reshape(-1, 32, 16)
    step = (oracle.dequantize_e4m3(w_scale, 1.0) * unit)[..., None]
    near = _near(np.where(step > 0, g / np.where(step > 0, step, 1.0), 0.0), oracle.E2M1_VALUES[:8], max(room, 2.0 ** -22))
    same = (scale == w_scale)[..., None]
    assert np.all((code == w_code) | near | ~same)
    assert np.mean(scale == w_scale) > 0.99 or scale.size < 1000
    back = oracle.dequantize_e4m3(got[:, 288:], 1.0) * unit
    half = np.maximum(2.0 ** -4 * np.abs(pe), 2.0 ** -10 * unit)
    assert np.all(np.abs(back - np.clip(pe, -448 * unit, 448 * unit)) <= half + pe_room)


@pytest.mark.parametrize("kv_scale", [2.0 ** -6, 0.013])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("new,past", [([1], [0]), ([1] * 5, [63, 64, 0, 200, 1]), ([3, 0, 130, 1], [62, 7, 0, 127])])
def test_append(new, past, norm, kv_scale):
    import mla_absorbed_decode_gb300 as mla
    s = _append_case(new, past, seed=sum(new) + norm, norm=norm)
    d = {k: v.cuda() for k, v in s.items() if v is not None}
    kv = mla.cache_append_fp4(d["rows"][:, :512], d["rows"][:, 512:], d["kv"], kv_scale, d["table"], d["lens"],
                              new_offsets=d["offsets"], positions=d["positions"], sections=(16, 8, 8),
                              norm_weight=d.get("norm"))
    assert kv is d["kv"] and mla.get_device_status() == 0
    slots = oracle.append_slots(s["table"].numpy(), s["lens"].numpy(), s["offsets"].numpy())
    got, before = kv.cpu().numpy(), s["kv"].numpy()
    x = to_np(s["rows"])
    y = oracle.normed_latent(x[:, :512], to_np(s["norm"]), 1e-6) if norm else x[:, :512]
    pe = oracle.rope_axes(x[:, None, 512:], s["positions"].numpy(), (16, 8, 8))[:, 0]
    a = np.abs(x[:, 512:])
    pe_room = 2.0 ** -19 * np.repeat(a[:, 0::2] + a[:, 1::2], 2, axis=1) * 1.07
    rows = np.stack([got[page, slot] for _, page, slot in slots])
    order = [r for r, _, _ in slots]
    _check_rows(rows, y[order], pe[order], pe_room[order], kv_scale, not norm)
    written = np.zeros(got.shape[:2], dtype=bool)
    for _, page, slot in slots:
        written[page, slot] = True
    assert np.array_equal(got[~written], before[~written])


@pytest.mark.parametrize("spread", [1e-6, 1e-3, 1.0, 300.0, 1e6])
def test_append_small_and_large_values(spread):
    """Groups whose scales are 0, subnormal and saturated."""
    import mla_absorbed_decode_gb300 as mla
    s = _append_case([70, 3], [0, 61], seed=5, norm=False, spread=spread)
    s["rows"][4, :16] = 0.0
    s["rows"][5, 40] = float("nan")
    s["rows"][6, 33], s["rows"][6, 34] = float("inf"), float("-inf")
    d = {k: v.cuda() for k, v in s.items() if v is not None}
    kv = mla.cache_append_fp4(d["rows"][:, :512], d["rows"][:, 512:], d["kv"], 2.0 ** -6, d["table"], d["lens"],
                              new_offsets=d["offsets"])
    assert mla.get_device_status() == 0
    got = kv.cpu().numpy()
    want = oracle.pack_fp4(to_np(s["rows"]), 2.0 ** -6)
    for r, page, slot in oracle.append_slots(s["table"].numpy(), s["lens"].numpy(), s["offsets"].numpy()):
        assert np.array_equal(got[page, slot], want[r]), r


def test_append_strides_even_rows_and_padding():
    import mla_absorbed_decode_gb300 as mla
    s = _append_case([2, 2, 2], [5, 63, 126], seed=6)
    d = {k: v.cuda() for k, v in s.items() if v is not None}
    more = dict(positions=d["positions"], sections=(10, 11, 11), interleaved=True, norm_weight=d["norm"], norm_eps=1e-3)
    want = mla.cache_append_fp4(d["rows"][:, :512].contiguous(), d["rows"][:, 512:].contiguous(), d["kv"].clone(), 0.02,
                                d["table"], d["lens"], new_offsets=d["offsets"], **more)
    got = mla.cache_append_fp4(d["rows"][:, :512], d["rows"][:, 512:], d["kv"].clone(), 0.02, d["table"], d["lens"], **more)
    assert torch.equal(got, want)
    # a padded batch: rows behind the last request's, and a request without rows, leave the cache as it was
    rows = torch.cat((d["rows"], d["rows"][:3]))
    pos = torch.cat((d["positions"], d["positions"][:, :3]), dim=1)
    offsets = torch.tensor([0, 2, 4, 6, 6], dtype=torch.int32, device="cuda")
    table = torch.cat((d["table"], torch.full_like(d["table"][:1], -1)))
    lens = torch.cat((d["lens"], torch.zeros_like(d["lens"][:1])))
    got = mla.cache_append_fp4(rows[:, :512], rows[:, 512:], d["kv"].clone(), 0.02, table, lens, new_offsets=offsets,
                               **dict(more, positions=pos))
    assert torch.equal(got, want) and mla.get_device_status() == 0
    none = mla.cache_append_fp4(rows[:0, :512], rows[:0, 512:], d["kv"], 0.02, table, lens, new_offsets=offsets * 0)
    assert torch.equal(none, s["kv"].cuda())


def test_append_bad_rows_are_reported_and_not_written():
    import mla_absorbed_decode_gb300 as mla
    s = _append_case([2, 2], [62, 10], seed=7)
    d = {k: v.cuda() for k, v in s.items() if v is not None}
    call = lambda table, lens: mla.cache_append_fp4(d["rows"][:, :512], d["rows"][:, 512:], d["kv"].clone(), 2.0 ** -6, table,
                                                    lens)
    want = call(d["table"], d["lens"])
    assert mla.get_device_status() == 0
    for value in (-1, 10 ** 6):
        table = d["table"].clone()
        table[1, 0] = value
        got = call(table, d["lens"])
        assert mla.get_device_status() == 6
        mine = s["table"][1, 0]
        assert torch.equal(got[mine], d["kv"][mine])
        keep = torch.ones(len(got), dtype=torch.bool)
        keep[mine] = False
        assert torch.equal(got[keep.cuda()], want[keep.cuda()])
    for n in (1, 5000):    # the first row's token is -1, or beyond the table
        call(d["table"], torch.tensor([64, n], dtype=torch.int32, device="cuda"))
        assert mla.get_device_status() == 6


# ----------------------------------------------------------------------------------- together --
def test_append_and_decode_together():
    """Prompts, then steps: what is written is what is read, dense and by lists."""
    import mla_absorbed_decode_gb300 as mla
    g = torch.Generator().manual_seed(0)
    B, H, kv_scale = 3, 32, 2.0 ** -6
    prompt, steps = [100, 1, 64], 3
    table = torch.arange(3 * 4, dtype=torch.int32).view(3, 4).flip(1).contiguous().cuda()
    kv = torch.full((12, 64, 352), 0x7F, dtype=torch.uint8, device="cuda")
    lens = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    norm = torch.ones(512, dtype=BF, device="cuda")
    P = mla.num_sm_parts(1, H)
    rows = torch.randn((sum(prompt), 576), generator=g).to(BF).cuda()
    offsets = torch.tensor([0] + list(np.cumsum(prompt)), dtype=torch.int32, device="cuda")
    mla.cache_append_fp4(rows[:, :512], rows[:, 512:], kv, kv_scale, table, lens, new_offsets=offsets, norm_weight=norm)
    for _ in range(steps):
        new = torch.randn((B, 576), generator=g).to(BF).cuda()
        lens += 1
        pos = (lens - 1).to(torch.int32)
        mla.cache_append_fp4(new[:, :512], new[:, 512:], kv, kv_scale, table, lens, positions=pos, norm_weight=norm)
        q = torch.randn((B, 1, H, 576), generator=g).to(BF).cuda()
        meta = mla.decode_metadata(lens, 1, H, False, P)
        got = mla.decode_fp4(q, kv, kv_scale, table, lens, SCALE, False, meta, P)
        k = torch.tensor([7, 2, 33], dtype=torch.int32, device="cuda").clamp(max=lens)
        idx = torch.stack([torch.randperm(int(n), generator=g)[:1].repeat(33) for n in lens.tolist()]).to(torch.int32).cuda()
        sp = mla.decode_sparse_fp4(q, kv, kv_scale, table, lens, idx, k, SCALE, False, mla.decode_metadata(k, 1, H, False, P), P)
        assert mla.get_device_status() == 0
        inp = dict(q=q.cpu(), kv=kv.cpu(), kv_scale=kv_scale, table=table.cpu(), seqlens=lens.cpu(), causal=False)
        _compare(inp, [t.cpu() for t in got], _ref(inp))
        inp.update(indices=idx.cpu(), topk_lens=k.cpu())
        _compare(inp, [t.cpu() for t in sp], _ref(inp))


def test_full_size_sampled():
    """The benchmark's shape in its launch configuration, some requests against the oracle."""
    import mla_absorbed_decode_gb300 as mla
    g = torch.Generator(device="cuda").manual_seed(0)
    B, H, L = W.V3.B, W.V3.H, W.V3.seqlen
    table = torch.randperm(B * L // 64, generator=g, device="cuda").to(torch.int32).view(B, L // 64)
    kv = torch.randint(0, 256, (B * L // 64, 64, 352), generator=g, device="cuda", dtype=torch.uint8)
    kv[..., 256:] &= 0xB7                                                 # no NaN, scales and rope codes below 1
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    q = torch.randn((B, 1, H, 576), generator=g, device="cuda").to(BF)
    P = mla.num_sm_parts(1, H)
    out, lse = mla.decode_fp4(q, kv, 0.5, table, lens, SCALE, False, mla.decode_metadata(lens, 1, H, False, P), P)
    assert mla.get_device_status() == 0
    sel = [0, 17, B - 1]
    inp = dict(q=q[sel].cpu(), kv=kv.cpu(), kv_scale=0.5, table=table[sel].cpu(), seqlens=lens[sel].cpu(), causal=False)
    _compare(inp, (out[sel].cpu(), lse[sel].cpu()), _ref(inp))
