"""Cases of the operators on a latent cache held in 4 bits, for timing and comparison:

* ``append``: a step's new rows, their latent normalised and k_pe rotated on the way, into the cache
  (``cache_append_fp4``);
* ``decode``: absorbed decode over that cache (``decode_fp4``);
* ``sparse``: the same over each request's list of token positions (``decode_sparse_fp4``).

A cached token is 352 bytes: 512 E2M1 codes of the latent (256 bytes, an even dim in the low half of its byte), 32 E4M3
scales of 16 latent values each, 64 E4M3 codes of the rope key.  A latent value is code * scale * kv_scale, a value
of the rope key code * kv_scale.  ``run`` computes the operators in elementary torch operations where ``own`` is
false and by the library's calls where it is true; ``exact`` restates them in 64 bits.
"""
import math

import torch

own = False

PAGE, DIM, LATENT, ROPE, GROUP = 64, 576, 512, 64, 16
CODES, SCALES, ROW = 256, 32, 352                # bytes of a row: latent codes, their scales, all of it
THETA = 10000.0
EPS = 1e-6
SCALE = 1.0 / math.sqrt(192.0)                   # softmax scale: the un-absorbed q/k width is 128 + 64
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # values of the codes 0..7; code 8 + i is -E2M1[i]


# ------------------------------------------------------------------------------------ cases --
def listed():
    return [
        # one new token of each of 64 requests, where latency counts
        dict(name="append_decode_b64", op="append", B=64, new=1, ragged=False, past=4096, sections="32", norm=True,
             kv_scale=2.0 ** -6),
        # the prompts of 16 requests, 1 to 1024 tokens each, with three position axes
        dict(name="append_prefill_b16", op="append", B=16, new=1024, ragged=True, past=0, sections="16,8,8", norm=True,
             kv_scale=2.0 ** -6),
        # long prompts, rows that come normalised, a scale that is no power of two
        dict(name="append_prefill_b4_t8192", op="append", B=4, new=8192, ragged=False, past=0, sections="32", norm=False,
             kv_scale=0.013),
        # a small batch on a small model, where latency counts
        dict(name="decode_b2_h16_l300", op="decode", B=2, s_q=1, H=16, length=300, ragged=True, empty=False,
             outliers=False, kv_scale=2.0 ** -6),
        # the decode step of 64 requests of 4096 tokens (the benchmark's shape)
        dict(name="decode_b64_h128_l4096", op="decode", B=64, s_q=1, H=128, length=4096, ragged=False, empty=False,
             outliers=False, kv_scale=2.0 ** -6),
        # the same with the heads dealt out to eight GPUs, of which this is one
        dict(name="decode_b64_h16_l4096", op="decode", B=64, s_q=1, H=16, length=4096, ragged=False, empty=False,
             outliers=False, kv_scale=2.0 ** -6),
        # a ragged batch, 1 to 8192 tokens
        dict(name="decode_b128_h128_l1_8192", op="decode", B=128, s_q=1, H=128, length=8192, ragged=True, empty=False,
             outliers=False, kv_scale=2.0 ** -6),
        # two new tokens a request, causal among them
        dict(name="decode_b64_sq2_h128_l8192", op="decode", B=64, s_q=2, H=128, length=8192, ragged=False, empty=False,
             outliers=False, kv_scale=2.0 ** -6),
        # four long contexts, 1% of the tokens eight times as large
        dict(name="decode_b4_h128_l131072", op="decode", B=4, s_q=1, H=128, length=131072, ragged=False, empty=False,
             outliers=True, kv_scale=2.0 ** -5),
        # top 2048 of 16384 tokens
        dict(name="sparse_b64_h128_l16384_top2048", op="sparse", B=64, s_q=1, H=128, length=16384, ragged=False,
             empty=False, topk=2048, kv_scale=2.0 ** -6),
        # short lists of two query positions in a small batch, where latency counts
        dict(name="sparse_b8_sq2_h16_l2000_top100", op="sparse", B=8, s_q=2, H=16, length=2000, ragged=True, empty=False,
             topk=100, kv_scale=2.0 ** -6),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _sections(rng):
    axes = rng.randint(1, 4)
    cuts = sorted(rng.sample(range(1, 32), axes - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [32]))


def draw(rng):
    op = rng.choice(("append", "decode", "decode", "sparse"))
    kv_scale = rng.choice((2.0 ** -6, 2.0 ** -5, 0.013))
    B = _log(rng, 1, 128)
    if op == "append":
        return dict(op=op, B=B, new=_log(rng, 1, max(1, 16384 // B)), ragged=rng.random() < 0.5,
                    past=rng.choice((0, _log(rng, 1, 4096))), sections=_sections(rng), norm=rng.random() < 0.7,
                    kv_scale=kv_scale)
    s_q, H = rng.choice((1, 1, 2, 3, 4)), _log(rng, 1, 128)
    if op == "sparse":
        topk = _log(rng, 1, max(1, min(4096, 64 * 2048 * 256 // (B * s_q * H))))
        return dict(op=op, B=B, s_q=s_q, H=H, length=_log(rng, topk, max(topk, 64 * 16384 // B)),
                    ragged=rng.random() < 0.5, empty=rng.random() < 0.3, topk=topk, kv_scale=kv_scale)
    length = _log(rng, 1, max(1, min(131072, 64 * 8192 // B, 64 * 8192 * 256 // (B * s_q * H))))
    return dict(op=op, B=B, s_q=s_q, H=H, length=length, ragged=rng.random() < 0.5, empty=rng.random() < 0.3,
                outliers=rng.random() < 0.3, kv_scale=kv_scale)


# ----------------------------------------------------------------------------------- inputs --
def _lengths(case, g):
    """int32 [B]: the requests' lengths."""
    B, most = case["B"], case["length"]
    if not case["ragged"]:
        n = torch.full((B,), most, dtype=torch.int32, device="cuda")
    else:
        n = torch.randint(1, most + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    if case["empty"]:   # a batch padded with requests that have no token
        n[1:][torch.rand((B - 1,), generator=g, device="cuda") < 0.25] = 0
    return n


def _table(pages, most, g):
    """A random page pool that holds B requests of up to `most` pages: (pages in it, block_table [B, most] int32,
    -1 past a request's pages)."""
    pool = math.ceil(1.03 * pages.numel() * most)
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    first = pages.cumsum(0) - pages
    k = torch.arange(most, device="cuda")
    at = (first[:, None] + k).clamp(max=pool - 1)
    return pool, torch.where(k < pages[:, None], perm[at], torch.full_like(perm[at], -1))


def _cache(pool, kv_scale, outliers, g):
    """uint8 [pool, 64, 352]: rows of N(0, 1) values, 1% of them eight times as large where wanted."""
    kv = torch.empty((pool, PAGE, ROW), dtype=torch.uint8, device="cuda")
    for part in kv.split(2048):   # 2048 pages a turn: 300 MB of fp32
        x = torch.randn((part.shape[0], PAGE, DIM), generator=g, device="cuda")
        if outliers:
            x[torch.rand(x.shape[:2], generator=g, device="cuda") < 0.01] *= 8.0
        part.copy_(_pack(x, kv_scale))
    return kv


def _positions(sections, N, g):
    """int32 [axes, N]: a time axis that runs to 131071, the others (height, width, ...) to 255."""
    axes = len(sections)
    p = torch.randint(0, 256, (axes, N), generator=g, device="cuda", dtype=torch.int32)
    p[0] = torch.randint(0, 131072, (N,), generator=g, device="cuda", dtype=torch.int32)
    return p


def _lists(n, topk, ragged, g):
    """(int32 [B, topk]: each request's listed positions in ascending order, -1 past its list; int32 [B]: their number)."""
    B = n.numel()
    k = n.clamp(max=topk)
    if ragged:
        k[1:] = (torch.rand((B - 1,), generator=g, device="cuda") * (k[1:] + 1).float()).int().clamp(max=k[1:])
    out = torch.full((B, topk), -1, dtype=torch.int32, device="cuda")
    for b, (m, length) in enumerate(zip(k.tolist(), n.tolist())):
        out[b, :m] = torch.randperm(length, generator=g, device="cuda")[:m].sort().values.int()
    return out, k.int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(op=op, case=case)
    # the two values of every byte of latent codes, as a pair of E4M3 numbers
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    byte = torch.arange(256, device="cuda")
    s["pairs"] = torch.stack((value[byte & 15], value[byte >> 4]), dim=1).to(torch.float8_e4m3fn).view(torch.int16)[:, 0]
    B = case["B"]
    if op == "append":
        s["sections"] = tuple(int(v) for v in case["sections"].split(","))
        s["axis"] = torch.tensor([a for a, n in enumerate(s["sections"]) for _ in range(n)], device="cuda")
        new = torch.randint(1, case["new"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if case["ragged"] \
            else torch.full((B,), case["new"], dtype=torch.int32, device="cuda")
        past = torch.randint(0, case["past"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["seqlens"] = past + new
        s["offsets"] = torch.cat([torch.zeros(1, device="cuda"), new.cumsum(0)]).to(torch.int32)
        N = int(new.sum())
        # the step writes a request's last pages only: the pool holds those, the table's other entries are not read
        first, last = past // PAGE, (s["seqlens"] + PAGE - 1) // PAGE
        pool, tail = _table(last - first, (case["new"] + PAGE - 2) // PAGE + 1, g)
        k = torch.arange((case["past"] + case["new"] + PAGE - 1) // PAGE, device="cuda")
        at = (k - first[:, None]).clamp(min=0, max=tail.shape[1] - 1)
        s["block_table"] = torch.where((k >= first[:, None]) & (k < last[:, None]), tail.gather(1, at.long()),
                                       torch.full_like(at, -1).int()).contiguous()
        s["kv"] = _cache(pool, case["kv_scale"], False, g)
        # one row of the down-projection: the latent next to the rope key
        s["rows"] = torch.randn((N, DIM), generator=g, device="cuda").to(torch.bfloat16)
        s["positions"] = _positions(s["sections"], N, g)
        s["norm"] = (1.0 + 0.2 * torch.randn((LATENT,), generator=g, device="cuda")).to(torch.bfloat16) if case["norm"] \
            else None
        return s
    n = _lengths(case, g)
    pool, s["block_table"] = _table((n + PAGE - 1) // PAGE, (case["length"] + PAGE - 1) // PAGE, g)
    s["seqlens"] = n
    s["kv"] = _cache(pool, case["kv_scale"], bool(case.get("outliers", False)), g)
    s_q, H = case["s_q"], case["H"]
    s["q"] = torch.randn((B, s_q, H, DIM), generator=g, device="cuda").to(torch.bfloat16)
    s["causal"] = s_q > 1
    if op == "sparse":
        s["indices"], s["topk_lens"] = _lists(n, case["topk"], case["ragged"], g)
    if own:   # the step's plan and scratch memory, which a program makes once for all layers
        import mla_absorbed_decode_gb300 as mla
        s["parts"] = mla.num_sm_parts(s_q, H)
        s["plan"] = mla.decode_metadata(s["topk_lens"] if op == "sparse" else n, s_q, H, s["causal"], s["parts"])
        s["workspace"] = torch.empty(mla.decode_workspace_size(B, s_q, H, s["parts"]), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------ plain forms --
def _pack(x, kv_scale):
    """Rows of values [..., 576] fp32 as rows of 352 bytes.  A group's scale is the E4M3 number nearest to the one that
    puts its largest value at E2M1's largest; codes are the nearest to the even one, everything saturates."""
    unit = torch.full((), kv_scale, dtype=torch.float32, device=x.device)
    c = x[..., :LATENT].unflatten(-1, (LATENT // GROUP, GROUP))
    scale = (c.abs().amax(dim=-1) / (6.0 * unit)).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = (scale.float() * unit)[..., None]
    y = torch.where(step > 0, c / step, torch.zeros_like(c))
    a = y.abs()
    code = (a > 0.25).to(torch.uint8)
    for least, even in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += a >= least if even else a > least   # halfway goes to the code whose last bit is 0
    code += torch.signbit(y).to(torch.uint8) * 8
    code = code.flatten(-2)
    rope = (x[..., LATENT:] / unit).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return torch.cat((code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8), rope.view(torch.uint8)), dim=-1)


def _codes(kv, pairs):
    """The values of the latent's codes, as E4M3 numbers [..., 512]."""
    return pairs[kv[..., :CODES].int()].view(torch.float8_e4m3fn)


def _values(kv, pairs, kv_scale):
    """A cache's values [..., 576] in fp32."""
    code = _codes(kv, pairs).float().unflatten(-1, (LATENT // GROUP, GROUP))
    scale = kv[..., CODES:CODES + SCALES].contiguous().view(torch.float8_e4m3fn).float()
    rope = kv[..., CODES + SCALES:].contiguous().view(torch.float8_e4m3fn).float()
    return torch.cat(((code * scale[..., None]).flatten(-2), rope), dim=-1) * kv_scale


def _shown(s):
    """What the cache holds, by its parts."""
    kv = s["kv"]
    return dict(latent=_codes(kv, s["pairs"]), scales=kv[..., CODES:CODES + SCALES].view(torch.float8_e4m3fn),
                rope=kv[..., CODES + SCALES:].view(torch.float8_e4m3fn))


def _rotate(x, positions, axis):
    """x [N, 64] fp32 rotated by the pairs' angles, which are formed in 64 bits."""
    j = torch.arange(32, device=x.device, dtype=torch.float64)
    angle = positions[axis].double().T * THETA ** (-j / 32.0)
    cos, sin = angle.cos().float(), angle.sin().float()
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)


def _plain_append(s):
    x = s["rows"].float()
    c = x[:, :LATENT]
    if s["norm"] is not None:
        c = c * torch.rsqrt(c.square().mean(dim=1, keepdim=True) + EPS) * s["norm"].float()
    row = torch.cat((c, _rotate(x[:, LATENT:], s["positions"], s["axis"])), dim=1)
    r = torch.arange(x.shape[0], device="cuda")
    b = torch.searchsorted(s["offsets"][1:].contiguous(), r, right=True)
    t = s["seqlens"][b].long() - s["offsets"][b + 1].long() + r
    at = s["block_table"][b, t // PAGE].long() * PAGE + t % PAGE
    s["kv"].view(-1, ROW)[at] = _pack(row, s["case"]["kv_scale"])
    return _shown(s)


def _plain_decode(s):
    q, table, n = s["q"], s["block_table"].clamp(min=0).long(), s["seqlens"].long()
    B, s_q, H, _ = q.shape
    if s["op"] == "sparse":
        t = s["indices"].clamp(min=0).long()
        held = torch.arange(t.shape[1], device="cuda") < s["topk_lens"][:, None]
        rows = s["kv"].view(-1, ROW)[table.gather(1, t // PAGE) * PAGE + t % PAGE]
    else:
        rows = s["kv"][table].flatten(1, 2)
        t = torch.arange(rows.shape[1], device="cuda").expand(B, -1)
        held = t < n[:, None]
    k = _values(rows, s["pairs"], s["case"]["kv_scale"])
    last = n[:, None].expand(B, s_q)
    if s["causal"]:
        last = last - (s_q - 1 - torch.arange(s_q, device="cuda"))
    seen = (held[:, None, :] & (t[:, None, :] < last[..., None])).repeat_interleave(H, dim=1)
    score = torch.matmul(q.float().flatten(1, 2), k.transpose(1, 2)) * SCALE
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    most = score.amax(dim=2, keepdim=True)
    p = torch.where(seen, torch.exp(score - torch.where(most > -math.inf, most, torch.zeros_like(most))),
                    torch.zeros_like(score))
    total = p.sum(dim=2, keepdim=True)
    out = torch.matmul(p, k[..., :LATENT]) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.where(total > 0, most + torch.log(total), torch.full_like(total, -math.inf))
    return out.view(B, s_q, H, LATENT).to(torch.bfloat16), lse.view(B, s_q, H)


# -------------------------------------------------------------------------------------- run --
def run(s):
    op = s["op"]
    if not own:
        return _plain_append(s) if op == "append" else _plain_decode(s)
    import mla_absorbed_decode_gb300 as mla
    kv, table, seqlens, kv_scale = s["kv"], s["block_table"], s["seqlens"], s["case"]["kv_scale"]
    if op == "append":
        mla.cache_append_fp4(s["rows"][:, :LATENT], s["rows"][:, LATENT:], kv, kv_scale, table, seqlens,
                             new_offsets=s["offsets"], positions=s["positions"], sections=s["sections"], rope_theta=THETA,
                             norm_weight=s["norm"], norm_eps=EPS)
        return _shown(s)
    more = dict(softmax_scale=SCALE, causal=s["causal"], metadata=s["plan"], parts=s["parts"], workspace=s["workspace"])
    if op == "sparse":
        return mla.decode_sparse_fp4(s["q"], kv, kv_scale, table, seqlens, s["indices"], s["topk_lens"], **more)
    return mla.decode_fp4(s["q"], kv, kv_scale, table, seqlens, **more)


# ------------------------------------------------------------------------------------- work --
def work(case):
    """Bytes and flops that a pass cannot do without (ragged lengths at their mean)."""
    B = case["B"]
    if case["op"] == "append":
        N = B * ((1 + case["new"]) / 2 if case["ragged"] else case["new"])
        return dict(bytes=N * (DIM * 2 + ROW + 4 * len(case["sections"].split(","))) + 8 * B, flops=N * (5 * LATENT + 3 * ROPE))
    rows = case["s_q"] * case["H"]
    mean = (1 + case["length"]) / 2 if case["ragged"] else case["length"]
    live = B * (0.75 if case["empty"] else 1.0)
    tokens = min(mean, case["topk"]) * (0.5 if case["ragged"] else 1.0) if case["op"] == "sparse" else mean
    index = 4 * tokens if case["op"] == "sparse" else tokens / 16
    return dict(bytes=live * (tokens * ROW + index + rows * DIM * 2) + B * rows * (LATENT * 2 + 4),
                flops=live * rows * tokens * 2 * (DIM + LATENT))


# ------------------------------------------------------------------------------------ exact --
def _nearest(x, mantissa, least, most):
    """x (64 bits) rounded to the nearest number of `mantissa` fraction bits, halves to even, with 2^least the smallest
    normal one and +-most the largest."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=least) - mantissa)
    return (torch.round(x / step) * step).clamp(-most, most)


def exact(case, seed):
    """The operators' definitions in 64 bits, request by request and pair by pair."""
    s = prepare(case, seed)
    kv, unit = s["kv"], float(torch.tensor(case["kv_scale"], dtype=torch.float32))
    at = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
    value = torch.tensor(at, dtype=torch.float64, device="cuda")

    def parts(rows):   # [..., 352] bytes: latent codes, scales and rope codes as numbers
        low, high = (rows[..., :CODES] & 15).long(), (rows[..., :CODES] >> 4).long()
        eight = rows[..., CODES:].contiguous().view(torch.float8_e4m3fn).double()
        return torch.stack((value[low], value[high]), dim=-1).flatten(-2), eight[..., :SCALES], eight[..., SCALES:]

    if case["op"] == "append":
        latent, scales, rope = parts(kv)
        x = s["rows"].double()
        c = x[:, :LATENT]
        if s["norm"] is not None:
            c = c / (c.square().sum(dim=1, keepdim=True) / LATENT + EPS).sqrt() * s["norm"].double()
        y = torch.empty_like(x[:, LATENT:])
        for j in range(32):
            turn = s["positions"][int(s["axis"][j])].double() / THETA ** (2 * j / 64)
            z = torch.polar(torch.ones_like(turn), turn) * torch.complex(x[:, LATENT + 2 * j], x[:, LATENT + 2 * j + 1])
            y[:, 2 * j], y[:, 2 * j + 1] = z.real, z.imag
        offsets, lens = s["offsets"].tolist(), s["seqlens"].tolist()
        for b in range(case["B"]):
            r0, r1 = offsets[b], offsets[b + 1]
            t = torch.arange(lens[b] - (r1 - r0), lens[b], device="cuda")
            page, slot = s["block_table"][b].long()[torch.div(t, PAGE, rounding_mode="floor")], t % PAGE
            group = c[r0:r1].reshape(r1 - r0, LATENT // GROUP, GROUP)
            sc = _nearest(group.abs().amax(dim=2) / 6.0 / unit, 3, -6, 448.0)
            code = torch.where(sc[..., None] > 0, group / sc[..., None].clamp(min=2.0 ** -9) / unit, 0.0)
            latent[page, slot] = _nearest(code, 1, 0, 6.0).flatten(1)
            scales[page, slot] = sc
            rope[page, slot] = _nearest(y[r0:r1] / unit, 3, -6, 448.0)
        return dict(latent=latent, scales=scales, rope=rope)
    s_q, H, q = case["s_q"], case["H"], s["q"]
    out = torch.zeros((case["B"], s_q, H, LATENT), dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"], s_q, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["seqlens"].tolist()):
        t = s["indices"][b, : int(s["topk_lens"][b])].long() if case["op"] == "sparse" else torch.arange(n, device="cuda")
        code, scale, rope = parts(kv[s["block_table"][b].long()[torch.div(t, PAGE, rounding_mode="floor")], t % PAGE])
        c = code * scale.repeat_interleave(GROUP, dim=1) * unit
        for i in range(s_q):
            see = t <= n - s_q + i if s["causal"] else torch.ones_like(t, dtype=torch.bool)
            if not bool(see.any()):
                continue
            e = (q[b, i, :, :LATENT].double() @ c[see].T + q[b, i, :, LATENT:].double() @ rope[see].T * unit) * SCALE
            lse[b, i] = torch.logsumexp(e, dim=1)
            out[b, i] = (e - lse[b, i, :, None]).exp() @ c[see]
    return out, lse
