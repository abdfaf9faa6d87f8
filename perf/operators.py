"""Cases of the operators that manage the latent cache of an MLA layer, for timing and comparison:

* ``rope``: the multi-axis rotation of q_pe (``rope_axes``), forwards and, for gradients, backwards;
* ``append``: a step's new rows into the paged cache (``cache_append``, ``cache_append_fp8``);
* ``weights``: the attention weight that a step gives every cached token (``attn_weights``, ``attn_weights_fp8``);
* ``evict``: dropping the cached tokens of least accumulated weight (``evict``, ``evict_fp8``).

``run`` computes them in elementary torch operations where ``own`` is false and by the library's calls
where it is true; ``exact`` restates them in 64 bits.
"""
import math

import torch

own = False

PAGE, DIM, LATENT, ROPE = 64, 576, 512, 64
THETA = 10000.0
SCALE = 1.0 / math.sqrt(192.0)   # softmax scale: the un-absorbed q/k width is 128 + 64
KV_SCALE = 2.0 ** -6             # FP8 cache: value = code value * KV_SCALE


# ------------------------------------------------------------------------------------ cases --
def listed():
    return [
        # the query side of one decode step of 64 requests, written into the tail of the decode query
        dict(name="rope_decode_b64_h128", op="rope", N=64, H=128, sections="16,8,8", interleaved=False, inverse=False,
             tail=True),
        # the gradient of q_pe for 4096 tokens of a prefill
        dict(name="rope_backward_t4096_h128", op="rope", N=4096, H=128, sections="16,8,8", interleaved=True,
             inverse=True, tail=False),
        # one new token of each of 64 requests into a bf16 cache
        dict(name="append_decode_b64", op="append", B=64, new=1, ragged=False, past=4096, sections="16,8,8", fp8=False),
        # the prompts of 16 requests, 1 to 1024 tokens each, into an FP8 cache
        dict(name="append_prefill_fp8_b16", op="append", B=16, new=1024, ragged=True, past=0, sections="16,8,8",
             fp8=True),
        # a small batch on a small model, where latency counts
        dict(name="weights_b2_h16_l300", op="weights", B=2, s_q=1, H=16, length=300, ragged=True, empty=False, fp8=False),
        # the decode step of 64 requests of 4096 tokens (the benchmark's shape)
        dict(name="weights_b64_h128_l4096", op="weights", B=64, s_q=1, H=128, length=4096, ragged=False, empty=False,
             fp8=False),
        # a ragged batch, 1 to 8192 tokens
        dict(name="weights_b128_h128_l1_8192", op="weights", B=128, s_q=1, H=128, length=8192, ragged=True, empty=False,
             fp8=False),
        # two new tokens a request, causal among them
        dict(name="weights_b64_sq2_h128_l8192", op="weights", B=64, s_q=2, H=128, length=8192, ragged=False, empty=False,
             fp8=False),
        # the benchmark's shape over an FP8 cache
        dict(name="weights_fp8_b64_h128_l4096", op="weights", B=64, s_q=1, H=128, length=4096, ragged=False, empty=False,
             fp8=True),
        # every 64 decode steps: 64 tokens over the budget leave
        dict(name="evict_b64_l2112_to_2048", op="evict", B=64, length=2112, ragged=False, empty=False, budget=2048, sink=4,
             recent=256, fp8=False),
        # halving the cache of a batch after its prefill
        dict(name="evict_b64_l4096_to_2048", op="evict", B=64, length=4096, ragged=False, empty=False, budget=2048, sink=4,
             recent=256, fp8=False),
        # four long contexts over an FP8 cache down to an eighth
        dict(name="evict_fp8_b4_l131072_to_16384", op="evict", B=4, length=131072, ragged=False, empty=False, budget=16384,
             sink=64, recent=4096, fp8=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _sections(rng):
    axes = rng.randint(1, 4)
    cuts = sorted(rng.sample(range(1, 32), axes - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [32]))


def draw(rng):
    op = rng.choice(("rope", "append", "weights", "weights", "evict"))
    if op == "rope":
        H = _log(rng, 1, 128)
        return dict(op=op, N=_log(rng, 1, 4096), H=H, sections=_sections(rng), interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, tail=rng.random() < 0.5)
    if op == "append":
        B = _log(rng, 1, 256)
        return dict(op=op, B=B, new=_log(rng, 1, max(1, 8192 // B)), ragged=rng.random() < 0.5,
                    past=rng.choice((0, _log(rng, 1, 4096))), sections=_sections(rng), fp8=rng.random() < 0.5)
    if op == "weights":
        B, s_q = _log(rng, 1, 128), rng.choice((1, 1, 2, 3, 4))
        H = _log(rng, 1, 128)
        length = _log(rng, 1, max(1, min(131072, 64 * 8192 // B, 64 * 8192 * 256 // (B * s_q * H))))
        return dict(op=op, B=B, s_q=s_q, H=H, length=length, ragged=rng.random() < 0.5, empty=rng.random() < 0.3,
                    fp8=rng.random() < 0.4)
    B = _log(rng, 1, 128)
    length = _log(rng, 32, min(131072, 64 * 4096 // B))
    budget = max(1, int(length * rng.uniform(0.1, 1.0)))
    sink = rng.choice((0, rng.randint(0, budget // 8)))
    return dict(op=op, B=B, length=length, ragged=rng.random() < 0.5, empty=rng.random() < 0.3, budget=budget, sink=sink,
                recent=rng.choice((0, rng.randint(0, budget // 2))), fp8=rng.random() < 0.5)


# ----------------------------------------------------------------------------------- inputs --
def _lengths(case, g):
    """int32 [B]: the requests' lengths."""
    B, most = case["B"], case["length"]
    if not case["ragged"]:
        n = torch.full((B,), most, dtype=torch.int32, device="cuda")
    else:
        n = torch.randint(1, most + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    if case["empty"]:   # a batch padded with requests that have no token
        n[torch.rand((B,), generator=g, device="cuda") < 0.25] = 0
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


def _codes(x):
    return (x / KV_SCALE).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _cache(pool, fp8, g):
    kv = torch.randn((pool, PAGE, DIM), generator=g, device="cuda")
    return _codes(kv) if fp8 else kv.to(torch.bfloat16)


def _values(kv):
    """A cache's values in fp32."""
    return kv.view(torch.float8_e4m3fn).float() * KV_SCALE if kv.dtype == torch.uint8 else kv.float()


def _positions(sections, N, g):
    """int32 [axes, N]: a time axis that runs to 131071, the others (height, width, ...) to 255."""
    axes = len(sections)
    p = torch.randint(0, 256, (axes, N), generator=g, device="cuda", dtype=torch.int32)
    p[0] = torch.randint(0, 131072, (N,), generator=g, device="cuda", dtype=torch.int32)
    return p


def _mix(sections, interleaved):
    """The axis of each of the 32 rotated pairs: sections one after the other, or dealt out in turn while they last."""
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while len(out) < 32:
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(op=op, case=case)
    if op in ("rope", "append"):
        s["sections"] = tuple(int(v) for v in case["sections"].split(","))
        s["interleaved"] = bool(case.get("interleaved", False))
        s["axis"] = torch.tensor(_mix(s["sections"], s["interleaved"]), device="cuda")
    if op == "rope":
        N, H = case["N"], case["H"]
        s["x"] = torch.randn((N, H, ROPE), generator=g, device="cuda").to(torch.bfloat16)
        s["positions"] = _positions(s["sections"], N, g)
        s["out"] = torch.zeros((N, H, DIM), dtype=torch.bfloat16, device="cuda")[..., LATENT:] if case["tail"] else \
            torch.zeros((N, H, ROPE), dtype=torch.bfloat16, device="cuda")
        return s
    if op == "append":
        B = case["B"]
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
        s["kv"] = _cache(pool, case["fp8"], g)
        # one row of the down-projection: the latent next to the rope key
        s["rows"] = torch.randn((N, DIM), generator=g, device="cuda").to(torch.bfloat16)
        s["positions"] = _positions(s["sections"], N, g)
        return s
    n = _lengths(case, g)
    B = case["B"]
    pool, s["block_table"] = _table((n + PAGE - 1) // PAGE, (case["length"] + PAGE - 1) // PAGE, g)
    s["seqlens"] = n
    s["kv"] = _cache(pool, case["fp8"], g)
    S = s["block_table"].shape[1] * PAGE
    held = torch.arange(S, device="cuda") < n[:, None]
    tail = torch.exp(1.5 * torch.randn((B, S), generator=g, device="cuda"))   # attention weight is heavy-tailed
    if op == "weights":
        s_q, H = case["s_q"], case["H"]
        s["q"] = torch.randn((B, s_q, H, DIM), generator=g, device="cuda").to(torch.bfloat16)
        s["causal"] = s_q > 1
        score, _ = _scores(s)
        s["lse"] = torch.logsumexp(score, dim=2).view(B, s_q, H)
        del score
        share = s_q * H / n.clamp(min=1).float()[:, None] / 3.0   # what an earlier step left
        s["weights"] = torch.where(held, tail * share, torch.zeros_like(tail))
        return s
    # weights as some steps have left them: a part of the slots has had none yet
    seen = torch.rand((B, S), generator=g, device="cuda") < 0.95
    s["weights"] = torch.where(held & seen, tail, torch.zeros_like(tail))
    # the cache has been evicted from before: its slots are no longer in the order of arrival
    order = torch.where(held, torch.rand((B, S), generator=g, device="cuda"), torch.full((B, S), 2.0, device="cuda"))
    order = torch.where(torch.arange(S, device="cuda") >= n[:, None] // 2, 1.0 + torch.arange(S, device="cuda") / S, order)
    rank = order.argsort(dim=1).argsort(dim=1)
    s["arrival"] = (3 * rank).to(torch.int32)
    s["width"] = (min(case["budget"], S) + 255) // 64 * 64   # room for the steps up to the next eviction
    return s


# ------------------------------------------------------------------------------ plain forms --
def _rotate(x, positions, axis, inverse):
    """x [N, H, 64] fp32 rotated by the pairs' angles, which are formed in 64 bits."""
    j = torch.arange(32, device=x.device, dtype=torch.float64)
    angle = positions[axis].double().T * THETA ** (-j / 32.0)
    if inverse:
        angle = -angle
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)


def _scores(s):
    """(scaled scores [B, rows, S] fp32 with -inf where a row does not see a slot, which slots it sees)."""
    q = s["q"]
    B, s_q, H, _ = q.shape
    table = s["block_table"].clamp(min=0).long()
    k = _values(s["kv"][table].flatten(1, 2))
    t = torch.arange(k.shape[1], device="cuda")
    last = s["seqlens"].long()[:, None].expand(B, s_q)
    if s["causal"]:
        last = last - (s_q - 1 - torch.arange(s_q, device="cuda"))
    seen = (t < last[..., None]).repeat_interleave(H, dim=1)
    score = torch.matmul(q.float().flatten(1, 2), k.transpose(1, 2)) * SCALE
    return torch.where(seen, score, torch.full_like(score, -math.inf)), seen


def _plain_append(s):
    N = s["rows"].shape[0]
    x = s["rows"].float()
    pe = _rotate(x[:, None, LATENT:], s["positions"], s["axis"], False)[:, 0]
    row = torch.cat((x[:, :LATENT], pe), dim=1)
    r = torch.arange(N, device="cuda")
    b = torch.searchsorted(s["offsets"][1:].contiguous(), r, right=True)
    t = s["seqlens"][b].long() - s["offsets"][b + 1].long() + r
    at = s["block_table"][b, t // PAGE].long() * PAGE + t % PAGE
    fp8 = s["kv"].dtype == torch.uint8
    s["kv"].view(-1, DIM)[at] = _codes(row) if fp8 else row.to(torch.bfloat16)
    return s["kv"].view(torch.float8_e4m3fn) if fp8 else s["kv"]


def _plain_weights(s):
    score, seen = _scores(s)
    lse = s["lse"].flatten(1)[..., None]
    p = torch.where(seen & (lse > -math.inf), torch.exp(score - lse), torch.zeros_like(score))
    s["weights"] += p.sum(dim=1)
    return s["weights"]


def _plain_evict(s):
    case, n, w, arrival = s["case"], s["seqlens"].long(), s["weights"], s["arrival"].long()
    B, S = w.shape
    budget, W = case["budget"], s["width"]
    t = torch.arange(S, device="cuda")
    held = t < n[:, None]
    first = torch.where(held, arrival, torch.full_like(arrival, -1)).amax(dim=1) + 1   # the next token's number
    guarded = (arrival < case["sink"]) | (arrival >= first[:, None] - case["recent"])
    key = torch.where(held, torch.where(guarded, torch.full_like(w, math.inf), w), torch.full_like(w, -1.0))
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, t.expand(B, S).contiguous())
    left = n.clamp(max=budget)
    keep = held & (rank < left[:, None])
    b, hole = (~keep & (t < left[:, None])).nonzero(as_tuple=True)
    source = (keep & (t >= left[:, None])).nonzero(as_tuple=True)[1]
    j = torch.arange(W, device="cuda")
    kept = torch.where(j < left[:, None], j, torch.full_like(j, -1))
    kept[b, hole] = source
    rows = s["kv"].view(-1, DIM)
    table = s["block_table"].long()
    rows[table[b, hole // PAGE] * PAGE + hole % PAGE] = rows[table[b, source // PAGE] * PAGE + source % PAGE]
    some = kept >= 0
    at = kept.clamp(min=0)
    later = first[:, None] + (j - left[:, None])   # the numbers of the tokens that will fill the other slots
    return dict(kv=_shown(s["kv"]), seqlens=left.to(torch.int32), kept=kept.to(torch.int32),
                weights=torch.where(some, w.gather(1, at), torch.zeros_like(w[:, :1])),
                arrival=torch.where(some, arrival.gather(1, at), later).to(torch.int32))


def _shown(kv):
    return kv.view(torch.float8_e4m3fn) if kv.dtype == torch.uint8 else kv


# -------------------------------------------------------------------------------------- run --
def run(s):
    op, case = s["op"], s["case"]
    if not own:
        if op == "rope":
            s["out"].copy_(_rotate(s["x"].float(), s["positions"], s["axis"], case["inverse"]))
            return s["out"]
        return {"append": _plain_append, "weights": _plain_weights, "evict": _plain_evict}[op](s)
    import mla_absorbed_decode_gb300 as mla
    if op == "rope":
        return mla.rope_axes(s["x"], s["positions"], s["sections"], out=s["out"], rope_theta=THETA,
                             interleaved=s["interleaved"], inverse=case["inverse"])
    kv, table, seqlens = s["kv"], s["block_table"], s["seqlens"]
    if op == "append":
        c, k_pe = s["rows"][:, :LATENT], s["rows"][:, LATENT:]
        more = dict(new_offsets=s["offsets"], positions=s["positions"], sections=s["sections"], rope_theta=THETA)
        if case["fp8"]:
            mla.cache_append_fp8(c, k_pe, kv, KV_SCALE, table, seqlens, **more)
        else:
            mla.cache_append(c, k_pe, kv, table, seqlens, **more)
        return _shown(kv)
    if op == "weights":
        if case["fp8"]:
            return mla.attn_weights_fp8(s["q"], s["lse"], kv, KV_SCALE, table, seqlens, SCALE, s["causal"], s["weights"])
        return mla.attn_weights(s["q"], s["lse"], kv, table, seqlens, SCALE, s["causal"], s["weights"])
    call = mla.evict_fp8 if case["fp8"] else mla.evict
    left, kept, weights, arrival = call(kv, table, seqlens, s["weights"], case["budget"], sink=case["sink"],
                                        recent=case["recent"], arrival=s["arrival"], width=s["width"])
    return dict(kv=_shown(kv), seqlens=left, kept=kept, weights=weights, arrival=arrival)


# ------------------------------------------------------------------------------------- work --
def work(case):
    """Bytes and flops that a pass cannot do without (ragged lengths at their mean)."""
    op = case["op"]
    row = DIM * (1 if case.get("fp8") else 2)
    if op == "rope":
        n = case["N"] * case["H"] * ROPE
        return dict(bytes=2 * n * 2 + 4 * case["N"] * len(case["sections"].split(",")), flops=3 * n)
    if op == "append":
        N = case["B"] * ((1 + case["new"]) / 2 if case["ragged"] else case["new"])
        return dict(bytes=N * (DIM * 2 + row + 4 * len(case["sections"].split(","))) + 8 * case["B"], flops=3 * ROPE * N)
    mean = (1 + case["length"]) / 2 if case["ragged"] else case["length"]
    B = case["B"] * (0.75 if case["empty"] else 1.0)
    if op == "weights":
        rows = case["s_q"] * case["H"]
        return dict(bytes=B * (mean * (row + 8) + mean / 16 + rows * (DIM * 2 + 4)), flops=B * rows * mean * (2 * DIM + 2))
    # kept tokens past the budget move: the recent ones, and of the others their share
    left = min(mean, case["budget"])
    guarded = min(left, case["sink"] + case["recent"])
    over = mean - left
    share = (left - guarded) / max(1.0, mean - guarded)
    moved = min(over, case["recent"]) + share * max(0.0, over - case["recent"])
    width = (min(case["budget"], case["length"]) + 255) // 64 * 64
    return dict(bytes=B * (mean * 8 + moved * 2 * row + mean / 16) + case["B"] * (width * 12 + 8), flops=B * mean)


# ------------------------------------------------------------------------------------ exact --
def exact(case, seed):
    """The operators' definitions in 64 bits, request by request and pair by pair."""
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rope", "append"):
        sections = s["sections"]
        axis = _mix(sections, s["interleaved"])
        x = s["x"].double() if op == "rope" else s["rows"].double()[:, None, LATENT:]
        y = torch.empty_like(x)
        sign = -1.0 if op == "rope" and case["inverse"] else 1.0
        for j in range(32):
            turn = sign * s["positions"][axis[j]].double() / THETA ** (2 * j / 64)
            z = torch.polar(torch.ones_like(turn), turn)[:, None] * torch.complex(x[..., 2 * j], x[..., 2 * j + 1])
            y[..., 2 * j], y[..., 2 * j + 1] = z.real, z.imag
        if op == "rope":
            return y
        kv = s["kv"].view(torch.float8_e4m3fn).double() if case["fp8"] else s["kv"].double()
        unit = KV_SCALE if case["fp8"] else 1.0
        offsets, lens = s["offsets"].tolist(), s["seqlens"].tolist()
        for b in range(case["B"]):
            r0, r1 = offsets[b], offsets[b + 1]
            t = torch.arange(lens[b] - (r1 - r0), lens[b], device="cuda")
            page = s["block_table"][b].long()[torch.div(t, PAGE, rounding_mode="floor")]
            kv[page, t % PAGE] = torch.cat((s["rows"][r0:r1, :LATENT].double(), y[r0:r1, 0]), dim=1) / unit
        return kv.clamp(-448.0, 448.0) if case["fp8"] else kv
    lens = s["seqlens"].tolist()
    if op == "weights":
        out = s["weights"].double()
        s_q, H = case["s_q"], case["H"]
        for b, n in enumerate(lens):
            pages = s["block_table"][b, : -(-n // PAGE)].long()
            k = s["kv"][pages].flatten(0, 1)[:n]
            k = k.view(torch.float8_e4m3fn).double() * KV_SCALE if case["fp8"] else k.double()
            for i in range(s_q):
                m = n - (s_q - 1 - i) if s["causal"] else n
                if m > 0:
                    e = torch.einsum("hd,td->ht", s["q"][b, i].double(), k[:m]) * SCALE - s["lse"][b, i].double()[:, None]
                    out[b, :m] += e.exp().sum(dim=0)
        return out
    W, budget = s["width"], case["budget"]
    out = torch.zeros((case["B"], W), dtype=torch.float64)
    weights, arrival = s["weights"].double().cpu(), s["arrival"].cpu()
    for b, n in enumerate(lens):
        w, a = weights[b, :n].tolist(), arrival[b, :n].tolist()
        end = max(a, default=-1) + 1
        best = sorted(range(n), key=lambda i: (not (a[i] < case["sink"] or a[i] >= end - case["recent"]), -w[i] if not (
            a[i] < case["sink"] or a[i] >= end - case["recent"]) else 0.0, i))[:budget]
        chosen = set(best)
        more = iter(sorted(i for i in chosen if i >= len(best)))
        out[b, : len(best)] = torch.tensor([w[j] if j in chosen else w[next(more)] for j in range(len(best))],
                                           dtype=torch.float64)
    return dict(kv=None, seqlens=None, kept=None, weights=out.cuda(), arrival=None)
