"""The calls on a 4-bit latent cache where programs use them: on streams of their own, in graphs that share buffers, in a
decode step, over caches beyond 2^32 bytes, with pages that never arrive, and with tensors that are refused."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
from mla_absorbed_decode_gb300 import workloads as W

from _harness import OUT_ABS, make, to_np
from test_gpu_fp4 import SCALE, _case, _compare, _ref, _run

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_absorbed_decode_gb300 import build_lib
    build_lib.build()
    yield


class _Call:
    """A decode with buffers of its own: prepared once, run on any stream, refilled in place."""

    def __init__(self, inp, parts=None, workspace=None):
        import mla_absorbed_decode_gb300 as mla
        self.causal, self.kv_scale = inp["causal"], inp["kv_scale"]
        self.q, self.kv, self.table, self.n = (inp[k].cuda() for k in ("q", "kv", "table", "seqlens"))
        self.lists = (inp["indices"].cuda(), inp["topk_lens"].cuda()) if "indices" in inp else ()
        B, s_q, H, _ = self.q.shape
        self.parts = mla.num_sm_parts(s_q, H) if parts is None else parts
        self.meta = mla.decode_metadata(self.lists[1] if self.lists else self.n, s_q, H, self.causal, self.parts)
        self.out = torch.empty((B, s_q, H, 512), dtype=BF, device="cuda")
        self.lse = torch.empty((B, s_q, H), device="cuda")
        size = mla.decode_workspace_size(B, s_q, H, self.parts)
        self.workspace = torch.empty(size, dtype=torch.uint8, device="cuda") if workspace is None else workspace
        assert self.workspace.numel() >= size

    def __call__(self, stream=None):
        import mla_absorbed_decode_gb300 as mla
        call = mla.decode_sparse_fp4 if self.lists else mla.decode_fp4
        call(self.q, self.kv, self.kv_scale, self.table, self.n, *self.lists, SCALE, self.causal, self.meta, self.parts,
             workspace=self.workspace, out=self.out, lse=self.lse, stream=stream)

    def result(self):
        return self.out.cpu(), self.lse.cpu()


def _equal(a, b):
    return torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def _two():
    return (_case([700, 64, 1, 4000], H=128, seed=51), _case([900, 300], s_q=2, H=16, topk=[400, 129], seed=52))


# ----------------------------------------------------------------------------------- streams --
@pytest.mark.parametrize("which", [0, 1])
def test_on_a_stream_of_its_own(which):
    inp = _two()[which]
    want = _run(inp)
    a = _Call(inp)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a(stream=side)
    side.synchronize()
    assert _equal(a.result(), want)
    with torch.cuda.stream(side):
        a.out.zero_()
        a()
    side.synchronize()
    assert _equal(a.result(), want)


def test_two_calls_at_once():
    inputs = _two()
    want = [_run(i) for i in inputs]
    calls = [_Call(i) for i in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        for c, s in zip(calls, streams):
            c(stream=s)
    torch.cuda.synchronize()
    import mla_absorbed_decode_gb300 as mla
    assert mla.get_device_status() == 0
    for c, w in zip(calls, want):
        assert _equal(c.result(), w)


def test_two_graphs_that_share_a_workspace():
    """Captured calls of different shapes on one workspace, replayed in turn, with inputs refilled in place between."""
    import mla_absorbed_decode_gb300 as mla
    inputs = _two()
    calls = [_Call(i) for i in inputs]
    shared = torch.empty(max(c.workspace.numel() for c in calls), dtype=torch.uint8, device="cuda")
    for c in calls:
        c.workspace = shared
        c()
    torch.cuda.synchronize()
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c()
        graphs.append(g)
    for step in range(3):
        for c, inp in zip(calls, inputs):
            inp["q"] = torch.randn(inp["q"].shape, generator=torch.Generator().manual_seed(step)).to(BF)
            c.q.copy_(inp["q"])
            c.out.fill_(7.0)
        shared.fill_(0xFF)
        for g in graphs + graphs:
            g.replay()
        assert mla.get_device_status() == 0
        for c, inp in zip(calls, inputs):
            assert _equal(c.result(), _run(inp))


def test_many_short_requests_and_a_large_batch():
    """More requests than parts, most of them a page or none."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 4, size=1500) * 33
    lens[[0, 7, 1499]] = 0, 513, 0
    inp = _case(lens.tolist(), H=16, seed=53)
    got = _run(inp)
    sel = [0, 1, 7, 700, 1498, 1499]
    part = dict(inp, q=inp["q"][sel], table=inp["table"][sel], seqlens=inp["seqlens"][sel])
    _compare(part, [t[sel] for t in got], _ref(part))


def test_a_page_held_by_two_requests():
    """A shared prompt: two requests whose tables name the same pages."""
    inp = _case([300, 300], H=32, seed=54)
    inp["table"][1, :4] = inp["table"][0, :4]
    _compare(inp, _run(inp), _ref(inp))


def test_no_query_rows_is_no_launch():
    import mla_absorbed_decode_gb300 as mla
    kv = torch.zeros((2, 64, 352), dtype=torch.uint8, device="cuda")
    n = torch.zeros(0, dtype=torch.int32, device="cuda")
    meta = torch.zeros(64, dtype=torch.int32, device="cuda")
    out, lse = mla.decode_fp4(torch.empty((0, 1, 16, 576), dtype=BF, device="cuda"), kv, 0.5,
                              torch.empty((0, 2), dtype=torch.int32, device="cuda"), n, SCALE, False, meta, 1)
    assert out.shape == (0, 1, 16, 512) and lse.shape == (0, 1, 16)
    c = torch.empty((0, 576), dtype=BF, device="cuda")
    table = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    mla.cache_append_fp4(c[:, :512], c[:, 512:], kv, 0.5, table, torch.ones(1, dtype=torch.int32, device="cuda"))
    assert mla.get_device_status() == 0 and not kv.any()


# ------------------------------------------------------------------------------- large caches --
def test_offsets_beyond_32_bits():
    """A cache of 5.6 GB: the same pages at its far end give the same bits, written, read whole and read by lists."""
    import mla_absorbed_decode_gb300 as mla
    blocks = 250_000
    assert blocks * 64 * 352 > 2 ** 32
    inputs = [_case([300, 1000], H=16, seed=55), _case([300, 1000], H=16, topk=[100, 512], seed=55)]
    pool = inputs[0]["kv"].shape[0]
    big = torch.empty((blocks, 64, 352), dtype=torch.uint8, device="cuda")
    for inp in inputs:
        a = _Call(inp)
        a()
        want = a.result()
        big[blocks - pool:] = a.kv
        a.kv = big
        a.table += blocks - pool
        a()
        assert mla.get_device_status() == 0
        assert _equal(a.result(), want)
    g = torch.Generator().manual_seed(0)
    rows = torch.randn((4, 576), generator=g).to(BF).cuda()
    n = inputs[0]["seqlens"].cuda()
    small = inputs[0]["kv"].cuda()
    table = inputs[0]["table"].cuda()
    for kv, t in ((small, table), (big, table + (blocks - pool))):
        mla.cache_append_fp4(rows[:, :512], rows[:, 512:], kv, 0.5, t, n)
    assert mla.get_device_status() == 0
    assert torch.equal(big[blocks - pool:], small)


# ----------------------------------------------------------------------------------- timeouts --
@pytest.mark.parametrize("which", [0, 1])
def test_gives_up_when_a_page_never_arrives(which):
    """The test hook withholds every part's first page: the call reports it and ends, and the calls after it are right."""
    import mla_absorbed_decode_gb300 as mla
    inp = _two()[which]
    good = _run(inp)
    a = _Call(inp)
    mla.debug_withhold_first_load(True)
    a()
    assert mla.get_device_status() == 5          # MLA_ERR_TIMEOUT
    assert mla.get_device_status() == 0
    for _ in range(3):
        a()
        assert _equal(a.result(), good)


def test_metadata_of_a_larger_batch_is_reported():
    import mla_absorbed_decode_gb300 as mla
    inp = _case([300, 100], H=16, seed=56)
    good = _run(inp)
    a = _Call(inp)
    more = torch.tensor([300] * 40, dtype=torch.int32, device="cuda")
    a.meta = mla.decode_metadata(more, 1, 16, False, a.parts)
    a()
    assert mla.get_device_status() == 6          # MLA_ERR_DEVICE_BOUNDS
    assert _equal(_run(inp), good)


# --------------------------------------------------------------------------------- decode step --
@pytest.mark.parametrize("s_q", [1, 2])
def test_step_chain_and_graph_vs_expanded_definition(s_q):
    """DecodeStep over a 4-bit cache: the step's rows appended with their norm and rotation, absorbed decode, un-absorption;
    eagerly and from a graph.  What the cache then holds (the append is tested by itself) is what the expanded definition is
    taken over; the chain's bf16 roundings of q, of the latent output and of o are those of the FP8 step, so are the bounds."""
    import mla_absorbed_decode_gb300 as mla
    w = dataclasses.replace(W.small_variant(W.FP8, B=3, seqlen=700), s_q=s_q)
    inp = make(w)
    B, H, kv_scale = w.B, w.H, 2.0 ** -6
    blocks = inp["kv_cache"].shape[0]
    g = torch.Generator().manual_seed(1)
    kv = torch.from_numpy(oracle.pack_fp4(torch.randn((blocks, 64, 576), generator=g).numpy(), kv_scale)).cuda()
    n = inp["seqlens"].cuda()
    # the last s_q tokens of every request are the step's
    pos = torch.stack([torch.arange(int(k) - s_q, int(k)) for k in inp["seqlens"]]).flatten().to(torch.int32).cuda()
    rows, norm = torch.randn((B * s_q, 576), generator=g).to(BF).cuda(), (1 + 0.1 * torch.randn(512, generator=g)).to(BF).cuda()
    step = mla.DecodeStep(B, s_q, H, n, s_q > 1, w.softmax_scale, kv_scale=kv_scale, kv_bits=4)
    args = (inp["q_nope"].cuda(), inp["q_pe"].cuda(), inp["w_uk"].cuda(), inp["w_uv"].cuda(), kv, inp["block_table"].cuda())
    append = lambda: step.append(rows[:, :512], rows[:, 512:], kv, args[5], positions=pos, norm_weight=norm)
    append()
    after = kv.clone()
    mla.cache_append_fp4(rows[:, :512], rows[:, 512:], kv, kv_scale, args[5], n, positions=pos, norm_weight=norm)
    assert torch.equal(kv, after)
    o = step.run(*args, positions=pos).clone()
    out, lse = step.out.clone(), step.lse.clone()
    got = mla.decode_fp4(step.q, kv, kv_scale, args[5], n, w.softmax_scale, s_q > 1, step.metadata, step.parts)
    assert torch.equal(out, got[0]) and torch.equal(lse, got[1])
    assert mla.get_device_status() == 0
    for b in range(B):   # the graph writes the rows too
        t = int(inp["seqlens"][b]) - 1
        kv[args[5][b, t // 64], t % 64] = 0
    step.capture(*args, positions=pos, before=append)
    o2 = step.replay().clone()
    torch.cuda.synchronize()
    assert mla.get_device_status() == 0
    assert torch.equal(o, o2) and torch.equal(kv, after)
    qp = np.swapaxes(oracle.rope_interleaved(np.swapaxes(to_np(inp["q_pe"]), 0, 1), pos.cpu().numpy()), 0, 1)
    ref, _ = oracle.decode_expanded(to_np(inp["q_nope"]).reshape(B, s_q, H, 128), qp.reshape(B, s_q, H, 64), to_np(inp["w_uk"]),
                                    to_np(inp["w_uv"]), oracle.unpack_fp4(kv.cpu().numpy(), kv_scale), inp["block_table"].numpy(),
                                    inp["seqlens"].numpy(), w.softmax_scale, **({"causal": True} if s_q > 1 else {}))
    d = np.abs(to_np(o.view(B, s_q, H, 128).cpu()) - ref)
    assert d.max() <= OUT_ABS, d.max()
    assert np.linalg.norm(d) / np.linalg.norm(ref) <= 2e-2


def test_step_refuses_what_a_4_bit_cache_has_not():
    import mla_absorbed_decode_gb300 as mla
    n = torch.ones(1, dtype=torch.int32, device="cuda")
    step = mla.DecodeStep(1, 1, 16, n, False, 0.1, kv_scale=0.5, kv_bits=4)
    kv = torch.zeros((1, 64, 352), dtype=torch.uint8, device="cuda")
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    weights = torch.zeros((1, 64), device="cuda")
    with pytest.raises(ValueError, match="4-bit"):
        step.accumulate_weights(kv, table, weights)
    with pytest.raises(ValueError, match="4-bit"):
        step.evict(kv, table, weights, 10)
    row = torch.zeros((1, 576), dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="norm"):
        mla.DecodeStep(1, 1, 16, n, False, 0.1, kv_scale=0.5).append(
            row[:, :512], row[:, 512:], torch.zeros((1, 64, 576), dtype=torch.uint8, device="cuda"), table,
            norm_weight=torch.ones(512, dtype=BF, device="cuda"))


# ----------------------------------------------------------------------------------- refusals --
def _tensors(B=2, H=16):
    return dict(q=torch.zeros((B, 1, H, 576), dtype=BF), kv=torch.zeros((4, 64, 352), dtype=torch.uint8),
                table=torch.zeros((B, 2), dtype=torch.int32), n=torch.ones(B, dtype=torch.int32),
                idx=torch.zeros((B, 5), dtype=torch.int32), k=torch.ones(B, dtype=torch.int32),
                meta=torch.zeros(4096, dtype=torch.int32))


def _refused(sparse, match, out=None, lse=None, workspace=None, **more):
    import mla_absorbed_decode_gb300 as mla
    t = {k: v.cuda() for k, v in dict(_tensors(), **more).items()}
    own = {k: v.cuda() for k, v in dict(out=out, lse=lse, workspace=workspace).items() if v is not None}
    with pytest.raises((ValueError, TypeError, RuntimeError), match=match):
        if sparse:
            mla.decode_sparse_fp4(t["q"], t["kv"], 0.5, t["table"], t["n"], t["idx"], t["k"], 0.1, False, t["meta"], 4, **own)
        else:
            mla.decode_fp4(t["q"], t["kv"], 0.5, t["table"], t["n"], 0.1, False, t["meta"], 4, **own)


@pytest.mark.parametrize("sparse", [False, True])
def test_decode_tensors_that_are_refused(sparse):
    t = _tensors()
    for q in (t["q"].float(), torch.zeros((2, 1, 32, 576), dtype=BF, device="cuda")[:, :, ::2],
              torch.zeros((3, 1, 16, 576), dtype=BF), torch.zeros((2, 1, 16, 512), dtype=BF)):
        _refused(sparse, "q", q=q)
    for kv in (t["kv"].view(torch.int8).to(torch.int16), torch.zeros((4, 64, 576), dtype=torch.uint8),
               torch.zeros((4, 32, 352), dtype=torch.uint8), torch.zeros((4, 64, 352), dtype=BF)):
        _refused(sparse, "kv_cache", kv=kv)
    _refused(sparse, "block_table", table=t["table"].long())
    _refused(sparse, "seqlens", n=t["n"].long())
    _refused(sparse, "metadata", meta=torch.zeros(3, dtype=torch.int32))
    _refused(sparse, "out", out=torch.zeros((2, 1, 16, 576), dtype=BF))
    _refused(sparse, "out", out=torch.zeros((2, 1, 16, 512)))
    _refused(sparse, "lse", lse=torch.zeros((2, 1, 17)))
    _refused(sparse, "lse", lse=torch.zeros((2, 1, 16), dtype=BF))
    _refused(sparse, "mla_decode", workspace=torch.zeros(1024, dtype=torch.uint8))


def test_decode_lists_that_are_refused():
    _refused(True, "indices", idx=torch.zeros((2, 5)))
    _refused(True, "indices", idx=torch.zeros((3, 5), dtype=torch.int32))
    _refused(True, "topk_lens", k=torch.ones(2, dtype=torch.int64))
    _refused(True, "topk_lens", k=torch.ones(3, dtype=torch.int32))
    import mla_absorbed_decode_gb300 as mla
    t = {k: v.cuda() for k, v in _tensors().items()}
    for idx, match in ((torch.zeros((2, 10), dtype=torch.int32, device="cuda")[:, ::2], "indices"),
                       (torch.zeros(5, dtype=torch.int32, device="cuda").expand(2, 5), "overlap")):
        with pytest.raises(ValueError, match=match):
            mla.decode_sparse_fp4(t["q"], t["kv"], 0.5, t["table"], t["n"], idx, t["k"], 0.1, False, t["meta"], 4)


def test_append_tensors_that_are_refused():
    import mla_absorbed_decode_gb300 as mla
    t = {k: v.cuda() for k, v in _tensors().items()}

    def refused(match, c=(2, 512), c_type=BF, pe=(2, 64), kv=t["kv"], **more):
        with pytest.raises((ValueError, TypeError), match=match):
            mla.cache_append_fp4(torch.zeros(c, dtype=c_type, device="cuda"), torch.zeros(pe, dtype=BF, device="cuda"), kv, 0.5,
                                 t["table"], t["n"], **more)

    refused("c", c_type=torch.float32)
    refused("k_pe", pe=(2, 32))
    refused("kv_cache", kv=torch.zeros((4, 64, 576), dtype=torch.uint8, device="cuda"))
    for norm in (torch.ones(512), torch.ones(256, dtype=BF), torch.ones(1024, dtype=BF)[::2]):
        refused("norm_weight", norm_weight=norm.cuda() if norm.is_contiguous() else torch.ones(1024, dtype=BF, device="cuda")[::2])
    refused("norm_weight", norm_weight=torch.ones(512, dtype=BF))      # not on the GPU


# ------------------------------------------------------------------------------------ rounding --
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("kv_scale", [2.0 ** -6, 0.013])
def test_append_codes_are_those_of_64_bits(norm, kv_scale):
    """Latent codes and scales from values that are known to 2^-40 of themselves (sums of two floats): none of the 2.1 million
    differs from the oracle's, whose 64 bits would have to lie within that of a halfway point (expected: 4e-6 of them)."""
    import mla_absorbed_decode_gb300 as mla
    g = torch.Generator().manual_seed(9)
    N, blocks = 4096, 64
    rows = torch.randn((N, 576), generator=g).to(BF)
    w = (1 + 0.3 * torch.randn(512, generator=g)).to(BF)
    kv = torch.zeros((blocks, 64, 352), dtype=torch.uint8, device="cuda")
    table = torch.arange(blocks, dtype=torch.int32, device="cuda").view(1, blocks)
    mla.cache_append_fp4(rows[:, :512].cuda(), rows[:, 512:].cuda(), kv, kv_scale, table,
                         torch.tensor([N], dtype=torch.int32, device="cuda"), norm_weight=w.cuda() if norm else None)
    assert mla.get_device_status() == 0
    x = to_np(rows)
    if norm:
        x = np.concatenate((oracle.normed_latent(x[:, :512], to_np(w), float(np.float32(1e-6))), x[:, 512:]), axis=1)
    assert np.array_equal(kv.view(N, 352).cpu().numpy(), oracle.pack_fp4(x, kv_scale))
