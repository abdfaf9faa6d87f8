"""What the merge of split requests makes of rows that are NaN: the 4-bit decode's come out as NaN, while the bf16 and FP8 decodes give
such a row's partials an lse of -inf, with which it merges to 0 and -inf; rows beside it keep their bits in all of them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_absorbed_decode_gb300 import build_lib
    build_lib.build()
    yield


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("parts", [None, 7])
def test_a_nan_row_of_a_split_request(kind, parts):
    import mla_absorbed_decode_gb300 as mla
    g = torch.Generator(device="cuda").manual_seed(0)
    lens, H, scale = [6000, 2500, 3100], 24, (0.5,)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    table = torch.randperm(300, generator=g, device="cuda").to(torch.int32).view(3, 100)
    if kind == "fp4":
        kv = torch.randint(0, 256, (300, 64, 352), generator=g, device="cuda", dtype=torch.uint8)
        kv[..., 256:] &= 0xB7                                             # no NaN, scales and rope codes below 1
    else:
        kv = torch.randn((300, 64, 576), generator=g, device="cuda").to(BF if kind == "bf16" else torch.float8_e4m3fn)
        if kind == "fp8":
            kv = kv.view(torch.uint8)
        else:
            scale = ()
    q = torch.randn((3, 1, H, 576), generator=g, device="cuda").to(BF)
    P = mla.num_sm_parts(1, H) if parts is None else parts
    meta = mla.decode_metadata(n, 1, H, False, P)
    assert bool((meta[8 * P:8 * P + 4].diff() > 1).any())                # some request is split
    split = (meta[8 * P:8 * P + 4].diff() > 1).tolist()
    call = getattr(mla, "decode" if kind == "bf16" else "decode_" + kind)
    clean = call(q, kv, *scale, table, n, 192 ** -0.5, False, meta, P)
    q = q.clone()
    q[:, 0, 5, 77] = float("nan")
    out, lse = call(q, kv, *scale, table, n, 192 ** -0.5, False, meta, P)
    assert mla.get_device_status() == 0
    rest = [h for h in range(H) if h != 5]
    assert torch.equal(out[:, :, rest], clean[0][:, :, rest]) and torch.equal(lse[:, :, rest], clean[1][:, :, rest])
    for b in range(3):
        if kind == "fp4":
            assert out[b, 0, 5].isnan().all() and lse[b, 0, 5].isnan()
        else:
            assert lse[b, 0, 5].isneginf()
            if split[b]:
                assert not out[b, 0, 5].any()
