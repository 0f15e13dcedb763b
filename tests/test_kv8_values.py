"""Values at the edge of the 8-bit cache's format (GPU), with expectations written out."""
import pytest
import torch

from tests import kv8_util as U
from tests.test_kv8 import H, cfg, i32  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 10])
def test_infinities_without_a_finite_value_to_scale_by(H, cuda, D, dtype):  # noqa: F811
    # a page and head whose finite values are all zero has scale 0: an infinity is +-448 * 0
    # there, a NaN stays a NaN, and a later token's scale finds zeros
    Hkv, page, inf, nan = 2, 16, float("inf"), float("nan")
    rows = torch.zeros(5, Hkv, D)
    rows[0, 0, 1], rows[2, 0, 3], rows[3, 0, 9], rows[3, 0, 0] = inf, -inf, inf, -0.0
    rows[1, 1, 2], rows[4, 1, 4] = inf, nan
    rows = rows.to(dtype).to(cuda)
    cache = U.to_device(U.make_cache([9], Hkv, D, page, 1, stale_nan=False), cuda)
    c, kv = cfg(H, Hkv, Hkv, D, page, dtype), H.kv8_view(cache)
    H.hspec_kv8_write(c, rows, -rows, i32([0, 5], cuda), i32([0], cuda), kv)
    out = [torch.full((5, Hkv, D), -7.0, dtype=dtype, device=cuda) for _ in range(2)]
    H.hspec_kv8_read(c, kv, i32([0, 5], cuda), None, *out)
    assert H.hspec_sync_status() == 0
    p = int(cache["page_table"][0, 0])
    assert bool((cache["k_scales"][p] == 0).all()) and bool((cache["v_scales"][p] == 0).all())
    for o in out:
        assert torch.equal(o.isnan(), rows.isnan()) and bool((o.nan_to_num(0.0) == 0).all())
    # tokens 5 .. 8 of ordinary size: the scale rises, what was there stays zero or NaN
    more = torch.ones(4, Hkv, D, dtype=dtype, device=cuda)
    H.hspec_kv8_write(c, more, more, i32([0, 4], cuda), i32([5], cuda), kv)
    out = [torch.full((9, Hkv, D), -7.0, dtype=dtype, device=cuda) for _ in range(2)]
    H.hspec_kv8_read(c, kv, i32([0, 9], cuda), None, *out)
    assert H.hspec_sync_status() == 0
    for o in out:
        assert torch.equal(o[:5].isnan(), rows.isnan()) and bool((o[:5].nan_to_num(0.0) == 0).all())
        assert bool((o[5:] == 1).all())


def test_read_rounds_once_whatever_the_scale(H, cuda):  # noqa: F811
    # scales of 24 bits for which code * scale, rounded to fp32, is a tie in bf16 that the product
    # is not; and scales below the normal range
    g = torch.Generator().manual_seed(5)
    codes = torch.randint(1, 127, (4_000_000,), generator=g)
    s = (1.0 + torch.rand(codes.numel(), generator=g)) * 2.0 ** -7
    tiny = torch.arange(codes.numel()) % 8 == 0
    s = torch.where(tiny, s * 2.0 ** -125, s)
    exact = U.VALUES[codes] * s.double()
    # one rounding of a double to bf16's 8 bits, ties to even (a step of 2^-133 at least)
    step = torch.exp2((torch.floor(torch.log2(exact)) - 7).clamp_min(-133.0))
    once = (torch.round(exact / step) * step).to(torch.bfloat16)
    twice = (U.VALUES[codes].float() * s).to(torch.bfloat16)
    hard = (once != twice).nonzero().flatten()
    assert hard.numel() >= 8 and bool(tiny[hard].any())
    pick = torch.cat([hard[:64], torch.arange(64)])
    n, D = pick.numel(), 16
    cache = {"page_table": torch.arange(n, dtype=torch.int32).view(1, n), "k_scales": s[pick].view(n, 1),
             "v_scales": -0.0 + s[pick].view(n, 1)}
    cache["k_codes"] = codes[pick].to(torch.uint8).view(n, 1, 1, 1).expand(n, 1, 1, D).contiguous()
    cache["v_codes"] = cache["k_codes"] | 0x80
    dev = U.to_device(cache, cuda)
    out = [torch.full((n, 1, D), -7.0, dtype=torch.bfloat16, device=cuda) for _ in range(2)]
    H.hspec_kv8_read(cfg(H, 1, 1, D, 1), H.kv8_view(dev), i32([0, n], cuda), None, *out)
    assert H.hspec_sync_status() == 0
    want = once[pick].view(n, 1, 1).expand(n, 1, D)
    assert torch.equal(out[0].cpu(), want) and torch.equal(out[1].cpu(), -want)
