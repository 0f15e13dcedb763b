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
