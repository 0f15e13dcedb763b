"""Attention over the 8-bit cache for batches at their ends: no key anywhere, and more requests
than a grid's z extent holds (GPU)."""
import pytest
import torch

from tests import kv8_util as U
from tests.test_kv8 import H, attend, cfg, check_attention, i32, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [1, 17])
def test_no_request_has_a_key(H, cuda, K, dtype):  # noqa: F811
    lens = [0, 0, 0]
    out = check_attention(H, cuda, lens, K, 8, 2, 128, 16, dtype, False, False)
    assert bool((out == 0).all())
    check_attention(H, cuda, lens, K, 8, 2, 128, 16, dtype, True, True)  # the block's keys alone


def test_more_requests_than_65535(H, cuda):  # noqa: F811
    # the tensor-core path takes them: each request gives what it gives in a small batch
    C, D, page = 66000, 64, 16
    g = torch.Generator().manual_seed(3)
    few = U.make_cache([5, 16, 0, 1], 1, D, page, 2)
    pick = torch.randint(0, 4, (C,), generator=g)
    dev = U.to_device(dict(few, page_table=few["page_table"][pick]), cuda)
    q = randn((C, 1, 1, D), 4, torch.bfloat16).to(cuda)
    lens = torch.tensor([5, 16, 0, 1])[pick]
    out = attend(H, cfg(H, 1, 1, D, page), q, dev, lens.tolist(), None, None)
    assert H.hspec_sync_status() == 0
    some = torch.cat([torch.arange(40), torch.randint(0, C, (100,), generator=g), torch.arange(C - 40, C)])
    part = dict(dev, page_table=dev["page_table"][some.to(cuda)].contiguous())
    want = attend(H, cfg(H, 1, 1, D, page), q[some.to(cuda)], part, lens[some].tolist(), None, None)
    assert H.hspec_sync_status() == 0
    assert torch.equal(out[some.to(cuda)], want)
    ref, A, S = U.attention(q[some.to(cuda)].cpu(), dict(few, page_table=few["page_table"][pick[some]]),
                            lens[some].tolist(), None, None, False)
    assert bool(((want.cpu().double() - ref).abs() <= U.attention_bound(ref, A, S, torch.bfloat16, 16, D)).all())
