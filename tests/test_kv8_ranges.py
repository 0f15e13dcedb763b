"""What a write and a read of the 8-bit cache do for the sound requests of a call that has a bad
one (GPU): everything, unless offsets fall, and then never more than their own."""
import pytest
import torch

from tests import kv8_util as U
from tests.test_kv8 import H, cfg, i32, randn  # noqa: F401

pytestmark = pytest.mark.gpu

HKV, D, PAGE = 2, 64, 16


def run(H, cuda, cu, first, T, lens, poke=None):  # noqa: F811
    """(cache before, cache after, rows written, rows read) of a write and a read of the same ranges."""
    cache = U.make_cache(lens, HKV, D, PAGE, 8, stale_nan=False)
    if poke is not None:
        cache["page_table"][poke] = 10 ** 6
    rows = randn((T, HKV, D), 1, torch.bfloat16)
    dev, c = U.to_device(cache, cuda), cfg(H, HKV, HKV, D, PAGE)
    r = rows.to(cuda)
    H.hspec_kv8_write(c, r, r, i32(cu, cuda), i32(first, cuda), H.kv8_view(dev))
    assert H.hspec_sync_status() == H.HSPEC_ERR_DEVICE_CHECK
    out = torch.full((T, HKV, D), -7.0, dtype=torch.bfloat16, device=cuda)
    H.hspec_kv8_read(c, H.kv8_view(dev), i32(cu, cuda), i32(first, cuda), out, out.clone())
    assert H.hspec_sync_status() == H.HSPEC_ERR_DEVICE_CHECK
    return cache, {k: v.cpu() for k, v in dev.items()}, rows, out.cpu()


@pytest.mark.parametrize("cu,first,T,bad,poke", [
    ([0, 100, 220, 330], [0, 0, 3], 329, [2], None),          # past the rows
    ([-40, 100, 220, 329], [0, 5, 3], 329, [0], None),
    ([0, 100, 220, 329], [0, 300, 3], 329, [1], None),        # past the table
    ([0, 100, 220, 329], [-1, 0, 3], 329, [0], None),
    ([0, 100, 5000, 5100], [2, 0, 3], 329, [1, 2], None),     # offsets past the rows, rising
    ([0, 100, 220, 329], [0, 0, 3], 329, [1], (1, 0)),        # a bad page: only its tokens
])
def test_the_sound_requests_are_complete(H, cuda, cu, first, T, bad, poke):  # noqa: F811
    cache, after, rows, out = run(H, cuda, cu, first, T, [400, 400, 400], poke)
    for c in range(3):
        if c in bad:
            continue
        one = U.write(cache, rows, rows, cu[c:c + 2], first[c:c + 1])
        if c:  # (the reference numbers its requests from 0)
            one = U.write(dict(cache, page_table=cache["page_table"][c:]), rows, rows, cu[c:c + 2], first[c:c + 1])
        pages = cache["page_table"][c].long()
        for x in ("k", "v"):
            assert torch.equal(after[x + "_codes"][pages], one[x + "_codes"][pages])
            assert torch.equal(after[x + "_scales"][pages], one[x + "_scales"][pages])
        n = cu[c + 1] - cu[c]
        want = U.gather(dict(one, page_table=cache["page_table"][c:]), "k", 0, first[c], first[c] + n)
        assert torch.equal(out[cu[c]:cu[c + 1]].double(), want)


@pytest.mark.parametrize("cu", [[0, 1000, 10, 20], [0, 10, 5, 900], [700, 20, 1000, 990]])
def test_offsets_that_fall_touch_no_others_pages(H, cuda, cu):  # noqa: F811
    # which of the sound requests' pages are written is open; no other page is, and a page that
    # is written holds its request's rows
    T = 1000
    cache, after, rows, out = run(H, cuda, cu, [0, 0, 0], T, [1000, 1000, 1000])
    for c in range(3):
        pages = cache["page_table"][c].long()
        sound = 0 <= cu[c] <= cu[c + 1] <= T
        one = U.write(dict(cache, page_table=cache["page_table"][c:]), rows, rows, cu[c:c + 2], [0]) if sound else cache
        for x in ("k", "v"):
            for p in pages.tolist():
                got = after[x + "_codes"][p]
                assert torch.equal(got, cache[x + "_codes"][p]) or torch.equal(got, one[x + "_codes"][p])
    free = torch.ones(cache["k_codes"].shape[0], dtype=torch.bool)
    free[cache["page_table"].flatten().long()] = False
    assert torch.equal(after["k_codes"][free], cache["k_codes"][free])
