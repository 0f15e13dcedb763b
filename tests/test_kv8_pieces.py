"""Attention over the 8-bit cache with whole contexts in one piece (GPU).

The automatic partition cuts the small batches of the other tests into pieces of a tile or two;
with a large attn_split_tokens one piece holds a context, so that the running references rise,
come down and are looked at again within it."""
import math

import pytest
import torch

from tests import kv8_util as U
from tests.test_kv8 import H, attend, cfg, check_attention, randn  # noqa: F401

pytestmark = pytest.mark.gpu

WHOLE = 1 << 20  # one chunk holds the batch
# K, Hq, Hkv: 4, 20, 32, 60, 68 and 128 query rows a kv head: every width of the query side
WIDTHS = [(1, 4, 1), (5, 4, 1), (8, 8, 2), (15, 4, 1), (17, 4, 1), (32, 4, 1)]


def run(H, cuda, cache, q, lens, **kw):  # noqa: F811
    C, K, Hq, D = q.shape
    Hkv, page = cache["k_codes"].shape[1:3]
    c = cfg(H, Hq, Hkv, D, page, attn_split_tokens=WHOLE, **kw)
    out = attend(H, c, q.to(cuda), U.to_device(cache, cuda), lens, None, None)
    assert H.hspec_sync_status() == 0
    return out.cpu().double()


def small_weights(q, cache, lens):
    """What the parts of small weights may lose, [C, K, Hq, D], by the format stated in the header.

    A weight p_t enters the product with V as P_t = 8 p_t sv_t / Mv, in units of 2^(its reference), sv_t
    its page's V scale and Mv the largest of the request and head.  The low part's smallest step
    is 2^-9 / 32, so P_t is off by half of that at most, and by no more than itself; the
    references never exceed the row's maximum.  Undone: min(p_t, 2^-18 p_max Mv / sv_t) |v_t|."""
    C, K, Hq, D = q.shape
    out = torch.zeros(C, K, Hq, D, dtype=torch.float64)
    page, G = cache["v_codes"].shape[2], Hq // cache["v_codes"].shape[1]
    for c, n in enumerate(lens):
        k, v = U.gather(cache, "k", c, 0, n), U.gather(cache, "v", c, 0, n).abs()
        sv = cache["v_scales"][cache["page_table"][c, torch.arange(n) // page].long()].double()  # [n, Hkv]
        ratio = sv.amax(0) / sv
        for j in range(K):
            for h in range(Hq):
                p = torch.softmax(k[:, h // G] @ q[c, j, h].double() / math.sqrt(D), 0)
                out[c, j, h] = torch.minimum(p, 2.0 ** -18 * p.max() * ratio[:, h // G]) @ v[:, h // G]
    return out


def over(got, ref, A, S, keys, D, lost=0.0):
    bound = U.attention_bound(ref, A, S, torch.bfloat16, keys, D) + lost
    return float(((got - ref).abs() / bound).nan_to_num(1e9).max())


def lay(cache, c, x, t, code):
    """Token t of request c gets `code` in every dim of every head."""
    page = cache[x + "_codes"].shape[2]
    cache[x + "_codes"][int(cache["page_table"][c, t // page]), :, t % page] = code


@pytest.mark.parametrize("K,Hq,Hkv", WIDTHS)
@pytest.mark.parametrize("D", [64, 128])
def test_maxima_that_jump(H, cuda, K, Hq, Hkv, D):  # noqa: F811
    # the scores' scale grows from tile to tile by steps of 2^0 .. 2^9: maxima that creep, and
    # jumps by far more than a weight's range (a weight under the old maximum overflows)
    lens, page = [1300, 700], 16
    cache = U.make_cache(lens, Hkv, D, page, 21)
    for r, n in enumerate(lens):
        for i in range((n + page - 1) // page):
            cache["k_scales"][int(cache["page_table"][r, i])] = 2.0 ** (-14 + (i // 8) * (r + 1))
    q = randn((2, K, Hq, D), 1, torch.bfloat16)
    ref, A, S = U.attention(q, cache, lens, None, None, False)
    assert over(run(H, cuda, cache, q, lens), ref, A, S, 1300, D, small_weights(q, cache, lens)) <= 1.0


@pytest.mark.parametrize("K,Hq,Hkv", WIDTHS)
def test_maxima_that_rise_and_fall(H, cuda, K, Hq, Hkv):  # noqa: F811
    # scales of the scores that wander over 2^-14 .. 2^2 from page to page, V scales over 2^6
    lens, D, page = [5000, 130, 2100], 128, 16
    g = torch.Generator().manual_seed(K)
    cache = U.make_cache(lens, Hkv, D, page, 5)
    for r, n in enumerate(lens):
        for i in range((n + page - 1) // page):
            p = int(cache["page_table"][r, i])
            cache["k_scales"][p] = 2.0 ** int(-14 + 16 * torch.rand(1, generator=g) ** 6)
            cache["v_scales"][p] *= 2.0 ** int(torch.randint(0, 7, (1,), generator=g))
    q = randn((3, K, Hq, D), 1, torch.bfloat16)
    ref, A, S = U.attention(q, cache, lens, None, None, False)
    assert over(run(H, cuda, cache, q, lens), ref, A, S, 5000, D, small_weights(q, cache, lens)) <= 1.0


@pytest.mark.parametrize("K,Hq,Hkv", WIDTHS)
def test_long_contexts(H, cuda, K, Hq, Hkv):  # noqa: F811
    # ordinary data, hundreds of tiles a piece; with a causal block as well
    check_attention(H, cuda, [9000, 17], K, Hq, Hkv, 128, 16, torch.bfloat16, False, False, attn_split_tokens=WHOLE)
    check_attention(H, cuda, [2000, 640], K, Hq, Hkv, 64, 32, torch.bfloat16, True, True, attn_split_tokens=WHOLE)


def one_key(n, Hkv, at, below, count=1):
    """A cache of n tokens and queries of ones: `count` keys at `at` (tiles in a row, one each),
    all others 2^-below of one of those in weight, values >= 0."""
    D, page = 128, 16
    cache = U.make_cache([n], Hkv, D, page, 3)
    cache["k_codes"][:], cache["k_scales"][:] = 0, 2.0 ** -12  # scores of zero
    cache["v_codes"][:], cache["v_scales"][:] = 0x38, 1.0      # values of one
    for i in range(count):
        lay(cache, 0, "k", at + 128 * i, 0x7E)  # 448 * 2^-12 in every dim
    return cache, below * math.log(2.0) / (448 * 2.0 ** -12 * D / math.sqrt(D))


@pytest.mark.parametrize("K,Hq,Hkv", WIDTHS)
@pytest.mark.parametrize("at,below,count", [
    (67 * 128 + 5, 17.05, 1), (67 * 128 + 5, 18.05, 1), (67 * 128 + 5, 16.5, 1), (66 * 128, 17.05, 1), (0, 17.05, 1),
    (3 * 128, 17.5, 1), (32 * 128 + 127, 19.0, 1), (64 * 128, 17.05, 4), (66 * 128, 17.05, 10), (2 * 128, 17.05, 20),
    (126 * 128, 17.05, 1),
])
def test_keys_that_outweigh_all_others(H, cuda, K, Hq, Hkv, at, below, count):  # noqa: F811
    # what is lost of the small weights that follow shows in the sum: every value is 1, and so is
    # the output
    n = 128 * 128
    cache, scale = one_key(n, Hkv, at, below, count)
    q = torch.full((1, K, Hq, 128), scale).to(torch.bfloat16)
    got = run(H, cuda, cache, q, [n])
    # A = 1; weights' parts 2^-8 and the store 2^-8 (as attention_bound without its terms in S)
    err = float((got - 1.0).abs().max())
    assert err <= 2.0 ** -7, err


@pytest.mark.parametrize("K,Hq,Hkv", [(1, 8, 1), (16, 4, 1), (17, 4, 1)])
@pytest.mark.parametrize("split", [0, WHOLE])
def test_error_of_long_contexts_in_the_mean(H, cuda, K, Hq, Hkv, split):  # noqa: F811
    """The error's RMS against the output's.

    A weight's two parts are off by up to 2^-8 of it and the store by up to 2^-8 of the output;
    an error spread evenly over +-h has RMS h / sqrt(3), and one whose distribution falls off
    towards +-h less.  The values are independent of sign zero mean, so a weight error of RMS e
    p_t gives the output's RMS times e.  Together at most sqrt(2 / 3) 2^-8 = 3.2e-3."""
    lens, D = [20000, 3000], 128
    cache = U.make_cache(lens, Hkv, D, 16, 7)
    q = randn((2, K, Hq, D), 1, torch.bfloat16)
    ref, _, _ = U.attention(q, cache, lens, None, None, False)
    c = cfg(H, Hq, Hkv, D, 16, attn_split_tokens=split)
    got = attend(H, c, q.to(cuda), U.to_device(cache, cuda), lens, None, None).cpu().double()
    assert H.hspec_sync_status() == 0
    rel = (((got - ref) ** 2).mean((1, 2, 3)) / (ref ** 2).mean((1, 2, 3))).sqrt()
    print("rel", rel.tolist())
    assert float(rel.max()) <= 3.2e-3
