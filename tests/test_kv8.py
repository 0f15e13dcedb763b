"""The 8-bit paged KV cache on the GPU: writing, reading back and attending, each against
plain double arithmetic (kv8_util), and the three in a row as a decoding target uses them."""
import pytest
import torch

from tests import kv8_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def H(cuda):
    from hybrid_mamba_attention_b200 import hspec
    return hspec


def cfg(H, Hq, Hkv, D, page, dtype=torch.bfloat16, causal=False, **kw):
    return H.hspec_cfg(d_model=Hq * D, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=D, page_size=page, n_layers=1,
                       layer_kinds=b"A", dtype=H.HSPEC_DTYPE_BF16 if dtype == torch.bfloat16 else H.HSPEC_DTYPE_F32,
                       flags=H.HSPEC_FLAG_CAUSAL_BLOCK if causal else 0, **kw)


def i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def offsets(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return cu


def randn(shape, seed, dtype, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def assert_same_cache(got, want, what=""):
    for x in ("k", "v"):
        assert torch.equal(got[x + "_scales"].cpu().nan_to_num(-1.0), want[x + "_scales"].nan_to_num(-1.0)), what
        a, b = U.VALUES[got[x + "_codes"].cpu().long()], U.VALUES[want[x + "_codes"].long()]
        bad = ~((a == b) | (a.isnan() & b.isnan()))
        assert not bad.any(), f"{what} {x}: {int(bad.sum())} codes differ, first at {bad.nonzero()[0].tolist()}"


# ------------------------------------------------------------------------- write, read

WRITES = [
    # (first, new tokens), Hkv, D, page
    ([0, 0, 0], [1, 0, 33], 2, 128, 16),
    ([5, 16, 31, 47], [1, 1, 1, 1], 8, 128, 16),     # one token each: inside, at and before a page's edge
    ([3, 0, 250, 7], [17, 64, 40, 9], 3, 64, 16),
    ([1, 70], [100, 129], 2, 128, 64),
    ([4, 2], [11, 30], 2, 66, 5),                     # odd page, rows not in multiples of eight
    ([0, 9], [300, 1], 1, 256, 128),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("first,new,Hkv,D,page", WRITES)
def test_write_then_read(H, cuda, first, new, Hkv, D, page, dtype):
    lens = [a + b for a, b in zip(first, new)]
    cache = U.make_cache(lens, Hkv, D, page, 3, stale_nan=False)
    cu = offsets(new)
    # magnitudes from far below to far above the old pages'
    spread = torch.exp2(torch.arange(cu[-1]) % 9 - 4.0)[:, None, None]
    k = (randn((cu[-1], Hkv, D), 4, torch.float32) * spread).to(dtype)
    v = (randn((cu[-1], Hkv, D), 5, torch.float32) / spread).to(dtype)
    v[:, 0] = 0  # a head of zeros: scale 0 in a fresh page
    want = U.write(cache, k, v, cu, first)
    dev = U.to_device(cache, cuda)
    c = cfg(H, Hkv, Hkv, D, page, dtype)
    H.hspec_kv8_write(c, k.to(cuda), v.to(cuda), i32(cu, cuda), i32(first, cuda), H.kv8_view(dev))
    assert H.hspec_sync_status() == 0
    assert_same_cache(dev, want)
    # read everything back, from token 0 and from the middle
    for start in ([0] * len(lens), first):
        n = [a - b for a, b in zip(lens, start)]
        co = offsets(n)
        ko = torch.full((co[-1] + 2, Hkv, D), -7.0, dtype=dtype, device=cuda)
        vo = ko.clone()
        H.hspec_kv8_read(c, H.kv8_view(dev), i32(co, cuda), None if start[0] == 0 == max(start) else i32(start, cuda),
                         ko, vo)
        assert H.hspec_sync_status() == 0
        for x, o in (("k", ko), ("v", vo)):
            ref = torch.cat([U.gather(want, x, r, start[r], lens[r]) for r in range(len(lens))])
            assert torch.equal(o[:co[-1]].cpu(), ref.to(dtype)) and bool((o[co[-1]:] == -7.0).all())


def test_write_rows_of_a_wider_projection(H, cuda):
    Hkv, D, page = 2, 128, 16
    first, new = [6, 0], [20, 3]
    cache = U.make_cache([26, 3], Hkv, D, page, 9)
    wide = randn((25, 4 * 128 + 2 * 2 * Hkv * D), 1, torch.bfloat16)
    k = wide[:, 512:512 + Hkv * D].view(25, Hkv, D)
    v = wide[:, 512 + Hkv * D:512 + 2 * Hkv * D].view(25, Hkv, D)
    want = U.write(cache, k, v, [1, 21, 24], first)  # rows 0 and 24 belong to nobody
    dev, w = U.to_device(cache, cuda), wide.to(cuda)
    w[0] = float("nan")
    H.hspec_kv8_write(cfg(H, 4, Hkv, D, page), w[:, 512:768].view(25, Hkv, D), w[:, 768:1024].view(25, Hkv, D),
                      i32([1, 21, 24], cuda), i32(first, cuda), H.kv8_view(dev))
    assert H.hspec_sync_status() == 0
    assert_same_cache(dev, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_write_special_values(H, cuda, dtype):
    # NaN, infinities, the largest and the smallest numbers, zeros, ties, each in its own page
    Hkv, D, page = 1, 64, 16
    cache = U.make_cache([16 * 6 + 3], Hkv, D, page, 2)
    k = randn((99, Hkv, D), 3, torch.float32)
    k[3, 0, 5], k[17, 0, 0], k[18, 0, 1] = float("nan"), float("inf"), -float("inf")
    k[32:48] *= 2.0 ** 126
    k[33, 0, 3] = torch.finfo(dtype).max
    k[48:64] *= 2.0 ** -130
    k[64:80] = 0.0
    k[80:96] = (torch.arange(1024).reshape(16, 1, 64) - 512) / 64.0  # multiples of 1/64 up to 8: many ties
    k = k.to(dtype)
    v = (-k).contiguous()
    want = U.write(cache, k, v, [0, 99], [0])
    dev = U.to_device(cache, cuda)
    H.hspec_kv8_write(cfg(H, 1, Hkv, D, page, dtype), k.to(cuda), v.to(cuda), i32([0, 99], cuda), i32([0], cuda),
                      H.kv8_view(dev))
    assert H.hspec_sync_status() == 0
    assert_same_cache(dev, want)


def test_token_by_token_equals_the_definition(H, cuda):
    # 40 appended tokens, growing magnitudes: every page is rescaled several times
    Hkv, D, page = 2, 128, 16
    cache = U.make_cache([40, 43], Hkv, D, page, 6)
    dev, c = U.to_device(cache, cuda), cfg(H, 2, Hkv, D, page)
    want = cache
    for t in range(40):
        k = randn((2, Hkv, D), 100 + t, torch.bfloat16, 2.0 ** (t % 7 - 3))
        v = randn((2, Hkv, D), 200 + t, torch.bfloat16, 2.0 ** (3 - t % 5))
        want = U.write(want, k, v, [0, 1, 2], [t, 3 + t])
        H.hspec_kv8_write(c, k.to(cuda), v.to(cuda), i32([0, 1, 2], cuda), i32([t, 3 + t], cuda), H.kv8_view(dev))
    assert H.hspec_sync_status() == 0
    assert_same_cache(dev, want)


def test_write_and_read_report_bad_ranges_and_pages(H, cuda):
    Hkv, D, page = 2, 64, 16
    c = cfg(H, 2, Hkv, D, page)

    def fresh():
        return U.make_cache([40, 40, 40], Hkv, D, page, 8)

    k = randn((30, Hkv, D), 1, torch.bfloat16)
    for cu, first, bad, poke in (([0, 10, 5, 15], [0, 0, 0], 1, None),     # falling offsets
                                 ([0, 10, 20, 31], [0, 0, 0], 2, None),    # past the rows
                                 ([-3, 10, 20, 30], [0, 0, 0], 0, None),
                                 ([0, 10, 20, 30], [0, 39, 0], 1, None),   # past the table's 48 slots
                                 ([0, 10, 20, 30], [0, -1, 0], 1, None),
                                 ([0, 10, 20, 30], [0, 0, 0], 1, 77),      # page ids outside the pool
                                 ([0, 10, 20, 30], [0, 0, 0], 1, -1)):
        cache = fresh()
        if poke is not None:
            cache["page_table"][1, 0] = poke
        dev = U.to_device(cache, cuda)
        before = {n: t.clone() for n, t in dev.items()}
        H.hspec_kv8_write(c, k.to(cuda), k.to(cuda), i32(cu, cuda), i32(first, cuda), H.kv8_view(dev))
        assert H.hspec_sync_status() == H.HSPEC_ERR_DEVICE_CHECK
        # pages that no sound request owns keep their bytes
        mine = set(cache["page_table"][[r for r in range(3) if r != bad]].flatten().tolist())
        other = [p for p in range(before["k_codes"].shape[0]) if p not in mine]
        assert torch.equal(dev["k_codes"][other], before["k_codes"][other])
        o = torch.full((30, Hkv, D), -7.0, dtype=torch.bfloat16, device=cuda)
        o2 = o.clone()
        H.hspec_kv8_read(c, H.kv8_view(dev), i32(cu, cuda), i32(first, cuda), o, o2)
        assert H.hspec_sync_status() == H.HSPEC_ERR_DEVICE_CHECK
        if poke is not None:
            assert bool((o[10:20] == 0).all())
    assert H.hspec_sync_status() == 0


# --------------------------------------------------------------------------- attention

def attend(H, c, q, dev, lens, kb, vb, ws=None):
    C, K = q.shape[:2]
    kv = H.kv8_view(dev)
    if ws is None:
        ws = H.alloc_workspace(H.hspec_attn_kv8_workspace_size(c, C, K, kv.max_pages))
        ws.fill_(0xFF)  # NaN everywhere: nothing unwritten may be read
    out = torch.full_like(q, float("nan"))
    H.hspec_attn_paged_block_kv8(c, q, kv, i32(lens, q.device), kb, vb, out, ws)
    return out


def check_attention(H, cuda, lens, K, Hq, Hkv, D, page, dtype, block, causal, seed=0, pow2=True, scale=1.0, **kw):
    cache = U.make_cache(lens, Hkv, D, page, seed + 11, pow2=pow2)
    q = randn((len(lens), K, Hq, D), seed + 1, dtype, scale)
    kb = randn((len(lens), K, Hkv, D), seed + 2, dtype) if block else None
    vb = randn((len(lens), K, Hkv, D), seed + 3, dtype) if block else None
    ref, A, S = U.attention(q, cache, lens, kb, vb, causal)
    dev = U.to_device(cache, cuda)
    to = lambda t: None if t is None else t.to(cuda)  # noqa: E731
    out = attend(H, cfg(H, Hq, Hkv, D, page, dtype, causal, **kw), q.to(cuda), dev, lens, to(kb), to(vb))
    assert H.hspec_sync_status() == 0
    got = out.cpu().double()
    bound = U.attention_bound(ref, A, S, dtype, max(lens) + K, D)
    over = ((got - ref).abs() / bound).nan_to_num(1e9)
    assert over.max() <= 1.0, f"{float(over.max()):.2f} times the bound at {(over == over.max()).nonzero()[0].tolist()}"
    return out


FAST = [
    # lens, K, Hq, Hkv, D, page: what the tensor-core path takes in bf16
    ([1], 1, 4, 1, 128, 16),
    ([0, 1, 2, 127, 128, 129, 640], 1, 8, 2, 128, 16),
    ([64, 700, 15, 0, 333], 16, 8, 2, 128, 16),
    ([300, 16, 17], 17, 4, 1, 128, 16),      # 68 rows
    ([257, 90], 33, 4, 1, 128, 32),          # 132 rows: two row blocks
    ([500], 64, 8, 2, 128, 64),              # 256 rows
    ([40, 411], 5, 7, 1, 128, 128),          # group of 7
    ([200, 31], 8, 16, 16, 128, 16),         # one query head per kv head
    ([130, 0, 65], 9, 8, 2, 64, 16),
    ([1000, 5], 24, 32, 1, 64, 48),          # 768 rows, pages of 48
]
ODD = [
    ([33, 0, 7], 3, 4, 2, 96, 16),
    ([100, 41], 7, 6, 2, 128, 5),
    ([77], 64, 12, 4, 256, 8),
    ([19, 64], 2, 2, 1, 10, 3),
]


@pytest.mark.parametrize("block,causal", [(True, False), (True, True), (False, False), (False, True)])
@pytest.mark.parametrize("lens,K,Hq,Hkv,D,page", FAST + ODD)
def test_attention_bf16(H, cuda, lens, K, Hq, Hkv, D, page, block, causal):
    check_attention(H, cuda, lens, K, Hq, Hkv, D, page, torch.bfloat16, block, causal)


@pytest.mark.parametrize("block,causal", [(True, True), (False, True), (False, False)])
@pytest.mark.parametrize("lens,K,Hq,Hkv,D,page", FAST[1:4] + ODD)
def test_attention_f32(H, cuda, lens, K, Hq, Hkv, D, page, block, causal):
    check_attention(H, cuda, lens, K, Hq, Hkv, D, page, torch.float32, block, causal)


@pytest.mark.parametrize("K,G", [(1, 1), (3, 3), (15, 1), (2, 12), (11, 3), (7, 6), (7, 7), (13, 5), (16, 5), (16, 6),
                                 (33, 3), (43, 3), (50, 3)])
def test_attention_query_rows(H, cuda, K, G):
    # 1 .. 150 query rows a kv head: every width of the query side, filled to the last column or not
    check_attention(H, cuda, [300, 5, 0, 140], K, 2 * G, 2, 128, 16, torch.bfloat16, True, True, seed=K)
    check_attention(H, cuda, [300, 70], K, 2 * G, 2, 64, 32, torch.bfloat16, False, False, seed=K + 1)


@pytest.mark.parametrize("D", [64, 100, 128, 256])
@pytest.mark.parametrize("K,G", [(8, 4), (11, 3), (16, 4), (13, 5), (29, 8)])
def test_attention_query_rows_f32(H, cuda, K, G, D):
    # 32 .. 232 query rows a kv head on the CUDA cores
    check_attention(H, cuda, [100, 5, 0, 170], K, 2 * G, 2, D, 16, torch.float32, True, True, seed=K)


@pytest.mark.parametrize("page", [80, 112, 144, 256, 1024])
def test_attention_page_sizes(H, cuda, page):
    # tiles that begin inside pages, pages of several tiles
    check_attention(H, cuda, [1500, 255, 257, 1], 3, 8, 2, 128, page, torch.bfloat16, True, True, seed=page)
    check_attention(H, cuda, [2100, 1024], 1, 8, 2, 64, page, torch.bfloat16, False, False, seed=page)


@pytest.mark.parametrize("split", [0, 64, 128, 512])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_split_lengths(H, cuda, split, dtype):
    check_attention(H, cuda, [900, 70, 0, 2000], 4, 8, 2, 128, 16, dtype, True, True, attn_split_tokens=split)


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -60, 12.0])
def test_attention_small_and_large_queries(H, cuda, scale):
    # flat weights (zero and tiny queries) and weights that sit on a few keys
    check_attention(H, cuda, [600, 45], 4, 8, 2, 128, 16, torch.bfloat16, True, False, scale=scale)


def test_attention_maxima_that_jump(H, cuda):
    # the scores' scale grows from tile to tile by steps of 2^0 .. 2^9: maxima that creep, and
    # jumps by far more than a weight's range (a weight under the old maximum overflows)
    lens, K, Hq, Hkv, D, page = [1300, 700], 4, 8, 2, 128, 16
    cache = U.make_cache(lens, Hkv, D, page, 21)
    for r, n in enumerate(lens):
        for i in range((n + page - 1) // page):
            cache["k_scales"][int(cache["page_table"][r, i])] = 2.0 ** (-14 + (i // 8) * (r + 1))
    q = randn((2, K, Hq, D), 1, torch.bfloat16)
    ref, A, S = U.attention(q, cache, lens, None, None, False)
    out = attend(H, cfg(H, Hq, Hkv, D, page), q.to(cuda), U.to_device(cache, cuda), lens, None, None)
    assert H.hspec_sync_status() == 0
    over = (out.cpu().double() - ref).abs() / U.attention_bound(ref, A, S, torch.bfloat16, 1300, D)
    assert float(over.nan_to_num(1e9).max()) <= 1.0


@pytest.mark.parametrize("K,first", [(1, 0), (20, 0), (1, 4000)])
def test_attention_one_key_against_many(H, cuda, K, first):
    # one key (a context's first, or one within) holds half of the weight and some 24000 others,
    # each 2^-14 or less of it, share the rest with values of one sign: what is lost of small
    # weights, or of their sum, shows
    n, Hq, Hkv, D, page = 24000, 4, 1, 128, 16
    cache = U.make_cache([n], Hkv, D, page, 3)
    cache["k_scales"][:] = 2.0 ** -12  # scores near zero
    cache["v_codes"] &= 0x7F           # values >= 0
    q = torch.ones(1, K, Hq, D).to(torch.bfloat16)
    p, slot = int(cache["page_table"][0, first // page]), first % page
    cache["k_codes"][p, 0, slot] = 0x7E  # 448 * 2^-12 in every dim
    s = 448 * 2.0 ** -12 * 128 / 128 ** 0.5  # its score
    q = q * (14.6 * 0.6931 / s)
    ref, A, S = U.attention(q, cache, [n], None, None, False)
    out = attend(H, cfg(H, Hq, Hkv, D, page), q.to(cuda), U.to_device(cache, cuda), [n], None, None)
    assert H.hspec_sync_status() == 0
    # (the sums' 2^-24 a key of the general bound, 24000 of them, is below 2^-9 of A)
    over = (out.cpu().double() - ref).abs() / U.attention_bound(ref, A, S, torch.bfloat16, n, D)
    assert float(over.nan_to_num(1e9).max()) <= 1.0


def test_attention_foreign_scales(H, cuda):
    check_attention(H, cuda, [333, 129], 6, 8, 2, 128, 16, torch.bfloat16, True, False, pow2=False)


def test_attention_smallest_scales(H, cuda):
    # V scales below the normal range (their inverse is not finite), zero, and one normal page
    # among them; values of 448 keep the outputs normal
    lens, K, Hq, Hkv, D, page = [333, 40, 17], 6, 8, 2, 128, 16
    cache = U.make_cache(lens, Hkv, D, page, 8)
    cache["v_codes"][:] = 0x7E
    for r, e in enumerate((2.0 ** -132, 2.0 ** -131, 0.0)):
        cache["v_scales"][cache["page_table"][r, :(lens[r] + page - 1) // page].long()] = e
    q = randn((3, K, Hq, D), 1, torch.bfloat16)
    for normal in (False, True):
        if normal:
            cache["v_scales"][cache["page_table"][0, 20].long()] = 2.0 ** -125
        ref, A, S = U.attention(q, cache, lens, None, None, False)
        out = attend(H, cfg(H, Hq, Hkv, D, page), q.to(cuda), U.to_device(cache, cuda), lens, None, None)
        assert H.hspec_sync_status() == 0
        over = (out.cpu().double() - ref).abs() / U.attention_bound(ref, A, S, torch.bfloat16, 333, D)
        assert float(over[:2].nan_to_num(1e9).max()) <= 1.0
        assert bool((out[2] == 0).all())


def test_attention_rows_without_keys_are_zero(H, cuda):
    # causal over the cache alone with fewer tokens than positions: the first rows see nothing
    for lens, K in (([2, 0, 5], 5), ([1, 63, 0], 64)):
        out = check_attention(H, cuda, lens, K, 8, 2, 128, 16, torch.bfloat16, False, True)
        for c, n in enumerate(lens):
            assert bool((out[c, :K - n] == 0).all())


def test_attention_hidden_and_stale_nan(H, cuda):
    # a NaN token is seen by the rows at or after it alone; stale slots and slack pages
    # (NaN in every make_cache) by none
    lens, K, Hq, Hkv, D, page = [200, 37], 8, 8, 2, 128, 16
    cache = U.make_cache(lens, Hkv, D, page, 5)
    q = randn((2, K, Hq, D), 1, torch.bfloat16)
    for x in ("k", "v"):
        dirty = {n: t.clone() for n, t in cache.items()}
        t = lens[0] - 3  # seen by positions K - 3, K - 2, K - 1
        dirty[x + "_codes"][dirty["page_table"][0, t // page].long(), :, t % page] = U.NAN_CODE
        ref, A, S = U.attention(q, dirty, lens, None, None, True)
        out = attend(H, cfg(H, Hq, Hkv, D, page, causal=True), q.to(cuda), U.to_device(dirty, cuda), lens, None, None)
        assert H.hspec_sync_status() == 0
        got = out.cpu().double()
        assert torch.equal(got.isnan(), ref.isnan()), x
        assert int(ref.isnan().sum()) == 3 * Hq * D
        fine = ~ref.isnan()
        assert bool(((got - ref).abs() <= U.attention_bound(ref, A, S, torch.bfloat16, 200, D))[fine].all())
        # the same in a draft block
        kb, vb = randn((2, K, Hkv, D), 2, torch.bfloat16), randn((2, K, Hkv, D), 3, torch.bfloat16)
        (kb if x == "k" else vb)[1, 5] = float("nan")
        ref, A, S = U.attention(q, cache, lens, kb, vb, True)
        out = attend(H, cfg(H, Hq, Hkv, D, page, causal=True), q.to(cuda), U.to_device(cache, cuda), lens,
                     kb.to(cuda), vb.to(cuda))
        assert H.hspec_sync_status() == 0
        got = out.cpu().double()
        assert torch.equal(got.isnan(), ref.isnan()), x


def test_attention_zero_pages_and_mixed_v_scales(H, cuda):
    # pages of zeros (scale 0) in front and behind, V scales that fall and rise by 2^6
    lens, K, Hq, Hkv, D, page = [400, 160], 3, 8, 2, 128, 16
    cache = U.make_cache(lens, Hkv, D, page, 5)
    for r, n in enumerate(lens):
        for i in range(n // page):
            p = int(cache["page_table"][r, i])
            if i % 5 == 0:
                cache["v_codes"][p], cache["v_scales"][p] = 0, 0.0
                cache["k_codes"][p], cache["k_scales"][p] = 0, 0.0
            else:
                cache["v_scales"][p] *= 2.0 ** (i % 7)
    q = randn((2, K, Hq, D), 1, torch.bfloat16)
    ref, A, S = U.attention(q, cache, lens, None, None, False)
    out = attend(H, cfg(H, Hq, Hkv, D, page), q.to(cuda), U.to_device(cache, cuda), lens, None, None)
    assert H.hspec_sync_status() == 0
    assert bool(((out.cpu().double() - ref).abs() <= U.attention_bound(ref, A, S, torch.bfloat16, 400, D)).all())


def test_attention_bad_pages_and_lengths_are_reported(H, cuda):
    lens, Hq, Hkv, D, page = [100, 50, 20], 4, 1, 128, 16
    cache = U.make_cache(lens, Hkv, D, page, 5)
    q = randn((3, 2, Hq, D), 1, torch.bfloat16)
    good = attend(H, cfg(H, Hq, Hkv, D, page), q.to(cuda), U.to_device(cache, cuda), lens, None, None)
    assert H.hspec_sync_status() == 0
    for poke in (-1, 10 ** 6):
        dirty = {n: t.clone() for n, t in cache.items()}
        dirty["page_table"][1, 1] = poke
        out = attend(H, cfg(H, Hq, Hkv, D, page), q.to(cuda), U.to_device(dirty, cuda), lens, None, None)
        assert H.hspec_sync_status() == H.HSPEC_ERR_DEVICE_CHECK
        assert torch.equal(out[0], good[0])
    for bad in (-1, 7 * 16 + 1):
        out = attend(H, cfg(H, Hq, Hkv, D, page), q.to(cuda), U.to_device(cache, cuda), [100, bad, 20], None, None)
        assert H.hspec_sync_status() == H.HSPEC_ERR_DEVICE_CHECK
        assert bool((out[1] == 0).all())
    assert H.hspec_sync_status() == 0


def test_write_attend_verify_in_a_row(H, cuda):
    """A target's round over its 8-bit cache: prompt written, drafts attended as a block
    (the drafter), then written and verified causally (the target), on one stream, eagerly
    and replayed from a CUDA graph."""
    lens, K, Hq, Hkv, D, page = [90, 33, 250], 8, 8, 2, 128, 16
    C = len(lens)
    cache = U.make_cache([n + K for n in lens], Hkv, D, page, 4)
    for x in ("k", "v"):  # empty pages
        cache[x + "_codes"][:], cache[x + "_scales"][:] = U.NAN_CODE, float("nan")
    prompt_cu, draft_cu = offsets(lens), offsets([K] * C)
    pk, pv = randn((sum(lens), Hkv, D), 1, torch.bfloat16), randn((sum(lens), Hkv, D), 2, torch.bfloat16)
    q = randn((C, K, Hq, D), 3, torch.bfloat16)
    kb, vb = randn((C, K, Hkv, D), 5, torch.bfloat16), randn((C, K, Hkv, D), 6, torch.bfloat16)
    w1 = U.write(cache, pk, pv, prompt_cu, [0] * C)
    ref1 = U.attention(q, w1, lens, kb, vb, True)
    w2 = U.write(w1, kb.flatten(0, 1), vb.flatten(0, 1), draft_cu, lens)
    after = [n + K for n in lens]
    ref2 = U.attention(q, w2, after, None, None, True)

    c = cfg(H, Hq, Hkv, D, page, causal=True)
    dev = U.to_device(cache, cuda)
    kv = H.kv8_view(dev)
    ws = H.alloc_workspace(H.hspec_attn_kv8_workspace_size(c, C, K, kv.max_pages))
    t = {n: x.to(cuda) for n, x in dict(pk=pk, pv=pv, q=q, kb=kb, vb=vb).items()}
    zero, l0, l1 = i32([0] * C, cuda), i32(lens, cuda), i32(after, cuda)
    pcu, dcu = i32(prompt_cu, cuda), i32(draft_cu, cuda)
    o1, o2 = torch.empty_like(t["q"]), torch.empty_like(t["q"])
    kf, vf = t["kb"].flatten(0, 1), t["vb"].flatten(0, 1)

    def step():
        H.hspec_kv8_write(c, t["pk"], t["pv"], pcu, zero, kv)
        H.hspec_attn_paged_block_kv8(c, t["q"], kv, l0, t["kb"], t["vb"], o1, ws)
        H.hspec_kv8_write(c, kf, vf, dcu, l0, kv)
        H.hspec_attn_paged_block_kv8(c, t["q"], kv, l1, None, None, o2, ws)

    step()
    assert H.hspec_sync_status() == 0
    assert_same_cache(dev, w2)
    for o, (ref, A, S) in ((o1, ref1), (o2, ref2)):
        assert bool(((o.cpu().double() - ref).abs() <= U.attention_bound(ref, A, S, torch.bfloat16, 300, D)).all())
    e1, e2 = o1.clone(), o2.clone()
    for x in ("k", "v"):
        dev[x + "_codes"].fill_(U.NAN_CODE)
        dev[x + "_scales"].fill_(float("nan"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(2):
        o1.zero_(), o2.zero_()
        graph.replay()
        assert H.hspec_sync_status() == 0
        assert torch.equal(o1, e1) and torch.equal(o2, e2)
        assert_same_cache(dev, w2)


# ------------------------------------------------------------------- the calls' manners

def test_outputs_stay_inside(H, cuda):
    # a read's rows and an attention's output between guards; every byte of a pool that the
    # write has no business with keeps its value
    Hkv, D, page, lens = 2, 128, 16, [37, 5, 90]
    cache = U.make_cache(lens, Hkv, D, page, 7)
    dev, c = U.to_device(cache, cuda), cfg(H, 8, Hkv, D, page)
    for what, shape in (("read", (sum(lens), Hkv, D)), ("attn", (3, 5, 8, D))):
        n, g = int(torch.tensor(shape).prod()), 4096
        bufs = [torch.full((n + 2 * g,), -7.0, dtype=torch.bfloat16, device=cuda) for _ in range(2)]
        outs = [b[g:g + n].view(shape) for b in bufs]
        if what == "read":
            H.hspec_kv8_read(c, H.kv8_view(dev), i32(offsets(lens), cuda), None, *outs)
        else:
            size = H.hspec_attn_kv8_workspace_size(c, 3, 5, dev["page_table"].shape[1])
            wbuf = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device=cuda)
            H.hspec_attn_paged_block_kv8(c, randn(shape, 1, torch.bfloat16).to(cuda), H.kv8_view(dev), i32(lens, cuda),
                                         None, None, outs[0], wbuf[256:256 + size])
            outs[1].zero_()
            assert bool((wbuf[:256] == 0xA5).all()) and bool((wbuf[256 + size:] == 0xA5).all())
        assert H.hspec_sync_status() == 0
        for b, o in zip(bufs, outs):
            assert bool((b[:g] == -7.0).all()) and bool((b[-g:] == -7.0).all()) and not bool((o == -7.0).any())


def test_another_stream_and_two_workspaces(H, cuda):
    # two calls in flight on two streams, each with its own workspace, and two captured graphs
    # replayed in turn, give what each gives alone
    Hq, Hkv, D, page = 8, 2, 128, 16
    jobs = []
    for i, lens in enumerate(([3000, 700], [40, 2500])):
        dev = U.to_device(U.make_cache(lens, Hkv, D, page, i), cuda)
        q = randn((2, 4, Hq, D), 10 + i, torch.bfloat16).to(cuda)
        c = cfg(H, Hq, Hkv, D, page)
        ws = H.alloc_workspace(H.hspec_attn_kv8_workspace_size(c, 2, 4, dev["page_table"].shape[1]))
        jobs.append((c, q, H.kv8_view(dev), i32(lens, cuda), torch.empty_like(q), ws, dev))

    def call(j, stream=None):
        H.hspec_attn_paged_block_kv8(j[0], j[1], j[2], j[3], None, None, j[4], j[5], stream=stream)

    want = []
    for j in jobs:
        call(j)
        assert H.hspec_sync_status() == 0
        want.append(j[4].clone())
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        for j, s in zip(jobs, streams):
            call(j, s)
    torch.cuda.synchronize()
    for j, x in zip(jobs, want):
        assert torch.equal(j[4], x)
    graphs = []
    for j, s in zip(jobs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(j)
        graphs.append(g)
    for _ in range(3):
        for g, j in zip(graphs, jobs):
            j[4].zero_()
            g.replay()
    assert H.hspec_sync_status() == 0
    for j, x in zip(jobs, want):
        assert torch.equal(j[4], x)


def test_attention_wait_runs_out(H, cuda):
    # a 1 ns limit, which no wait for a copy from HBM meets: the call reports the timeout, the
    # context stays usable and the next call gives the same output as before
    lens, Hq, Hkv, D, page = [700, 4096, 1, 3000, 0, 2500], 8, 2, 128, 16
    dev = U.to_device(U.make_cache(lens, Hkv, D, page, 4), cuda)
    for K in (4, 20):
        q = randn((len(lens), K, Hq, D), 1, torch.bfloat16).to(cuda)
        want = attend(H, cfg(H, Hq, Hkv, D, page), q, dev, lens, None, None)
        assert H.hspec_sync_status() == 0
        attend(H, cfg(H, Hq, Hkv, D, page, wait_limit_ns=1), q, dev, lens, None, None)
        assert H.hspec_sync_status() == H.HSPEC_ERR_DEVICE_CHECK
        assert int(H.hspec_last_error().split("bits 0x")[1].split()[0], 16) & 8
        assert H.hspec_sync_status() == 0
        got = attend(H, cfg(H, Hq, Hkv, D, page), q, dev, lens, None, None)
        assert H.hspec_sync_status() == 0 and torch.equal(got, want)


def test_attention_of_many_short_and_few_long(H, cuda):
    # 300 requests of 0 .. 40 tokens; two of 30000 and 17000 over many chunks
    g = torch.Generator().manual_seed(5)
    short = torch.randint(0, 41, (300,), generator=g).tolist()
    check_attention(H, cuda, short, 2, 4, 1, 128, 16, torch.bfloat16, True, True, seed=3)
    check_attention(H, cuda, [30000, 17001], 1, 2, 1, 128, 64, torch.bfloat16, False, False, seed=4)


def test_empty_write_and_read(H, cuda):
    c = cfg(H, 2, 2, 64, 16)
    dev = U.to_device(U.make_cache([20], 2, 64, 16, 1), cuda)
    before = {n: t.clone() for n, t in dev.items()}
    k = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=cuda)
    H.hspec_kv8_write(c, k, k, i32([0, 0], cuda), i32([20], cuda), H.kv8_view(dev))
    H.hspec_kv8_read(c, H.kv8_view(dev), i32([0, 0], cuda), None, k, k)
    assert H.hspec_sync_status() == 0
    for x in ("k_codes", "v_codes", "page_table"):
        assert torch.equal(dev[x], before[x])
