"""The 8-bit paged cache in plain double arithmetic: its format, random caches, and the
three operators (write, read, attention) from their definitions.

A cache is a dict of CPU tensors: k_codes, v_codes uint8 [pages, Hkv, page, D], k_scales,
v_scales fp32 [pages, Hkv], page_table int32 [C, width] (unused entries -1).
"""
import math

import torch

E4M3 = torch.float8_e4m3fn
NAN_CODE = 0x7F


def value_table():
    """The 256 e4m3 values from the format: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    out = []
    for c in range(256):
        s, e, m = -1.0 if c & 128 else 1.0, (c >> 3) & 15, c & 7
        v = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        out.append(float("nan") if (c & 127) == 127 else s * v)
    return torch.tensor(out, dtype=torch.float64)


VALUES = value_table()


def encode(x):
    """Codes (uint8) of the double tensor x rounded to nearest, ties to even; NaN stays NaN."""
    grid = VALUES[:127]  # increasing magnitudes
    a = x.abs().clamp_max(448.0)
    hi = torch.searchsorted(grid, torch.nan_to_num(a).contiguous()).clamp(max=126)
    lo = (hi - 1).clamp_min(0)
    dl, dh = a - grid[lo], grid[hi] - a
    pick = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    code = pick + torch.where(torch.signbit(x), 128, 0)
    return torch.where(torch.isnan(x), torch.full_like(code, NAN_CODE), code).to(torch.uint8)


def scale_of(top: float) -> float:
    if top == 0.0:
        return 0.0
    k = -126
    while 448.0 * 2.0 ** k < top:
        k += 1
    return 2.0 ** k


def values(codes, scales):
    """[pages, Hkv, page, D] doubles."""
    return VALUES[codes.long()] * scales.double()[:, :, None, None]


def make_cache(lens, Hkv, D, page, seed, pow2=True, stale_nan=True, width=None, slack=2):
    """A cache holding `lens` random tokens per request in shuffled pages.  Slots past a
    request's end and the slack pages hold NaN codes (and NaN scales for slack pages)."""
    g = torch.Generator().manual_seed(seed)
    need = [(n + page - 1) // page for n in lens]
    total = max(sum(need) + slack, 1)
    width = width or max(max(need), 1)
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    out, at, owned = {}, 0, []
    for c, n in enumerate(need):
        table[c, :n] = order[at:at + n]
        owned += order[at:at + n].tolist()
        at += n
    for x in ("k", "v"):
        codes = encode((torch.randn(total, Hkv, page, D, generator=g) * 96.0).double())
        e = torch.randint(-9, -6, (total, Hkv), generator=g)
        scales = torch.ldexp(torch.ones(total, Hkv), e)
        if not pow2:
            scales = scales * (1.0 + torch.rand(total, Hkv, generator=g))
        free = torch.ones(total, dtype=torch.bool)
        free[torch.tensor(owned, dtype=torch.long)] = False
        codes[free] = NAN_CODE
        scales[free] = float("nan")
        if stale_nan:
            for c, n in enumerate(lens):
                if n % page:
                    codes[table[c, n // page].long(), :, n % page:] = NAN_CODE
        out[x + "_codes"], out[x + "_scales"] = codes, scales
    out["page_table"] = table
    return out


def to_device(cache, dev):
    return {k: v.to(dev) for k, v in cache.items()}


def gather(cache, x, c, t0, t1):
    """Tokens [t0, t1) of request c: [t1 - t0, Hkv, D] doubles."""
    page = cache[x + "_codes"].shape[2]
    if t1 <= t0:
        return torch.zeros(0, cache[x + "_codes"].shape[1], cache[x + "_codes"].shape[3], dtype=torch.float64)
    p = cache["page_table"][c, t0 // page:(t1 + page - 1) // page].long()
    v = values(cache[x + "_codes"][p], cache[x + "_scales"][p]).transpose(1, 2)
    return v.reshape(-1, v.shape[2], v.shape[3])[t0 % page:t0 % page + t1 - t0]


def write(cache, k_new, v_new, cu, first):
    """The write's definition; returns a new cache dict (CPU)."""
    out = {k: v.clone() for k, v in cache.items()}
    page = cache["k_codes"].shape[2]
    for x, new in (("k", k_new), ("v", v_new)):
        codes, scales = out[x + "_codes"], out[x + "_scales"]
        for c in range(len(first)):
            pos, end = first[c], first[c] + cu[c + 1] - cu[c]
            while pos < end:
                p, slot = int(cache["page_table"][c, pos // page]), pos % page
                n = min(page - slot, end - pos)
                rows = new[cu[c] + pos - first[c]:][:n].double().transpose(0, 1)  # [Hkv, n, D]
                for h in range(rows.shape[0]):
                    fine = rows[h][torch.isfinite(rows[h])].abs()
                    s = scale_of(float(fine.max()) if fine.numel() else 0.0)
                    old = float(scales[p, h])
                    if slot > 0:
                        if old > s:
                            s = old
                        elif s != old:
                            ratio = (scales[p, h] / torch.tensor(s)).double() if s > 0 else 0.0
                            codes[p, h, :slot] = encode((VALUES[codes[p, h, :slot].long()] * ratio).float().double())
                    r = rows[h] / s if s > 0 else torch.where(torch.isnan(rows[h]), rows[h], rows[h] * 0.0)
                    codes[p, h, slot:slot + n] = encode(r)
                    scales[p, h] = s
                pos += n
    return out


def attention(q, cache, lens, k_blk, v_blk, causal):
    """(out, A, S): the attention in double, [C, K, Hq, D]; A = sum_t p_t |v_t|, the scale of
    an error in the weights; S [C, K, Hq] = the largest sum_d |q_d k_d| / sqrt(D) of a seen key.

    For bf16, A holds 2^-9 max_d |v_td| more for each block key.  The tensor-core path takes
    block values as two e4m3 parts of a row scaled so that its largest element lies in
    [128, 256): hi, then the rest, whose rounding is 2^-4 of it (2^-8 of the element) or half of
    e4m3's smallest step, 2^-10, which is 2^-17 of a largest element of 128 or more.  The
    bound takes 2^-8 of A, so 2^-9 of that element makes up for it."""
    C, K, Hq, D = q.shape
    Hkv = cache["k_codes"].shape[1]
    out, A = torch.zeros(C, K, Hq, D, dtype=torch.float64), torch.zeros(C, K, Hq, D, dtype=torch.float64)
    S = torch.zeros(C, K, Hq, dtype=torch.float64)
    for c, n in enumerate(lens):
        k, v = gather(cache, "k", c, 0, n), gather(cache, "v", c, 0, n)
        if k_blk is not None:
            k, v = torch.cat([k, k_blk[c].double()]), torch.cat([v, v_blk[c].double()])
        for j in range(K):
            if k_blk is not None:
                seen = n + j + 1 if causal else n + K
            else:
                seen = n - (K - 1) + j if causal else n
            if seen <= 0:
                continue
            for h in range(Hq):
                kk, vv = k[:seen, h // (Hq // Hkv)], v[:seen, h // (Hq // Hkv)]
                qk = kk * q[c, j, h].double()
                p = torch.softmax(qk.sum(1) / math.sqrt(D), 0)
                out[c, j, h] = p @ vv
                A[c, j, h] = p @ vv.abs()
                if k_blk is not None and q.dtype == torch.bfloat16 and seen > n:
                    A[c, j, h] += p[n:] @ (vv[n:].abs().amax(1, keepdim=True) * 2.0 ** -9)
                S[c, j, h] = qk.abs().sum(1).max() / math.sqrt(D)
    return out, A, S


def attention_bound(ref, A, S, dtype, keys: int, D: int):
    """How far an output element may be from `ref`.

    Scores: the dot product of D terms and the scaling, each a rounding of 2^-24 relative to
    S; a weight's relative error is ln-linear in its score's, and the sums over `keys` keys
    add 2^-24 a term (the partial merges and exp a few more).  bf16: the query enters as two
    e4m3 parts that hold its 8 bits down to 2^-17.8 of the row's largest element (D of them
    in a score: below 2^-12 of S plus 2^-12 for the inputs used here), the weights as two
    parts, each rounding 2^-4 relative: 2^-8; then the store's half step, 2^-8 |ref|."""
    eps = 2.0 ** -24
    w = eps * ((D + 8) * S[..., None] * 2.0 + keys + 64)
    if dtype == torch.bfloat16:
        return 2.0 ** -8 * ref.abs() + (w + 2.0 ** -8 + 2.0 ** -12 * (1 + S[..., None])) * A + 1e-30
    return eps * ref.abs() + w * A + 1e-30
