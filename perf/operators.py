"""The operators of an 8-bit paged KV cache: cases to measure them on, and their plain forms.

Three operators share one cache (a target model's keys and values held as e4m3 codes with a
power-of-two scale for each page and kv head):

  write  quantises new tokens' keys and values into the pages as they are written (hspec_kv8_write)
  read   gathers tokens back out of the pages as ordinary values               (hspec_kv8_read)
  attn   paged block attention over the cache in place                         (hspec_attn_paged_block_kv8)

`own` False: elementary torch operations in 32 bits.  `own` True: the library's calls.

Cache layout: codes [num_pages, Hkv, page, D] (torch.float8_e4m3fn), scales [num_pages, Hkv] fp32,
value = code * scale; token t of request c lies in page table[c, t // page], slot t % page.
Scale of a page and head: 0 if all its values are zero, else 2^k with the least k >= -126 for which
every magnitude is at most 448 * 2^k.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------- cases

def _attn(name, C, K, lo, hi, Hq=32, Hkv=8, D=128, page=16, dtype="bf16", block=True, causal=False):
    return {"name": name, "op": "attn", "C": C, "K": K, "lo": lo, "hi": hi, "Hq": Hq, "Hkv": Hkv, "D": D,
            "page": page, "dtype": dtype, "block": block, "causal": causal}


def _move(name, op, C, lo, hi, old_lo, old_hi, Hkv=8, D=128, page=16, dtype="bf16"):
    return {"name": name, "op": op, "C": C, "lo": lo, "hi": hi, "old_lo": old_lo, "old_hi": old_hi, "Hkv": Hkv,
            "D": D, "page": page, "dtype": dtype}


def listed():
    return [
        # one request decoding one token after a short prompt: latency
        _attn("attn_decode_c1", 1, 1, 512, 512, block=False),
        # the small fp32 drafter shapes, two requests
        _attn("attn_draft_tiny_f32", 2, 8, 64, 77, Hq=4, Hkv=2, D=64, dtype="f32"),
        # one request drafting a block of 16 after 2048 tokens
        _attn("attn_draft_c1", 1, 16, 2048, 2048),
        # a target verifying 16 drafts (17 positions, causal) for 32 requests, tokens already in the cache
        _attn("attn_verify_c32", 32, 17, 512, 8192, block=False, causal=True),
        # 64 query heads, long contexts, one decoded token each: bandwidth
        _attn("attn_decode_c64_g8", 64, 1, 1024, 32768, Hq=64, block=False),
        # 128 requests drafting blocks of 16 over mixed contexts: the largest
        _attn("attn_draft_c128", 128, 16, 512, 16384),
        # one new token for each of 128 requests, appended inside partly filled pages
        _move("write_decode_c128", "write", 128, 1, 1, 512, 16384),
        # accepted drafts: 1..17 tokens for each of 32 requests
        _move("write_accept_c32", "write", 32, 1, 17, 512, 8192),
        # prompts of 8 new requests written whole
        _move("write_prompt_c8", "write", 8, 512, 16384, 0, 0),
        # one prefix of 2048 tokens read back
        _move("read_c1", "read", 1, 2048, 2048, 0, 0),
        # ragged prefixes of 16 requests, starting in the middle of pages
        _move("read_c16", "read", 16, 512, 8192, 0, 100),
    ]


def draw(rng):
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    op = rng.choice(["attn", "attn", "attn", "write", "read"])
    Hq, Hkv = rng.choice([(32, 8), (64, 8), (32, 32), (28, 4), (8, 1), (4, 2)])
    D, page = rng.choice([128, 128, 64]), rng.choice([16, 16, 32, 64])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "attn":
        K = log(1, 48)
        # at most the largest listed case's key bytes, and its products
        most = min(10_000_000 * 128 // (Hkv * D), 330_000_000 * 128 // (Hq * K * D))
        if dtype == "f32":
            K, most = min(K, 256 * Hkv // Hq, 32), most // 64
        hi = max(K, log(33, max(64, min(20000, most))))
        lo = max(K, rng.randint(1, hi))
        C = max(1, min(128, most // hi, log(1, 128)))
        block = rng.random() < 0.6
        return _attn("", C, K, lo, hi, Hq, Hkv, D, page, dtype, block, rng.random() < 0.5)
    hi = log(1, 16000)
    lo = rng.randint(1, hi)
    C = max(1, min(128, 65536 // hi, log(1, 128)))
    old = rng.choice([0, 100, 2000])
    return _move("", op, C, lo, hi, 0, old, Hkv, D, page, dtype)


# --------------------------------------------------------------------------- inputs

def _spread(C, lo, hi):
    """C lengths spread evenly over [lo, hi] (the same multiset for every seed)."""
    return [lo + (hi - lo) * (2 * i + 1) // (2 * C) for i in range(C)] if C > 1 else [(lo + hi) // 2]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _cache(case, g, tokens, dev):
    """Pools whose pages 0.. hold earlier tokens, and a shuffled page table for `tokens` per request."""
    page, Hkv, D = case["page"], case["Hkv"], case["D"]
    need = [(t + page - 1) // page for t in tokens]
    total, width = sum(need) + max(1, sum(need) // 16), max(1, max(need))
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(tokens), width), -1, dtype=torch.int32)
    at = 0
    order = order.cpu()
    for c, n in enumerate(need):
        table[c, :n] = order[at:at + n]
        at += n
    out = {"page_table": table.to(dev)}
    for x in ("k", "v"):
        codes = torch.empty((total, Hkv, page, D), dtype=E4M3, device=dev)
        for a in range(0, total, 1 << 13):
            b = min(total, a + (1 << 13))
            r = torch.randn((b - a, Hkv, page, D), generator=g, device=dev)
            codes[a:b].copy_(r.mul_(96.0).clamp_(-448.0, 448.0))
        # values of the order of one: magnitudes differ by up to 4 from page to page
        e = torch.randint(-8, -5, (total, Hkv), generator=g, device=dev)
        out[x + "_codes"], out[x + "_scales"] = codes, torch.ldexp(torch.ones((), device=dev), e)
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 17)
    dt, C, Hkv, D = _dtype(case), case["C"], case["Hkv"], case["D"]
    mix = torch.randperm(C, generator=g, device=dev).tolist()
    lens = [_spread(C, case["lo"], case["hi"])[i] for i in mix]
    rand = lambda *s: torch.randn(s, generator=g, device=dev).to(dt)  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    s = {"case": dict(case)}
    if case["op"] == "attn":
        K, Hq = case["K"], case["Hq"]
        s.update(_cache(case, g, lens, dev))
        s["ctx_lens"] = i32(lens)
        s["q"] = rand(C, K, Hq, D)
        s["k_blk"] = rand(C, K, Hkv, D) if case["block"] else None
        s["v_blk"] = rand(C, K, Hkv, D) if case["block"] else None
        s["out"] = torch.empty_like(s["q"])
    else:
        old = [_spread(C, case["old_lo"], case["old_hi"])[i] for i in mix]
        s.update(_cache(case, g, [a + b for a, b in zip(old, lens)], dev))
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["first"], s["cu"], s["T"] = i32(old), i32(cu), cu[-1]
        if case["op"] == "write":
            # new tokens of other magnitudes than the old ones, so that scales grow in some pages
            s["k_new"] = rand(s["T"], Hkv, D) * 2
            s["v_new"] = rand(s["T"], Hkv, D)
        else:
            s["k_out"] = torch.empty((s["T"], Hkv, D), dtype=dt, device=dev)
            s["v_out"] = torch.empty_like(s["k_out"])
    return s


# ---------------------------------------------------------------------- plain forms

def _tokens(s):
    """(physical page, slot) of each of the T ragged tokens."""
    T, page = s["T"], s["case"]["page"]
    row = torch.arange(T, device=s["cu"].device)
    c = torch.searchsorted(s["cu"].long(), row, right=True) - 1
    pos = s["first"].long()[c] + row - s["cu"].long()[c]
    return s["page_table"].long()[c, pos // page], pos % page


def _bytes(x):
    return x.view(torch.uint8)


def _write_plain(s, x):
    codes, scales, new = s[x + "_codes"], s[x + "_scales"], s[x + "_new"].float()
    P, Hkv, page, D = codes.shape
    pg, slot = _tokens(s)
    amax = torch.zeros((P, Hkv), device=new.device).index_reduce_(0, pg, new.abs().amax(-1), "amax")
    first = torch.full((P,), page, device=new.device).index_reduce_(0, pg, slot, "amin")  # page: nothing written
    f, e = torch.frexp(amax)
    e = torch.where(f <= 0.875, e - 9, e - 8).clamp_min(-126)
    grown = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax))
    grown = torch.where((first > 0)[:, None], torch.maximum(grown, scales), grown)
    now = torch.where((first < page)[:, None], grown, scales)
    ratio = torch.where(now > 0, scales / now, torch.zeros_like(now))
    kept = torch.arange(page, device=new.device)[None, :] < first[:, None]
    kept = kept & (first < page)[:, None]
    again = (codes.float() * ratio[:, :, None, None]).to(E4M3)
    _bytes(codes).copy_(torch.where(kept[:, None, :, None], _bytes(again), _bytes(codes)))
    sc = now[pg]
    inv = torch.where(sc > 0, 1.0 / sc, torch.zeros_like(sc))
    _bytes(codes)[pg, :, slot] = _bytes((new * inv[:, :, None]).to(E4M3))
    scales.copy_(now)
    return codes, scales


def _read_plain(s, x):
    pg, slot = _tokens(s)
    v = _bytes(s[x + "_codes"])[pg, :, slot].view(E4M3).float()
    return (v * s[x + "_scales"][pg][:, :, None]).to(s[x + "_out"].dtype)


def _attn_plain(s):
    c = s["case"]
    C, K, Hq, Hkv, D, page = c["C"], c["K"], c["Hq"], c["Hkv"], c["D"], c["page"]
    table = s["page_table"].long().clamp_min(0)

    def gathered(x):
        v = _bytes(s[x + "_codes"])[table].view(E4M3).float()
        v = v * s[x + "_scales"][table][..., None, None]  # [C, pages, Hkv, page, D]
        v = v.transpose(1, 2).reshape(C, Hkv, -1, D)
        return torch.cat([v, s[x + "_blk"].float().transpose(1, 2)], 2) if c["block"] else v

    q = s["q"].float().reshape(C, K, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(C, Hkv, -1, D)
    score = (q @ gathered("k").transpose(2, 3)) * (1.0 / math.sqrt(D))
    N = table.shape[1] * page
    j = torch.arange(K, device=q.device).repeat_interleave(Hq // Hkv)
    t = torch.arange(score.shape[-1], device=q.device)
    ctx = s["ctx_lens"].long()[:, None, None]
    if c["block"]:
        seen = t[None, None, :] < ctx
        blk = (t[None, :] >= N) & ((t[None, :] - N <= j[:, None]) if c["causal"] else (t[None, :] >= N))
        seen = seen & (t < N) | blk[None]
    elif c["causal"]:
        seen = t[None, None, :] < ctx - (K - 1) + j[None, :, None]
    else:
        seen = t[None, None, :] < ctx
    score = score.masked_fill_(~seen[:, None], float("-inf"))
    p = torch.exp(score - score.amax(-1, keepdim=True))
    out = (p @ gathered("v")) / p.sum(-1, keepdim=True)
    return out.reshape(C, Hkv, K, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(C, K, Hq, D).to(s["q"].dtype)


# ------------------------------------------------------------------ the library's calls

def _handles(s):
    """What a program keeps: the configuration, the view of the cache and the workspace."""
    if "cfg" not in s:
        from hybrid_mamba_attention_b200 import hspec as H
        c = s["case"]
        s["H"] = H
        s["cfg"] = H.hspec_cfg(
            d_model=c.get("Hq", c["Hkv"]) * c["D"], n_q_heads=c.get("Hq", c["Hkv"]), n_kv_heads=c["Hkv"],
            head_dim=c["D"], page_size=c["page"], n_layers=1, layer_kinds=b"A",
            dtype=H.HSPEC_DTYPE_BF16 if c["dtype"] == "bf16" else H.HSPEC_DTYPE_F32,
            flags=H.HSPEC_FLAG_CAUSAL_BLOCK if c.get("causal") else 0)
        s["kv8"] = H.kv8_view(s)
        if c["op"] == "attn":
            n = H.hspec_attn_kv8_workspace_size(s["cfg"], c["C"], c["K"], s["page_table"].shape[1])
            s["ws"] = H.alloc_workspace(n)
    return s["H"]


def run(s):
    op = s["case"]["op"]
    if own:
        H = _handles(s)
        if op == "attn":
            H.hspec_attn_paged_block_kv8(s["cfg"], s["q"], s["kv8"], s["ctx_lens"], s["k_blk"], s["v_blk"], s["out"],
                                         s["ws"])
            return s["out"]
        if op == "write":
            H.hspec_kv8_write(s["cfg"], s["k_new"], s["v_new"], s["cu"], s["first"], s["kv8"])
        else:
            H.hspec_kv8_read(s["cfg"], s["kv8"], s["cu"], s["first"], s["k_out"], s["v_out"])
            return {"k": s["k_out"], "v": s["v_out"]}
    elif op == "attn":
        return _attn_plain(s)
    elif op == "read":
        return {"k": _read_plain(s, "k"), "v": _read_plain(s, "v")}
    else:
        _write_plain(s, "k")
        _write_plain(s, "v")
    return {k: s[k] for k in ("k_codes", "k_scales", "v_codes", "v_scales")}


# ------------------------------------------------------------------------------ work

def work(case):
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    E = 2 if case["dtype"] == "bf16" else 4
    lens = _spread(case["C"], case["lo"], case["hi"])
    if case["op"] == "attn":
        C, K, Hq = case["C"], case["K"], case["Hq"]
        pages = sum((n + page - 1) // page for n in lens)
        cache = 2 * sum(lens) * Hkv * D + pages * (2 * Hkv * 4 + 4)
        rows = 2 * C * K * Hq * D * E + (2 * C * K * Hkv * D * E if case["block"] else 0)
        keys = sum(lens) + (C * K if case["block"] else 0)
        return {"bytes": cache + rows, "flops": 4 * K * Hq * D * keys}
    old = _spread(case["C"], case["old_lo"], case["old_hi"])
    pages = sum((o + n + page - 1) // page - o // page for o, n in zip(old, lens))
    moved = 2 * sum(lens) * Hkv * D * (E + 1) + pages * (2 * Hkv * 4 + 4)
    return {"bytes": moved, "flops": 4 * sum(lens) * Hkv * D}


# ------------------------------------------------------------------------- 64 bits

def _e4m3_value(x):
    """x (double) rounded to the nearest e4m3 value, ties to even."""
    mag = x.abs()
    e = torch.floor(torch.log2(mag.clamp_min(2.0 ** -40))).clamp_min(-6.0)
    step = torch.exp2(e - 3.0)
    return torch.sign(x) * (torch.round(mag / step) * step).clamp_max(448.0)


def _exact_write(s, x):
    codes, scales, new = s[x + "_codes"].double(), s[x + "_scales"].double(), s[x + "_new"].double()
    page = codes.shape[2]
    cu, first, table = s["cu"].tolist(), s["first"].tolist(), s["page_table"].tolist()
    for c in range(len(first)):
        pos, end = first[c], first[c] + cu[c + 1] - cu[c]
        while pos < end:
            p, slot = table[c][pos // page], pos % page
            n = min(page - slot, end - pos)
            at = cu[c] + pos - first[c]
            rows = new[at:at + n].transpose(0, 1)  # [Hkv, n, D]
            top = rows.abs().amax((1, 2))
            k = torch.ceil(torch.log2(top.clamp_min(2.0 ** -149) / 448.0)).clamp_min(-126.0)
            k = torch.where((torch.exp2(k - 1) * 448.0 >= top) & (k > -126), k - 1, k)
            k = torch.where(torch.exp2(k) * 448.0 < top, k + 1, k)
            sc = torch.where(top > 0, torch.exp2(k), torch.zeros_like(k))
            if slot > 0:
                sc = torch.maximum(sc, scales[p])
                old = codes[p, :, :slot] * scales[p][:, None, None]
                codes[p, :, :slot] = _e4m3_value(old / sc.clamp_min(2.0 ** -1000)[:, None, None])
            codes[p, :, slot:slot + n] = _e4m3_value(rows / sc.clamp_min(2.0 ** -1000)[:, None, None])
            scales[p] = sc
            pos += n
    return codes, scales


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        out = {}
        for x in ("k", "v"):
            out[x + "_codes"], out[x + "_scales"] = _exact_write(s, x)
        return out
    page, D = case["page"], case["D"]
    table = s["page_table"].long()

    def tokens(x, c, t0, t1):
        """[t1 - t0, Hkv, D] of request c's cache, in double."""
        p0 = t0 // page
        p = table[c, p0:(t1 + page - 1) // page]
        v = s[x + "_codes"].view(torch.uint8)[p].view(E4M3).double() * s[x + "_scales"][p].double()[:, :, None, None]
        return v.transpose(1, 2).reshape(-1, v.shape[1], D)[t0 - p0 * page:t1 - p0 * page]

    if case["op"] == "read":
        cu, first = s["cu"].tolist(), s["first"].tolist()
        return {x: torch.cat([tokens(x, c, first[c], first[c] + cu[c + 1] - cu[c]) for c in range(case["C"])])
                for x in ("k", "v")}
    K, G = case["K"], case["Hq"] // case["Hkv"]
    outs = []
    for c, n in enumerate(s["ctx_lens"].tolist()):
        k, v = tokens("k", c, 0, n), tokens("v", c, 0, n)
        last = torch.arange(K, device=k.device)  # the last key that query j sees
        if case["block"]:
            k, v = torch.cat([k, s["k_blk"][c].double()]), torch.cat([v, s["v_blk"][c].double()])
            last = last + n if case["causal"] else torch.full_like(last, n + K - 1)
        else:
            last = last + n - K if case["causal"] else torch.full_like(last, n - 1)
        kk, vv = k.repeat_interleave(G, 1).transpose(0, 1), v.repeat_interleave(G, 1).transpose(0, 1)  # [Hq, t, D]
        score = s["q"][c].double().transpose(0, 1) @ kk.transpose(1, 2) / math.sqrt(D)  # [Hq, K, t]
        hide = torch.arange(kk.shape[1], device=k.device)[None, :] > last[:, None]
        score = score.masked_fill(hide[None], float("-inf"))
        outs.append((torch.softmax(score, -1) @ vv).transpose(0, 1))
    return torch.stack(outs)
