"""The draft step over 8-bit target caches (GPU): against the oracle on caches of the same
values, captured and replayed, and in a decoding target's round."""
from dataclasses import replace

import numpy as np
import pytest
import torch

import oracle
from hybrid_mamba_attention_b200 import inputs as I
from tests import kv8_util as U
from tests.parity_util import host, host_weights, rel_max, rel_rms, F32_TOL

pytestmark = pytest.mark.gpu

SMALL = I.Shapes("small", d=256, Hq=4, Hkv=2, D=64, H=4, P=64, N=32, dtype="bf16", rope_theta=1e4, layers="MAMA",
                 d_ff=512, vocab=1000)


@pytest.fixture(scope="module")
def H(cuda):
    from hybrid_mamba_attention_b200 import hspec
    return hspec


def setup(H, cuda, sh, lens, K, seed=0, width=None):
    """Weights, step inputs and per attention layer an 8-bit cache and one of the same values."""
    wl = I.Workload("kv8", sh, C=len(lens), K=K, ctx_lo=min(lens), ctx_hi=max(lens), seed=seed)
    st = I.make_step_inputs(wl, cuda)
    st["ctx_lens"] = torch.tensor(lens, dtype=torch.int32, device=cuda)
    kv8, plain = [], []
    for i in range(sh.layers.count("A")):
        c = U.make_cache(lens, sh.Hkv, sh.D, sh.page, seed + 50 + i, width=width)
        # code * 2^k has four bits: the values are exact in bf16
        pools = {x: U.values(c[x + "_codes"], c[x + "_scales"]).transpose(1, 2).to(sh.torch_dtype).contiguous()
                 for x in ("k", "v")}
        kv8.append(U.to_device(c, cuda))
        plain.append({"k_pool": pools["k"], "v_pool": pools["v"], "page_table": c["page_table"]})
    return st, kv8, plain


def outputs(H, cuda, sh, C, K):
    t = {"hidden": torch.full((C, K, sh.d), float("nan"), device=cuda),
         "layer_hidden": torch.full((len(sh.layers), C, K, sh.d), float("nan"), device=cuda)}
    if sh.vocab:
        t["draft_tokens"] = torch.full((C, K), -7, dtype=torch.int32, device=cuda)
    return t, H.hspec_step_out(**{n: x.data_ptr() for n, x in t.items()})


@pytest.mark.parametrize("sh,lens,K", [
    (replace(I.TINY, layers="MA"), [64, 0, 17], 8),
    (replace(I.TINY, layers="AMA", page=5, causal_block=True), [33, 70], 3),
    (SMALL, [40, 100, 0], 8),
    (replace(SMALL, D=128, page=32, causal_block=True), [300, 1], 17),
])
def test_step_matches_the_oracle(H, cuda, sh, lens, K):
    st, kv8, plain = setup(H, cuda, sh, lens, K)
    dr = H.Drafter(sh, st["weights"])
    width = max(c["page_table"].shape[1] for c in kv8)
    ws = H.alloc_workspace(dr.workspace_size_kv8(len(lens), K, width), cuda)
    ws.fill_(0xFF)
    t, so = outputs(H, cuda, sh, len(lens), K)
    si = dr.step_in(len(lens), K, st["h_last"], st["ctx_lens"], [], tokens=st["tokens"], x_in=st["x_in"])
    dr.step_kv8(si, kv8, so, ws)
    assert H.hspec_sync_status() == 0
    kv = [dict(c, num_pages=c["k_pool"].shape[0]) for c in plain]
    ref = oracle.draft_step(sh, host_weights(st["weights"]), kv, host(st["h_last"]), host(st["ctx_lens"]),
                            tokens=None if st["tokens"] is None else host(st["tokens"]),
                            x_in=None if st["x_in"] is None else host(st["x_in"]))
    got = t["hidden"].double().cpu().numpy()
    assert np.isfinite(got).all()
    if sh.dtype == "f32":
        assert rel_max(got, ref["hidden"]) <= F32_TOL
    else:
        # the bound of the step over a bf16 cache end to end (its roundings cascade through
        # the layers); the attention's weights add 2^-8 of each attention output to a store
        # that rounds by 2^-8 already
        assert rel_rms(got, ref["hidden"]) <= 3e-2
    dr.close()


def test_step_replayed_from_a_graph(H, cuda):
    sh, lens, K = SMALL, [150, 33, 90], 8
    st, kv8, _ = setup(H, cuda, sh, lens, K)
    dr = H.Drafter(sh, st["weights"])
    ws = H.alloc_workspace(dr.workspace_size_kv8(3, K, kv8[0]["page_table"].shape[1]), cuda)
    t, so = outputs(H, cuda, sh, 3, K)
    si = dr.step_in(3, K, st["h_last"], st["ctx_lens"], [], tokens=st["tokens"])
    dr.step_kv8(si, kv8, so, ws)
    assert H.hspec_sync_status() == 0
    want = {n: x.clone() for n, x in t.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dr.step_kv8(si, kv8, so, ws)
    for _ in range(2):
        for x in t.values():
            x.zero_()
        graph.replay()
        assert H.hspec_sync_status() == 0
        for n in t:
            assert torch.equal(t[n], want[n]), n
    dr.close()


def test_rounds_of_drafting_and_verifying(H, cuda):
    """Three rounds on one stream: the accepted tokens' keys and values go into every layer's
    8-bit cache, the drafter reads it in place, the target's logits decide what is accepted."""
    sh, K, C = SMALL, 8, 3
    lens = [30, 47, 5]
    st, kv8, _ = setup(H, cuda, sh, lens, K, width=16)
    for c in kv8:  # every request has the pages of its whole row
        c["page_table"] = torch.arange(C * 16, dtype=torch.int32, device=cuda).view(C, 16).flip(1).contiguous()
        for x in ("k", "v"):
            c[x + "_codes"] = torch.full((C * 16, sh.Hkv, sh.page, sh.D), U.NAN_CODE, dtype=torch.uint8, device=cuda)
            c[x + "_scales"] = torch.full((C * 16, sh.Hkv), float("nan"), device=cuda)
    dr = H.Drafter(sh, st["weights"])
    ws = H.alloc_workspace(dr.workspace_size_kv8(C, K, 16), cuda)
    vws = H.alloc_workspace(H.hspec_verify_workspace_size(dr.cfg, C, K))
    t, so = outputs(H, cuda, sh, C, K)
    si = dr.step_in(C, K, st["h_last"], st["ctx_lens"], [], tokens=st["tokens"])
    g = torch.Generator(device=cuda).manual_seed(1)
    accepted, nxt = torch.zeros(C, dtype=torch.int32, device=cuda), torch.zeros(C, dtype=torch.int32, device=cuda)
    first = torch.zeros(C, dtype=torch.int32, device=cuda)
    counts = list(lens)
    for _ in range(3):
        cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=cuda)
        rows = torch.randn(int(cu[-1]), 2 * len(kv8), sh.Hkv, sh.D, generator=g, device=cuda).to(torch.bfloat16)
        for i, c in enumerate(kv8):
            H.hspec_kv8_write(dr.cfg, rows[:, 2 * i], rows[:, 2 * i + 1], cu, first, H.kv8_view(c))
        dr.step_kv8(si, kv8, so, ws)
        assert H.hspec_sync_status() == 0
        assert torch.isfinite(t["hidden"]).all()
        logits = torch.randn(C, K + 1, sh.vocab, generator=g, device=cuda).to(torch.bfloat16)
        for r, n in enumerate((0, 3, K)):  # logits that agree with the first n drafts
            for j in range(n):
                logits[r, j, t["draft_tokens"][r, j]] = 100.0
        first.copy_(st["ctx_lens"])
        H.hspec_verify_greedy(dr.cfg, logits, t["draft_tokens"], accepted, nxt, vws, ctx_lens=st["ctx_lens"])
        assert H.hspec_sync_status() == 0
        assert accepted.tolist()[2] == K and accepted.tolist()[1] >= 3
        counts = [n + 1 for n in accepted.tolist()]
        assert torch.equal(st["ctx_lens"] - first, accepted + 1)
    dr.close()


def test_wrong_number_of_caches_is_refused(H, cuda):
    st, kv8, _ = setup(H, cuda, SMALL, [20], 4)
    dr = H.Drafter(SMALL, st["weights"])
    si = dr.step_in(1, 4, st["h_last"], st["ctx_lens"], [], tokens=st["tokens"])
    with pytest.raises(ValueError):
        dr.step_kv8(si, kv8[:1], H.hspec_step_out(), torch.empty(256, dtype=torch.uint8, device=cuda))
    with pytest.raises(H.HspecError):  # a workspace too small
        t, so = outputs(H, cuda, SMALL, 1, 4)
        dr.step_kv8(si, kv8, so, torch.empty(256, dtype=torch.uint8, device=cuda))
    dr.close()
