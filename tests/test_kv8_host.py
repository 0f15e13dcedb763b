"""CPU checks of the 8-bit cache's entry points: struct layout, workspace sizes and the
refusal of bad arguments before anything is launched; and of the plain arithmetic that
the GPU tests compare with (no GPU is touched here)."""
import ctypes as ct
import os
import subprocess

import pytest
import torch

from tests import kv8_util as U

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def H():
    from hybrid_mamba_attention_b200 import hspec
    return hspec


def cfg(H, **kw):
    f = dict(d_model=512, n_q_heads=4, n_kv_heads=2, head_dim=128, page_size=16, n_layers=1, layer_kinds=b"A",
             dtype=H.HSPEC_DTYPE_BF16)
    f.update(kw)
    return H.hspec_cfg(**f)


def view(H, **kw):
    f = dict(k_codes=256, v_codes=256, k_scales=256, v_scales=256, num_pages=4, page_table=256, max_pages=4)
    f.update(kw)
    return H.hspec_kv8_view(**f)


def test_view_layout_matches_the_header(H, tmp_path):
    fields = ["v_codes", "k_scales", "v_scales", "num_pages", "page_table", "max_pages"]
    src = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{ROOT}/include/hspec.h"', "int main(void){",
           'printf("%zu\\n", sizeof(hspec_kv8_view));']
    src += [f'printf("%zu\\n", offsetof(hspec_kv8_view, {f}));' for f in fields] + ["return 0;}"]
    (tmp_path / "sz.c").write_text("\n".join(src))
    subprocess.run(["gcc", str(tmp_path / "sz.c"), "-o", str(tmp_path / "sz")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "sz")], capture_output=True, text=True,
                                          check=True).stdout.split()]
    cls = H.hspec_kv8_view
    assert got == [ct.sizeof(cls)] + [getattr(cls, f).offset for f in fields]


def test_write_and_read_refusals(H):
    L, n0 = H._lib, H.hspec_launch_count()
    INV, OOB, UNS, SHP = (H.HSPEC_ERR_INVALID_ARG, H.HSPEC_ERR_PAGE_OOB, H.HSPEC_ERR_UNSUPPORTED,
                          H.HSPEC_ERR_SHAPE_MISMATCH)

    def write(c=None, k=256, v=256, rs=0, cu=256, first=256, C=2, T=5, kv=None):
        kv = kv if kv is not None else view(H)
        return L.hspec_kv8_write(ct.byref(c or cfg(H)), k, v, rs, cu, first, C, T, ct.byref(kv), None)

    def read(c=None, k=256, v=256, rs=0, cu=256, first=256, C=2, T=5, kv=None):
        kv = kv if kv is not None else view(H)
        return L.hspec_kv8_read(ct.byref(c or cfg(H)), ct.byref(kv), cu, first, C, T, k, v, rs, None)

    for call in (write, read):
        assert call(k=None) == INV and call(v=None) == INV and call(cu=None) == INV
        assert call(C=0) == INV and call(T=-1) == INV
        assert call(rs=255) == INV and "row_stride" in H.hspec_last_error()
        assert call(kv=view(H, k_codes=None)) == INV and call(kv=view(H, v_scales=None)) == INV
        assert call(kv=view(H, k_codes=264)) == INV and "aligned" in H.hspec_last_error()
        assert call(kv=view(H, num_pages=0)) == OOB and call(kv=view(H, max_pages=0)) == OOB
        assert call(kv=view(H, max_pages=1 << 27)) == UNS
        assert call(c=cfg(H, n_kv_heads=3)) == SHP
        assert call(c=cfg(H, page_size=0)) == INV
        assert call(c=cfg(H, dtype=5)) == INV
        assert call(T=(1 << 30) + 1) == UNS
    assert write(first=None) == INV
    assert L.hspec_kv8_write(None, 256, 256, 0, 256, 256, 1, 1, ct.byref(view(H)), None) == INV
    assert L.hspec_kv8_write(ct.byref(cfg(H)), 256, 256, 0, 256, 256, 1, 1, None, None) == INV
    assert H.hspec_launch_count() == n0


def test_pages_too_large_are_refused(H):
    # a page and head's codes are counted in 32 bits
    L, n0, kv = H._lib, H.hspec_launch_count(), view(H, max_pages=1)
    for page, D, ok in ((1 << 23, 128, True), ((1 << 23) + 1, 128, False), (1 << 29, 2, True), (1 << 30, 2, False)):
        c = cfg(H, page_size=page, head_dim=D)
        want = H.HSPEC_OK if ok else H.HSPEC_ERR_UNSUPPORTED
        assert L.hspec_kv8_write(ct.byref(c), 256, 256, 0, 256, 256, 1, 0, ct.byref(kv), None) == want
        assert L.hspec_kv8_read(ct.byref(c), ct.byref(kv), 256, 256, 1, 0, 256, 256, 0, None) == want
        if not ok:
            st = L.hspec_attn_paged_block_kv8(ct.byref(c), 256, ct.byref(kv), 256, 256, 256, 1, 1, 256, 256, 1 << 50, None)
            assert st == want and "page_size" in H.hspec_last_error()
    assert H.hspec_launch_count() == n0


def test_attention_refusals(H):
    L, n0 = H._lib, H.hspec_launch_count()
    INV, UNS, WSP = H.HSPEC_ERR_INVALID_ARG, H.HSPEC_ERR_UNSUPPORTED, H.HSPEC_ERR_WORKSPACE

    def attn(c=None, q=256, kv=None, lens=256, kb=256, vb=256, C=2, K=4, out=256, ws=256, n=1 << 40):
        kv = kv if kv is not None else view(H)
        return L.hspec_attn_paged_block_kv8(ct.byref(c or cfg(H)), q, ct.byref(kv), lens, kb, vb, C, K, out, ws, n,
                                            None)

    assert attn(q=None) == INV and attn(lens=None) == INV and attn(out=None) == INV
    assert attn(kb=None) == INV and attn(vb=None) == INV and "both" in H.hspec_last_error()
    assert attn(q=260) == INV and attn(out=264) == INV and attn(kb=258) == INV
    assert attn(K=0) == UNS and attn(K=65) == UNS and attn(C=0) == UNS
    assert attn(c=cfg(H, head_dim=258)) == UNS and "head_dim" in H.hspec_last_error()
    assert attn(ws=None) == WSP and attn(ws=272) == WSP
    need = H.hspec_attn_kv8_workspace_size(cfg(H), 2, 4, 4)
    assert need > 0 and need % 256 == 0
    assert attn(n=need - 1) == WSP
    assert attn(kv=view(H, v_codes=257)) == INV
    assert H.hspec_attn_kv8_workspace_size(cfg(H), 0, 4, 4) == 0
    assert H.hspec_attn_kv8_workspace_size(cfg(H), 2, 65, 4) == 0
    assert H.hspec_attn_kv8_workspace_size(cfg(H), 2, 4, 0) == 0
    assert H.hspec_launch_count() == n0


def test_binding_refuses_unlike_rows(H):
    a, b = torch.zeros(4, 2, 128), torch.zeros(4, 3, 128)
    wide = torch.zeros(4, 1024)
    k, v = wide[:, :256].view(4, 2, 128), wide[:, 512:768].view(4, 2, 128)
    assert H._row_stride(k, v, 128) == 1024 and H._row_stride(a, a, 128) == 256
    for x, y in ((a, b), (a, k), (a.transpose(0, 1), a.transpose(0, 1))):
        with pytest.raises(ValueError):
            H._row_stride(x, y, 128)


def test_plain_codes_match_the_format():
    # torch's own cast of values already on the grid, and of midpoints (ties to even)
    v = U.VALUES[torch.isfinite(U.VALUES)]
    assert torch.equal(U.VALUES[U.encode(v).long()], v)
    x = (torch.rand(20000, generator=torch.Generator().manual_seed(0)) * 2 - 1).double()
    x = (x * torch.exp2(torch.arange(20000).double() % 20 - 11)).float().double()
    grid = U.VALUES[:127]
    x = torch.cat([x, (grid[1:] + grid[:-1]) / 2, -(grid[1:] + grid[:-1]) / 2])
    assert torch.equal(U.VALUES[U.encode(x).long()], x.float().to(U.E4M3).double())


def test_plain_scale():
    assert U.scale_of(0.0) == 0.0 and U.scale_of(448.0) == 1.0 and U.scale_of(448.5) == 2.0
    assert U.scale_of(224.0) == 0.5 and U.scale_of(2.0 ** -140) == 2.0 ** -126


def test_every_touched_page_has_one_slot():
    # the write's and the read's numbering of touched pages: request c owns the slots
    # [cu[c] / page + 2c, cu[c+1] / page + 2(c + 1)), whatever its range's start
    g = torch.Generator().manual_seed(0)
    for _ in range(200):
        page = int(torch.randint(1, 40, (1,), generator=g))
        C = int(torch.randint(1, 70, (1,), generator=g))
        n = torch.randint(0, 90, (C,), generator=g) * torch.randint(0, 2, (C,), generator=g)
        first = torch.randint(0, 200, (C,), generator=g).tolist()
        cu = [0] + torch.cumsum(n, 0).tolist()
        slots = cu[-1] // page + 2 * C
        seen = {}
        for u in range(slots):
            # the kernels' 32-way search
            c, m = 0, C
            while m > 1:
                step = (m + 31) // 32
                hits = sum(1 for lane in range(32)
                           if lane * step < m and cu[c + lane * step] // page + 2 * (c + lane * step) <= u)
                if hits == 0:
                    c = None
                    break
                c, m = c + (hits - 1) * step, min(step, m - (hits - 1) * step)
            if c is None:
                continue
            i, f, e = u - (cu[c] // page + 2 * c), first[c], first[c] + cu[c + 1] - cu[c]
            if i < 0 or e == f or f // page + i > (e - 1) // page:
                continue
            assert (c, f // page + i) not in seen
            seen[(c, f // page + i)] = u
        want = {(c, p) for c in range(C) if cu[c + 1] > cu[c]
                for p in range(first[c] // page, (first[c] + cu[c + 1] - cu[c] - 1) // page + 1)}
        assert set(seen) == want


def test_step_kv8_refusals(H):
    L, n0 = H._lib, H.hspec_launch_count()
    assert L.hspec_draft_step_kv8(None, None, None, None, None, 0, None) == H.HSPEC_ERR_INVALID_ARG
    c = cfg(H, n_ssm_heads=4, ssm_head_dim=64, d_state=32, vocab=0)
    assert H.hspec_step_kv8_workspace_size(c, 2, 4, 8) >= H.hspec_attn_kv8_workspace_size(c, 2, 4, 8) > 0
    assert H.hspec_step_kv8_workspace_size(c, 2, 65, 8) == 0 and H.hspec_step_kv8_workspace_size(c, 0, 4, 8) == 0
    h = H.hspec_drafter_create(c, weights(H))
    si = H.hspec_step_in(C=2, K=4, x_in=256, ctx_lens=256)
    so = H.hspec_step_out()
    views = (H.hspec_kv8_view * 1)(view(H))

    def step(v):
        return L.hspec_draft_step_kv8(h, ct.byref(si), v, ct.byref(so), 256, 1 << 40, None)

    assert step(None) == H.HSPEC_ERR_INVALID_ARG and "kv8" in H.hspec_last_error()
    views[0] = view(H, v_codes=None)
    assert step(views) == H.HSPEC_ERR_INVALID_ARG
    views[0] = view(H, num_pages=0)
    assert step(views) == H.HSPEC_ERR_PAGE_OOB
    views[0] = view(H)
    assert L.hspec_draft_step_kv8(h, ct.byref(si), views, ct.byref(so), 256, 256, None) == H.HSPEC_ERR_WORKSPACE
    H.hspec_drafter_destroy(h)
    assert H.hspec_launch_count() == n0


def weights(H):
    mw = H.hspec_model_weights()
    mw.layers[0].norm = mw.layers[0].W_qkv = mw.layers[0].W_o = 256
    return mw
