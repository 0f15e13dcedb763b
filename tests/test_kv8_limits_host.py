"""CPU checks that sizes the 8-bit cache's attention cannot launch are refused by every entry
point before anything is launched (no GPU is touched here)."""
import ctypes as ct

import pytest


@pytest.fixture(scope="module")
def H():
    from hybrid_mamba_attention_b200 import hspec
    return hspec


def cfg(H, Hq=4, Hkv=2, D=64, page=16, dtype=None, **kw):
    return H.hspec_cfg(d_model=64, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=D, page_size=page, n_layers=1,
                       layer_kinds=b"A", dtype=H.HSPEC_DTYPE_BF16 if dtype is None else dtype, **kw)


# configuration, C, K, num_pages, max_pages, whether it runs
CASES = [
    (dict(dtype=0), 65535, 1, 4, 4, True),
    (dict(dtype=0), 65536, 1, 4, 4, False),                   # requests on the CUDA-core path
    (dict(D=96), 65536, 1, 4, 4, False),
    (dict(), 65536, 1, 4, 4, True),                           # not on the tensor-core path
    (dict(dtype=0, Hq=65536, Hkv=65536), 1, 1, 4, 4, False),  # heads
    (dict(dtype=0, Hq=4096, Hkv=1), 1, 16, 4, 4, True),       # 1024 row blocks
    (dict(Hq=16, Hkv=16), 255, 1, 4, 1 << 21, True),          # 255 * 16 * (2^18 + 5) units of the line, below 2^30
    (dict(Hq=16, Hkv=16), 256, 1, 4, 1 << 21, False),
    (dict(Hq=16, Hkv=16), 4200, 1, 4, 1 << 16, True),
    (dict(Hq=16, Hkv=16), 4200, 1, 4, 1 << 17, False),
    (dict(Hq=16, Hkv=16), 4, 1, (1 << 27) - 1, 4, True),      # pages of the pool
    (dict(Hq=16, Hkv=16), 4, 1, 1 << 27, 4, False),
    (dict(Hq=1 << 20, Hkv=1 << 20), 2100, 1, 4, 1, False),    # query heads in all
    (dict(D=258), 1, 1, 4, 4, False),
]


@pytest.mark.parametrize("kw,C,K,num_pages,max_pages,runs", CASES)
def test_limits(H, kw, C, K, num_pages, max_pages, runs):
    assert H.HSPEC_DTYPE_F32 == 0
    L, n0, c = H._lib, H.hspec_launch_count(), cfg(H, **kw)
    v = H.hspec_kv8_view(k_codes=256, v_codes=256, k_scales=256, v_scales=256, num_pages=num_pages, page_table=256,
                         max_pages=max_pages)
    # too small a workspace is refused last, after every limit
    st = L.hspec_attn_paged_block_kv8(ct.byref(c), 256, ct.byref(v), 256, 256, 256, C, K, 256, 256, 0, None)
    assert st == (H.HSPEC_ERR_WORKSPACE if runs else H.HSPEC_ERR_UNSUPPORTED), H.hspec_last_error()
    size, step = H.hspec_attn_kv8_workspace_size(c, C, K, max_pages), H.hspec_step_kv8_workspace_size(c, C, K, max_pages)
    assert (size > 0 and step > size) if runs else (size == step == 0 or num_pages > 4)
    mw = H.hspec_model_weights()
    mw.layers[0].norm = mw.layers[0].W_qkv = mw.layers[0].W_o = 256
    h = H.hspec_drafter_create(c, mw)
    si, so = H.hspec_step_in(C=C, K=K, x_in=256, ctx_lens=256), H.hspec_step_out()
    st = L.hspec_draft_step_kv8(h, ct.byref(si), ct.byref(v), ct.byref(so), 256, 0 if runs else 1 << 60, None)
    assert st == (H.HSPEC_ERR_WORKSPACE if runs else H.HSPEC_ERR_UNSUPPORTED), H.hspec_last_error()
    H.hspec_drafter_destroy(h)
    assert H.hspec_launch_count() == n0
