"""CPU checks that a draft step's workspace, sized for the widest of its attention layers' page
tables, holds the split partials of every narrower layer (no GPU is touched here)."""
import pytest

SHAPES = [
    # C, K, Hq, Hkv, D, page: CUDA-core attention in both kinds of cache (fp32), or in 8-bit ones
    (2, 8, 4, 2, 64, 16), (8, 8, 32, 8, 64, 16), (1, 1, 2, 1, 64, 16), (3, 5, 4, 2, 64, 5), (33, 16, 8, 1, 128, 16),
]
WIDTHS = list(range(1, 1300)) + list(range(1300, 20000, 7))


@pytest.fixture(scope="module")
def H():
    from hybrid_mamba_attention_b200 import hspec
    return hspec


def cfg(H, dtype, Hq, Hkv, D, page, split=0):
    return H.hspec_cfg(d_model=64, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=D, page_size=page, n_layers=2,
                       layer_kinds=b"AA", dtype=dtype, attn_split_tokens=split)


def check(step, attn):
    """step(w) must cover attn(v) and the step's other buffers, which no width changes, for v <= w."""
    rest = step(1) - attn(1)
    most = 0
    for w in WIDTHS:
        most = max(most, attn(w))
        assert step(w) >= rest + most, w


@pytest.mark.parametrize("split", [0, 64, 528])
@pytest.mark.parametrize("C,K,Hq,Hkv,D,page", SHAPES)
def test_kv8_step_covers_narrower_tables(H, C, K, Hq, Hkv, D, page, split):
    for dtype, dim in ((H.HSPEC_DTYPE_F32, D), (H.HSPEC_DTYPE_BF16, 96), (H.HSPEC_DTYPE_BF16, D)):
        c = cfg(H, dtype, Hq, Hkv, dim, page, split)
        check(lambda w: H.hspec_step_kv8_workspace_size(c, C, K, w),
              lambda w: H.hspec_attn_kv8_workspace_size(c, C, K, w))


@pytest.mark.parametrize("split", [0, 64, 528])
@pytest.mark.parametrize("C,K,Hq,Hkv,D,page", SHAPES)
def test_step_covers_narrower_tables(H, C, K, Hq, Hkv, D, page, split):
    for dtype in (H.HSPEC_DTYPE_F32, H.HSPEC_DTYPE_BF16):
        c = cfg(H, dtype, Hq, Hkv, D, page, split)
        check(lambda w: H.hspec_step_workspace_size(c, C, K, w), lambda w: H.hspec_attn_workspace_size(c, C, K, w))


def test_attention_alone_needs_its_own_width_only(H):
    # (the allocation-free entry point's fixed scratch takes what it took before)
    c = cfg(H, H.HSPEC_DTYPE_F32, 4, 2, 64, 16)
    a, b = H.hspec_attn_workspace_size(c, 2, 8, 2367), H.hspec_attn_workspace_size(c, 2, 8, 2368)
    assert b < 0.6 * a and H.hspec_step_workspace_size(c, 2, 8, 2368) > a
