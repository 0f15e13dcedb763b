"""CPU checks of what the Python binding of the 8-bit cache's write and read refuses: rows that
the library would read past their ends (no GPU is touched here)."""
import pytest
import torch


@pytest.fixture(scope="module")
def H():
    from hybrid_mamba_attention_b200 import hspec
    return hspec


def cfg(H, Hkv, D, dtype=None):
    return H.hspec_cfg(d_model=64, n_q_heads=Hkv, n_kv_heads=Hkv, head_dim=D, page_size=16, n_layers=1,
                       layer_kinds=b"A", dtype=H.HSPEC_DTYPE_BF16 if dtype is None else dtype)


def calls(H, c, rows, first=(0, 0)):
    kv = H.hspec_kv8_view(k_codes=256, v_codes=256, k_scales=256, v_scales=256, num_pages=4, page_table=256, max_pages=4)
    cu, first = torch.tensor([0, 1, 4], dtype=torch.int32), torch.tensor(first, dtype=torch.int32)
    yield lambda: H.hspec_kv8_write(c, rows, rows, cu, first, kv, stream=0)
    yield lambda: H.hspec_kv8_read(c, kv, cu, first, rows, rows, stream=0)


def zeros(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("Hkv,D,rows", [
    (2, 64, zeros(1, 2, 64).expand(4, 2, 64)),                       # one row for all: stride 0
    (2, 64, zeros(512).as_strided((4, 2, 64), (64, 64, 1))),         # rows that overlap
    (2, 64, zeros(4, 3, 64)), (3, 64, zeros(4, 2, 64)),              # other heads than the cache's
    (1, 64, zeros(4, 1, 32)), (2, 64, zeros(4, 2, 128)),             # other head sizes
    (1, 128, zeros(4, 256)[:, :64].unsqueeze(1)),                    # narrow rows of a wide tensor
    (2, 64, zeros(4, 128)),                                          # not [T, Hkv, D]
])
def test_rows_of_other_shapes_are_refused(H, Hkv, D, rows):
    n0 = H.hspec_launch_count()
    for call in calls(H, cfg(H, Hkv, D), rows):
        with pytest.raises(ValueError):
            call()
    assert H.hspec_launch_count() == n0


def test_rows_of_another_type_and_short_starts_are_refused(H):
    n0 = H.hspec_launch_count()
    for c, rows, first in ((cfg(H, 2, 64, H.HSPEC_DTYPE_F32), zeros(4, 2, 64), (0, 0)),
                           (cfg(H, 2, 64), torch.zeros(4, 2, 64), (0, 0)),
                           (cfg(H, 2, 64), zeros(4, 2, 64), (0,))):
        for call in calls(H, c, rows, first):
            with pytest.raises(ValueError):
                call()
    assert H.hspec_launch_count() == n0


def test_rows_that_are_fine(H):
    c = cfg(H, 2, 64)
    wide = zeros(4, 512)
    for rows, stride in ((zeros(4, 2, 64), 128), (wide[:, 128:256].view(4, 2, 64), 512), (zeros(1, 2, 64), 0),
                         (zeros(0, 2, 64), 0)):
        assert H._rows(c, rows, rows, torch.zeros(3), torch.zeros(2)) == (2, rows.shape[0], stride)
    assert H._rows(cfg(H, 1, 64), wide[:, :64].unsqueeze(1), wide[:, 64:128].unsqueeze(1), torch.zeros(1), None) == (0, 4, 512)


def test_current_stream_with_and_without_the_raw_handle(H, monkeypatch):
    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(H, "_raw_stream", lambda device: 100 + device)
    assert H._stream(None) == 103 and H._stream(5) == 5 and H._stream(Stream()) == 77
    monkeypatch.setattr(H, "_raw_stream", None)
    assert H._stream(None) == 77 and H._stream(5) == 5 and H._stream(Stream()) == 77


def test_views_of_strided_pools_are_refused(H):
    def cache(**kw):
        c = {"k_codes": torch.zeros(4, 2, 16, 64, dtype=torch.uint8), "v_codes": torch.zeros(4, 2, 16, 64, dtype=torch.uint8),
             "k_scales": torch.zeros(4, 2), "v_scales": torch.zeros(4, 2), "page_table": torch.zeros(3, 4, dtype=torch.int32)}
        return dict(c, **kw)

    assert H.kv8_view(cache()).max_pages == 4
    assert H.kv8_view(cache(k_codes=torch.zeros(4, 2, 16, 64).to(torch.float8_e4m3fn))).num_pages == 4
    for bad in (dict(k_codes=torch.zeros(1, 2, 16, 64, dtype=torch.uint8).expand(4, 2, 16, 64)),
                dict(v_codes=torch.zeros(4, 4, 16, 64, dtype=torch.uint8)[:, :2]),
                dict(v_codes=zeros(4, 2, 16, 64)), dict(k_scales=torch.zeros(2, 4).T), dict(v_scales=zeros(4, 2)),
                dict(page_table=torch.zeros(3, 4, dtype=torch.int64)),
                dict(page_table=torch.zeros(3, 8, dtype=torch.int32)[:, :4])):
        with pytest.raises(ValueError):
            H.kv8_view(cache(**bad))


def test_attention_operands_of_other_shapes_are_refused(H):
    n0 = H.hspec_launch_count()
    c = H.hspec_cfg(d_model=64, n_q_heads=4, n_kv_heads=2, head_dim=64, page_size=16, n_layers=1, layer_kinds=b"A",
                    dtype=H.HSPEC_DTYPE_BF16)
    kv = H.hspec_kv8_view(k_codes=256, v_codes=256, k_scales=256, v_scales=256, num_pages=4, page_table=256, max_pages=4)

    def attn(q=None, out=None, kb=None, vb=None, lens=2):
        q = zeros(2, 3, 4, 64) if q is None else q
        H.hspec_attn_paged_block_kv8(c, q, kv, torch.zeros(lens, dtype=torch.int32),
                                     zeros(2, 3, 2, 64) if kb is None else kb, zeros(2, 3, 2, 64) if vb is None else vb,
                                     zeros(2, 3, 4, 64) if out is None else out, torch.zeros(256, dtype=torch.uint8), stream=0)

    for kw in (dict(q=zeros(1, 3, 4, 64).expand(2, 3, 4, 64)), dict(q=zeros(2, 3, 8, 64)[:, :, :4]),
               dict(q=zeros(2, 3, 2, 64)), dict(q=torch.zeros(2, 3, 4, 64)), dict(out=zeros(2, 3, 64, 4).transpose(2, 3)),
               dict(kb=zeros(1, 3, 2, 64).expand(2, 3, 2, 64)), dict(vb=zeros(2, 2, 2, 64)), dict(lens=1)):
        with pytest.raises(ValueError):
            attn(**kw)
    with pytest.raises(H.HspecError):  # nothing wrong but the workspace's size (or its alignment)
        attn()
    assert H.hspec_launch_count() == n0
