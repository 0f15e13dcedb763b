"""The draft step with attention layers whose page tables differ in width (GPU): one workspace,
sized for the widest, between guards.

1184 pages of 16 tokens are where the automatic split length doubles (2 requests of 8
positions, 2 kv heads), so the layer with 1183 pages has twice the splits."""
from dataclasses import replace

import pytest
import torch

from hybrid_mamba_attention_b200 import inputs as I
from tests import kv8_util as U
from tests.parity_util import rel_max, rel_rms, F32_TOL

pytestmark = pytest.mark.gpu

LENS, K, WIDE = [1183 * 16, 1183 * 16 - 5], 8, 1184
F32 = replace(I.TINY, layers="AA")
BF16_96 = replace(I.TINY, layers="AA", D=96, dtype="bf16")


@pytest.fixture(scope="module")
def H(cuda):
    from hybrid_mamba_attention_b200 import hspec
    return hspec


def widened(cache, width):
    t = cache["page_table"]
    out = torch.full((t.shape[0], width), -1, dtype=torch.int32, device=t.device)
    out[:, :t.shape[1]] = t
    return dict(cache, page_table=out)


def run_step(H, cuda, sh, dr, size, step):
    """hidden [C, K, d] of step(step_out, workspace) and whether the guards hold."""
    guard = 16 << 20
    buf = torch.full((2 * guard + size,), 0xA5, dtype=torch.uint8, device=cuda)
    hidden = torch.full((len(LENS), K, sh.d), float("nan"), device=cuda)
    step(H.hspec_step_out(hidden=hidden.data_ptr()), buf[guard:guard + size])
    assert H.hspec_sync_status() == 0
    assert bool((buf[:guard] == 0xA5).all()) and bool((buf[-guard:] == 0xA5).all())
    return hidden


def close(sh, got, want):
    got, want = got.double().cpu().numpy(), want.double().cpu().numpy()
    if sh.dtype == "f32":
        return rel_max(got, want) <= F32_TOL
    return rel_rms(got, want) <= 3e-2  # as the step over a bf16 cache end to end


@pytest.mark.parametrize("sh", [F32, BF16_96])
def test_kv8_tables_of_two_widths(H, cuda, sh):
    st = I.make_step_inputs(I.Workload("w", sh, C=2, K=K, ctx_lo=16, ctx_hi=16, seed=0), cuda)
    lens = torch.tensor(LENS, dtype=torch.int32, device=cuda)
    caches = [U.to_device(U.make_cache(LENS, sh.Hkv, sh.D, sh.page, 50 + i), cuda) for i in range(2)]
    dr = H.Drafter(sh, st["weights"])
    si = dr.step_in(2, K, st["h_last"], lens, [], x_in=st["x_in"])
    size = dr.workspace_size_kv8(2, K, WIDE)
    outs = []
    for widths in ((WIDE, WIDE), (WIDE, WIDE - 1), (WIDE - 1, WIDE)):
        tables = [widened(c, w) for c, w in zip(caches, widths)]
        outs.append(run_step(H, cuda, sh, dr, size, lambda so, ws: dr.step_kv8(si, tables, so, ws)))
    assert torch.isfinite(outs[0]).all()
    assert close(sh, outs[1], outs[0]) and close(sh, outs[2], outs[0])
    dr.close()


def test_plain_tables_of_two_widths(H, cuda):
    # the fp32 step over ordinary caches: its split length doubles at 2368 pages
    lens = torch.tensor([2367 * 16, 2367 * 16 - 5], dtype=torch.int32, device=cuda)
    st = I.make_step_inputs(I.Workload("w", F32, C=2, K=K, ctx_lo=2367 * 16, ctx_hi=2367 * 16, seed=0), cuda)
    dr = H.Drafter(F32, st["weights"])
    size = dr.workspace_size(2, K, 2368)
    outs = []
    for widths in ((2368, 2368), (2368, 2367), (2367, 2368)):
        tables = [widened(c, w) for c, w in zip(st["kv"], widths)]
        si = dr.step_in(2, K, st["h_last"], lens, tables, x_in=st["x_in"])
        outs.append(run_step(H, cuda, F32, dr, size, lambda so, ws: dr.step(si, so, ws)))
    assert torch.isfinite(outs[0]).all()
    assert close(F32, outs[1], outs[0]) and close(F32, outs[2], outs[0])
    dr.close()
