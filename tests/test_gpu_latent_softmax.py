"""The softmax of the latent attention where its parts differ most: the two halves of
a tile's rows, one tile and the next.  Tolerances as in test_gpu_latent_mla.py."""
import numpy as np
import pytest
import torch

import oracle
import sparse_attention_token_misa_b200 as misa
from test_gpu_latent_mla import FORMS, SCALE, _check, _draw_idx, _i32, _prefix_idx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,L", [(160, 64 * 5 + 7), (80, 64 * 2), (3, 64 * 40)])
def test_halves_and_tiles_of_different_size(form, T, L):
    """Every half tile (32 rows) has its own size of score, some 20 apart, so that a
    maximum taken from another tile or half would be far off: in a cluster's first
    tiles, in several items a cluster, in items of several lengths.  The same bits
    every time."""
    g = torch.Generator().manual_seed(T)
    q = torch.randn(T, 128, 576, generator=g) * 0.5
    q[:, :, 512:] = 1.0
    rows = torch.randn(1, L, 576, generator=g) * 0.3
    size = torch.tensor([20.0, -20.0, -20.0, 0.0, -20.0, 20.0, 0.0, 7.0])
    rows[0, :, 512:] += (size[torch.arange(L) // 32 % 8] / (64 * SCALE))[:, None]
    q, rows = q.bfloat16(), rows.bfloat16()
    cache = misa.alloc_kv_cache(1, L, form)
    misa.append_kv(cache, _i32([0]), rows.cuda())
    held = oracle.latent_values(rows.double().numpy(), form)
    lens = [L - (37 * t) % L for t in range(T)]
    args = (q.cuda(), cache, _i32([0] * T), _i32(lens), SCALE)
    ws = misa.alloc_workspace(misa.workspace_bytes(misa.OP_PREFIX_MLA, T, 128, L, 0))
    out, lse = misa.prefix_mla(*args, want_lse=True, workspace=ws)
    assert misa.error_query(ws) == 0
    _check(out, lse, q, held, np.zeros(T, np.int64), _prefix_idx(lens, L), SCALE)
    for _ in range(20):
        again, lse2 = misa.prefix_mla(*args, want_lse=True, workspace=ws)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("scale", [0.0, 1e-45, 1e-39, 2.0 ** -126])
def test_smallest_scales(form, scale):
    """Scores of 1e37, which only a scale of exactly what was asked for makes alike."""
    T, L = 3, 300
    g = torch.Generator().manual_seed(50)
    q = (torch.randn(T, 128, 576, generator=g) * 1e19).bfloat16()
    rows = (torch.randn(1, L, 576, generator=g) * 1e17).bfloat16()
    cache = misa.alloc_kv_cache(1, L, form)
    misa.append_kv(cache, _i32([0]), rows.cuda())
    held = oracle.latent_values(rows.double().numpy(), form)
    scale = float(np.float32(scale))
    lens = [300, 129, 40]
    out, lse = misa.prefix_mla(q.cuda(), cache, _i32([0] * T), _i32(lens), scale, want_lse=True)
    _check(out, lse, q, held, np.zeros(T, np.int64), _prefix_idx(lens, L), scale)
    if form != "bf16":
        idx = _draw_idx(50, T, L, 130, 3)
        idx[0] = -1
        out, lse = misa.sparse_mla_q(q.cuda(), cache, _i32([0] * T), _i32(idx), scale, want_lse=True)
        assert not out[0].any() and torch.isneginf(lse[0]).all()
        _check(out, lse, q, held, np.zeros(T, np.int64), idx, scale)


@pytest.mark.parametrize("form", FORMS)
def test_scale_of_zero_keeps_nan_and_infinities(form):
    """0 * s is NaN where the score is not finite; a row that is not seen stays out."""
    q = torch.ones(2, 128, 576, dtype=torch.bfloat16)
    rows = torch.randn(1, 100, 576, generator=torch.Generator().manual_seed(51)).bfloat16()
    rows[0, 70, 520] = float("inf")      # a rotary entry, which every form keeps
    cache = misa.alloc_kv_cache(1, 100, form)
    misa.append_kv(cache, _i32([0]), rows.cuda())
    held = oracle.latent_values(rows.double().numpy(), form)
    out, lse = misa.prefix_mla(q.cuda(), cache, _i32([0, 0]), _i32([70, 71]), 0.0, want_lse=True)
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    _check(out[:1], lse[:1], q[:1], held[:, :70], np.zeros(1, np.int64), _prefix_idx([70], 70), 0.0)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("L", [70, 3000])
def test_scores_that_are_not_finite(form, L):
    """-inf has no weight, alone it is a query without rows; +inf gives NaN.  In one
    part and in several."""
    g = torch.Generator().manual_seed(52)
    q = torch.randn(4, 128, 576, generator=g).bfloat16()
    rows = torch.randn(4, L, 576, generator=g).bfloat16()
    q[:, :, 570] = 1.0
    rows[0, :, 570] = -float("inf")
    rows[1, :, 570] = -float("inf")
    rows[1, 65:68, 570] = 0.5
    rows[2, 3, 570] = float("inf")
    cache = misa.alloc_kv_cache(4, L, form)
    misa.append_kv(cache, _i32([0] * 4), rows.cuda())
    held = oracle.latent_values(rows.double().numpy(), form)
    out, lse = misa.prefix_mla(q.cuda(), cache, _i32([0, 1, 2, 3]), _i32([L] * 4), SCALE, want_lse=True)
    assert not out[0].any() and torch.isneginf(lse[0]).all()
    assert torch.isnan(out[2]).all() and torch.isnan(lse[2]).all()
    keep = np.full((2, L), -1)
    keep[0, :3], keep[1] = [65, 66, 67], np.arange(L)
    _check(out[[1, 3]], lse[[1, 3]], q[[1, 3]], held, np.array([1, 3]), keep, SCALE)
