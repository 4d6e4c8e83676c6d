"""Workspaces, buffers and lengths that a program keeps between calls of the latent
attention: used for other sizes, with old contents, one call after the other."""
import numpy as np
import pytest
import torch

import oracle
import sparse_attention_token_misa_b200 as misa
from test_gpu_latent_mla import FORMS, SCALE, _check, _draw_idx, _i32, _prefix_idx, _setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", FORMS)
def test_workspace_of_a_larger_batch(form):
    """One workspace, sized for the largest batch and never cleared behind its error
    word, serves smaller ones, whose rows are split into more parts; so do calls that
    bring none."""
    L, Hq = 2048, 64
    q, cache, held = _setup(40, 2, L, form, 70, Hq)
    ws = misa.alloc_workspace(misa.workspace_bytes(misa.OP_PREFIX_MLA, 70, Hq, L, 0))
    for T in (70, 32, 3, 1):
        ws[256:].fill_(0xFF)
        seq, lens = np.arange(T) % 2, [L - 5 * t for t in range(T)]
        args = (q[:T].cuda(), cache, _i32(seq), _i32(lens), SCALE)
        out, lse = misa.prefix_mla(*args, want_lse=True, workspace=ws)
        assert misa.error_query(ws) == 0
        alone, lse_alone = misa.prefix_mla(*args, want_lse=True)
        assert torch.equal(out, alone) and torch.equal(lse, lse_alone)
        _check(out, lse, q[:T], held, seq, _prefix_idx(lens, L), SCALE)


@pytest.mark.parametrize("form", ["mx8", "mx4"])
def test_shorter_lists_in_the_workspace_of_longer_ones(form):
    L, k = 6000, 4737
    q, cache, held = _setup(41, 1, L, form, 1, 128)
    ws = misa.alloc_workspace(misa.workspace_bytes(misa.OP_SPARSE_MLA_Q, 1, 128, L, 0, k))
    for n in (4737, 4736, 2048, 1):
        ws[256:].fill_(0xFF)
        idx = _draw_idx(n, 1, L, n, 0)
        out, lse = misa.sparse_mla_q(q.cuda(), cache, _i32([0]), _i32(idx), SCALE, want_lse=True, workspace=ws)
        assert misa.error_query(ws) == 0
        _check(out, lse, q, held, np.array([0]), idx, SCALE)


@pytest.mark.parametrize("form", FORMS)
def test_listed_and_prefix_side_by_side(form):
    """Both attentions of a step, compared behind it: each with its own oracle value."""
    T, L, k, Hq = 3, 500, 200, 128
    g = torch.Generator().manual_seed(42)
    rows, q = torch.randn(T, L, 576, generator=g).bfloat16(), torch.randn(T, Hq, 576, generator=g).bfloat16()
    held = oracle.latent_values(rows.double().numpy(), form)
    lc = misa.LatentCache(T, L, form, T, Hq, k)
    lc.append(rows.cuda())
    idx, seq = _draw_idx(42, T, L, k, 20), _i32(range(T))
    listed = lc.attend(q.cuda(), seq, _i32(idx), SCALE)
    prefix = lc.attend_prefix(q.cuda(), seq, lc.lens, SCALE)
    # the bf16 form of the listed tokens rounds its weights before their sum too
    more = dict(roundings=3, lse_more=1.01 * 2.0 ** -8) if form == "bf16" else {}
    _check(*listed, q, held, np.arange(T), idx, SCALE, **more)
    _check(*prefix, q, held, np.arange(T), _prefix_idx([L] * T, L), SCALE)


@pytest.mark.parametrize("counted", [False, True])
def test_lengths_and_rows_advance_together(counted):
    """Where append moves a length it has written the rows, and nowhere else."""
    L, n = 16, 3
    lens = [-1, 0, 5, 13, 14, 16, 17, 2 ** 31 - 1, -2 ** 31]
    counts = [3, 0, 2, 3, 2, 1, 0, 3, 3] if counted else [n] * len(lens)
    rows = torch.randn(len(lens), n, 576, generator=torch.Generator().manual_seed(43)).bfloat16()
    lc = misa.LatentCache(len(lens), L, "mx8", T=1, Hq=1, k=1)
    lc.rows.fill_(0x5A)
    lc.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    want = lc.rows.cpu()
    held = torch.from_numpy(oracle.latent_bytes(rows.double().numpy(), "mx8"))
    new = []
    for b, (l, c) in enumerate(zip(lens, counts)):
        fits = 0 <= c <= n and l >= 0 and l + c <= L
        if fits:
            want[b, l:l + c] = held[b, :c]
        new.append(l + c if fits else l)
    lc.append(rows.cuda(), counts=_i32(counts) if counted else None)
    assert lc.lens.tolist() == new and torch.equal(lc.rows.cpu(), want)
    assert misa.error_query(lc.ws) == misa._native.DEVERR_BAD_LEN


@pytest.mark.parametrize("form", FORMS)
def test_a_step_allocates_nothing(form):
    T, L, k, Hq = 2, 64, 8, 16
    lc = misa.LatentCache(T, L, form, T, Hq, k)
    rows, q = torch.randn(T, 3, 576, device="cuda").bfloat16(), torch.randn(T, Hq, 576, device="cuda").bfloat16()
    counts, seq, idx = _i32([2, 3]), _i32([0, 1]), _i32([[0, 1, -1, -1, -1, -1, -1, -1]] * T)

    def step():
        lc.append(rows)
        lc.append(rows, counts=counts)
        lc.attend(q, seq, idx, SCALE)
        lc.attend_prefix(q, seq, lc.lens, SCALE)

    step()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    step()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    assert lc.lens.tolist() == [10, 12]
