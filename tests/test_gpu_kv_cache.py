"""append_kv and read_kv against the table-driven oracle: bytes and values have to
be equal, everything else of the cache and behind the last row untouched."""
import numpy as np
import pytest
import torch

import oracle
import sparse_attention_token_misa_b200 as misa
from sparse_attention_token_misa_b200 import _native as nat

pytestmark = pytest.mark.gpu

FORMS = ["bf16", "mx8", "mx4"]
QUANT = ["mx8", "mx4"]


def _rows(seed, *shape, spread=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, 576, generator=g)
    if spread:
        x = torch.ldexp(x, torch.randint(-spread, spread + 1, (*shape, 576), generator=g))
    return x.bfloat16()


def _held(rows, form):
    """What the cache should hold, as the cache's own element type."""
    return rows if form == "bf16" else torch.from_numpy(oracle.latent_bytes(rows.double().numpy(), form))


def _cache(nseq, L, form, fill=0x5A):
    c = misa.alloc_kv_cache(nseq, L, form)
    c.view(torch.uint8).fill_(fill)
    return c


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("nseq,n,L,lens,counts", [
    (1, 1, 1, [0], None),
    (3, 1, 70, [0, 69, 33], None),
    (2, 37, 64, [27, 3], [37, 0]),
    (4, 130, 300, [0, 1, 170, 99], [130, 129, 130, 1]),
])
def test_append_writes_the_rows_and_nothing_else(form, nseq, n, L, lens, counts):
    rows = _rows(n, nseq, n, spread=3)
    cache = _cache(nseq, L, form)
    want = cache.clone().cpu()
    held = _held(rows, form)
    for b in range(nseq):
        c = n if counts is None else counts[b]
        want[b, lens[b]:lens[b] + c] = held[b, :c]
    ws = misa.alloc_workspace(256)
    misa.append_kv(cache, _i32(lens), rows.cuda(), counts=None if counts is None else _i32(counts), workspace=ws)
    assert _same(cache.cpu(), want)
    assert misa.error_query(ws) == 0


@pytest.mark.parametrize("form", QUANT)
def test_every_bf16_number(form):
    """All finite bf16 numbers, in groups of like and of mixed size."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = bits[torch.isfinite(bits.float())]
    x = torch.cat([x, x[torch.randperm(len(x), generator=torch.Generator().manual_seed(1))]])
    x = torch.cat([x, torch.zeros(-len(x) % 512, dtype=torch.bfloat16)]).reshape(-1, 512)
    rows = torch.cat([x, _rows(2, len(x))[:, 512:]], 1)[None]
    cache = _cache(1, rows.shape[1], form)
    misa.append_kv(cache, _i32([0]), rows.cuda())
    assert _same(cache.cpu(), _held(rows, form))
    back = misa.read_kv(cache, _i32([0]), n=rows.shape[1])
    want = torch.from_numpy(oracle.latent_values(rows.double().numpy(), form)).bfloat16()
    assert torch.equal(back.cpu(), want)


@pytest.mark.parametrize("form", QUANT)
def test_ties_and_borders(form):
    """Halfway cases of every element, with the group's largest entry pinned."""
    t = oracle.latent_elements(form)
    mids = np.concatenate([t, (t[1:] + t[:-1]) / 2])
    mids = mids[torch.from_numpy(mids).bfloat16().double().numpy() == mids]
    rows = np.zeros((1, len(mids) // 8 + 1, 576))
    for i, v in enumerate(np.pad(mids, (0, -len(mids) % 8 + 8))[:rows.shape[1] * 8]):
        g = i % 8 * 2
        rows[0, i // 8, 32 * g:32 * g + 3] = (v, -v, t[-1])
        rows[0, i // 8, 32 * g + 32:32 * g + 34] = (t[-1] * 2 ** -20, v * 2 ** -20)
    rows = torch.from_numpy(rows).bfloat16()
    cache = _cache(1, rows.shape[1], form)
    misa.append_kv(cache, _i32([0]), rows.cuda())
    assert _same(cache.cpu(), _held(rows, form))


@pytest.mark.parametrize("form", QUANT)
def test_non_finite_groups_read_back_as_nan(form):
    rows = _rows(5, 1, 4)
    rows[0, 0, 3], rows[0, 1, 64], rows[0, 2, 511], rows[0, 3, 575] = float("inf"), float("nan"), -float("inf"), float("nan")
    cache = _cache(1, 4, form)
    misa.append_kv(cache, _i32([0]), rows.cuda())
    back = misa.read_kv(cache, _i32([0]), n=4).cpu()
    want = torch.from_numpy(oracle.latent_values(rows.double().numpy(), form)).bfloat16()
    assert torch.equal(torch.isnan(back), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(back.float()), torch.nan_to_num(want.float()))


def test_bad_lengths_are_skipped_and_recorded():
    rows = _rows(6, 5, 4)
    cache = _cache(5, 20, "mx8")
    before = cache.clone()
    ws = misa.alloc_workspace(256)
    misa.append_kv(cache, _i32([-1, 17, 0, 0, 16]), rows.cuda(), counts=_i32([4, 4, 5, -1, 4]), workspace=ws)
    assert misa.error_query(ws) == nat.DEVERR_BAD_LEN
    assert _same(cache[:4], before[:4])
    assert _same(cache[4, 16:].cpu(), _held(rows[4], "mx8"))


@pytest.mark.parametrize("form", FORMS)
def test_read_listed_and_ranges(form):
    nseq, L = 3, 50
    rows = _rows(7, nseq, L)
    # a cache inside a larger buffer: sequences further apart than their rows
    wide = _cache(nseq, L + 13, form)
    cache = wide[:, :L]
    misa.append_kv(cache, _i32([0] * nseq), rows.cuda())
    val = torch.from_numpy(oracle.latent_values(rows.double().numpy(), form)).bfloat16()
    zero = torch.zeros(576, dtype=torch.bfloat16)
    ws = misa.alloc_workspace(256)
    seq = [2, 0, 0, 1]
    idx = torch.tensor([[49, 0, -1, 7, 7], [-1] * 5, [3, 2, 1, 0, 49], [48, -1, 5, 6, 9]], dtype=torch.int32)
    wide_idx = torch.full((4, 9), -77, dtype=torch.int32)
    wide_idx[:, 2:7] = idx
    got = misa.read_kv(cache, _i32(seq), idx=wide_idx.cuda()[:, 2:7], workspace=ws).cpu()
    want = torch.stack([torch.stack([val[b, i] if i >= 0 else zero for i in row]) for b, row in zip(seq, idx.tolist())])
    assert torch.equal(got, want)
    first, end = [0, 45, 50, 10], [50, 60, 50, 12]
    got = misa.read_kv(cache, _i32(seq), first=_i32(first), n=7, prefix_len=_i32(end), workspace=ws).cpu()
    want = torch.stack([torch.stack([val[b, f + i] if f + i < min(e, L) else zero for i in range(7)])
                        for b, f, e in zip(seq, first, end)])
    assert torch.equal(got, want)
    assert torch.equal(misa.read_kv(cache, _i32([1]), n=L, workspace=ws).cpu()[0], val[1])
    assert misa.error_query(ws) == 0


def test_read_bad_arguments_are_recorded():
    cache = misa.alloc_kv_cache(2, 8, "mx4")
    rows = _rows(8, 2, 8)
    misa.append_kv(cache, _i32([0, 0]), rows.cuda())
    val = torch.from_numpy(oracle.latent_values(rows.double().numpy(), "mx4")).bfloat16()
    ws = misa.alloc_workspace(256)
    got = misa.read_kv(cache, _i32([0, 1]), idx=_i32([[8, 3], [-2, 2 ** 31 - 1]]), workspace=ws).cpu()
    assert misa.error_query(ws) == nat.DEVERR_BAD_INDEX
    assert torch.equal(got[0, 1], val[0, 3]) and not got[0, 0].any() and not got[1].any()
    misa.error_reset(ws)
    got = misa.read_kv(cache, _i32([2, 1]), first=_i32([0, -1]), n=2, workspace=ws).cpu()
    assert misa.error_query(ws) == nat.DEVERR_BAD_SEQ | nat.DEVERR_BAD_INDEX and not got.any()


def test_offsets_behind_2_31():
    """Rows whose byte offset does not fit 32 bits."""
    L = (1 << 31) // 656 + 1000
    cache = torch.empty((1, L, 656), dtype=torch.uint8, device="cuda")
    rows = _rows(9, 1, 3)
    at = L - 5
    cache[0, at - 1:] = 0x33
    misa.append_kv(cache, _i32([at]), rows.cuda())
    val = torch.from_numpy(oracle.latent_values(rows.double().numpy(), "mx8")).bfloat16()
    got = misa.read_kv(cache, _i32([0]), idx=_i32([[at, at + 1, at + 2]])).cpu()
    assert torch.equal(got, val)
    assert (cache[0, at - 1] == 0x33).all() and (cache[0, at + 3:] == 0x33).all()


def test_append_in_a_graph_advances():
    lc = misa.LatentCache(2, 16, "mx8", T=2, Hq=8, k=4)
    rows = torch.zeros(2, 2, 576, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lc.append(rows)
    torch.cuda.current_stream().wait_stream(side)
    lc.lens.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lc.append(rows)
    want = []
    for step in range(9):          # the ninth no longer fits: recorded, nothing moves
        new = _rows(20 + step, 2, 2)
        rows.copy_(new)
        g.replay()
        want.append(new)
    assert lc.lens.tolist() == [16, 16] and misa.error_query(lc.ws) == nat.DEVERR_BAD_LEN
    assert _same(lc.rows.cpu(), _held(torch.cat(want[:8], 1), "mx8"))


@pytest.mark.parametrize("form", QUANT)
def test_another_stream(form):
    """A call on a stream of its own, with the workspace left to the call."""
    rows = _rows(30, 2, 64)
    cache = _cache(2, 64, form)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    misa.append_kv(cache, _i32([0, 0]), rows.cuda(), stream=s)
    torch.cuda.synchronize()
    back = misa.read_kv(cache, _i32([0, 1]), n=64, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(back.cpu(), torch.from_numpy(oracle.latent_values(rows.double().numpy(), form)).bfloat16())
