"""The latent attention over caches and batches laid out otherwise: sequences further
apart than their rows, far offsets, far more room than rows, other orders of the same
queries.  Tolerances as in test_gpu_latent_mla.py."""
import numpy as np
import pytest
import torch

import oracle
import sparse_attention_token_misa_b200 as misa
from sparse_attention_token_misa_b200 import _native as nat
from test_gpu_latent_mla import FORMS, SCALE, _check, _draw_idx, _i32, _prefix_idx, _setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("L,room,T,Hq", [(130, 141, 6, 128), (300, 513, 80, 20), (3001, 3003, 3, 128)])
def test_sequences_further_apart_than_their_rows(form, L, room, T, Hq):
    """A cache inside a larger buffer, NaN between its sequences."""
    nseq = 3
    g = torch.Generator().manual_seed(room)
    rows, q = torch.randn(nseq, L, 576, generator=g).bfloat16(), torch.randn(T, Hq, 576, generator=g).bfloat16()
    wide = misa.alloc_kv_cache(nseq, room, form)
    wide.view(torch.uint8).fill_(0xFF)          # bf16 and e4m3 NaN, e2m1 under a NaN scale
    cache = wide[:, :L]
    misa.append_kv(cache, _i32([0] * nseq), rows.cuda())
    held = oracle.latent_values(rows.double().numpy(), form)
    seq = np.arange(T) * 2 % nseq
    lens = [L - (t * 29) % L for t in range(T)]
    out, lse = misa.prefix_mla(q.cuda(), cache, _i32(seq), _i32(lens), SCALE, want_lse=True)
    _check(out, lse, q, held, seq, _prefix_idx(lens, L), SCALE)
    idx = _draw_idx(room, T, L, 100, 7)
    attend = nat.sparse_mla if form == "bf16" else misa.sparse_mla_q
    out, lse = attend(q.cuda(), cache, _i32(seq), _i32(idx), SCALE, want_lse=True)
    # the bf16 form rounds its weights before their sum too
    more = dict(roundings=3, lse_more=1.01 * 2.0 ** -8) if form == "bf16" else {}
    _check(out, lse, q, held, seq, idx, SCALE, **more)


@pytest.mark.parametrize("form", FORMS)
def test_sequences_behind_2_31_bytes(form):
    """seq * cache_seq_stride does not fit 32 bits: the last of three sequences 2 GB apart."""
    row = misa.kv_row_bytes(form)
    stride, L = ((1 << 31) // row + 1) * row, 200
    flat = torch.empty(2 * stride + L * row, dtype=torch.uint8, device="cuda")
    for b in range(3):
        flat[b * stride:b * stride + L * row].fill_(0)
    cache = flat.as_strided((3, L, row), (stride, row, 1))
    if form == "bf16":
        cache = cache.view(torch.bfloat16)
    g = torch.Generator().manual_seed(60)
    rows, q = torch.randn(3, L, 576, generator=g).bfloat16(), torch.randn(2, 128, 576, generator=g).bfloat16()
    misa.append_kv(cache, _i32([0] * 3), rows.cuda())
    held = oracle.latent_values(rows.double().numpy(), form)
    seq, lens = np.array([2, 1]), [L, 77]
    out, lse = misa.prefix_mla(q.cuda(), cache, _i32(seq), _i32(lens), SCALE, want_lse=True)
    _check(out, lse, q, held, seq, _prefix_idx(lens, L), SCALE)
    back = misa.read_kv(cache, _i32(seq), n=L).cpu()
    assert np.array_equal(back.double().numpy(), held[seq])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T", [1, 7, 32])
def test_far_more_room_than_rows(form, T):
    """The normal state of a cache that grows: rows are split for its room, so most
    parts have none."""
    room, Hq = 60000, 48
    g = torch.Generator().manual_seed(T)
    lens = ([1, 500, 63, 0, 64, 65, 129] * 5)[:T] if T > 1 else [70]
    rows, q = torch.randn(1, 500, 576, generator=g).bfloat16(), torch.randn(T, Hq, 576, generator=g).bfloat16()
    cache = misa.alloc_kv_cache(1, room, form)
    misa.append_kv(cache, _i32([0]), rows.cuda())
    cache[0, 500:].view(torch.uint8).fill_(0xFF)
    held = oracle.latent_values(rows.double().numpy(), form)
    seq = np.zeros(T, np.int64)
    out, lse = misa.prefix_mla(q.cuda(), cache, _i32(seq), _i32(lens), SCALE, want_lse=True)
    _check(out, lse, q, held, seq, _prefix_idx(lens, 500), SCALE)


@pytest.mark.parametrize("form", FORMS)
def test_one_long_query_among_short_ones(form):
    """64 queries, so that none is split: one takes nearly all of the work."""
    T, L, Hq = 64, 9001, 32
    q, cache, held = _setup(61, 2, L, form, T, Hq)
    lens = [100 + t for t in range(T)]
    lens[20] = L
    seq = np.arange(T) % 2
    out, lse = misa.prefix_mla(q.cuda(), cache, _i32(seq), _i32(lens), SCALE, want_lse=True)
    _check(out, lse, q, held, seq, _prefix_idx(lens, L), SCALE)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,L", [(5, 700), (90, 200)])
def test_queries_in_another_order_give_the_same_bits(form, T, L):
    """With as many queries and as much room, a query's result does not depend on its
    place among them (rows split over clusters, and whole)."""
    q, cache, _ = _setup(62, 3, L, form, T, 128)
    g = torch.Generator().manual_seed(T)
    lens, seq = torch.randint(0, L + 1, (T,), generator=g).int(), torch.randint(0, 3, (T,), generator=g).int()
    idx = torch.from_numpy(_draw_idx(62, T, L, L, 10))
    order = torch.randperm(T, generator=g)
    a = misa.prefix_mla(q.cuda(), cache, seq.cuda(), lens.cuda(), SCALE, want_lse=True)
    b = misa.prefix_mla(q[order].cuda(), cache, seq[order].cuda(), lens[order].cuda(), SCALE, want_lse=True)
    assert torch.equal(a[0][order.cuda()], b[0]) and torch.equal(a[1][order.cuda()], b[1])
    if form != "bf16":
        a = misa.sparse_mla_q(q.cuda(), cache, seq.cuda(), idx.cuda(), SCALE, want_lse=True)
        b = misa.sparse_mla_q(q[order].cuda(), cache, seq[order].cuda(), idx[order].cuda(), SCALE, want_lse=True)
        assert torch.equal(a[0][order.cuda()], b[0]) and torch.equal(a[1][order.cuda()], b[1])


@pytest.mark.parametrize("form", ["mx8", "mx4"])
@pytest.mark.parametrize("T,L", [(3, 900), (80, 260)])
def test_a_listed_cache_gives_what_the_prefix_does(form, T, L):
    """All rows listed in order: the same rows in the same parts and order, so the same
    bits.  A shorter prefix, listed, falls into other parts: the same within the tolerance."""
    q, cache, held = _setup(63, 2, L, form, T, 128)
    seq = np.arange(T) % 2
    every = np.tile(np.arange(L, dtype=np.int32), (T, 1))
    a = misa.prefix_mla(q.cuda(), cache, _i32(seq), _i32([L] * T), SCALE, want_lse=True)
    b = misa.sparse_mla_q(q.cuda(), cache, _i32(seq), _i32(every), SCALE, want_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    every[:, 100:] = -1
    for out, lse in (misa.prefix_mla(q.cuda(), cache, _i32(seq), _i32([100] * T), SCALE, want_lse=True),
                     misa.sparse_mla_q(q.cuda(), cache, _i32(seq), _i32(every), SCALE, want_lse=True)):
        _check(out, lse, q, held, seq, _prefix_idx([100] * T, L), SCALE)


@pytest.mark.parametrize("form", ["mx8", "mx4"])
def test_longest_lists(form):
    T, L, k = 2, 20000, 16384
    q, cache, held = _setup(64, 1, L, form, T, 128)
    idx = _draw_idx(64, T, L, k, 0)
    idx[1, 5:16000] = -1
    out, lse = misa.sparse_mla_q(q.cuda(), cache, _i32([0, 0]), _i32(idx), SCALE, want_lse=True)
    _check(out, lse, q, held, np.zeros(T, np.int64), idx, SCALE)


@pytest.mark.parametrize("form", FORMS)
def test_very_many_queries(form):
    """Hundreds of items a cluster, a third of them without rows, one head each."""
    T, L = 30000, 90
    q, cache, held = _setup(65, 2, L, form, T, 1)
    rng = np.random.default_rng(65)
    lens = np.where(rng.random(T) < 0.3, 0, rng.integers(1, L + 1, T))
    lens[200:4000] = 0
    seq = rng.integers(0, 2, T)
    out, lse = misa.prefix_mla(q.cuda(), cache, _i32(seq), _i32(lens), SCALE, want_lse=True)
    _check(out, lse, q, held, seq, _prefix_idx(lens, L), SCALE)


@pytest.mark.parametrize("form", FORMS)
def test_captured_with_everything_left_to_the_call(form):
    """Outputs and workspace allocated inside the capture; replayed on new inputs."""
    T, L = 3, 2100
    q, cache, held = _setup(66, 2, L, form, T, 128)
    qd, lens, seq, kept = torch.zeros(T, 128, 576, dtype=torch.bfloat16, device="cuda"), _i32([L, 5, 900]), _i32([0, 1, 0]), []
    graph = misa.indexer.capture_graph(lambda: kept.append(misa.prefix_mla(qd, cache, seq, lens, SCALE, want_lse=True)))
    out, lse = kept[-1]
    for _ in range(2):
        q = q.flip(0).contiguous()
        qd.copy_(q)
        graph.replay()
        _check(out, lse, q, held, np.array([0, 1, 0]), _prefix_idx([L, 5, 900], L), SCALE)


@pytest.mark.parametrize("form", ["mx8", "mx4"])
def test_listed_calls_at_once(form):
    """Rows split over clusters on two streams, with a workspace each: the same bits as alone."""
    q, cache, _ = _setup(67, 2, 3000, form, 4, 128)
    sets = [(q.cuda(), cache, _i32([0, 1, 0, 1]), _i32(_draw_idx(s, 4, 3000, 2048, 100 * s)), SCALE) for s in (0, 1)]
    alone = [misa.sparse_mla_q(*x, want_lse=True) for x in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        both = [misa.sparse_mla_q(*x, want_lse=True, stream=s) for x, s in zip(sets, streams)]
        torch.cuda.synchronize()
        for one, other in zip(alone, both):
            assert torch.equal(one[0], other[0]) and torch.equal(one[1], other[1])
