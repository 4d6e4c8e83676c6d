"""sparse_mla_q and prefix_mla against the fp64 oracle on what the cache holds.

Tolerance, from the arithmetic.  Scores are fp32 sums of 576 products of bf16
numbers, off by at most d = 576 * 2^-24 * scale * max sum |q k|.  An error of d in
every score moves a weighted mean by at most 2 d A, A = sum p |v| / sum p.  bf16 keeps
8 significant bits, so a rounding to it is off by at most 2^-8 of the value.  The
weights of the numerator are rounded to it (their sum is not), and the output once
more; 2^-12 is left for the exponential and the fp32 sums: (2 d + 2 * 2^-8 + 2^-12) A.
lse carries d, its own rounding (2^-24 of it, twice) and the fp32 sum of the weights:
d + 1e-4 + 2^-22 |lse|.
"""
import numpy as np
import pytest
import torch

import oracle
import sparse_attention_token_misa_b200 as misa
from sparse_attention_token_misa_b200 import _native as nat

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
FORMS = ["bf16", "mx8", "mx4"]


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def _setup(seed, nseq, L, form, T, Hq, row_scale=1.0):
    g = torch.Generator().manual_seed(seed)
    rows = (torch.randn(nseq, L, 576, generator=g) * row_scale).bfloat16()
    q = torch.randn(T, Hq, 576, generator=g).bfloat16()
    cache = misa.alloc_kv_cache(nseq, L, form)
    misa.append_kv(cache, _i32([0] * nseq), rows.cuda())
    return q, cache, oracle.latent_values(rows.double().numpy(), form)


def _check(out, lse, q, held, seq_of, idx, scale, roundings=2, lse_more=0.0):
    q64 = q.double().cpu().numpy()
    ref, ref_lse = oracle.sparse_attention(q64, held, seq_of, idx, scale, 512)
    A = oracle.sparse_attention_abs_weights(q64, held, seq_of, idx, scale, 512)
    size = max((np.abs(q64[t]) @ np.abs(held[b][idx[t][idx[t] >= 0]]).T).max(initial=0.0) for t, b in enumerate(seq_of))
    d = 576 * 2.0 ** -24 * scale * size
    bound = (2 * d + roundings * 2.0 ** -8 + 2.0 ** -12) * A + 1e-6
    err = np.abs(out.double().cpu().numpy() - ref)
    assert np.isfinite(err).all()
    assert (err <= bound).all(), f"{(err > bound).sum()} outputs off, worst excess {(err - bound).max():.3g}"
    if lse is not None:
        lse = lse.double().cpu().numpy()
        fin = np.isfinite(ref_lse)
        assert np.array_equal(np.isneginf(lse), ~fin)
        assert (np.abs(lse[fin] - ref_lse[fin]) <= d + 1e-4 + lse_more + 2.0 ** -22 * np.abs(ref_lse[fin])).all()


def _prefix_idx(lens, L):
    width = max(1, max(min(n, L) for n in lens))
    return np.array([[i if i < min(n, L) else -1 for i in range(width)] for n in lens])


def _draw_idx(seed, T, L, k, pad):
    rng = np.random.default_rng(seed)
    idx = np.full((T, k), -1, dtype=np.int32)
    for t in range(T):
        n = max(0, min(k - pad, L))
        idx[t, :n] = np.sort(rng.choice(L, size=n, replace=False))
    return idx


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("nseq,L,T,Hq,lens", [
    (1, 1, 1, 128, [1]),
    (1, 777, 1, 128, [777]),
    (3, 130, 3, 128, [130, 0, 64]),
    (4, 700, 4, 64, [1, 63, 128, 700]),
    (2, 300, 2, 65, [129, 299]),
    (2, 300, 2, 1, [257, 300]),
    (1, 260, 9, 20, [252, 253, 254, 255, 256, 257, 258, 259, 260]),
    (1, 200, 3, 128, [-4, 200, 900]),              # below zero: empty; past the cache: all of it
])
def test_prefix_parity(form, nseq, L, T, Hq, lens):
    q, cache, held = _setup(L + Hq, nseq, L, form, T, Hq)
    seq_of = np.arange(T) % nseq
    ws = misa.alloc_workspace(misa.workspace_bytes(misa.OP_PREFIX_MLA, T, Hq, L, 0))
    out, lse = misa.prefix_mla(q.cuda(), cache, _i32(seq_of), _i32(lens), SCALE, want_lse=True, workspace=ws)
    assert misa.error_query(ws) == 0
    _check(out, lse, q, held, seq_of, _prefix_idx(lens, L), SCALE)


@pytest.mark.parametrize("form", FORMS)
def test_prefix_long(form):
    L, lens = 20011, [20011, 10243]
    q, cache, held = _setup(5, 2, L, form, 2, 128)
    out, lse = misa.prefix_mla(q.cuda(), cache, _i32([1, 0]), _i32(lens), SCALE, want_lse=True)
    _check(out, lse, q, held, np.array([1, 0]), _prefix_idx(lens, L), SCALE)


@pytest.mark.parametrize("form", FORMS)
def test_prefix_many_queries(form):
    """A prompt: more queries than SMs, each attending to those up to itself."""
    T, L = 333, 340
    q, cache, held = _setup(6, 1, L, form, T, 16)
    lens = [L - T + 1 + t for t in range(T)]
    out, lse = misa.prefix_mla(q.cuda(), cache, _i32([0] * T), _i32(lens), SCALE, want_lse=True)
    _check(out, lse, q, held, np.zeros(T, np.int64), _prefix_idx(lens, L), SCALE)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,L,Hq", [(160, 500, 13), (20, 4000, 13), (5, 4000, 9), (75, 130, 128)])
def test_prefix_uneven_lengths(form, T, L, Hq):
    """Several queries a cluster, some without rows; rows split few and many ways
    with heads that fill no group."""
    q, cache, held = _setup(8, 2, L, form, T, Hq)
    rng = np.random.default_rng(T)
    lens = rng.integers(0, L + 1, T)
    lens[[0, T // 2, T - 1]] = 0, 1, 0
    lens[T // 3] = L
    seq_of = rng.integers(0, 2, T)
    out, lse = misa.prefix_mla(q.cuda(), cache, _i32(seq_of), _i32(lens), SCALE, want_lse=True)
    _check(out, lse, q, held, seq_of, _prefix_idx(lens, L), SCALE)


@pytest.mark.parametrize("form", FORMS)
def test_two_calls_at_once(form):
    """On two streams with a workspace each, several times over: the same bits as alone."""
    q, cache, _ = _setup(9, 2, 3000, form, 6, 128)
    a, b = (q.cuda(), _i32([0, 1, 0, 1, 0, 1]), _i32([3000, 17, 0, 2999, 64, 65])), (q.flip(0).contiguous().cuda(), _i32([1] * 6), _i32([3000] * 6))
    alone = [misa.prefix_mla(x[0], cache, x[1], x[2], SCALE, want_lse=True) for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        both = [misa.prefix_mla(x[0], cache, x[1], x[2], SCALE, want_lse=True, stream=s) for x, s in zip((a, b), streams)]
        torch.cuda.synchronize()
        for one, other in zip(alone, both):
            assert torch.equal(one[0], other[0]) and torch.equal(one[1], other[1])


@pytest.mark.parametrize("form", ["mx8", "mx4"])
@pytest.mark.parametrize("nseq,L,T,Hq,k,pad,scale", [
    (1, 5, 1, 128, 1, 0, SCALE),
    (3, 3000, 3, 128, 700, 50, SCALE),
    (1, 1000, 2, 16, 100, 0, SCALE),
    (2, 5000, 4, 64, 1300, 300, 4 * SCALE),      # peaked weights; whole tiles of padding
    (2, 600, 2, 128, 256, 0, 0.0),               # the plain mean
    (2, 40000, 2, 128, 2048, 0, SCALE),
    (1, 300, 1, 100, 17, 0, SCALE),
    (1, 300, 200, 128, 129, 1, SCALE),
])
def test_sparse_parity(form, nseq, L, T, Hq, k, pad, scale):
    q, cache, held = _setup(k + T, nseq, L, form, T, Hq)
    idx = _draw_idx(k, T, L, k, pad)
    seq_of = np.arange(T) % nseq
    ws = misa.alloc_workspace(misa.workspace_bytes(misa.OP_SPARSE_MLA_Q, T, Hq, L, 0, k))
    out, lse = misa.sparse_mla_q(q.cuda(), cache, _i32(seq_of), _i32(idx), scale, want_lse=True, workspace=ws)
    assert misa.error_query(ws) == 0
    _check(out, lse, q, held, seq_of, idx, scale)


def test_sparse_empty_rows_repeats_and_bad_ids():
    q, cache, held = _setup(9, 2, 500, "mx8", 5, 128)
    idx = _draw_idx(9, 5, 500, 400, 0)
    idx[0] = -1                       # no valid slot
    idx[1, 128:256] = -1              # a tile without one
    idx[1, :128] = -1                 # ... and the first one
    idx[2, 7] = idx[2, 6]             # listed twice: counts twice
    idx[3] = idx[3][::-1]             # any order
    idx[4, 3], idx[4, 300] = 500, -9
    ws = misa.alloc_workspace(misa.workspace_bytes(misa.OP_SPARSE_MLA_Q, 5, 128, 500, 0, 400))
    seq_of = np.array([0, 1, 0, 1, 0])
    wide = torch.full((5, 411), 12345, dtype=torch.int32)
    wide[:, 4:404] = torch.from_numpy(idx.copy())
    out, lse = misa.sparse_mla_q(q.cuda(), cache, _i32(seq_of), wide.cuda()[:, 4:404], SCALE, want_lse=True, workspace=ws)
    assert misa.error_query(ws) == nat.DEVERR_BAD_INDEX
    assert not out[0].any() and torch.isneginf(lse[0]).all()
    idx[4, 3] = idx[4, 300] = -1
    _check(out, lse, q, held, seq_of, idx, SCALE)


@pytest.mark.parametrize("form", FORMS)
def test_bad_sequence_is_empty(form):
    q, cache, held = _setup(11, 2, 100, form, 3, 128)
    ws = misa.alloc_workspace(misa.workspace_bytes(misa.OP_PREFIX_MLA, 3, 128, 100, 0))
    out, lse = misa.prefix_mla(q.cuda(), cache, _i32([2, 1, -1]), _i32([100, 100, 100]), SCALE, want_lse=True, workspace=ws)
    assert misa.error_query(ws) == nat.DEVERR_BAD_SEQ
    assert not out[0].any() and not out[2].any() and torch.isneginf(lse[0]).all()
    _check(out[1:2], lse[1:2], q[1:2], held, np.array([1]), _prefix_idx([100], 100), SCALE)


@pytest.mark.parametrize("form", FORMS)
def test_rows_past_the_prefix_do_not_matter(form):
    """NaN behind the prefix, and in rows that no query lists, stays there."""
    q, cache, held = _setup(12, 1, 200, form, 2, 128)
    lens = [70, 131]
    cache[0, 131:].view(torch.uint8).fill_(0xFF)
    out, lse = misa.prefix_mla(q.cuda(), cache, _i32([0, 0]), _i32(lens), SCALE, want_lse=True)
    _check(out, lse, q, held, np.zeros(2, np.int64), _prefix_idx(lens, 200), SCALE)
    if form != "bf16":
        idx = _draw_idx(3, 2, 131, 60, 5)
        out, lse = misa.sparse_mla_q(q.cuda(), cache, _i32([0, 0]), _i32(idx), SCALE, want_lse=True)
        _check(out, lse, q, held, np.zeros(2, np.int64), idx, SCALE)


@pytest.mark.parametrize("form", FORMS)
def test_nan_in_a_seen_row_shows(form):
    q, cache, held = _setup(13, 2, 300, form, 2, 128)
    rows = torch.full((2, 1, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    misa.append_kv(cache, _i32([200, 0]), rows, counts=_i32([1, 0]))
    out, lse = misa.prefix_mla(q.cuda(), cache, _i32([0, 1]), _i32([300, 300]), SCALE, want_lse=True)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    _check(out[1:], lse[1:], q[1:], held, np.array([1]), _prefix_idx([300], 300), SCALE)


@pytest.mark.parametrize("form", FORMS)
def test_growing_scores(form):
    """Scores that keep rising along the prefix, by far more than a running
    maximum may lag, and that fall: the sums are carried over rightly."""
    L, Hq = 1500, 128
    g = torch.Generator().manual_seed(14)
    q = torch.randn(2, Hq, 576, generator=g).bfloat16()
    rows = torch.randn(2, L, 576, generator=g) * 0.1
    ramp = torch.linspace(-60, 60, L)
    rows[0, :, 512:] += ramp[:, None]
    rows[1, :, 512:] -= ramp[:, None]
    q[:, :, 512:] = 0.25
    rows = rows.bfloat16()
    cache = misa.alloc_kv_cache(2, L, form)
    misa.append_kv(cache, _i32([0, 0]), rows.cuda())
    held = oracle.latent_values(rows.double().numpy(), form)
    out, lse = misa.prefix_mla(q.cuda(), cache, _i32([0, 1]), _i32([L, L]), SCALE, want_lse=True)
    _check(out, lse, q, held, np.arange(2), _prefix_idx([L, L], L), SCALE)


@pytest.mark.parametrize("form", FORMS)
def test_single_row_is_exact(form):
    q, cache, held = _setup(15, 1, 300, form, 3, 128)
    out, _ = misa.prefix_mla(q.cuda(), cache, _i32([0] * 3), _i32([1] * 3), SCALE)
    assert np.array_equal(out.double().cpu().numpy(), np.broadcast_to(held[0, 0, :512], (3, 128, 512)))
    if form != "bf16":
        idx = np.full((3, 200), -1)
        idx[:, 150] = [5, 299, 0]
        out, _ = misa.sparse_mla_q(q.cuda(), cache, _i32([0] * 3), _i32(idx), SCALE)
        assert np.array_equal(out.double().cpu().numpy()[:, 0], held[0, [5, 299, 0], :512])


@pytest.mark.parametrize("form", FORMS)
def test_same_bits_every_time_and_in_any_batch(form):
    """The same call gives the same bits; a listed prefix gives what the prefix does."""
    q, cache, held = _setup(16, 3, 900, form, 3, 128)
    args = (cache, _i32([0, 1, 2]), _i32([900, 555, 128]), SCALE)
    a, la = misa.prefix_mla(q.cuda(), *args, want_lse=True)
    for _ in range(3):
        b, lb = misa.prefix_mla(q.cuda(), *args, want_lse=True)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_decode_step_in_order():
    """The calls of a decode step, as they are used together: the new token's
    latent row is written, the indexer picks tokens, attention reads them; and the
    dense form beside it.  Eagerly, then captured and replayed on new inputs."""
    T, H, L, B, k, Hq = 4, 64, 640, 128, 256, 128
    g = torch.Generator().manual_seed(17)
    for form in FORMS:
        prompt = torch.randn(T, 600, 576, generator=g).bfloat16()
        lc = misa.LatentCache(T, L, form, T, Hq, k)
        lc.append(prompt.cuda(), counts=_i32([600, 511, 300, 17]))
        keys = torch.randn(T, L, 128, generator=g).bfloat16().cuda()
        ix = misa.DenseIndexer(T, H, L, k)
        qi, w = torch.randn(T, H, 128, generator=g).bfloat16().cuda(), torch.randn(T, H, generator=g).cuda()
        row, q = torch.randn(T, 1, 576, generator=g).bfloat16().cuda(), torch.randn(T, Hq, 576, generator=g).bfloat16().cuda()
        seq = _i32(np.arange(T))
        dense = torch.empty(T, Hq, 512, dtype=torch.bfloat16, device="cuda")

        def step():
            lc.append(row)
            idx = ix.run(qi, w, keys, seq, lc.lens)
            lc.attend_prefix(q, seq, lc.lens, SCALE)
            dense.copy_(lc.out)
            lc.attend(q, seq, idx, SCALE)

        graph = misa.indexer.capture_graph(step)      # runs the step once, eagerly
        held_rows = [list(prompt[b, :n]) + [row[b, 0].cpu()] for b, n in enumerate([600, 511, 300, 17])]
        for i in range(2):
            if i:
                row.copy_(torch.randn(T, 1, 576, generator=g).bfloat16())
                q.copy_(torch.randn(T, Hq, 576, generator=g).bfloat16())
                graph.replay()
                for b in range(T):
                    held_rows[b].append(row[b, 0].cpu())
            lens = [len(r) for r in held_rows]
            assert lc.lens.tolist() == lens
            held = np.zeros((T, L, 576))
            for b in range(T):
                held[b, :lens[b]] = oracle.latent_values(torch.stack(held_rows[b]).double().numpy(), form)
            idx = ix.idx.cpu().numpy()
            # misa_sparse_mla (the bf16 form) sums the weights as it rounded them to bf16: each, and so their sum,
            # is off by at most 2^-8 of itself (a third rounding), its logarithm by 2^-8 (and 2^-16 of second order)
            more = dict(roundings=3, lse_more=1.01 * 2.0 ** -8) if form == "bf16" else {}
            _check(lc.out, lc.lse, q, held, np.arange(T), idx, SCALE, **more)
            _check(dense, None, q, held, np.arange(T), _prefix_idx(lens, L), SCALE)
        for ws in (lc.ws, lc.ws_prefix, lc.ws_sparse):
            assert misa.error_query(ws) == 0


def test_two_graphs_share_a_workspace():
    """Replayed in turn on one stream, two captured calls may share a workspace."""
    L, Hq = 4000, 128
    q, cache, held = _setup(18, 2, L, "mx8", 2, Hq)
    qa, qb = q.cuda(), torch.randn(2, Hq, 576, generator=torch.Generator().manual_seed(3)).bfloat16()
    qb_d = qb.cuda()
    ws = misa.alloc_workspace(misa.workspace_bytes(misa.OP_PREFIX_MLA, 2, Hq, L, 0))
    outs = [torch.empty(2, Hq, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lses = [torch.empty(2, Hq, device="cuda") for _ in range(2)]
    so, lens = _i32([0, 1]), [_i32([L, 1000]), _i32([3, 3333])]
    graphs = [misa.indexer.capture_graph(lambda i=i: misa.prefix_mla((qa, qb_d)[i], cache, so, lens[i], SCALE, out=outs[i],
                                                                   lse=lses[i], workspace=ws)) for i in range(2)]
    for o in outs:
        o.zero_()
    for i in (0, 1, 0):
        graphs[i].replay()
    for i in range(2):
        _check(outs[i], lses[i], (q, qb)[i], held, np.arange(2), _prefix_idx(lens[i].tolist(), L), SCALE)


def test_another_stream_and_workspace_left_to_the_call():
    q, cache, held = _setup(19, 2, 2000, "mx4", 2, 128)
    idx = _draw_idx(1, 2, 2000, 1024, 0)
    s = torch.cuda.Stream()
    qd, so, ix = q.cuda(), _i32([0, 1]), _i32(idx)
    s.wait_stream(torch.cuda.current_stream())
    out, lse = misa.sparse_mla_q(qd, cache, so, ix, SCALE, want_lse=True, stream=s)
    s.synchronize()
    _check(out, lse, q, held, np.arange(2), idx, SCALE)


def test_offsets_behind_2_31():
    """Rows whose byte offset does not fit 32 bits."""
    L = (1 << 31) // 400 + 3000
    cache = torch.zeros((1, L, 400), dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(20)
    rows = torch.randn(1, 300, 576, generator=g).bfloat16()
    misa.append_kv(cache, _i32([L - 300]), rows.cuda())
    q = torch.randn(1, 128, 576, generator=g).bfloat16()
    idx = np.arange(L - 300, L)[None]
    out, lse = misa.sparse_mla_q(q.cuda(), cache, _i32([0]), _i32(idx), SCALE, want_lse=True)
    held = oracle.latent_values(rows.double().numpy(), "mx4")
    _check(out, lse, q, held, np.array([0]), idx - (L - 300), SCALE)
