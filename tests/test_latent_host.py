"""The latent-cache calls on the host: the header and the binding agree, sizes
follow their formula, and bad arguments are refused before anything is launched
(the addresses below are never touched)."""
import os
import re

import pytest
import torch

import sparse_attention_token_misa_b200 as misa
from sparse_attention_token_misa_b200 import _native as nat

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P, MIS = 1 << 20, (1 << 20) + 4
BIG = 1 << 40


def test_header_and_binding_agree():
    text = open(os.path.join(ROOT, "include", "misa_latent.h"), encoding="utf-8").read()
    names = re.findall(r"MISA_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)
    assert len(names) == 5 and set(names) == set(nat.LATENT_SIGNATURES)
    for n in names:
        assert hasattr(misa.lib(), n)
    for name in ("OP_APPEND_KV", "OP_READ_KV", "OP_SPARSE_MLA_Q", "OP_PREFIX_MLA"):
        assert int(re.search(rf"#define MISA_{name} (\d+)", text).group(1)) == getattr(misa, name)


def test_row_bytes():
    assert [misa.kv_row_bytes(f) for f in ("bf16", "mx8", "mx4")] == [1152, 512 + 16 + 128, 256 + 16 + 128]
    assert misa.lib().misa_kv_row_bytes(3) == 0 and misa.lib().misa_kv_row_bytes(-1) == 0
    with pytest.raises(ValueError, match="form"):
        misa.kv_row_bytes("fp6")


def test_workspace_sizes():
    assert misa.workspace_bytes(misa.OP_APPEND_KV, 5, 5, 5, 5) == 256
    assert misa.workspace_bytes(misa.OP_READ_KV, 5, 5, 5, 5) == 256
    assert misa.workspace_bytes(misa.OP_SPARSE_MLA_Q, 3, 16, 0, 0, 0) == 0
    for op in (misa.OP_SPARSE_MLA_Q, misa.OP_PREFIX_MLA):
        sizes = [misa.workspace_bytes(op, T, 128, 4096, 0, 4096) for T in (1, 4, 32)]
        assert all(s >= 256 for s in sizes)


def append(rows=P, nseq=2, n_new=3, counts=None, lens=P, fmt=1, cache=P, stride=656 * 10, L=10, ws=P, wsb=256):
    return misa.lib().misa_append_kv(rows, nseq, n_new, counts, lens, fmt, cache, stride, L, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=None), INVALID), (dict(lens=None), INVALID), (dict(cache=None), INVALID),
    (dict(nseq=0), INVALID), (dict(n_new=0), INVALID), (dict(L=0), INVALID),
    (dict(fmt=3), INVALID), (dict(fmt=-1), INVALID),
    (dict(rows=MIS), INVALID), (dict(cache=MIS), INVALID), (dict(stride=656 * 10 - 8), INVALID),
    (dict(stride=656 * 9), INVALID), (dict(fmt=0), INVALID), (dict(stride=-16), INVALID),
    (dict(nseq=1 << 20, n_new=1 << 12), UNSUPPORTED), (dict(L=1 << 31, stride=1 << 42), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(wsb=255), WORKSPACE), (dict(ws=MIS), INVALID),
])
def test_append_refuses(kw, status):
    assert append(**kw) == status


def read(cache=P, fmt=1, nseq=2, stride=656 * 10, L=10, seq_of=P, T=2, idx=None, idx_stride=0, first=None, plen=None,
         n=4, out=P, ws=P, wsb=256):
    return misa.lib().misa_read_kv(cache, fmt, nseq, stride, L, seq_of, T, idx, idx_stride, first, plen, n, out, ws,
                                   wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(cache=None), INVALID), (dict(seq_of=None), INVALID), (dict(out=None), INVALID), (dict(T=0), INVALID),
    (dict(n=0), INVALID), (dict(idx=P, idx_stride=3), INVALID), (dict(idx=P, idx_stride=4, first=P), INVALID),
    (dict(idx=P, idx_stride=4, plen=P), INVALID), (dict(out=MIS), INVALID), (dict(stride=656 * 9), INVALID),
    (dict(n=1 << 31), UNSUPPORTED), (dict(T=1 << 16, n=1 << 15), UNSUPPORTED), (dict(ws=None), WORKSPACE),
])
def test_read_refuses(kw, status):
    assert read(**kw) == status


def sparse(q=P, cache=P, fmt=1, nseq=2, stride=656 * 10, L=10, seq_of=P, T=2, Hq=128, idx=P, k=8, idx_stride=8,
           scale=0.1, out=P, lse=None, ws=P, wsb=BIG):
    return misa.lib().misa_sparse_mla_q(q, cache, fmt, nseq, stride, L, seq_of, T, Hq, idx, k, idx_stride, scale, out,
                                        lse, ws, wsb, None)


def prefix(q=P, cache=P, fmt=1, nseq=2, stride=656 * 10, L=10, seq_of=P, plen=P, T=2, Hq=128, scale=0.1, out=P,
           lse=None, ws=P, wsb=BIG):
    return misa.lib().misa_prefix_mla(q, cache, fmt, nseq, stride, L, seq_of, plen, T, Hq, scale, out, lse, ws, wsb,
                                      None)


COMMON = [
    (dict(q=None), INVALID), (dict(cache=None), INVALID), (dict(seq_of=None), INVALID), (dict(out=None), INVALID),
    (dict(T=0), INVALID), (dict(Hq=0), INVALID), (dict(Hq=129), UNSUPPORTED), (dict(L=0), INVALID),
    (dict(q=MIS), INVALID), (dict(cache=MIS), INVALID), (dict(out=MIS), INVALID), (dict(stride=656 * 9), INVALID),
    (dict(scale=-0.1), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(T=1 << 24, Hq=128), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(wsb=255), WORKSPACE),
    (dict(fmt=7), INVALID),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(idx=None), INVALID), (dict(k=0), INVALID), (dict(idx_stride=7), INVALID), (dict(k=16385, idx_stride=16385), UNSUPPORTED),
    (dict(fmt=0, stride=1152 * 10), UNSUPPORTED)])
def test_sparse_refuses(kw, status):
    assert sparse(**kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [(dict(plen=None), INVALID)])
def test_prefix_refuses(kw, status):
    assert prefix(**kw) == status


# ------------------------------------------------------------------------ the binding
bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8


def z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses():
    cache = z(2, 10, 656, dtype=u8)
    lens, rows = z(2, dtype=i32), z(2, 3, 576, dtype=bf)
    for bad in (z(2, 10, 655, dtype=u8), z(2, 10, 576, dtype=torch.float16), z(10, 656, dtype=u8)):
        with pytest.raises(ValueError, match="expected shape"):
            misa.append_kv(bad, lens, rows)
    with pytest.raises(ValueError, match="contiguous"):
        misa.append_kv(z(2, 20, 656, dtype=u8)[:, ::2], lens, rows)
    for kw in (dict(rows=z(2, 3, 512, dtype=bf)), dict(rows=z(3, 3, 576, dtype=bf)), dict(lens=z(3, dtype=i32)),
               dict(counts=z(3, dtype=i32))):
        with pytest.raises(ValueError, match="expected"):
            misa.append_kv(cache, **{"lens": lens, "rows": rows, **kw})
    with pytest.raises(TypeError):
        misa.append_kv(cache, z(2, dtype=torch.int64), rows)
    so = z(2, dtype=i32)
    for kw in (dict(), dict(idx=z(2, 4, dtype=i32), first=so), dict(idx=z(3, 4, dtype=i32)),
               dict(n=4, first=z(3, dtype=i32)), dict(n=4, out=z(2, 3, 576, dtype=bf))):
        with pytest.raises(ValueError):
            misa.read_kv(cache, so, **kw)
    q, idx = z(2, 128, 576, dtype=bf), z(2, 8, dtype=i32)
    with pytest.raises(ValueError, match="sparse_mla reads bf16"):
        misa.sparse_mla_q(q, z(2, 10, 576, dtype=bf), so, idx, 0.1)
    for bad in (-1.0, float("nan")):
        with pytest.raises(ValueError, match="scale"):
            misa.sparse_mla_q(q, cache, so, idx, bad)
    for kw in (dict(q=z(2, 128, 512, dtype=bf)), dict(idx=z(3, 8, dtype=i32)), dict(seq_of=z(1, dtype=i32)),
               dict(out=z(2, 128, 576, dtype=bf)), dict(lse=z(2, 127))):
        with pytest.raises(ValueError, match="expected"):
            misa.sparse_mla_q(**{"q": q, "cache": cache, "seq_of": so, "idx": idx, "scale": 0.1, **kw})
    with pytest.raises(ValueError, match="expected"):
        misa.prefix_mla(q, cache, so, z(3, dtype=i32), 0.1)


def test_binding_stops_at_cpu_tensors():
    cache, so = z(2, 10, 656, dtype=u8), z(2, dtype=i32)
    for call in (lambda: misa.append_kv(cache, so, z(2, 3, 576, dtype=bf)), lambda: misa.read_kv(cache, so, n=3),
                 lambda: misa.prefix_mla(z(2, 4, 576, dtype=bf), cache, so, so, 0.1),
                 lambda: misa.sparse_mla_q(z(2, 4, 576, dtype=bf), cache, so, z(2, 8, dtype=i32), 0.1)):
        with pytest.raises(ValueError, match="device tensors"):
            call()
