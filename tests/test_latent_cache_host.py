"""LatentCache on the host: what it passes to the library's calls, which are replaced
by stand-ins, and what it keeps between them."""
import contextlib

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import sparse_attention_token_misa_b200 as misa
from sparse_attention_token_misa_b200 import _native as nat
from sparse_attention_token_misa_b200 import latent

bf, i32 = torch.bfloat16, torch.int32
FORMS = ["bf16", "mx8", "mx4"]


def cache(form, nseq=2, L=16, T=2, Hq=4, k=8):
    return misa.LatentCache(nseq, L, form, T, Hq, k, device="cpu")


def attention(value):
    """Stands for an attention call: fills the outputs it is given."""
    def call(q, rows, seq_of, per_query, scale, out, lse, workspace, stream=None):
        out.fill_(value); lse.fill_(value)
        return out, lse
    return call


@pytest.fixture
def calls(monkeypatch):
    monkeypatch.setattr(nat, "sparse_mla", attention(1.0))
    monkeypatch.setattr(latent, "sparse_mla_q", attention(1.0))
    monkeypatch.setattr(latent, "prefix_mla", attention(2.0))
    monkeypatch.setattr(latent, "_on", lambda first, stream, *others: contextlib.nullcontext(0))


QUERY = (torch.zeros(2, 4, 576, dtype=bf), torch.zeros(2, dtype=i32))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("listed_first", [True, False])
def test_the_two_results_stand_side_by_side(calls, form, listed_first):
    """The comparison of the listed tokens with the whole prefix: neither call's
    result is the other's.  `out` and `lse` are the last call's."""
    lc = cache(form)
    for name in ("attend", "attend_prefix") if listed_first else ("attend_prefix", "attend"):
        r = getattr(lc, name)(*QUERY, torch.zeros(2, 8, dtype=i32) if name == "attend" else QUERY[1], 0.1)
        assert lc.out is r[0] and lc.lse is r[1]
        if name == "attend":
            listed = r
        else:
            prefix = r
    for a, b in zip(listed, prefix):
        assert (a == 1).all() and (b == 2).all()


def test_bf16_attention_runs_on_the_tensors_device(calls, monkeypatch):
    """sparse_mla launches on the current device: attend makes the cache's device the
    current one around it, and refuses tensors of another, as the other calls do."""
    lc, idx, made = cache("bf16"), torch.zeros(2, 8, dtype=i32), []

    @contextlib.contextmanager
    def on(first, stream, *others):
        made.append((stream, {first.data_ptr(), *(t.data_ptr() for t in others)}))
        yield 77
        made.append("left")

    def sparse_mla(q, rows, seq_of, idx, scale, out, lse, workspace, stream):
        assert len(made) == 1 and stream == 77
        return out, lse

    monkeypatch.setattr(latent, "_on", on)
    monkeypatch.setattr(nat, "sparse_mla", sparse_mla)
    out, lse = lc.attend(*QUERY, idx, 0.1)
    used = {t.data_ptr() for t in (*QUERY, lc.rows, idx, out, lse, lc.ws_sparse)}
    assert made == [(None, used), "left"]


def kernel_rule(lens, n, counts, L):
    """Lengths behind an append by misa_append_kv's rule, one sequence at a time."""
    out = []
    for b, l in enumerate(lens):
        c = n if counts is None else counts[b]
        out.append(l + c if 0 <= c <= n and l >= 0 and l + c <= L else l)
    return out


@pytest.mark.parametrize("n", [1, 3, 16, 17])
def test_lengths_advance_where_rows_were_written(calls, monkeypatch, n):
    """For every length and count at the borders, those out of range included."""
    monkeypatch.setattr(latent, "append_kv", lambda *a, **kw: None)
    top = 2 ** 31 - 1
    lens = [-top - 1, -n, -1, 0, 1, 16 - n, 17 - n, 15, 16, 17, top - 1, top]
    for counts in (None, -top - 1, -1, 0, 1, n - 1, n, n + 1, 16, top):
        lc = cache("mx8", nseq=len(lens))
        lc.lens.copy_(torch.tensor(lens, dtype=i32))
        each = None if counts is None else [counts] * len(lens)
        lc.append(torch.zeros(len(lens), n, 576, dtype=bf), counts=None if each is None else torch.tensor(each, dtype=i32))
        assert lc.lens.tolist() == kernel_rule(lens, n, each, 16), counts


class Fresh(TorchDispatchMode):
    """Counts operations whose result stands in memory that none of their arguments had."""

    def __init__(self):
        super().__init__()
        self.made = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        given = {t.untyped_storage().data_ptr() for t in (*args, *(kwargs or {}).values()) if isinstance(t, torch.Tensor)}
        if isinstance(out, torch.Tensor) and out.untyped_storage().data_ptr() not in given:
            self.made.append(str(func))
        return out


@pytest.mark.parametrize("n", [0, 1, 3, 17])
def test_append_makes_no_tensors(calls, monkeypatch, n):
    monkeypatch.setattr(latent, "append_kv", lambda *a, **kw: None)
    lc, rows = cache("mx8", nseq=4), torch.zeros(4, n, 576, dtype=bf)
    for counts in (None, torch.tensor([0, 1, n, 2], dtype=i32)):
        with Fresh() as f:
            lc.append(rows, counts=counts)
        assert f.made == []
