"""Limits of the latent attention.  Workspaces: one sized for a batch serves every
smaller call (fewer queries, heads, listed tokens or rows), and its size is a formula.
Scales: those whose product with log2(e) fp32 does not hold are refused (the addresses
below are never touched)."""
import pytest

import sparse_attention_token_misa_b200 as misa

OPS = {"sparse": misa.OP_SPARSE_MLA_Q, "prefix": misa.OP_PREFIX_MLA}
SIZES = [1, 2, 3, 63, 64, 65, 128, 129, 256, 511, 1153, 1152, 2047, 2048, 4736, 4737, 8200, 16384, 131072]
QUERIES = [1, 2, 3, 4, 5, 8, 16, 31, 32, 33, 60, 74, 75, 99, 100, 147, 148, 149, 296, 1000, 100000]


def size(op, T, Hq, n):
    return misa.workspace_bytes(OPS[op], T, Hq, 1 << 20, 0, n) if op == "sparse" else misa.workspace_bytes(OPS[op], T, Hq, n, 0)


@pytest.mark.parametrize("op", OPS)
def test_larger_calls_need_no_less(op):
    for T in QUERIES:
        sizes = [size(op, T, 128, n) for n in sorted(SIZES)]
        assert sizes == sorted(sizes), T
    for n in SIZES:
        sizes = [size(op, T, 128, n) for T in QUERIES]
        assert sizes == sorted(sizes), n
    assert [size(op, 4, h, 5000) for h in range(1, 129)] == sorted(size(op, 4, h, 5000) for h in range(1, 129))


@pytest.mark.parametrize("op", OPS)
def test_neighbouring_sizes(op):
    """Where a tile or a cluster more changes the plan."""
    for T in (1, 2, 3, 7, 37):
        sizes = [size(op, T, 128, n) for n in range(1, 8192, 9)]
        assert sizes == sorted(sizes), T
    for n in (2048, 32768, 131072):
        sizes = [size(op, T, 128, n) for T in range(1, 310)]
        assert sizes == sorted(sizes), n


@pytest.mark.parametrize("op", OPS)
def test_formula(op):
    """256 bytes, and 514 floats a head of each partial result: at most 128 a query,
    at most one for each 64 rows, at most 296 in all, and none where a query is whole."""
    for T in QUERIES:
        for n in SIZES:
            parts = [t * min(128, -(-n // 64), 296 // t) for t in range(1, min(T, 148) + 1)
                     if min(128, -(-n // 64), 296 // t) > 1]
            assert size(op, T, 96, n) == 256 + max(parts, default=0) * 96 * 514 * 4, (T, n)


P = 1 << 20


@pytest.mark.parametrize("scale", [2.36e38, 3.4e38])
def test_scales_too_large_are_refused(scale):
    tail = (scale, P, None, P, 1 << 40, None)
    assert misa.lib().misa_sparse_mla_q(P, P, 1, 2, 6560, 10, P, 2, 128, P, 8, 8, *tail) == 2     # unsupported
    assert misa.lib().misa_prefix_mla(P, P, 1, 2, 6560, 10, P, P, 2, 128, *tail) == 2
