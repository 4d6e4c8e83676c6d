"""What is measured of the latent key/value cache and the attention that reads it.

A latent row is 576 numbers, one row a token, shared by every query head: 512
latent entries and 64 rotary ones.  Keys are whole rows, values their first 512
entries.  A cache holds its rows in one of three forms:

* "bf16": the row as it is, 1152 bytes;
* "mx8": the 512 latent entries as e4m3 numbers in 16 groups of 32, each group
  with a power-of-two scale (one byte, the exponent + 127), then the 64 rotary
  entries in bf16: 512 + 16 + 128 = 656 bytes;
* "mx4": the same with e2m1 numbers, two a byte, the even entry in the low half:
  256 + 16 + 128 = 400 bytes.

A group's scale is 2^e with the smallest e for which no entry is above the
largest number of the element type (448 or 6), e within [-117, 119] (mx8) or
[-117, 125] (mx4); entries are rounded to nearest, ties to even.

The operators:

* write:  append_kv puts new rows into a cache, read_kv reads them back (what the
          cache holds is returned as the values it stands for);
* read:   read_kv of listed rows, or of a range of rows;
* sparse: sparse_mla_q, attention of every query head over its query's listed rows;
* prefix: prefix_mla, attention over all rows of a query's prefix.

    out[t, h] = sum_i p_i v_i / sum_i p_i,  p_i = exp(scale q[t, h] . k_i),
    lse[t, h] = log sum_i p_i.
"""
import math

import numpy as np
import torch

own = False

DQK, DV, GROUP = 576, 512, 32
NGROUPS = DV // GROUP
ROW_BYTES = {"bf16": 2 * DQK, "mx8": DV + NGROUPS + 128, "mx4": DV // 2 + NGROUPS + 128}
ELEM_MAX = {"mx8": 448.0, "mx4": 6.0}
E_RANGE = {"mx8": (-117, 119), "mx4": (-117, 125)}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SCALE = 192 ** -0.5    # 128 + 64 entries of a query-key product before the projection is absorbed


# ------------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step writes one token's row to each of 32 caches
        {"name": "write mx8, 32 x 1 row", "op": "write", "fmt": "mx8", "nseq": 32, "L": 4096, "n": 1},
        # four prompts of different lengths go into their caches
        {"name": "write mx4, 4 prompts", "op": "write", "fmt": "mx4", "nseq": 4, "L": 8200, "n": 8191},
        # the selected rows of a decode batch read back (32 sequences of 32768, 2048 of each)
        {"name": "read mx8, 32 x 2048 listed", "op": "read", "fmt": "mx8", "nseq": 32, "L": 32768, "n": 2048,
         "listed": True},
        # a stored prompt read back whole before its continuation
        {"name": "read mx4, 2 x 40001 rows", "op": "read", "fmt": "mx4", "nseq": 2, "L": 40001, "n": 40001,
         "listed": False},
        # the decode step behind the indexer: 32 sequences, 2048 selected tokens each
        {"name": "sparse mx8, decode", "op": "sparse", "fmt": "mx8", "nseq": 32, "L": 32768, "T": 32, "Hq": 128,
         "k": 2048},
        # the smallest call: one token, few heads on this GPU, a short selection
        {"name": "sparse mx4, one token", "op": "sparse", "fmt": "mx4", "nseq": 1, "L": 1000, "T": 1, "Hq": 16,
         "k": 256},
        # a prompt's chunk behind the indexer: 1024 queries over one shared cache
        {"name": "sparse mx4, prompt chunk", "op": "sparse", "fmt": "mx4", "nseq": 1, "L": 32768, "T": 1024,
         "Hq": 128, "k": 2048},
        # one sequence that is shorter than the selection: every token is attended
        {"name": "prefix bf16, one token", "op": "prefix", "fmt": "bf16", "nseq": 1, "L": 777, "T": 1, "Hq": 128},
        # a decode batch of short contexts of different lengths
        {"name": "prefix bf16, decode", "op": "prefix", "fmt": "bf16", "nseq": 32, "L": 4096, "T": 32, "Hq": 128},
        # a whole prompt of 2047 tokens, each attending to those up to itself
        {"name": "prefix bf16, prompt", "op": "prefix", "fmt": "bf16", "nseq": 1, "L": 2047, "T": 2047, "Hq": 128},
        # the dense comparison at the benchmark's context length
        {"name": "prefix mx8, long decode", "op": "prefix", "fmt": "mx8", "nseq": 16, "L": 32768, "T": 16,
         "Hq": 128},
        # few long sequences, half of the heads on this GPU
        {"name": "prefix mx4, 131071 tokens", "op": "prefix", "fmt": "mx4", "nseq": 4, "L": 131071, "T": 4, "Hq": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["write", "read", "sparse", "sparse", "prefix", "prefix"])
        fmt = rng.choice(["mx8", "mx4"] if op == "sparse" else ["bf16", "mx8", "mx4"])
        L = _log(rng, 100, 131072)
        case = {"op": op, "fmt": fmt, "nseq": _log(rng, 1, 64), "L": L}
        if op == "write":
            case["n"] = min(L, _log(rng, 1, 8192))
        elif op == "read":
            case["listed"] = rng.random() < 0.5
            case["n"] = min(L, _log(rng, 1, 4096)) if case["listed"] else L
        else:
            case["Hq"] = rng.choice([8, 16, 20, 32, 64, 96, 128, 128])
            if rng.random() < 0.3:   # one shared cache: a prompt or a part of one
                case["nseq"], case["T"] = 1, min(L, _log(rng, 2, 2048))
            else:
                case["T"] = case["nseq"]
            if op == "sparse":
                case["k"] = min(L, _log(rng, 1, 4096))
        w = work(case)
        if case["nseq"] * L * ROW_BYTES[fmt] <= 9e8 and w["bytes"] <= 2.5e8 and w["flops"] <= 4e11:
            return case


# ------------------------------------------------------------------------ shapes
def _lens(case):
    """What each query sees: the rows up to itself where queries share a cache,
    else lengths between half of the cache and all of it."""
    T, L = case["T"], case["L"]
    if T > 1 and case["nseq"] == 1:
        return [L - T + 1 + t for t in range(T)]
    return [L - (t * (L // 2)) // T for t in range(T)]


def _counts(case):
    """New rows of each sequence: n, or, in prompts, lengths between half of n and n."""
    nseq, n = case["nseq"], case["n"]
    return [n - (b * (n // 2)) // nseq for b in range(nseq)]


def work(case):
    fmt, rb = case["fmt"], ROW_BYTES[case["fmt"]]
    if case["op"] == "write":
        rows = sum(_counts(case))
        return {"bytes": rows * (2 * DQK + rb) + case["nseq"] * case["n"] * 2 * DQK, "flops": 4 * rows * DV}
    if case["op"] == "read":
        rows = case["nseq"] * case["n"]
        return {"bytes": rows * (rb + 2 * DQK + (4 if case["listed"] else 0)), "flops": 2 * rows * DV}
    T, Hq = case["T"], case["Hq"]
    seen = [min(n, case["k"]) for n in _lens(case)] if case["op"] == "sparse" else _lens(case)
    total = sum(seen)
    rows = min(total, case["L"]) if case["nseq"] == 1 else total
    extra = T * case["k"] * 4 if case["op"] == "sparse" else T * 4
    return {"bytes": rows * rb + T * Hq * (2 * DQK + 2 * DV + 4) + extra, "flops": 2 * Hq * (DQK + DV) * total}


# ------------------------------------------------------------------------ the cache's forms, plainly
def _encode(rows, fmt):
    """Rows [..., 576] bf16 -> what a cache of this form holds."""
    if fmt == "bf16":
        return rows
    x = rows[..., :DV].float().reshape(*rows.shape[:-1], NGROUPS, GROUP)
    m, e = torch.frexp(x.abs().amax(-1))                    # amax = m 2^e, m in [0.5, 1)
    top = 8 if fmt == "mx8" else 2                          # 448 = 1.75 2^8, 6 = 1.5 2^2
    e = e - 1 - top + (m > (0.875 if fmt == "mx8" else 0.75)).int()
    e = torch.where(m == 0, torch.full_like(e, -127), e).clamp(*E_RANGE[fmt])
    y = torch.ldexp(x, -e.unsqueeze(-1)).reshape(*rows.shape[:-1], DV)
    if fmt == "mx8":
        code = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        a = y.abs()
        c = (torch.signbit(y) * 8).to(torch.uint8)
        for limit, tie_up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                              (5.0, False)):
            c += (a >= limit) if tie_up else (a > limit)
        code = c[..., 0::2] | (c[..., 1::2] << 4)
    rope = rows[..., DV:].contiguous().view(torch.uint8)
    return torch.cat([code, (e + 127).to(torch.uint8), rope], -1)


def _decode(held, fmt):
    """What a cache of this form holds -> rows [..., 576] fp32."""
    if fmt == "bf16":
        return held.float()
    ncode = DV if fmt == "mx8" else DV // 2
    code, scale = held[..., :ncode], held[..., ncode:ncode + NGROUPS]
    rope = held[..., ncode + NGROUPS:].contiguous().view(torch.bfloat16).float()
    if fmt == "mx8":
        v = code.contiguous().view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float32, device=held.device)
        v = table[torch.stack([code & 15, code >> 4], -1).long()].reshape(*code.shape[:-1], DV)
    s = torch.exp2(scale.float() - 127.0)
    v = (v.reshape(*v.shape[:-1], NGROUPS, GROUP) * s.unsqueeze(-1)).reshape(*v.shape[:-1], DV)
    return torch.cat([v, rope], -1)


# ------------------------------------------------------------------------ inputs
def _rows(gen, *shape):
    """Latent rows: a normalised latent, a few entries of which are habitually
    large, and tokens that differ in size; rotary entries of unit size."""
    x = torch.randn(*shape, DQK, generator=gen, device="cuda")
    x[..., 5:DV:97] *= 6.0
    x[..., :DV] *= 0.5 + torch.rand(*shape, 1, generator=gen, device="cuda")
    return x.bfloat16()


def _cache(gen, case):
    out = None
    for b in range(case["nseq"]):
        for s in range(0, case["L"], 65536):
            e = min(case["L"], s + 65536)
            held = _encode(_rows(gen, e - s), case["fmt"])
            if out is None:
                out = torch.empty((case["nseq"], case["L"], held.shape[-1]), dtype=held.dtype, device="cuda")
            out[b, s:e] = held
    return out


def _ids(gen, n_rows, seen, k):
    """k distinct ids below `seen`, ascending, -1 behind the last."""
    m = min(seen, k)
    ids = torch.full((k,), -1, dtype=torch.int32, device="cuda")
    ids[:m] = torch.rand(seen, generator=gen, device="cuda").topk(m).indices.sort().values.int()
    return ids


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    d = {"case": case, "cache": _cache(gen, case)}
    nseq, L = case["nseq"], case["L"]
    if case["op"] == "write":
        n = case["n"]
        d["rows"] = _rows(gen, nseq, n)
        d["lens"] = torch.randint(0, L - n + 1, (nseq,), generator=gen, **i32)
        d["counts"] = torch.tensor(_counts(case), **i32)
        d["seq_of"] = torch.arange(nseq, **i32)
        d["end"] = d["lens"] + d["counts"]
    elif case["op"] == "read":
        d["seq_of"] = torch.arange(nseq, **i32)
        if case["listed"]:
            d["idx"] = torch.stack([_ids(gen, L, L, case["n"]) for _ in range(nseq)])
    else:
        T = case["T"]
        d["q"] = torch.randn(T, case["Hq"], DQK, generator=gen, device="cuda").bfloat16()
        d["seq_of"] = torch.arange(T, **i32) if nseq > 1 else torch.zeros(T, **i32)
        lens = _lens(case)
        d["prefix_len"] = torch.tensor(lens, **i32)
        if case["op"] == "sparse":
            d["idx"] = torch.stack([_ids(gen, L, seen, case["k"]) for seen in lens])
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    if own:
        import sparse_attention_token_misa_b200 as misa
        d["ws"] = misa.alloc_workspace(256)
        if case["op"] in ("sparse", "prefix"):
            op = misa.OP_SPARSE_MLA_Q if case["op"] == "sparse" else misa.OP_PREFIX_MLA
            k = case["k"] if case["op"] == "sparse" else 0
            d["ws"] = misa.alloc_workspace(misa.workspace_bytes(op, case["T"], case["Hq"], case["L"], 0, k))
    return d


# ------------------------------------------------------------------------ one pass
def run(d):
    return _run_own(d) if own else _run_plain(d)


def _run_own(d):
    import sparse_attention_token_misa_b200 as misa
    case = d["case"]
    if case["op"] == "write":
        misa.append_kv(d["cache"], d["lens"], d["rows"], counts=d["counts"], workspace=d["ws"])
        return misa.read_kv(d["cache"], d["seq_of"], first=d["lens"], n=case["n"], prefix_len=d["end"],
                            workspace=d["ws"])
    if case["op"] == "read":
        if case["listed"]:
            return misa.read_kv(d["cache"], d["seq_of"], idx=d["idx"], workspace=d["ws"])
        return misa.read_kv(d["cache"], d["seq_of"], n=case["n"], workspace=d["ws"])
    if case["op"] == "sparse":
        return misa.sparse_mla_q(d["q"], d["cache"], d["seq_of"], d["idx"], SCALE, want_lse=True, workspace=d["ws"])
    return misa.prefix_mla(d["q"], d["cache"], d["seq_of"], d["prefix_len"], SCALE, want_lse=True, workspace=d["ws"])


def _run_plain(d):
    case, cache = d["case"], d["cache"]
    fmt = case["fmt"]
    if case["op"] == "write":
        n = case["n"]
        place = d["lens"].long()[:, None] + torch.arange(n, device="cuda")
        new = torch.arange(n, device="cuda") < d["counts"][:, None]
        b, i = torch.nonzero(new, as_tuple=True)
        cache[b, place[b, i]] = _encode(d["rows"], fmt)[b, i]
        back = _decode(cache[d["seq_of"].long()[:, None], place], fmt).bfloat16()
        return torch.where(new[..., None], back, torch.zeros_like(back))
    if case["op"] == "read":
        if case["listed"]:
            return _decode(cache[d["seq_of"].long()[:, None], d["idx"].long()], fmt).bfloat16()
        return _decode(cache[:, :case["n"]], fmt).bfloat16()
    T, Hq, L = case["T"], case["Hq"], case["L"]
    out = torch.empty((T, Hq, DV), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((T, Hq), dtype=torch.float32, device="cuda")
    shared = _decode(cache[0], fmt) if case["nseq"] == 1 else None
    width = case["k"] if case["op"] == "sparse" else L
    step = max(1, 1 << 28 >> max(1, (width * max(Hq, DQK) - 1).bit_length()))   # about 1 GB of fp32 at a time
    for t in range(0, T, step):
        u = min(T, t + step)
        q = d["q"][t:u].float()
        if case["op"] == "sparse":
            ids = d["idx"][t:u].long()
            hidden = ids < 0
            ids = ids.clamp(min=0)
            kv = shared[ids] if shared is not None else _decode(cache[d["seq_of"][t:u].long()[:, None], ids], fmt)
        else:
            kv = shared if shared is not None else _decode(cache[d["seq_of"][t:u].long()], fmt)
            hidden = torch.arange(L, device="cuda") >= d["prefix_len"][t:u, None]
        s = (q @ kv.transpose(-1, -2)) * SCALE
        s = s.masked_fill(hidden[:, None, :], -math.inf)
        top = s.amax(-1, keepdim=True)
        p = torch.exp(s - top)
        total = p.sum(-1, keepdim=True)
        out[t:u] = ((p @ kv[..., :DV]) / total).bfloat16()
        lse[t:u] = (top + torch.log(total))[..., 0]
    return out, lse


# ------------------------------------------------------------------------ 64 bits, from the definition
def _value64(x, quantum_floor, bits, largest):
    """x rounded to a binary number of `bits` bits after its leading one, whose
    quanta stop shrinking at quantum_floor: nearest, ties to even."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(divide="ignore"):
        lead = np.floor(np.log2(np.abs(x), where=x != 0, out=np.full(x.shape, -200.0)))
    q = np.maximum(2.0 ** (lead - bits), quantum_floor)
    return np.clip(np.rint(x / q) * q, -largest, largest)


def _held64(rows, fmt):
    """The values, in 64 bits, that a cache holds of these rows (a numpy array [..., 576])."""
    rows = np.asarray(rows, dtype=np.float64)
    if fmt == "bf16":
        return rows
    out = rows.copy()
    lo, hi = E_RANGE[fmt]
    for g in range(NGROUPS):
        part = rows[..., g * GROUP:(g + 1) * GROUP]
        amax = np.abs(part).max(-1, keepdims=True)
        scale = 2.0 ** np.clip(np.ceil(np.log2(np.maximum(amax, 1e-300) / ELEM_MAX[fmt])), lo, hi)
        grid = (2.0 ** -9, 3, 448.0) if fmt == "mx8" else (0.5, 1, 6.0)
        out[..., g * GROUP:(g + 1) * GROUP] = _value64(part / scale, *grid) * scale
    return out


def _stands_for64(held, fmt):
    """Cache bytes [n, row] -> the numbers they stand for, [n, 576] in 64 bits."""
    if fmt == "bf16":
        return held.double()
    half = 1 if fmt == "mx8" else 2
    code = held[:, :DV // half]
    if half == 2:
        code = torch.stack([code & 15, code // 16], 2).reshape(len(held), DV)
        man, exp, sign, bias, nman = code & 1, (code >> 1) & 3, code >> 3, 1, 1
    else:
        man, exp, sign, bias, nman = code & 7, (code >> 3) & 15, code >> 7, 7, 3
    man, exp, sign = man.double(), exp.double(), sign.double()
    mag = torch.where(exp == 0, man * 2.0 ** (1 - bias - nman), (1 + man / 2 ** nman) * 2.0 ** (exp - bias))
    at = DV // half
    power = 2.0 ** (held[:, at:at + NGROUPS].double() - 127)
    latent = (1 - 2 * sign) * mag * power.repeat_interleave(GROUP, 1)
    bits = held[:, at + NGROUPS:].to(torch.int32)
    rope = ((bits[:, 0::2] + bits[:, 1::2] * 256) * 65536).view(torch.float32).double()
    return torch.cat([latent, rope], 1)


def exact(case, seed):
    d = _inputs(case, seed)
    fmt, cache = case["fmt"], d["cache"]
    if case["op"] == "write":
        back = torch.zeros(d["rows"].shape, dtype=torch.float64, device="cuda")
        for b, c in enumerate(_counts(case)):
            back[b, :c] = torch.from_numpy(_held64(d["rows"][b, :c].double().cpu().numpy(), fmt)).cuda()
        return back
    if case["op"] == "read":
        return torch.stack([_stands_for64(cache[b][d["idx"][b].long()] if case["listed"] else cache[b, :case["n"]], fmt)
                            for b in range(case["nseq"])])
    out = torch.empty((case["T"], case["Hq"], DV), dtype=torch.float64, device="cuda")
    lse = torch.empty((case["T"], case["Hq"]), dtype=torch.float64, device="cuda")
    whole = _stands_for64(cache[0], fmt) if case["nseq"] == 1 else None
    for t, n in enumerate(_lens(case)):
        if case["op"] == "sparse":
            ids = d["idx"][t][d["idx"][t] >= 0].long()
            rows = whole[ids] if whole is not None else _stands_for64(cache[t][ids], fmt)
        else:
            rows = whole[:n] if whole is not None else _stands_for64(cache[t, :n], fmt)
        s = torch.einsum("hd,nd->hn", d["q"][t].double(), rows) * SCALE
        lse[t] = torch.logsumexp(s, 1)
        out[t] = torch.einsum("hn,nd->hd", torch.exp(s - lse[t][:, None]), rows[:, :DV])
    return out, lse
