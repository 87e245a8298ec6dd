"""Cases of the operators of a latent cache held in 4 bits: rows quantised as
they are written into its pages, rows read back out of a paged cache (of 4 bits,
e4m3 or bf16), and the decode over it.

Each case is one pass through one operator, in its plain form (elementary torch
operations in 32 bits, rounded once at the end) or, with ``own`` set, through
the library.

A row of the 4-bit cache is 304 bytes: the 512 latent values and the 64 rope
values in 18 groups of 32, each value one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a
sign, times 2^(E - k) with an exponent E of the row and a shift k of the group.
  bytes 0 .. 287     72 words of 8 values: the index of value i's magnitude in
                     bits 4i .. 4i + 2; the signs of values 0 .. 3 in bits 8i + 7,
                     of values 4 .. 7 in bits 8 (i - 4) + 3
  bytes 288 .. 296   the shifts k (0 .. 14), 4 bits each, the lower half first
  byte 297           E + 127, E from -32 to 63; 255 in a row that held a NaN
  bytes 298 .. 303   zero
"""
import math

import numpy as np
import torch

own = False

D_CKV, D_KPE, D = 512, 64, 576
ROW, GROUPS = 304, 18
E_MIN, E_MAX, K_MAX = -32, 63, 14
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
INF = float("inf")
DTYPES = dict(bf16=torch.bfloat16, fp16=torch.float16, fp32=torch.float32)
SIZES = dict(bf16=2, fp16=2, fp32=4, fp8=1)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the new token of each request of a decode step
        dict(name="write_decode", op="write", tokens=64, page_size=64, dtype="bf16", padded=0),
        # a prefill chunk, its last places padded
        dict(name="write_prefill", op="write", tokens=8190, page_size=64, dtype="bf16", padded=2),
        # a long prompt whose rows a pass before left in 32 bits
        dict(name="write_long", op="write", tokens=131000, page_size=32, dtype="fp32", padded=0),
        # the context that a short chunk of a few requests attends to
        dict(name="read_small", op="read", batch=4, ctx=500, page_size=64, cache="q4", dtype="bf16", skip=0),
        # long contexts brought back for a prefill that multiplies them out
        dict(name="read_long", op="read", batch=16, ctx=8192, page_size=64, cache="q4", dtype="bf16", skip=0),
        # the same out of an e4m3 cache, the tokens past a first part that is there already
        dict(name="read_fp8", op="read", batch=16, ctx=8000, page_size=32, cache="fp8", dtype="fp16", skip=1000),
        # a small batch of one of eight head groups
        dict(name="decode_small", op="decode", batch=4, heads=16, ctx=2000, ragged=True, page_size=64, q_len=1),
        # long contexts, one of eight head groups
        dict(name="decode_long", op="decode", batch=4, heads=16, ctx=131072, ragged=False, page_size=64, q_len=1),
        # the same with four query tokens for each request (drafted tokens checked at once)
        dict(name="decode_drafted", op="decode", batch=4, heads=16, ctx=65536, ragged=True, page_size=32, q_len=4),
        # a decode batch with all heads
        dict(name="decode_batch", op="decode", batch=64, heads=128, ctx=4096, ragged=False, page_size=64, q_len=1),
        # many requests of all lengths in small pages
        dict(name="decode_ragged", op="decode", batch=128, heads=128, ctx=8192, ragged=True, page_size=16, q_len=1),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode"])
    page_size = rng.choice([16, 32, 64])
    if op == "write":
        tokens = _log_int(rng, 1, 131000)
        return dict(op=op, tokens=tokens, page_size=page_size, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    padded=rng.randint(0, tokens // 8))
    if op == "read":
        batch = _log_int(rng, 1, 64)
        ctx = _log_int(rng, 1, 131072 // batch)
        return dict(op=op, batch=batch, ctx=ctx, page_size=page_size, cache=rng.choice(["q4", "q4", "fp8", "bf16"]),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), skip=rng.randint(0, ctx // 2))
    batch = _log_int(rng, 1, 64)
    heads = rng.choice([1, 8, 16, 20, 32, 40, 64, 128])
    return dict(op=op, batch=batch, heads=heads, ctx=_log_int(rng, 8, min(131072, 524288 // batch)),
                ragged=rng.random() < 0.5, page_size=page_size,
                q_len=rng.choice([1, 1, 2, 4]) if heads <= 32 else 1)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _randint(g, lo, hi, *shape, dtype=torch.int32):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=dtype)


def _indptr(counts):
    out = torch.zeros(counts.numel() + 1, dtype=torch.int32, device="cuda")
    out[1:] = counts.cumsum(0)
    return out


def _channels(g):
    """The spread of the dims' magnitudes: most alike, a few that stand out."""
    c = torch.exp(0.4 * _randn(g, D))
    c[_randint(g, 0, D, 6).long()] *= 6.0
    return c


def _random_rows(g, n, dtype):
    return (_randn(g, n, D) * _channels(g)).to(dtype)


def _random_cache(g, pages, page_size, kind):
    """A paged cache: (rows of 4 bits, None), or (latent part, rope part)."""
    n = pages * page_size
    c = _channels(g)
    if kind == "q4":
        cache = torch.empty(n, ROW, dtype=torch.uint8, device="cuda")
        for i in range(0, n, 65536):
            cache[i:i + 65536] = _pack(_randn(g, min(65536, n - i), D) * c)
        return cache.view(pages, page_size, ROW), None
    x = (_randn(g, n, D, dtype=torch.bfloat16) * c.to(torch.bfloat16)).view(pages, page_size, D)
    if kind == "fp8":
        x = (x.float() / _scale(kind)).clamp_(-448, 448).to(torch.float8_e4m3fn)
        return x[..., :D_CKV].contiguous(), x[..., D_CKV:].contiguous()
    return x[..., :D_CKV].contiguous(), x[..., D_CKV:].contiguous()


def _scale(kind):
    return 0.125 if kind == "fp8" else 1.0


def _prepare_write(case, g):
    T, P = case["tokens"], case["page_size"]
    pages = max(4, -(-3 * T // (2 * P))) + 1                  # the last page takes no token
    x = _random_rows(g, T, DTYPES[case["dtype"]])            # the latent projection's output, normed and turned
    slots = torch.randperm((pages - 1) * P, generator=g, device="cuda")[:T].to(torch.int64)
    if case["padded"]:
        slots[T - case["padded"]:] = -1
    cache = _randint(g, 0, 256, pages, P, ROW, dtype=torch.uint8)
    return dict(ckv=x[:, :D_CKV], kpe=x[:, D_CKV:], slots=slots, cache=cache)


def _page_table(g, counts, spare):
    """Page lists of `counts` pages each out of a pool with `spare` more."""
    total = int(counts.sum())
    return _indptr(counts), torch.randperm(total + spare, generator=g, device="cuda")[:total].to(torch.int32)


def _read_ranges(case):
    """The contexts, from half the longest up, and where the rows of each begin."""
    B, ctx = case["batch"], case["ctx"]
    lens = [ctx - b * (ctx // 2) // B for b in range(B)]
    return lens, [min(37 * b % (case["skip"] + 1) if b else case["skip"], n - 1) for b, n in enumerate(lens)]


def _prepare_read(case, g):
    P = case["page_size"]
    lens, starts = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in _read_ranges(case))
    kv_indptr, kv_indices = _page_table(g, (lens + P - 1) // P, 3)
    pages = kv_indices.numel() + 3
    cache, kpe = _random_cache(g, pages, P, case["cache"])
    rows = lens - starts
    n = int(rows.sum()) + 5                                   # a few rows that no request fills
    dtype = DTYPES[case["dtype"]]
    return dict(cache=cache, kpe_cache=kpe, kind=case["cache"], page_size=P, kv_indptr=kv_indptr,
                kv_indices=kv_indices, starts=starts, row_indptr=_indptr(rows), kv_scale=_scale(case["cache"]),
                ckv_out=torch.zeros(n, D_CKV, dtype=dtype, device="cuda"),
                kpe_out=torch.zeros(n, D_KPE, dtype=dtype, device="cuda"))


def _prepare_decode(case, g):
    B, H, P, Q = case["batch"], case["heads"], case["page_size"], case["q_len"]
    lens = torch.full((B,), case["ctx"], dtype=torch.int32, device="cuda")
    if case["ragged"]:
        lens = _randint(g, Q, case["ctx"] + 1, B)
        lens[0] = case["ctx"]
    counts = (lens + P - 1) // P
    kv_indptr, kv_indices = _page_table(g, counts, 3)
    cache, _ = _random_cache(g, kv_indices.numel() + 3, P, "q4")
    # what lies behind a request's last token is left of other requests, or of nothing: NaN rows
    last = kv_indices[(kv_indptr[1:] - 1).long()].long()
    behind = torch.arange(P, device="cuda")[None] >= (lens - (counts - 1) * P)[:, None]
    cache[last] = torch.where(behind[..., None], 255, cache[last].int()).to(torch.uint8)
    q = _randn(g, B, Q, H, D).to(torch.bfloat16)
    if Q == 1:
        q = q[:, 0]
    state = dict(q_nope=q[..., :D_CKV].contiguous(), q_pe=q[..., D_CKV:].contiguous(), cache=cache, page_size=P,
                 q_len=Q, sm_scale=1 / math.sqrt(192.0), kv_indices=kv_indices, kv_indptr=kv_indptr.tolist(),
                 kv_len=lens.tolist())
    if own:                       # the plan that a serving loop keeps for the layers of a step
        from paged_mla_decode_02_gb300 import mla
        dec = mla.MLADecoder(B * Q, H, kernel="q4")
        dec.plan(state["kv_indptr"], kv_indices, state["kv_len"], P, state["sm_scale"], q_len=Q if Q > 1 else 0)
        state["decoder"] = dec
    return state


_PREPARE = dict(write=_prepare_write, read=_prepare_read, decode=_prepare_decode)


def prepare(case, seed):
    state = _PREPARE[case["op"]](case, _gen(seed))
    state["op"] = case["op"]
    return state


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _sign_shifts(device):
    return torch.tensor([7, 15, 23, 31, 3, 11, 19, 27], dtype=torch.int32, device=device)


def _pack(x):
    """fp32 rows [n, 576] -> their bytes [n, 304]."""
    n = x.shape[0]
    x = x.view(n, GROUPS, 32)
    nan = x.isnan().flatten(1).any(1)
    top = x.abs().nan_to_num(0.0, posinf=torch.finfo(torch.float32).max).amax(2)
    m, e = torch.frexp(top)                                   # top = m 2^e with m in [0.5, 1)
    e = torch.where(top > 0, e - torch.where(m <= 0.75, 3, 2), -1000)    # the least e with top <= 6 * 2^e
    row_e = e.amax(1).clamp(E_MIN, E_MAX)
    k = (row_e[:, None] - e).clamp(0, K_MAX)
    y = torch.ldexp(x, (k - row_e[:, None])[..., None])
    a = y.abs()
    mag = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
           + (a >= 3.5).int() + (a > 5).int())
    mag, sign = mag.view(n, 72, 8), torch.signbit(x).int().view(n, 72, 8)
    at = torch.arange(8, dtype=torch.int32, device=x.device)
    words = ((mag << 4 * at) | (sign << _sign_shifts(x.device))).sum(2, dtype=torch.int32)
    out = torch.zeros(n, ROW, dtype=torch.uint8, device=x.device)
    out[:, :288] = words.view(torch.uint8)
    out[:, 288:297] = (k[:, 0::2] | (k[:, 1::2] << 4)).to(torch.uint8)
    out[:, 297] = torch.where(nan, 255, row_e + 127).to(torch.uint8)
    return torch.where(nan[:, None] & (torch.arange(ROW, device=x.device) != 297), 0, out)


def _unpack(rows):
    """The bytes of rows [n, 304] -> fp32 [n, 576]."""
    n = rows.shape[0]
    words = rows[:, :288].contiguous().view(torch.int32).view(n, 72, 1)
    at = torch.arange(8, dtype=torch.int32, device=rows.device)
    table = torch.tensor(MAGNITUDES, device=rows.device)
    v = table[((words >> 4 * at) & 7).long()]
    v = torch.where(((words >> _sign_shifts(rows.device)) & 1) != 0, -v, v).view(n, GROUPS, 32)
    half = rows[:, 288:297].int()
    k = torch.stack([half & 15, half >> 4], 2).view(n, GROUPS)
    e = rows[:, 297].int()
    v = torch.ldexp(v, (e[:, None] - 127 - k)[..., None]).view(n, D)
    return torch.where(e[:, None] == 255, math.nan, v)


def _plain_write(s):
    flat, slots = s["cache"].view(-1, ROW), s["slots"]
    packed = _pack(torch.cat([s["ckv"], s["kpe"]], 1).float())
    spare = flat.shape[0] - 1                                 # no token's slot: takes the padded ones
    kept = flat[spare].clone()
    flat.index_copy_(0, torch.where(slots >= 0, slots, spare), packed)
    flat[spare] = kept
    return s["cache"]                                         # its bytes: whole numbers


def _plain_read(s):
    P = s["page_size"]
    n = s["ckv_out"].shape[0]
    i = torch.arange(n, device="cuda")
    real = (i < s["row_indptr"][-1])[:, None]
    b = torch.searchsorted(s["row_indptr"][1:].long(), i, right=True).clamp(max=s["starts"].numel() - 1)
    token = s["starts"][b].long() + i - s["row_indptr"][b].long()
    listed_ = (s["kv_indptr"][b].long() + token // P).clamp(max=s["kv_indices"].numel() - 1)
    slot = s["kv_indices"][listed_].long() * P + token % P
    if s["kind"] == "q4":
        x = _unpack(s["cache"].view(-1, ROW)[slot])
        ckv, kpe = x[:, :D_CKV], x[:, D_CKV:]
    else:
        ckv = s["cache"].view(-1, D_CKV)[slot].float() * s["kv_scale"]
        kpe = s["kpe_cache"].view(-1, D_KPE)[slot].float() * s["kv_scale"]
    return dict(ckv=torch.where(real, ckv.to(s["ckv_out"].dtype), s["ckv_out"]),
                kpe=torch.where(real, kpe.to(s["kpe_out"].dtype), s["kpe_out"]))


def _plain_decode(s):
    lead = s["q_nope"].shape[:-1]
    B, Q, P = lead[0], s["q_len"], s["page_size"]
    q = torch.cat([s["q_nope"], s["q_pe"]], -1).float().view(B, Q, -1, D)
    out = torch.empty(B, Q, q.shape[2], D_CKV, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, Q, q.shape[2], device="cuda")
    for b, n in enumerate(s["kv_len"]):
        pages = s["kv_indices"][s["kv_indptr"][b]:s["kv_indptr"][b + 1]].long()
        key = _unpack(s["cache"][pages].view(-1, ROW)[:n])
        for j in range(Q):
            seen = key[:n - Q + 1 + j]
            logit = torch.matmul(q[b, j], seen.t()) * s["sm_scale"]
            top = logit.amax(1, keepdim=True)
            p = torch.exp(logit - top)
            total = p.sum(1, keepdim=True)
            out[b, j] = torch.matmul(p, seen[:, :D_CKV]) / total
            lse[b, j] = (top + total.log())[:, 0]
    return dict(out=out.view(*lead, D_CKV), lse=lse.view(lead))


_PLAIN = dict(write=_plain_write, read=_plain_read, decode=_plain_decode)


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _own_pass(s):
    from paged_mla_decode_02_gb300 import mla
    if s["op"] == "write":
        mla.mla_quantize_append(s["ckv"], s["kpe"], s["slots"], s["cache"])
        return s["cache"]
    if s["op"] == "read":
        mla.mla_read_cache(s["cache"], s["kpe_cache"], s["kv_indptr"], s["kv_indices"], s["starts"],
                           s["row_indptr"], s["ckv_out"], s["kpe_out"], kv_scale=s["kv_scale"])
        return dict(ckv=s["ckv_out"], kpe=s["kpe_out"])
    out, lse = s["decoder"].run_q4(s["q_nope"], s["q_pe"], s["cache"])
    return dict(out=out, lse=lse)


def run(state):
    return _own_pass(state) if own else _PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    P = case["page_size"]
    if case["op"] == "write":
        T = case["tokens"]
        return dict(bytes=T * 8 + (T - case["padded"]) * (D * SIZES[case["dtype"]] + ROW), flops=0)
    if case["op"] == "read":
        rows = sum(n - a for n, a in zip(*_read_ranges(case)))
        width = ROW if case["cache"] == "q4" else D * SIZES[case["cache"]]
        return dict(bytes=rows * (width + D * SIZES[case["dtype"]] + 4 / P) + 12 * case["batch"], flops=0)
    tokens = case["batch"] * case["ctx"] * (0.5 if case["ragged"] else 1.0)
    rows = case["heads"] * case["q_len"]
    return dict(bytes=tokens * (ROW + 4 / P) + case["batch"] * rows * (2 * D + 2 * D_CKV + 4),
                flops=tokens * rows * 2 * (D + D_CKV))


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_bytes(x):
    """Rows quantised in 64 bits: each value divided by its unit and rounded to
    a multiple of the step of its binade; the bytes put together bit by bit."""
    x = x.double().reshape(-1, GROUPS, 32)
    n = x.shape[0]
    top = x.abs().amax(2)
    e = torch.where(top > 0, torch.ceil(torch.log2(top / 6)), -1e9)
    e = torch.where(top > 6 * torch.exp2(e), e + 1, torch.where(top <= 3 * torch.exp2(e), e - 1, e))
    row_e = e.amax(1, keepdim=True).clamp(E_MIN, E_MAX)
    k = (row_e - e).clamp(0, K_MAX)
    y = (x / torch.exp2(row_e - k)[..., None]).abs().clamp(max=6)
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = torch.round(y / step) * step
    index = torch.bucketize(y, torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)).view(n, 72, 8)
    neg = torch.signbit(x).view(n, 72, 8)
    bits = torch.zeros(n, 72, 32, dtype=torch.bool, device=x.device)
    for i in range(8):
        for b in range(3):
            bits[:, :, 4 * i + b] = (index[:, :, i] >> b) & 1 != 0
        bits[:, :, 8 * i + 7 if i < 4 else 8 * i - 29] = neg[:, :, i]
    weight = 2 ** torch.arange(8, device=x.device)
    out = torch.zeros(n, ROW, dtype=torch.uint8, device=x.device)
    for i in range(0, n, 16384):
        out[i:i + 16384, :288] = (bits[i:i + 16384].view(-1, 288, 8) * weight).sum(2).to(torch.uint8)
    out[:, 288:297] = (k[:, 0::2] + 16 * k[:, 1::2]).to(torch.uint8)
    out[:, 297] = (row_e[:, 0] + 127).to(torch.uint8)
    return out


def _exact_values(rows):
    """The values of rows of bytes in 64 bits: the bits spread out, the eight
    magnitudes as (2 + m) 2^(x - 1) / 4 with a mantissa bit m and a 2-bit exponent x."""
    n = rows.shape[0]
    bits = ((rows[:, :288, None] >> torch.arange(8, dtype=torch.uint8, device=rows.device)) & 1).view(n, 72, 32)
    sign = bits[:, :, [7, 15, 23, 31, 3, 11, 19, 27]].double()
    m, x = bits[:, :, 0::4].double(), (bits[:, :, 1::4] + 2 * bits[:, :, 2::4]).double()
    v = torch.where(x == 0, m / 2, (2 + m) * torch.exp2(x - 2)) * (1 - 2 * sign)
    k = torch.stack([rows[:, 288:297] % 16, rows[:, 288:297] // 16], 2).view(n, GROUPS, 1).double()
    unit = torch.exp2(rows[:, 297].double()[:, None, None] - 127 - k)
    return (v.view(n, GROUPS, 32) * unit).view(n, D)


def exact(case, seed):
    s = prepare(case, seed)
    P = case["page_size"]
    if case["op"] == "write":
        keep = case["tokens"] - case["padded"]
        out = s["cache"].clone().view(-1, ROW)
        for i in range(0, keep, 16384):
            j = min(keep, i + 16384)
            out[s["slots"][i:j]] = _exact_bytes(torch.cat([s["ckv"][i:j], s["kpe"][i:j]], 1))
        return out.view(s["cache"].shape)
    if case["op"] == "read":
        ckv, kpe = s["ckv_out"].double(), s["kpe_out"].double()
        lists, rows, starts = s["kv_indptr"].tolist(), s["row_indptr"].tolist(), s["starts"].tolist()
        for b in range(case["batch"]):
            pages = s["kv_indices"][lists[b]:lists[b + 1]].long()
            lo, hi = rows[b], rows[b + 1]
            mine = slice(starts[b], starts[b] + hi - lo)
            if case["cache"] == "q4":
                x = _exact_values(s["cache"][pages].view(-1, ROW)[mine])
                ckv[lo:hi], kpe[lo:hi] = x[:, :D_CKV], x[:, D_CKV:]
            else:
                ckv[lo:hi] = s["cache"][pages].view(-1, D_CKV)[mine].double() * s["kv_scale"]
                kpe[lo:hi] = s["kpe_cache"][pages].view(-1, D_KPE)[mine].double() * s["kv_scale"]
        return dict(ckv=ckv, kpe=kpe)
    Q, H = case["q_len"], case["heads"]
    q = torch.cat([s["q_nope"], s["q_pe"]], -1).double().view(case["batch"], Q * H, D)
    late = (Q - 1 - torch.arange(Q * H, device="cuda") // H)[:, None]     # tokens of the request behind this one
    outs, lses = [], []
    for b, n in enumerate(s["kv_len"]):
        pages = s["kv_indices"][s["kv_indptr"][b]:s["kv_indptr"][b + 1]].long()
        key = torch.cat([_exact_values(part) for part in s["cache"][pages].view(-1, ROW)[:n].split(16384)])
        logit = q[b] @ key.T * s["sm_scale"]
        logit.masked_fill_(torch.arange(n, device="cuda")[None] >= n - late, -INF)
        lses.append(torch.logsumexp(logit, 1))
        outs.append(torch.softmax(logit, 1) @ key[:, :D_CKV])
    lead = s["q_nope"].shape[:-1]
    return dict(out=torch.stack(outs).view(*lead, D_CKV), lse=torch.stack(lses).view(lead))
