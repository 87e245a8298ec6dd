"""Cases of the operators around the paged MLA decode: page tables built from
request lengths, rotary embedding with the cache append, page summaries, page
scores, page selection, and the sparse decode that they make together.

Each case is one pass through one operator, in its plain form (elementary torch
operations in 32 bits, rounded once at the end) or, with ``own`` set, through
the library.
"""
import math

import numpy as np
import torch

own = False

D_CKV, D_KPE, D = 512, 64, 576
NOPE = 128                       # no-rope width of a head's query, beside its 64 rope dims
INF = float("inf")


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a serving batch: one new token for every request
        dict(name="tables_decode", op="tables", batch=64, page_size=64, ctx=8192, chunk=1, prefills=0, released=0),
        # decoding and prefilling requests mixed, some finished ones give their pages back
        dict(name="tables_mixed", op="tables", batch=512, page_size=16, ctx=16384, chunk=509, prefills=16, released=20),
        # the new token of each decoding request: queries rotated, latent row normed and cached
        dict(name="append_decode", op="append", tokens=64, heads=128, axes=1, interleaved=True, fp8=False,
             page_size=64, padded=0),
        # a prefill chunk of text and image tokens (time, height, width) into an fp8 cache
        dict(name="append_prefill", op="append", tokens=8190, heads=128, axes=3, interleaved=False, fp8=True,
             page_size=64, padded=2),
        # the pages that a prefill chunk completes
        dict(name="summarize_chunk", op="summarize", tokens=8192, page_size=64, fp8=False),
        # a long prompt brought into an fp8 cache at once
        dict(name="summarize_long", op="summarize", tokens=131000, page_size=32, fp8=True),
        # few requests of one of eight head groups, short lists
        dict(name="scores_small", op="scores", rows=4, heads=16, pages=100, ragged=True),
        # a decode batch over caches of 64k tokens in pages of 64
        dict(name="scores_large", op="scores", rows=64, heads=128, pages=1024, ragged=False),
        # short lists: a small batch at 12k tokens
        dict(name="select_small", op="select", rows=8, pages=200, top_k=32, keep_first=1, keep_last=1, ragged=True),
        # half a million tokens in pages of 64
        dict(name="select_large", op="select", rows=64, pages=8192, top_k=256, keep_first=1, keep_last=4, ragged=True),
        # score, select and decode: a small batch of 16 heads
        dict(name="sparse_small", op="sparse", rows=4, heads=16, pages=256, page_size=64, top_k=32, keep_first=1,
             keep_last=1),
        # the same for a batch of 64 with 128 heads over 32k tokens each, an eighth of them read
        dict(name="sparse_large", op="sparse", rows=64, heads=128, pages=512, page_size=64, top_k=64, keep_first=1,
             keep_last=2),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "summarize", "scores", "select", "sparse"])
    page_size = rng.choice([16, 32, 64])
    if op == "tables":
        batch = _log_int(rng, 1, 512)
        prefills = rng.randint(0, min(batch, 16))
        return dict(op=op, batch=batch, page_size=page_size, ctx=_log_int(rng, 1, 1024 * page_size),
                    chunk=_log_int(rng, 1, 509), prefills=prefills, released=rng.randint(0, (batch - prefills) // 4))
    if op == "append":
        tokens = _log_int(rng, 1, 8190)
        return dict(op=op, tokens=tokens, heads=rng.choice([1, 8, 16, 20, 64, 128]), axes=rng.choice([1, 2, 3]),
                    interleaved=rng.random() < 0.5, fp8=rng.random() < 0.5, page_size=page_size,
                    padded=rng.randint(0, tokens // 8))
    if op == "summarize":
        return dict(op=op, tokens=_log_int(rng, 256, 65536), page_size=page_size, fp8=rng.random() < 0.5)
    if op == "scores":
        return dict(op=op, rows=_log_int(rng, 1, 64), heads=rng.choice([1, 8, 16, 20, 40, 64, 128]),
                    pages=_log_int(rng, 1, 1024), ragged=rng.random() < 0.5)
    top_k = _log_int(rng, 3, 256)
    keep_first, keep_last = rng.randint(0, 1), rng.randint(1, 2)
    if op == "select":
        return dict(op=op, rows=_log_int(rng, 1, 64), pages=_log_int(rng, 1, 8192), top_k=top_k,
                    keep_first=keep_first, keep_last=keep_last, ragged=rng.random() < 0.5)
    rows = _log_int(rng, 1, 64)
    return dict(op=op, rows=rows, heads=rng.choice([8, 16, 40, 128]), pages=_log_int(rng, 4, 512),
                page_size=page_size, top_k=min(top_k, 64), keep_first=keep_first, keep_last=keep_last)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _randint(g, lo, hi, *shape, dtype=torch.int32):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=dtype)


def _indptr(counts):
    out = torch.zeros(counts.numel() + 1, dtype=torch.int32, device="cuda")
    out[1:] = counts.cumsum(0)
    return out


def _fp8_scale(case):
    return 0.125 if case.get("fp8") else 1.0


def _random_cache(g, pages, page_size, fp8):
    def part(width):
        t = _randn(g, pages, page_size, width)
        return (t.float() / 0.125).clamp_(-448, 448).to(torch.float8_e4m3fn) if fp8 else t
    return part(D_CKV), part(D_KPE)


def _inv_freq():
    return 10000.0 ** (-np.arange(32, dtype=np.float64) / 32)


def _axis_of_pair(axes):
    """Frequency pairs dealt to the axes in sections: 32, or 16 + 16, or 8 + 12 + 12."""
    return {1: [0] * 32, 2: [0] * 16 + [1] * 16, 3: [0] * 8 + [1] * 12 + [2] * 12}[axes]


def _prepare_tables(case, g):
    B, P, ctx = case["batch"], case["page_size"], case["ctx"]
    kv_len = _randint(g, 0, ctx + 1, B)
    new_len = torch.ones(B, dtype=torch.int32, device="cuda")
    who = torch.randperm(B, generator=g, device="cuda")
    new_len[who[:case["prefills"]]] = _randint(g, 0, case["chunk"] + 1, case["prefills"])
    new_len[who[case["prefills"]:case["prefills"] + case["released"]]] = -1
    max_tokens = B + case["prefills"] * case["chunk"]
    max_pages = -(-(ctx + case["chunk"]) // P)
    num_pages = B * max_pages + 7
    ids = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    block_table = ids[:B * max_pages].reshape(B, max_pages).clone()
    held = (kv_len + P - 1) // P
    used = torch.arange(max_pages, device="cuda")[None] < held[:, None]
    free = torch.cat([block_table[~used], ids[B * max_pages:]])
    block_table[~used] = -1
    free_pages = torch.full((num_pages,), -1, dtype=torch.int32, device="cuda")
    free_pages[:free.numel()] = free
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(kv_len=kv_len, new_len=new_len, block_table=block_table, free_pages=free_pages,
                free_count=torch.tensor([free.numel()], **i32), page_size=P,
                kv_len_out=torch.zeros(B, **i32), free_count_out=torch.zeros(1, **i32),
                kv_indptr=torch.zeros(B + 1, **i32), kv_indices=torch.zeros(B * max_pages, **i32),
                q_indptr=torch.zeros(B + 1, **i32),
                slots=torch.zeros(max_tokens, dtype=torch.int64, device="cuda"),
                positions=torch.zeros(max_tokens, **i32), status=torch.zeros(1, **i32))


def _prepare_append(case, g):
    T, H, P = case["tokens"], case["heads"], case["page_size"]
    pages = max(4, -(-3 * T // (2 * P))) + 1                 # the last page takes no token
    q = _randn(g, T, H, NOPE + D_KPE)                        # the query projection's output
    kv_a = _randn(g, T, D)                                   # the latent projection's output
    weight = (1 + 0.1 * _randn(g, D_CKV, dtype=torch.float32)).to(torch.bfloat16)
    slots = torch.randperm((pages - 1) * P, generator=g, device="cuda")[:T].to(torch.int64)
    if case["padded"]:
        slots[T - case["padded"]:] = -1
    if case["axes"] == 1:
        positions = _randint(g, 0, 1 << 20, 1, T)
    else:                                                    # a start far in, then a grid of patches
        start = _randint(g, 0, 1 << 18, 1)
        t = torch.arange(T, device="cuda", dtype=torch.int32)
        positions = torch.stack([start + t // 1024, start + t // 32 % 32, start + t % 32][:case["axes"]])
    ckv_cache, kpe_cache = _random_cache(g, pages, P, case["fp8"])
    state = dict(q_pe=q[..., NOPE:], ckv=kv_a[:, :D_CKV], kpe=kv_a[:, D_CKV:], weight=weight, eps=1e-6, slots=slots,
                 positions=positions.contiguous(), ckv_cache=ckv_cache, kpe_cache=kpe_cache,
                 q_out=torch.zeros(T, H, D_KPE, dtype=torch.bfloat16, device="cuda"), kv_scale=_fp8_scale(case),
                 interleaved=case["interleaved"],
                 inv_freq=torch.from_numpy(_inv_freq()).cuda(),
                 axis=torch.tensor(_axis_of_pair(case["axes"]), device="cuda"))
    if own:
        from paged_mla_decode_02_gb300 import mla
        state["rope"] = mla.rope_spec(_inv_freq(), _axis_of_pair(case["axes"]), case["interleaved"])
    return state


def _prepare_summarize(case, g):
    T, P = case["tokens"], case["page_size"]
    first = P // 3                                           # the prompt starts inside a page
    n = -(-(T + first) // P)
    pages = n + 3
    table = torch.randperm(pages, generator=g, device="cuda")[:n]
    pos = first + torch.arange(T, device="cuda")
    ckv_cache, kpe_cache = _random_cache(g, pages, P, case["fp8"])
    return dict(slots=table[pos // P] * P + pos % P, ckv_cache=ckv_cache, kpe_cache=kpe_cache,
                kv_scale=_fp8_scale(case), summaries=torch.zeros(pages, D, dtype=torch.bfloat16, device="cuda"))


def _counts(case, g):
    n = case["pages"]
    counts = torch.full((case["rows"],), n, dtype=torch.int32, device="cuda")
    if case["ragged"]:
        counts = _randint(g, (n + 1) // 2, n + 1, case["rows"])
        counts[0] = n
    return counts


def _prepare_scores(case, g):
    counts = _counts(case, g)
    kv_indptr = _indptr(counts)
    total = case["rows"] * case["pages"]
    kv_indices = torch.randperm(total + 5, generator=g, device="cuda")[:total].to(torch.int32)
    return dict(q_nope=_randn(g, case["rows"], case["heads"], D_CKV), q_pe=_randn(g, case["rows"], case["heads"], D_KPE),
                summaries=(_randn(g, total + 5, D) * 0.3), kv_indptr=kv_indptr, kv_indices=kv_indices,
                scores=torch.zeros(case["rows"], case["pages"], device="cuda"))


def _prepare_select(case, g):
    counts = _counts(case, g)
    total = case["rows"] * case["pages"]
    # scores of few pages stand out of a crowd; many of them are alike
    scores = (_randn(g, case["rows"], case["pages"], dtype=torch.float32) * 4 + 12).to(torch.bfloat16).float()
    return dict(scores=scores, kv_indptr=_indptr(counts),
                kv_indices=torch.randperm(total, generator=g, device="cuda").to(torch.int32), top_k=case["top_k"],
                keep_first=case["keep_first"], keep_last=case["keep_last"],
                sel_indptr=torch.zeros(case["rows"] + 1, dtype=torch.int32, device="cuda"),
                sel_indices=torch.zeros(case["rows"] * case["top_k"], dtype=torch.int32, device="cuda"))


def _prepare_sparse(case, g):
    """Caches in which some pages of each request speak to its queries: their
    rows share a direction with them, the others do not."""
    R, H, N, P, k = case["rows"], case["heads"], case["pages"], case["page_size"], case["top_k"]
    counts = _randint(g, (N + 1) // 2, N + 1, R)
    counts[0] = N
    tail = _randint(g, 1, P + 1, R)
    kv_len = (counts - 1) * P + tail
    kv_indptr = _indptr(counts)
    total = R * N
    table = torch.randperm(total, generator=g, device="cuda").to(torch.int32).reshape(R, N)
    listed_ = torch.arange(N, device="cuda")[None] < counts[:, None]
    kv_indices = torch.zeros(total + 1, dtype=torch.int32, device="cuda")
    kv_indices.scatter_(0, torch.where(listed_, kv_indptr[:-1, None] + torch.arange(N, device="cuda")[None],
                                       total).long().reshape(-1), table.reshape(-1))
    u = torch.nn.functional.normalize(_randn(g, R, D, dtype=torch.float32), dim=1)
    q = (_randn(g, R, H, D, dtype=torch.float32) + 6 * u[:, None]).to(torch.bfloat16)
    kf, kl = case["keep_first"], case["keep_last"]
    order = torch.rand(R, N, generator=g, device="cuda")
    at = torch.arange(N, device="cuda")[None]
    order = torch.where((at >= kf) & (at < counts[:, None] - kl), order, INF)
    rank = order.argsort(1).argsort(1)
    speak = (rank < max(0, k - kf - kl)) & (order < INF)
    ckv, kpe = _random_cache(g, total, P, False)
    rows, cols = speak.nonzero(as_tuple=True)
    pages = table[rows, cols].long()
    ckv[pages] += (10 * u[rows, None, :D_CKV]).to(torch.bfloat16)
    kpe[pages] += (10 * u[rows, None, D_CKV:]).to(torch.bfloat16)
    summaries = torch.cat([ckv.mean(1, dtype=torch.float32), kpe.mean(1, dtype=torch.float32)], 1).to(torch.bfloat16)
    state = dict(q_nope=q[..., :D_CKV].contiguous(), q_pe=q[..., D_CKV:].contiguous(), ckv=ckv, kpe=kpe,
                 summaries=summaries, table=table, counts=counts, kv_len=kv_len, kv_indptr=kv_indptr,
                 kv_indices=kv_indices[:total], top_k=k, keep_first=kf, keep_last=kl, page_size=P,
                 sm_scale=1 / math.sqrt(192.0))
    if own:                       # the plan that a serving loop keeps for the layers of a step
        from paged_mla_decode_02_gb300 import mla
        dec = mla.MLASparseDecoder(R, H, N, k, kf, kl)
        dec.plan(kv_indptr.cpu(), state["kv_indices"], kv_len.cpu(), P, state["sm_scale"])
        state["decoder"] = dec
    return state


_PREPARE = dict(tables=_prepare_tables, append=_prepare_append, summarize=_prepare_summarize, scores=_prepare_scores,
                select=_prepare_select, sparse=_prepare_sparse)


def prepare(case, seed):
    state = _PREPARE[case["op"]](case, _gen(seed))
    state["op"] = case["op"]
    return state


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _plain_tables(s):
    P, table, kv_len, new_len = s["page_size"], s["block_table"], s["kv_len"].long(), s["new_len"].long()
    B, W = table.shape
    gone = new_len < 0
    add = new_len.clamp(min=0)
    old = (kv_len + P - 1) // P
    length = torch.where(gone, 0, kv_len + add)
    pages = (length + P - 1) // P
    fresh = torch.where(gone, 0, pages - old)
    freed = torch.where(gone, old, 0)
    zero = torch.zeros(1, dtype=torch.int64, device=table.device)
    fresh_at, freed_at = torch.cat([zero, fresh.cumsum(0)]), torch.cat([zero, freed.cumsum(0)])
    fc, A, R = s["free_count"].long(), fresh_at[-1:], freed_at[-1:]
    col = torch.arange(W, device=table.device)[None]
    n = s["free_pages"].numel()
    # the stack of free pages with the released ones on top
    stack = torch.cat([s["free_pages"], torch.zeros(B * W + 1, dtype=torch.int32, device=table.device)])
    to = torch.where(gone[:, None] & (col < old[:, None]), fc + freed_at[:-1, None] + col, stack.numel() - 1)
    stack = stack.scatter(0, to.reshape(-1), table.reshape(-1))
    # pages come off its top
    take = (fc + R - 1 - (fresh_at[:-1, None] + col - old[:, None])).clamp(0, stack.numel() - 1)
    given = (col >= old[:, None]) & (col < pages[:, None]) & ~gone[:, None]
    table = torch.where(given, stack[take], table)
    left = fc + R - A
    free_pages = torch.where(torch.arange(n, device=table.device) < left, stack[:n], s["free_pages"])
    indptr = torch.cat([zero, pages.cumsum(0)])
    indices = torch.zeros(s["kv_indices"].numel() + 1, dtype=torch.int32, device=table.device)
    to = torch.where(col < pages[:, None], indptr[:-1, None] + col, indices.numel() - 1)
    indices = indices.scatter(0, to.reshape(-1), table.reshape(-1))[:-1]
    q_indptr = torch.cat([zero, add.cumsum(0)])
    t = torch.arange(s["slots"].numel(), device=table.device)
    real = t < q_indptr[-1]
    b = torch.searchsorted(q_indptr[1:], t, right=True).clamp(max=B - 1)
    pos = kv_len[b] + t - q_indptr[b]
    page = table[b, (pos // P).clamp(max=W - 1)].long()
    slots = torch.where(real, page * P + pos % P, -1)
    short = (left < 0) | (pages.max() > W) | (indptr[-1] > s["kv_indices"].numel()) | (q_indptr[-1] > t.numel())
    i32 = torch.int32
    return dict(kv_len=length.to(i32), free_count=left.to(i32), free_pages=free_pages, block_table=table,
                kv_indptr=indptr.to(i32), kv_indices=indices, q_indptr=q_indptr.to(i32), slots=slots,
                positions=torch.where(real, pos, 0).to(i32), status=short.to(i32) * 3)


def _rotate(x, cos, sin, interleaved):
    x = x.float()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)


def _plain_append(s):
    angle = (s["positions"].double()[s["axis"]] * s["inv_freq"][:, None]).t()        # [T, 32]
    cos, sin = angle.cos().float(), angle.sin().float()
    real = s["slots"] >= 0
    q = _rotate(s["q_pe"], cos[:, None], sin[:, None], s["interleaved"]).to(torch.bfloat16)
    q_out = torch.where(real[:, None, None], q, s["q_out"])
    ckv = s["ckv"].float()
    ckv = ckv * torch.rsqrt(ckv.square().mean(1, keepdim=True) + s["eps"]) * s["weight"].float()
    kpe = _rotate(s["kpe"], cos, sin, s["interleaved"])
    caches = []
    for cache, x in ((s["ckv_cache"], ckv), (s["kpe_cache"], kpe)):
        if cache.dtype == torch.float8_e4m3fn:
            x = (x / s["kv_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            flat = cache.view(torch.uint8).view(-1, cache.shape[-1])
        else:
            x = x.to(cache.dtype)
            flat = cache.view(-1, cache.shape[-1])
        spare = flat.shape[0] - 1                        # no token's slot: takes the padded ones
        kept = flat[spare].clone()
        flat.index_copy_(0, torch.where(real, s["slots"], spare), x)
        flat[spare] = kept
        caches.append(cache)
    return dict(q_pe=q_out, ckv_cache=caches[0], kpe_cache=caches[1])


def _plain_summarize(s):
    P = s["ckv_cache"].shape[1]
    slots, out = s["slots"], s["summaries"]
    done = (slots >= 0) & (slots % P == P - 1)
    # completed pages, each once: one more row takes the tokens that complete none
    pages = out.shape[0]
    hit = torch.zeros(pages + 1, dtype=torch.bool, device=out.device)
    hit[torch.where(done, slots // P, pages)] = True
    mean = torch.cat([s["ckv_cache"].float().mean(1), s["kpe_cache"].float().mean(1)], 1) * s["kv_scale"]
    return torch.where(hit[:pages, None], mean.to(torch.bfloat16), out)


def _page_lists(s, width):
    """[rows, width] page ids and which of them are in the row's list."""
    counts = s["kv_indptr"][1:] - s["kv_indptr"][:-1]
    at = torch.arange(width, device=counts.device)[None]
    mine = at < counts[:, None]
    where = torch.where(mine, s["kv_indptr"][:-1, None] + at, 0)
    return s["kv_indices"][where].long(), mine, counts


def _plain_scores_of(s, width):
    pages, mine, counts = _page_lists(s, width)
    q = torch.cat([s["q_nope"], s["q_pe"]], -1).float()
    each = torch.matmul(s["summaries"][pages].float(), q.transpose(1, 2))            # [rows, pages, heads]
    each = torch.where(each.isnan(), -INF, each)
    return each.amax(-1), mine, counts, pages


def _plain_scores(s):
    score, mine, _, _ = _plain_scores_of(s, s["scores"].shape[1])
    return torch.where(mine, score, s["scores"])


def _plain_choice(s, scores, mine, counts):
    """[rows, width] truth of being kept."""
    at = torch.arange(scores.shape[1], device=scores.device)[None]
    rank = torch.where(scores.isnan(), -INF, scores)
    forced = (at < s["keep_first"]) | (at >= counts[:, None] - s["keep_last"])
    # the kept ends first, then by score, pages of other rows last; a stable sort keeps ties in order
    group = torch.where(mine, torch.where(forced, 0, 1), 2)
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices
    order = order.gather(1, torch.sort(group.gather(1, order), dim=1, stable=True).indices)
    place = torch.empty_like(order).scatter_(1, order, at.expand_as(order).contiguous())
    return (place < s["top_k"]) & mine


def _plain_packed(s, kept, pages, capacity):
    n = kept.sum(1)
    indptr = torch.cat([torch.zeros(1, dtype=torch.int64, device=n.device), n.cumsum(0)])
    to = torch.where(kept, indptr[:-1, None] + kept.cumsum(1) - 1, capacity)
    out = torch.zeros(capacity + 1, dtype=torch.int32, device=n.device)
    out.scatter_(0, to.reshape(-1), pages.to(torch.int32).reshape(-1))
    return indptr.to(torch.int32), out[:capacity]


def _plain_select(s):
    pages, mine, counts = _page_lists(s, s["scores"].shape[1])
    kept = _plain_choice(s, s["scores"], mine, counts)
    indptr, indices = _plain_packed(s, kept, pages, s["sel_indices"].numel())
    return dict(sel_indptr=indptr, sel_indices=indices)


def _plain_sparse(s):
    scores, mine, counts, pages = _plain_scores_of(s, s["table"].shape[1])
    kept = _plain_choice(s, scores, mine, counts)
    R, k, P = pages.shape[0], min(s["top_k"], pages.shape[1]), s["page_size"]
    at = torch.arange(pages.shape[1], device=pages.device)[None]
    places = torch.sort(torch.where(kept, at, pages.shape[1]), 1).values[:, :k]      # ascending; past the end: none
    none = places >= pages.shape[1]
    chosen = pages.gather(1, places.clamp(max=pages.shape[1] - 1))
    token = places[:, :, None] * P + torch.arange(P, device=pages.device)
    seen = ((token < s["kv_len"][:, None, None]) & ~none[:, :, None]).reshape(R, k * P)
    key_c = s["ckv"][chosen].float().reshape(R, k * P, D_CKV)
    key_p = s["kpe"][chosen].float().reshape(R, k * P, D_KPE)
    logit = torch.matmul(s["q_nope"].float(), key_c.transpose(1, 2))
    logit = (logit + torch.matmul(s["q_pe"].float(), key_p.transpose(1, 2))) * s["sm_scale"]
    logit = torch.where(seen[:, None], logit, -INF)
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - top)
    total = p.sum(-1, keepdim=True)
    key_c = torch.where(seen[:, :, None], key_c, 0)
    out = torch.matmul(p, key_c) / total
    indptr, indices = _plain_packed(s, kept, pages, R * s["top_k"])
    return dict(out=out.to(torch.bfloat16), lse=(top + total.log())[..., 0], sel_indptr=indptr, sel_indices=indices)


_PLAIN = dict(tables=_plain_tables, append=_plain_append, summarize=_plain_summarize, scores=_plain_scores,
              select=_plain_select, sparse=_plain_sparse)


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _own_pass(s):
    from paged_mla_decode_02_gb300 import mla
    op = s["op"]
    if op == "tables":
        mla.mla_build_tables(s["kv_len"], s["new_len"], s["block_table"], s["free_pages"], s["free_count"],
                             s["page_size"], s["kv_indptr"], s["kv_indices"], s["q_indptr"], s["slots"],
                             s["positions"], s["status"], kv_len_out=s["kv_len_out"],
                             free_count_out=s["free_count_out"])
        return dict(kv_len=s["kv_len_out"], free_count=s["free_count_out"], free_pages=s["free_pages"],
                    block_table=s["block_table"], kv_indptr=s["kv_indptr"], kv_indices=s["kv_indices"],
                    q_indptr=s["q_indptr"], slots=s["slots"], positions=s["positions"], status=s["status"])
    if op == "append":
        mla.mla_rope_append(s["rope"], s["positions"], s["slots"], s["q_pe"], s["ckv"], s["kpe"], s["weight"],
                            s["eps"], s["ckv_cache"], s["kpe_cache"], q_pe_out=s["q_out"], kv_scale=s["kv_scale"])
        return dict(q_pe=s["q_out"], ckv_cache=s["ckv_cache"], kpe_cache=s["kpe_cache"])
    if op == "summarize":
        mla.mla_summarize_pages(s["slots"], s["ckv_cache"], s["kpe_cache"], s["summaries"], kv_scale=s["kv_scale"])
        return s["summaries"]
    if op == "scores":
        mla.mla_page_scores(s["q_nope"], s["q_pe"], s["summaries"], s["kv_indptr"], s["kv_indices"], s["scores"])
        return s["scores"]
    if op == "select":
        mla.mla_select_pages(s["scores"], s["kv_indptr"], s["kv_indices"], s["top_k"], s["keep_first"],
                             s["keep_last"], s["sel_indptr"], s["sel_indices"])
        return dict(sel_indptr=s["sel_indptr"], sel_indices=s["sel_indices"])
    dec = s["decoder"]
    out, lse = dec.run(s["q_nope"], s["q_pe"], s["ckv"], s["kpe"], s["summaries"])
    return dict(out=out, lse=lse, sel_indptr=dec.sel_indptr, sel_indices=dec.sel_indices)


def run(state):
    return _own_pass(state) if own else _PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "tables":
        B, P = case["batch"], case["page_size"]
        entries = B * (case["ctx"] / 2 / P + 0.5)
        tokens = B - case["prefills"] - case["released"] + case["prefills"] * case["chunk"] / 2
        return dict(bytes=8 * entries + 20 * B + 12 * tokens + 8 * tokens / P, flops=0)
    if op == "append":
        T, H = case["tokens"], case["heads"]
        row = H * D_KPE * 4 + D * (3 if case["fp8"] else 4) + 4 * case["axes"] + 8
        return dict(bytes=T * row + 2 * D_CKV, flops=T * (H + 1) * D_KPE * 3 + T * D_CKV * 4)
    if op == "summarize":
        P = case["page_size"]
        pages = (case["tokens"] + P // 3) // P
        return dict(bytes=pages * (P * D * (1 if case["fp8"] else 2) + 2 * D) + 8 * case["tokens"], flops=pages * P * D)
    share = 0.75 if case.get("ragged", True) else 1.0
    pages = case["rows"] * case["pages"] * share
    if op == "select":
        return dict(bytes=4 * pages + 8 * case["rows"] * min(case["top_k"], case["pages"] * share), flops=0)
    scores = dict(bytes=pages * (2 * D + 8) + case["rows"] * case["heads"] * 2 * D,
                  flops=pages * case["heads"] * 2 * D)
    if op == "scores":
        return scores
    tokens = case["rows"] * min(case["top_k"], case["pages"] * share) * case["page_size"]
    return dict(bytes=pages * (2 * D + 4) + tokens * 2 * D + case["rows"] * case["heads"] * (2 * D + 2 * D_CKV + 4),
                flops=scores["flops"] + tokens * case["heads"] * 2 * (D + D_CKV))


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_rope(x, angles, interleaved):
    """x [T, h, 64], angles [T, 32]: each pair as one complex number, turned."""
    x = x.double()
    pair = torch.complex(x[..., 0::2], x[..., 1::2]) if interleaved else torch.complex(x[..., :32], x[..., 32:])
    turned = pair * torch.polar(torch.ones_like(angles), angles)[:, None]
    if interleaved:
        return torch.view_as_real(turned).flatten(-2)
    return torch.cat([turned.real, turned.imag], -1)


def exact(case, seed):
    op = case["op"]
    if op in ("tables", "select"):
        return None                                   # whole numbers throughout
    s = prepare(case, seed)
    if op == "append":
        T = case["tokens"]
        angles = torch.empty(T, 32, dtype=torch.float64, device="cuda")
        for i, a in enumerate(_axis_of_pair(case["axes"])):
            angles[:, i] = s["positions"][a].double() * float(_inv_freq()[i])
        keep = T - case["padded"]
        q = s["q_out"].double()
        q[:keep] = _exact_rope(s["q_pe"], angles, case["interleaved"])[:keep]
        row = s["ckv"].double()
        row = row / (row.pow(2).sum(1, keepdim=True) / D_CKV + s["eps"]).sqrt() * s["weight"].double()
        kpe = _exact_rope(s["kpe"][:, None], angles, case["interleaved"])[:, 0]
        caches = []
        for cache, x in ((s["ckv_cache"], row), (s["kpe_cache"], kpe)):
            c = cache.double().reshape(-1, x.shape[1])
            c[s["slots"][:keep]] = x[:keep] / s["kv_scale"]
            caches.append(c.reshape(cache.shape))
        return dict(q_pe=q, ckv_cache=caches[0], kpe_cache=caches[1])
    if op == "summarize":
        P = case["page_size"]
        first = P // 3
        out = s["summaries"].double()
        ends = s["slots"][P - 1 - first::P] // P       # the tokens at which a page is full
        for c in ends.split(2048):
            out[c, :D_CKV] = s["ckv_cache"][c].double().sum(1) * (s["kv_scale"] / P)
            out[c, D_CKV:] = s["kpe_cache"][c].double().sum(1) * (s["kv_scale"] / P)
        return out
    rows, offsets = case["rows"], s["kv_indptr"].tolist()
    q = torch.cat([s["q_nope"], s["q_pe"]], -1).double()
    if op == "scores":
        out = s["scores"].double()
        for r in range(rows):
            pages = s["kv_indices"][offsets[r]:offsets[r + 1]].long()
            out[r, :pages.numel()] = (q[r] @ s["summaries"][pages].double().T).max(0).values
        return out
    outs, lses = [], []
    for r in range(rows):
        pages = s["kv_indices"][offsets[r]:offsets[r + 1]].long()
        n, P = pages.numel(), case["page_size"]
        score = (q[r] @ s["summaries"][pages].double().T).max(0).values
        score[:case["keep_first"]] = INF
        score[max(0, n - case["keep_last"]):] = INF
        places = torch.sort(score, descending=True, stable=True).indices[:case["top_k"]].sort().values
        last = n * P - int(s["kv_len"][r])             # empty places of the last page, which is always kept
        key = torch.cat([s["ckv"][pages[places]], s["kpe"][pages[places]]], -1).double().reshape(-1, D)
        key = key[:key.shape[0] - last]
        logit = q[r] @ key.T * s["sm_scale"]
        lses.append(torch.logsumexp(logit, 1))
        outs.append(torch.softmax(logit, 1) @ key[:, :D_CKV])
    return dict(out=torch.stack(outs), lse=torch.stack(lses), sel_indptr=None, sel_indices=None)
