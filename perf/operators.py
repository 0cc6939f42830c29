"""The operators of attention over a paged key/value cache: cases, inputs, plain forms.

Three operators, as one serving step calls them in turn:

* plan: the step's block tables, slot map and lengths from the requests' lengths and the
  pool of free pages (moe_paged_plan);
* append: the per-head QK-norm of the step's projected rows and the write of their keys and
  values into the cache's pages (moe_paged_append);
* attention: causal grouped-query attention of every request's new tokens over its pages
  (moe_paged_attention).

Lengths follow from a case alone, so that work(case) is exact; page placement and values
follow from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

HD = 128     # head width of the model's attention
EPS = 1e-6   # of the QK-norm
DEV = "cuda"


# ------------------------------------------------------------------------------- cases

def listed():
    heads = dict(n_head=8, n_kv_head=2)  # the model's grouping: four query heads per key/value head
    return [
        # One decode step's bookkeeping for a handful of requests: pure latency.
        dict(name="plan_decode_8", op="plan", requests=8, chunks=0, chunk=1, kv=2048, page_size=16, pad=0, lens=1),
        # A prompt batch admitted at once: four whole prompts of 2048 tokens.
        dict(name="plan_prompts_4", op="plan", requests=4, chunks=4, chunk=2048, kv=0, page_size=64, pad=0, lens=2),
        # A busy server's mixed step: decoding, prompt chunks, idle and ended requests, padded rows.
        dict(name="plan_mixed_1021", op="plan", requests=1021, chunks=24, chunk=300, kv=8192, page_size=16, pad=77,
             lens=3),
        # One decode step of 64 requests: one row each.
        dict(name="append_decode_64", op="append", tokens=64, page_size=16, pad=3, **heads),
        # The tokens of four prompts of 2048 in one step.
        dict(name="append_prompts_8192", op="append", tokens=8192, page_size=64, pad=0, **heads),
        # A single user's decode step: the latency of one token over a short context.
        dict(name="decode_1x2048", op="attention", requests=1, chunks=0, chunk=1, kv=2047, ragged=False,
             page_size=16, pad=0, lens=4, **heads),
        # A batch of decoding requests with ragged contexts in small pages: bound by reading the cache.
        dict(name="decode_64_ragged", op="attention", requests=64, chunks=0, chunk=1, kv=16000, ragged=True,
             page_size=16, pad=0, lens=5, **heads),
        # One token over a very long context: the work has to be split along the keys.
        dict(name="decode_1x131071", op="attention", requests=1, chunks=0, chunk=1, kv=131070, ragged=False,
             page_size=128, pad=0, lens=6, **heads),
        # A verification step: a few tokens per request, six query heads on two key/value heads, padded rows.
        dict(name="verify_13x5", op="attention", requests=13, chunks=13, chunk=5, kv=3001, ragged=True, page_size=32,
             pad=7, lens=7, n_head=6, n_kv_head=2),
        # Four whole prompts of 2048 tokens: the model's training shape, bound by the tensor cores.
        dict(name="prompts_4x2048", op="attention", requests=4, chunks=4, chunk=2048, kv=0, ragged=False,
             page_size=64, pad=0, lens=8, **heads),
        # Chunked prefill of long prompts at odd lengths.
        dict(name="chunk_2x2011_long", op="attention", requests=2, chunks=2, chunk=2011, kv=14000, ragged=True,
             page_size=32, pad=0, lens=9, **heads),
        # One prompt chunk riding along with decoding requests, as continuous batching schedules them.
        dict(name="mixed_32_and_500", op="attention", requests=33, chunks=1, chunk=500, kv=4096, ragged=True,
             page_size=16, pad=11, lens=10, **heads),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attention", "attention", "attention"])
    page = rng.choice([16, 32, 64, 128])
    pad = rng.choice([0, 0, rng.randint(1, 40)])
    if op == "plan":
        requests = _log_int(rng, 1, 1021)
        return dict(op=op, requests=requests, chunks=min(requests, rng.randint(0, 24)), chunk=_log_int(rng, 1, 300),
                    kv=_log_int(rng, 1, 8192), page_size=page, pad=pad, lens=rng.randint(100, 1 << 30))
    n_head, n_kv_head = rng.choice([(8, 2), (8, 2), (4, 1), (8, 8), (6, 2), (16, 2)])
    if op == "append":
        return dict(op=op, tokens=_log_int(rng, 1, 8192 * 8 // max(8, n_head)), page_size=page, pad=pad,
                    n_head=n_head, n_kv_head=n_kv_head, add=rng.randint(0, 1 << 20))
    kind = rng.choice(["decode", "chunk", "mixed"])
    lens = rng.randint(100, 1 << 30)
    if kind == "decode":  # keys in all up to those of 64 requests with 16000 each
        requests = _log_int(rng, 1, 64)
        kv = _log_int(rng, 16, min(131070, 1024000 // requests) * 2 // max(2, n_kv_head))
        return dict(op=op, requests=requests, chunks=0, chunk=1, kv=kv, ragged=rng.random() < 0.7, page_size=page,
                    pad=pad, lens=lens, n_head=n_head, n_kv_head=n_kv_head)
    if kind == "chunk":
        requests = _log_int(rng, 1, 4)
        chunk = _log_int(rng, 2, 2048 * 8 // max(8, n_head) * 2 // max(2, requests))
        kv = _log_int(rng, 1, 14000 * 2 // max(2, n_kv_head))
        return dict(op=op, requests=requests, chunks=requests, chunk=chunk, kv=kv, ragged=rng.random() < 0.7,
                    page_size=page, pad=pad, lens=lens, n_head=n_head, n_kv_head=n_kv_head)
    requests = _log_int(rng, 2, 33)
    return dict(op=op, requests=requests, chunks=1, chunk=_log_int(rng, 2, 500), kv=_log_int(rng, 16, 4096),
                ragged=True, page_size=page, pad=pad, lens=lens, n_head=n_head, n_kv_head=n_kv_head)


def _plan_lengths(case):
    """(ctx, new) of the plan's requests: chunk requests first admitted or mid-prompt, the others
    decoding one token; one in ten idle and one in ten ended (none in an all-chunk batch)."""
    rng = random.Random(case["lens"])
    ctx, new = [], []
    for r in range(case["requests"]):
        c = rng.randint(1, case["kv"]) if case["kv"] else 0
        kind = rng.random()
        if r < case["chunks"]:
            ctx.append(c if kind < 0.5 else 0)
            new.append(case["chunk"])
        else:
            ctx.append(c)
            new.append(-1 if kind < 0.1 else 0 if kind < 0.2 else 1)
    both = list(zip(ctx, new))
    rng.shuffle(both)
    return [c for c, _ in both], [n for _, n in both]


def _attn_lengths(case):
    """(keys before the step, new tokens) of the attention's requests, the chunk requests last."""
    rng = random.Random(case["lens"])
    ctx, new = [], []
    for r in range(case["requests"]):
        kv = case["kv"]
        ctx.append(rng.randint(kv // 16, kv) if case["ragged"] and kv else kv)
        new.append(case["chunk"] if r >= case["requests"] - case["chunks"] else 1)
    return ctx, new


def _pages(n, page):
    return -(-n // page)


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    page = case["page_size"]
    s = dict(case=case, kept={})
    if case["op"] == "plan":
        ctx, new = _plan_lengths(case)
        held = [_pages(c, page) for c in ctx]
        width = max(_pages(c + max(n, 0), page) for c, n in zip(ctx, new)) + 2
        taken = sum(_pages(c + max(n, 0), page) - h for c, n, h in zip(ctx, new, held))
        free = taken + 1 + len(ctx) // 8
        pages = sum(held) + free
        ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = torch.full((len(ctx), width), -1, dtype=torch.int32, device=DEV)
        col = torch.arange(width, device=DEV)[None, :]
        h = torch.tensor(held, device=DEV)[:, None]
        first = torch.cumsum(h, 0) - h
        table = torch.where(col < h, ids[(first + col).clamp(max=pages - 1)], table)
        head = int(torch.randint(0, pages, (1,), generator=g, device=DEV))
        pool = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
        pool[(head + torch.arange(free, device=DEV)) % pages] = ids[sum(held):]
        rows = sum(max(n, 0) for n in new)
        s.update(requests=len(ctx), tokens=max(1, rows + case["pad"]), pages=pages, width=width, ctx=_i32(ctx),
                 new=_i32(new), table=table.contiguous(), pool=pool, pool_state=_i32([head, free]))
        return s
    H, KV = case["n_head"], case["n_kv_head"]
    if case["op"] == "append":
        T = case["tokens"] + case["pad"]
        # Slots: the tokens of consecutive positions in randomly placed pages; padded rows have none.
        used = _pages(case["tokens"], page)
        pages = used + 3
        ids = torch.randperm(pages, generator=g, device=DEV)[:used]
        t = torch.arange(case["tokens"], device=DEV)
        slots = torch.full((T,), -1, dtype=torch.int32, device=DEV)
        slots[:case["tokens"]] = (ids[t // page] * page + t % page).to(torch.int32)
        qkv = torch.randn(T, (H + 2 * KV) * HD, generator=g, device=DEV).to(torch.bfloat16)
        # One page more than the operator is told of: where the plain form puts rows without a slot.
        caches = [torch.randn(pages + 1, KV, page, HD, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
        s.update(tokens=T, pages=pages, slots=slots, qkv=qkv, k_cache=caches[0], v_cache=caches[1],
                 q=torch.empty(T, H * HD, dtype=torch.bfloat16, device=DEV))
        return s
    ctx, new = _attn_lengths(case)
    R, rows = len(ctx), sum(new)
    T = rows + case["pad"]
    held = [_pages(c + n, page) for c, n in zip(ctx, new)]
    width, pages = max(held), sum(held) + 2
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    h = torch.tensor(held, device=DEV)[:, None]
    col = torch.arange(width, device=DEV)[None, :]
    table = torch.where(col < h, ids[(torch.cumsum(h, 0) - h + col).clamp(max=pages - 1)], -1).to(torch.int32)

    def values(*shape, normed):
        v = torch.randn(*shape, HD, generator=g, device=DEV)
        if normed:  # what the QK-norm leaves
            v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
        return v.to(torch.bfloat16)

    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s.update(requests=R, tokens=T, pages=pages, width=width, most_new=max(new),
             most_kv=max(c + n for c, n in zip(ctx, new)), q=values(T, H, normed=True).reshape(T, H * HD),
             k_cache=values(pages, KV, page, normed=True), v_cache=values(pages, KV, page, normed=False),
             table=table.contiguous(), row_start=_i32(starts), kv_len=_i32([c + n for c, n in zip(ctx, new)]))
    return s


# -------------------------------------------------------------------------- plain forms

def _plain_plan(s):
    page, pages, T, width = s["case"]["page_size"], s["pages"], s["tokens"], s["width"]
    ctx, new = s["ctx"].long(), s["new"].long()
    head, count = s["pool_state"][0].long(), s["pool_state"][1].long()
    n, ended = new.clamp(min=0), new < 0
    have = (ctx + page - 1) // page
    ends = torch.cumsum(n, 0)
    valid = (n > 0) & (ctx + n <= width * page) & (ends <= T)
    need = torch.where(valid, (ctx + n + page - 1) // page - have, 0)
    upto = torch.cumsum(need, 0)
    granted = valid & ((need == 0) | (upto <= count))
    taken = torch.where(granted, upto, 0).amax()
    got = torch.where(granted, need, 0)
    row_start = torch.cat([ends.new_zeros(1), ends]).clamp(max=T)
    col = torch.arange(width, device=DEV)[None, :]
    j = col - have[:, None]
    fresh = (j >= 0) & (j < got[:, None])
    from_pool = s["pool"][(head + (upto - need)[:, None] + j.clamp(min=0)) % pages]
    table = torch.where(fresh, from_pool, s["table"])
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(row_start[1:], t, right=True)
    inside = r < s["requests"]
    r = r.clamp(max=s["requests"] - 1)
    pos = (ctx[r] + t - row_start[r]).clamp(max=width * page - 1)
    slot = table[r, pos // page].long() * page + pos % page
    slot_map = torch.where(inside & granted[r], slot, -1)
    back = torch.where(ended, have, 0)
    back_first = torch.cumsum(back, 0) - back
    gone = col < back[:, None]
    # The ended requests' pages go behind the free ones; the other entries write the pool's last place anew.
    place = torch.where(gone, (head + count + back_first[:, None] + col) % pages, pages)
    pool = torch.cat([s["pool"], s["pool"].new_zeros(1)])
    pool = pool.scatter(0, place.flatten(), s["table"].flatten())[:pages]
    denied = ((n > 0) & ~granted).sum()
    out = dict(table=table, pool=pool, row_start=row_start, slot_map=slot_map,
               kv_len=torch.where(granted, ctx + n, torch.where(ended | (n > 0), 0, ctx)),
               next_ctx=torch.where(granted, ctx + n, torch.where(ended, 0, ctx)),
               pool_state=torch.stack([(head + taken) % pages, count - taken + back.sum()]),
               info=torch.stack([row_start[-1], taken, back.sum(), denied]))
    return {k: v.to(torch.int32) for k, v in out.items()}


def _plain_append(s):
    c = s["case"]
    H, KV, page, T = c["n_head"], c["n_kv_head"], c["page_size"], s["tokens"]
    u = s["qkv"].float().reshape(T, H + 2 * KV, HD)
    qk = u[:, :H + KV]
    qk = qk / torch.sqrt((qk * qk).mean(-1, keepdim=True) + EPS)
    slots = s["slots"].long()
    slots = torch.where(slots < 0, s["pages"] * page, slots)
    s["k_cache"][slots // page, :, slots % page] = qk[:, H:].to(torch.bfloat16)
    s["v_cache"][slots // page, :, slots % page] = u[:, H + KV:].to(torch.bfloat16)
    return dict(q=qk[:, :H].reshape(T, H * HD).to(torch.bfloat16), k_cache=s["k_cache"][:s["pages"]],
                v_cache=s["v_cache"][:s["pages"]])


def _plain_attention(s):
    c = s["case"]
    H, KV, page, T, R = c["n_head"], c["n_kv_head"], c["page_size"], s["tokens"], s["requests"]
    G, N, S = H // KV, s["most_new"], s["most_kv"]
    starts, kv_len = s["row_start"].long(), s["kv_len"].long()
    new = starts[1:] - starts[:-1]
    i = torch.arange(N, device=DEV)
    rows = (starts[:-1, None] + i).clamp(max=T - 1)
    q = s["q"].float().reshape(T, KV, G, HD)[rows].permute(0, 2, 3, 1, 4).reshape(R, KV, G * N, HD)
    p = torch.arange(S, device=DEV)
    slot_page = s["table"].long().clamp(min=0)[:, p // page]
    inside = (p < kv_len[:, None])[:, None, :, None]
    k = s["k_cache"][slot_page, :, p % page].float().permute(0, 2, 1, 3)
    v = torch.where(inside, s["v_cache"][slot_page, :, p % page].float().permute(0, 2, 1, 3), 0.0)
    x = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(HD)
    sees = p <= (kv_len - new)[:, None, None] + i[None, :, None]
    sees = sees & (p < kv_len[:, None, None]) & (kv_len >= new)[:, None, None]
    x = torch.where(sees[:, None, None], x.reshape(R, KV, G, N, S), -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.reshape(R, KV, G * N, S), v).reshape(R, KV, G, N, HD)
    o = o / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total))[..., 0]
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(starts[1:], t, right=True)
    inside = (r < R)[:, None, None]
    r = r.clamp(max=R - 1)
    i = (t - starts[r]).clamp(max=N - 1)
    out = torch.where(inside[..., None], o.permute(0, 3, 1, 2, 4)[r, i], 0.0).reshape(T, H * HD)
    lse = torch.where(inside, lse.permute(0, 3, 1, 2)[r, i], -math.inf).reshape(T, H)
    return dict(out=out.to(torch.bfloat16), lse=lse)


# ------------------------------------------------------------------ the framework's calls

def _keep(s):
    """What a serving program holds from step to step: the shape, the outputs, the workspace."""
    import aux_loss_free_gb300 as M
    c, k = s["case"], s["kept"]
    op = c["op"]
    k["M"] = M
    k["shape"] = M.make_paged_shape(s.get("requests", 1), s["tokens"], c.get("n_head", 8), c.get("n_kv_head", 2),
                                    c["page_size"], s["pages"], s.get("width", 1), eps=EPS)

    def i32(*shape):
        return torch.empty(*shape, dtype=torch.int32, device=DEV)

    if op == "plan":
        k.update(row_start=i32(s["requests"] + 1), slot_map=i32(s["tokens"]), kv_len=i32(s["requests"]),
                 next_ctx=i32(s["requests"]), pool_state=i32(2), info=i32(4))
    elif op == "attention":
        k.update(out=torch.empty_like(s["q"]),
                 lse=torch.empty(s["tokens"], c["n_head"], dtype=torch.float32, device=DEV),
                 workspace=torch.empty(M.moe_paged_attention_workspace_size(k["shape"]), dtype=torch.uint8,
                                       device=DEV))
    return k


def _own(s):
    k = s["kept"] or _keep(s)
    M, op = k["M"], s["case"]["op"]
    if op == "plan":
        M.moe_paged_plan(k["shape"], s["ctx"], s["new"], s["table"], s["pool"], s["pool_state"], k["pool_state"],
                         k["row_start"], k["slot_map"], k["kv_len"], k["next_ctx"], k["info"])
        return dict(table=s["table"], pool=s["pool"], row_start=k["row_start"], slot_map=k["slot_map"],
                    kv_len=k["kv_len"], next_ctx=k["next_ctx"], pool_state=k["pool_state"], info=k["info"])
    if op == "append":
        M.moe_paged_append(k["shape"], s["qkv"], s["slots"], s["q"], s["k_cache"], s["v_cache"])
        return dict(q=s["q"], k_cache=s["k_cache"][:s["pages"]], v_cache=s["v_cache"][:s["pages"]])
    M.moe_paged_attention(k["shape"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["row_start"], s["kv_len"],
                          k["out"], k["lse"], k["workspace"])
    return dict(out=k["out"], lse=k["lse"])


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "append": _plain_append, "attention": _plain_attention}[state["case"]["op"]](state)


# ------------------------------------------------------------------------ work and truth

def work(case):
    page = case["page_size"]
    if case["op"] == "plan":
        ctx, new = _plan_lengths(case)
        R, rows = len(ctx), sum(max(n, 0) for n in new)
        fresh = sum(_pages(c + max(n, 0), page) - _pages(c, page) for c, n in zip(ctx, new))
        back = sum(_pages(c, page) for c, n in zip(ctx, new) if n < 0)
        # Lengths and pool state in; table entries and pool moved; row starts, slots, lengths, state and info out.
        return dict(bytes=4 * (2 * R + 2 + 2 * fresh + 2 * back + (R + 1) + rows + case["pad"] + 2 * R + 6), flops=0)
    H, KV = case["n_head"], case["n_kv_head"]
    if case["op"] == "append":
        T, n = case["tokens"] + case["pad"], case["tokens"]
        moved = 2 * HD * (T * H + n * 2 * KV)  # a row without a slot has its query heads moved alone
        return dict(bytes=2 * moved + 4 * T, flops=3 * HD * (T * H + n * KV))
    ctx, new = _attn_lengths(case)
    T = sum(new) + case["pad"]
    keys = sum(c + n for c, n in zip(ctx, new))
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
    entries = sum(_pages(c + n, page) for c, n in zip(ctx, new))
    return dict(bytes=2 * HD * (2 * H * sum(new) + H * case["pad"] + 2 * KV * keys) + 4 * H * T
                + 4 * (entries + 2 * len(ctx) + 1), flops=4 * HD * H * pairs)


def _exact_plan(case, s):
    page, pages, T, width = case["page_size"], s["pages"], s["tokens"], s["width"]
    ctx, new = s["ctx"].tolist(), s["new"].tolist()
    table, pool = s["table"].cpu().numpy().copy(), s["pool"].cpu().numpy().copy()
    head, count = s["pool_state"].tolist()
    before = table.copy()
    slots = np.full(T, -1, np.int32)
    row, starts, kv_len, nxt = 0, [0], [], []
    asked = taken = returned = denied = 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        if n < 0:
            for j in range(_pages(c, page)):
                pool[(head + count + returned) % pages] = before[r, j]
                returned += 1
            kv_len.append(0)
            nxt.append(0)
        elif n == 0:
            kv_len.append(c)
            nxt.append(c)
        else:
            ok = c + n <= width * page and row + n <= T
            need = _pages(c + n, page) - _pages(c, page) if ok else 0
            asked += need
            ok = ok and (need == 0 or asked <= count)
            if ok:
                for j in range(need):
                    table[r, _pages(c, page) + j] = pool[(head + asked - need + j) % pages]
                taken = max(taken, asked)
                for i in range(n):
                    slots[row + i] = table[r, (c + i) // page] * page + (c + i) % page
            denied += not ok
            kv_len.append(c + n if ok else 0)
            nxt.append(c + n if ok else c)
            row += n
        starts.append(min(row, T))
    i32 = lambda v: np.asarray(v, np.int32)  # noqa: E731
    return dict(table=i32(table), pool=i32(pool), row_start=i32(starts), slot_map=slots, kv_len=i32(kv_len),
                next_ctx=i32(nxt), pool_state=i32([(head + taken) % pages, count - taken + returned]),
                info=i32([starts[-1], taken, returned, denied]))


def _exact_append(case, s):
    H, KV, page = case["n_head"], case["n_kv_head"], case["page_size"]
    u = s["qkv"].double().view(s["tokens"], -1, HD)
    norm = u / (u.pow(2).sum(-1, keepdim=True) / HD + EPS).pow(0.5)
    k, v = s["k_cache"].double(), s["v_cache"].double()
    keep = s["slots"] >= 0
    at = s["slots"][keep].long()
    page_of, off = torch.div(at, page, rounding_mode="floor"), at.remainder(page)
    for g in range(KV):
        k[page_of, g, off] = norm[keep, H + g]
        v[page_of, g, off] = u[keep, H + KV + g]
    return dict(q=norm[:, :H].flatten(1), k_cache=k[:s["pages"]], v_cache=v[:s["pages"]])


def _exact_attention(case, s):
    H, KV, page, T = case["n_head"], case["n_kv_head"], case["page_size"], s["tokens"]
    ctx, new = _attn_lengths(case)
    out = torch.zeros(T, H, HD, dtype=torch.float64, device=DEV)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=DEV)
    q = s["q"].double().view(T, H, HD)
    row = 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        held = s["table"][r, :_pages(c + n, page)].long()
        for g in range(KV):
            keys = s["k_cache"][held, g].double().flatten(0, 1)[:c + n]
            vals = s["v_cache"][held, g].double().flatten(0, 1)[:c + n]
            for h in range(g * (H // KV), (g + 1) * (H // KV)):
                for a in range(0, n, 512):  # positions c + a .. of this piece
                    b = min(n, a + 512)
                    z = q[row + a:row + b, h] @ keys[:c + b].T / HD ** 0.5
                    late = torch.ones(b - a, c + b, dtype=torch.bool, device=DEV).triu(c + a + 1)
                    z.masked_fill_(late, -math.inf)
                    norm = z.logsumexp(-1)
                    out[row + a:row + b, h] = (z - norm[:, None]).exp() @ vals[:c + b]
                    lse[row + a:row + b, h] = norm
        row += n
    return dict(out=out.flatten(1), lse=lse)


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "attention": _exact_attention}[case["op"]](case, s)
