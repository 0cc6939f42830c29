"""Oracle for the paged key/value cache: step plan, append, attention over pages.

TEST INFRASTRUCTURE.  Plain loops in Python integers and fp64; shares no code with the
CUDA path.  The method's source is the attention block's (attention_oracle); the paged
form is this library's own, and these functions restate its definition.
"""
from __future__ import annotations

import numpy as np

from .attention_oracle import rms_norm_heads


def step_plan(ctx_len, new_len, block_table, pool, pool_state, tokens: int, pages: int, page_size: int) -> dict:
    """One step's row starts, block table, slots, lengths and pool, request by request."""
    table = np.array(block_table, dtype=np.int64)
    pool = np.array(pool, dtype=np.int64)
    head, count = (int(v) for v in pool_state)
    max_pages = table.shape[1]
    slots = np.full(tokens, -1, np.int64)
    row, asked, taken, denied = 0, 0, 0, 0
    row_start, kv_len, next_ctx, returned = [0], [], [], []
    ceil = lambda n: -(-n // page_size)  # noqa: E731
    for r, (c, n) in enumerate(zip(map(int, ctx_len), map(int, new_len))):
        if n < 0:
            returned += [int(table[r, j]) for j in range(ceil(c))]
            kv, nxt = 0, 0
        elif n == 0:
            kv, nxt = c, c
        else:
            fits = 0 <= c and c + n <= max_pages * page_size and row + n <= tokens
            want = ceil(c + n) - ceil(c) if fits else 0
            asked += want
            if fits and (want == 0 or asked <= count):
                for j in range(want):
                    table[r, ceil(c) + j] = pool[(head + asked - want + j) % pages]
                for i in range(n):
                    p = c + i
                    slots[row + i] = table[r, p // page_size] * page_size + p % page_size
                if want:
                    taken = asked
                kv, nxt = c + n, c + n
            else:
                denied += 1
                kv, nxt = 0, c
            row += n
        row_start.append(min(row, tokens))
        kv_len.append(kv)
        next_ctx.append(nxt)
    for k, page in enumerate(returned):
        pool[(head + count + k) % pages] = page
    i32 = lambda v: np.asarray(v, dtype=np.int32)  # noqa: E731
    return dict(block_table=i32(table), pool=i32(pool), row_start=i32(row_start), slot_map=i32(slots),
                kv_len=i32(kv_len), next_ctx=i32(next_ctx),
                pool_state=i32([(head + taken) % pages, count - taken + len(returned)]),
                info=i32([row_start[-1], taken, len(returned), denied]))


def append(qkv, slot_map, n_head: int, n_kv_head: int, page_size: int, k_cache, v_cache, eps: float = 1e-6):
    """(q, k_cache, v_cache): QK-norm of the rows, keys and values into their slots (fp64)."""
    T = qkv.shape[0]
    u = np.asarray(qkv, np.float64).reshape(T, n_head + 2 * n_kv_head, -1)
    k_cache, v_cache = np.array(k_cache, np.float64), np.array(v_cache, np.float64)
    for t in range(T):
        if slot_map[t] >= 0:
            page, off = divmod(int(slot_map[t]), page_size)
            k_cache[page, :, off] = rms_norm_heads(u[t, n_head:n_head + n_kv_head], eps)
            v_cache[page, :, off] = u[t, n_head + n_kv_head:]
    return rms_norm_heads(u[:, :n_head], eps).reshape(T, -1), k_cache, v_cache


def paged_attention(q, k_cache, v_cache, block_table, row_start, kv_len, n_head: int, n_kv_head: int) -> dict:
    """out [T][n_head * hd], lse [T][n_head], and weight [T][n_head * hd]: the softmax's sum
    of |v| in place of v, which bounds what a relative error of its weights can do to out."""
    T = q.shape[0]
    page_size, hd = k_cache.shape[2], k_cache.shape[3]
    q = np.asarray(q, np.float64).reshape(T, n_head, hd)
    out = np.zeros((T, n_head, hd))
    weight = np.zeros((T, n_head, hd))
    lse = np.full((T, n_head), -np.inf)
    group = n_head // n_kv_head
    for r in range(len(kv_len)):
        a, n, kv = int(row_start[r]), int(row_start[r + 1] - row_start[r]), int(kv_len[r])
        if n == 0 or kv < n:
            continue
        ids = np.asarray(block_table[r, :-(-kv // page_size)], np.int64)
        k = np.asarray(k_cache[ids], np.float64).transpose(1, 0, 2, 3).reshape(n_kv_head, -1, hd)[:, :kv]
        v = np.asarray(v_cache[ids], np.float64).transpose(1, 0, 2, 3).reshape(n_kv_head, -1, hd)[:, :kv]
        seen = np.arange(kv)[None, :] <= (kv - n) + np.arange(n)[:, None]
        for h in range(n_head):
            g = h // group
            s = np.where(seen, q[a:a + n, h] @ k[g].T / np.sqrt(hd), -np.inf)
            top = s.max(axis=1, keepdims=True)
            e = np.exp(s - top)
            total = e.sum(axis=1, keepdims=True)
            out[a:a + n, h] = (e / total) @ v[g]
            weight[a:a + n, h] = (e / total) @ np.abs(v[g])
            lse[a:a + n, h] = (top + np.log(total))[:, 0]
    return dict(out=out.reshape(T, -1), lse=lse, weight=weight.reshape(T, -1))
