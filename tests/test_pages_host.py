"""Calls that branch rows, move and copy pages refuse what they cannot serve, before any launch (no GPU);
the classes refuse what they were not made for; and the oracles agree with hand-worked values."""
import ctypes
import gc
import weakref

import numpy as np
import pytest
import torch

import aux_loss_free_gb300 as M
from aux_loss_free_gb300 import build as B
from aux_loss_free_gb300 import paged
from oracle import paged_oracle as P

GOOD = dict(requests=3, tokens=20, n_head=8, n_kv_head=2, page_size=16, pages=10, max_pages=4)


@pytest.fixture(scope="module")
def lib():
    return M.load_library(B.build())


def _calls(lib, shape, p, ws=1 << 30, window=7, sinks=2):
    """The status of every call on `shape`, its pointers all p."""
    s, one = ctypes.byref(shape), (ctypes.c_void_p * 1)(p)
    return [lib.moe_paged_fork(s, p, p, window, sinks, *[p] * 9, p, ws, None),
            lib.moe_paged_release(s, p, window, sinks, *[p] * 5, p, ws, None),
            lib.moe_paged_compact(s, *[p] * 7, p, ws, None), lib.moe_paged_copy(s, p, p, 1, 1, one, None)]


BAD_SHAPES = [(dict(requests=0), 1), (dict(tokens=0), 1), (dict(n_kv_head=0), 1), (dict(page_size=0), 1),
              (dict(pages=0), 1), (dict(max_pages=0), 1), (dict(eps=0.0), 1), (dict(requests=4097), 2),
              (dict(head_dim=64), 2), (dict(n_head=9), 2), (dict(page_size=48), 2), (dict(pages=1 << 26), 2),
              (dict(max_pages=(1 << 20) + 1), 2)]


@pytest.mark.parametrize("change,code", BAD_SHAPES, ids=[str(c[0]) for c in BAD_SHAPES])
def test_bad_shapes_are_refused(lib, change, code):
    shape = M.make_paged_shape(**{**GOOD, **change})
    assert M.moe_paged_pages_workspace_size(shape) == 0
    assert _calls(lib, shape, ctypes.c_void_p(16)) == [code] * 4


def test_bad_pointers_windows_and_workspaces_are_refused(lib):
    shape = M.make_paged_shape(**GOOD)
    p, s = ctypes.c_void_p(16), ctypes.byref(shape)
    assert _calls(lib, shape, None) == [1] * 4
    assert _calls(lib, shape, ctypes.c_void_p(24)) == [1] * 4  # not 16-byte aligned
    assert _calls(lib, shape, p, window=-1)[:2] == [1] * 2
    assert _calls(lib, shape, p, sinks=-1)[:2] == [1] * 2
    need = M.moe_paged_pages_workspace_size(shape)
    assert need >= 4 * 3 * 4  # the rows' entries
    assert _calls(lib, shape, p, ws=need - 1)[:3] == [3] * 3
    off = ctypes.c_void_p(24)
    for bad in ((off, None), (None, off)):
        assert lib.moe_paged_fork(s, *bad, 0, 0, *[p] * 9, p, need, None) == 1
    one = (ctypes.c_void_p * 2)(16, 24)
    assert lib.moe_paged_copy(s, p, p, -1, 1, one, None) == 1
    assert lib.moe_paged_copy(s, p, p, 1, -1, one, None) == 1
    assert lib.moe_paged_copy(s, p, p, 1, 1, None, None) == 1
    assert lib.moe_paged_copy(s, p, p, 1, 2, one, None) == 1


def test_fork_oracle_on_a_worked_step():
    """Pages of 16, pages 0, 1, 9 free.  Rows: 0 has 40 tokens in 3, 4, 5; 1 has 20 in 6, 7; 2 has 5 in 8."""
    table = [[3, 4, 5, -1], [6, 7, -1, -1], [8, -1, -1, -1], [-1] * 4]
    pool = [1, 9, -1, -1, -1, -1, -1, -1, -1, 0]  # from place 9 on
    args = ([40, 20, 5, 0], table, pool, [9, 3], 10, 16)
    # 0 stays, 1 goes on from 0's first 36 tokens (page 5 copied), 2 from 0's 32 (whole pages), 3 from 1's 18 tokens:
    # page 7 has room left and 3 alone ends there.  Page 8 is free.
    r = P.fork([0, 0, 0, 1], [40, 36, 32, 18], *args)
    assert r["next_ctx"].tolist() == [40, 36, 32, 18]
    assert r["block_table"].tolist() == [[3, 4, 5, -1], [3, 4, 0, -1], [3, 4, -1, -1], [6, 7, -1, -1]]
    assert r["copies"].tolist() == [[5, 0, 4, 0]]
    assert r["info"].tolist() == [1, 1, 0, 6] and r["pool_state"].tolist() == [0, 3]
    assert r["pool"].tolist() == [1, 9, 8, -1, -1, -1, -1, -1, -1, 0]
    # Rejected tokens and an ended row: 0 cut to 17 tokens (page 5 back), 1 ended.
    r = P.fork([0, -1, 2, 3], [17, 20, 5, 0], *args)
    assert r["next_ctx"].tolist() == [17, 0, 5, 0] and r["info"].tolist() == [0, 3, 0, 3]
    assert r["pool"].tolist() == [1, 9, 5, 6, 7, -1, -1, -1, -1, 0] and r["pool_state"].tolist() == [9, 6]
    # Nothing free and four branches of row 2: page 8 stays row 0's, which is the lowest; the pages
    # given back go to rows 1 to 3.
    r = P.fork([2, 2, 2, 2], None, [40, 20, 5, 0], table, [-1] * 10, [4, 0], 10, 16)
    assert r["block_table"][:, 0].tolist() == [8, 3, 4, 5] and r["info"].tolist() == [3, 5, 0, 4]
    # One page free and none given back: the second branch is cut to whole pages.
    r = P.fork([0, 1, 1, 1], [40, 20, 20, 20], [40, 20, 5, 0], [[3, 4, 5, -1], [6, 7, -1, -1], [7, -1, -1, -1], [-1] * 4],
               [0] + [-1] * 9, [0, 1], 10, 16)
    assert r["next_ctx"].tolist() == [40, 20, 20, 16] and r["info"].tolist() == [1, 0, 1, 6]
    # A window of 9: of 40 tokens the next one sees 32 and later, page 3 holds a sink, page 4 nothing any more.
    r = P.fork(None, None, *args, window=9, sinks=3)
    assert r["block_table"][0].tolist() == [3, -1, 5, -1] and r["block_table"][1].tolist() == [6, 7, -1, -1]
    assert P.fork(None, None, *args, window=10, sinks=3)["block_table"][0].tolist() == [3, 4, 5, -1]


def test_release_and_compact_oracles():
    table = [[3, 4, 5], [3, 7, -1], [8, -1, -1]]
    pool = [1, 9, -1, -1, -1, -1, -1, -1, -1, 0]
    r = P.release([-1, 1, 0], [40, 20, 5], table, pool, [9, 3], 10, 16)
    assert r["next_ctx"].tolist() == [0, 20, 5] and r["pool"].tolist() == [1, 9, 4, 5, -1, -1, -1, -1, -1, 0]
    assert r["info"].tolist() == [0, 2, 0, 3] and r["pool_state"].tolist() == [9, 5]
    r = P.release([1, -1, -1], [40, 20, 5], table, pool, [9, 3], 10, 16, window=8, sinks=0)
    assert r["block_table"][0].tolist() == [-1, -1, 5] and r["info"].tolist() == [0, 4, 0, 1]
    r = P.compact([40, 20, 5], table, pool, 10, 16)
    assert r["block_table"].tolist() == [[3, 4, 0], [3, 1, -1], [2, -1, -1]]
    assert r["copies"].tolist() == [[5, 0, 16, 0], [7, 1, 16, 0], [8, 2, 16, 0]]
    assert r["pool"].tolist()[:5] == [5, 6, 7, 8, 9] and r["pool_state"].tolist() == [0, 5]
    assert r["info"].tolist() == [3, 0, 0, 5]


@pytest.fixture
def step(lib, monkeypatch):
    def reached(*_, **__):
        raise AssertionError("the library was called")

    for name in ("moe_paged_plan", "moe_paged_fork", "moe_paged_release", "moe_paged_compact", "moe_paged_copy",
                 "moe_attention_paged_fwd", "moe_attention_paged_window_fwd"):
        monkeypatch.setattr(paged.L, name, reached)
    return lambda **kw: paged.PagedStep(requests=2, pages=4, page_size=16, max_pages=2, max_tokens=8, device="cpu", **kw)


def test_the_step_refuses_windows_and_branches_that_it_was_not_made_for(step):
    for kw in (dict(window=-1, sharing=True), dict(sinks=-1, sharing=True), dict(window=4)):
        with pytest.raises(ValueError):
            step(**kw)
    plain = step()
    one = torch.tensor([0, 0], dtype=torch.int32)
    with pytest.raises(ValueError, match="sharing"):
        plain.fork(one)
    with pytest.raises(ValueError, match="sharing"):
        plain.compact()
    shared = step(sharing=True)
    for bad, why in ((one.long(), "type"), (one[:1], "size"), (torch.zeros(4, dtype=torch.int32)[::2], "contiguous"),
                     (torch.empty(2, dtype=torch.int32, device="meta"), "device"), (one, "CUDA device")):
        for kw in (dict(parent=bad), dict(keep=bad)):
            with pytest.raises(ValueError, match=why):
                shared.fork(**kw)
    with pytest.raises(ValueError, match="CUDA device"):
        shared.compact()
    with pytest.raises(ValueError, match="size"):
        shared.add_caches(2, torch.zeros(4, 1, 16, 128, dtype=torch.bfloat16))


def test_the_block_refuses_a_window_that_the_step_does_not_keep(step):
    w = [torch.zeros(512, 64, dtype=torch.bfloat16), torch.zeros(64, 256, dtype=torch.bfloat16)]

    def block(st, **kw):
        return paged.PagedAttention(st, 64, 2, 1, *w, **kw)

    kept = step(sharing=True, window=100, sinks=4)
    for kw in (dict(), dict(window=101), dict(window=100, sinks=5), dict(window=-1), dict(window=1, sinks=-1)):
        with pytest.raises(ValueError):
            block(kept, **kw)
    block(kept, window=100, sinks=4)
    block(step(), window=7, sinks=9)


def test_sizes_beyond_32_bits_are_refused(step):
    w = [torch.zeros(512, 64, dtype=torch.bfloat16), torch.zeros(64, 256, dtype=torch.bfloat16)]
    for kw in (dict(window=1 << 32), dict(window=(1 << 32) + 5), dict(window=9, sinks=1 << 32), dict(window=1 << 31)):
        with pytest.raises(ValueError):
            step(sharing=True, **kw)
        with pytest.raises(ValueError):
            paged.PagedAttention(step(), 64, 2, 1, *w, **kw)


def test_a_step_without_sharing_does_not_keep_a_layers_caches(step):
    w = [torch.zeros(512, 64, dtype=torch.bfloat16), torch.zeros(64, 256, dtype=torch.bfloat16)]
    st = step()
    layer = paged.PagedAttention(st, 64, 2, 1, *w)
    caches = [weakref.ref(layer.k_cache), weakref.ref(layer.v_cache)]
    del layer
    gc.collect()
    assert [c() for c in caches] == [None, None]


# --------------------------------------------------------- rows cut short behind a window

def _put(tensor, values):
    tensor.view(-1)[:np.asarray(values).size] = torch.as_tensor(np.asarray(values), dtype=torch.int32).view(-1)


def _oracle_calls(monkeypatch):
    """The step's calls answered by the oracles, on host tensors."""
    n = lambda *ts: [None if t is None else t.numpy().copy() for t in ts]  # noqa: E731

    def fork(shape, parent, keep, window, sinks, ctx, table, table_out, pool, state, state_out, next_ctx, copies, info,
             workspace, stream=None):
        got = P.fork(*n(parent, keep, ctx, table, pool, state), shape.pages, shape.page_size, window, sinks)
        for t, k in ((table_out, "block_table"), (pool, "pool"), (next_ctx, "next_ctx"), (state_out, "pool_state"),
                     (copies, "copies"), (info, "info")):
            _put(t, got[k])

    def release(shape, new_len, window, sinks, ctx, table, pool, state, info, workspace, stream=None):
        got = P.release(*n(new_len, ctx, table, pool, state), shape.pages, shape.page_size, window, sinks)
        for t, k in ((table, "block_table"), (pool, "pool"), (ctx, "next_ctx"), (state, "pool_state"), (info, "info")):
            _put(t, got[k])

    def plan(shape, ctx, new_len, table, pool, state, state_out, row_start, slot_map, kv_len, next_ctx, info, stream=None):
        got = P.step_plan(*n(ctx, new_len, table, pool, state), shape.tokens, shape.pages, shape.page_size)
        for t, k in ((table, "block_table"), (pool, "pool"), (next_ctx, "next_ctx"), (state_out, "pool_state"),
                     (info, "info")):
            _put(t, got[k])

    for name, call in (("fork", fork), ("release", release), ("plan", plan)):
        monkeypatch.setattr(paged.L, f"moe_paged_{name}", call)
    monkeypatch.setattr(paged, "_check_cuda", lambda device: None)


def _nothing_is_missing(st, window, sinks):
    """Every key that a row's next token sees is in a page of its own table, which is not free."""
    head, count = st._state.tolist()
    free = {int(st.pool[(head + i) % st.pages]) for i in range(count)}
    assert len(free) == count
    for r, length in enumerate(st.ctx_len.tolist()):
        for key in range(length):
            if length - key < window or key < sinks:
                page = int(st.block_table[r, key // st.page_size])
                assert 0 <= page < st.pages and page not in free, f"row {r} of {length} tokens: key {key} in page {page}"


@pytest.mark.parametrize("seed", range(24))
def test_rows_cut_short_behind_a_window_keep_what_their_next_token_sees(lib, monkeypatch, seed):
    """A search of eight rows behind a window in a pool that runs short, within what PagedStep allows: a row is cut
    back no further than it stood when it was last planned or forked."""
    _oracle_calls(monkeypatch)
    rng = np.random.default_rng(4200 + seed)
    R, page, cut = 8, 16, 0
    window, sinks = int(rng.choice([2, 9, 16, 17, 24, 40, 70])), int(rng.choice([0, 4, 20]))
    st = paged.PagedStep(requests=R, pages=-(-(window + sinks) // page) + int(rng.integers(5, 9)), page_size=page,
                         max_pages=60, max_tokens=400, device="cpu", sharing=True, window=window, sinks=sinks)
    stood = np.zeros(R, int)
    for turn in range(90):
        ctx = st.ctx_len.numpy().copy()
        if turn % 3:  # a row that is empty stays so, all of them but the first
            new = np.where(ctx > 0, rng.choice([0, 1, 2, 5], R), 0)
            new[0] = new[0] if ctx[0] else 20
            new[ctx > 850] = -1
            st.plan(torch.tensor(new, dtype=torch.int32), 400)
            stood = np.where(new < 0, 0, ctx)
        else:
            live = np.flatnonzero(ctx > 0) if ctx.any() else np.array([0])
            parent = np.where(rng.random(R) < 0.6, rng.choice(live, R), np.arange(R))
            back = np.where(rng.random(R) < 0.3, rng.integers(0, ctx - stood + 1), 0)
            st.fork(torch.tensor(parent, dtype=torch.int32), torch.tensor((ctx - back)[parent], dtype=torch.int32))
            cut += int(st.pages_info[2])
            stood = st.ctx_len.numpy().copy()
        _nothing_is_missing(st, window, sinks)
    assert cut > 0


def test_a_window_near_the_largest_is_kept(lib, monkeypatch):
    seen = []
    monkeypatch.setattr(paged, "_check_cuda", lambda device: None)
    monkeypatch.setattr(paged.L, "moe_paged_release", lambda shape, new, window, *_, **__: seen.append(window))
    monkeypatch.setattr(paged.L, "moe_paged_plan", lambda *_, **__: None)
    monkeypatch.setattr(paged.L, "moe_paged_fork", lambda shape, parent, keep, window, *_, **__: seen.append(window))
    for window in (0, 1, (1 << 31) - 1):
        st = paged.PagedStep(requests=2, pages=4, page_size=16, max_pages=2, max_tokens=8, device="cpu", sharing=True,
                             window=window)
        st.plan(torch.zeros(2, dtype=torch.int32), 8).fork()
    assert seen == [0, 0, 16, 16, (1 << 31) - 1, (1 << 31) - 1]
