"""GPU tests of rows that branch, are cut back and end, of pages moved together, and of page copies,
against oracle/paged_oracle.py.  Whole numbers and copies: everything is equal."""
import numpy as np
import pytest
import torch

import aux_loss_free_gb300 as M
from oracle import paged_oracle as P

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    M.load_library()
    yield
    assert M.moe_device_status() == 0


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def _state(rng, R, page, width, free, share=0.5, holes=0.0, extra=0):
    """A cache as earlier calls leave it: rows that share whole pages of a common beginning, a page with
    room left one row's alone, some pages given up, the pool's ring from a random place on."""
    ctx = rng.integers(0, width * page + 1, R)
    ctx[rng.random(R) < 0.1] = 0
    ctx[rng.random(R) < 0.2] = ctx[rng.random(R) < 0.2].max(initial=0) // page * page
    number = np.full((R, width), -1)
    used = 0
    for r in range(R):
        held = -(-int(ctx[r]) // page)
        common = 0
        if r and rng.random() < share:
            q = int(rng.integers(max(0, r - 5), r))
            common = int(rng.integers(0, min(ctx[r], ctx[q]) // page + 1))
            number[r, :common] = number[q, :common]
        number[r, common:held] = np.arange(used, used + held - common)
        used += held - common
    pages = used + free + extra
    ids = rng.permutation(max(pages, 1))
    table = np.where(number >= 0, ids[np.maximum(number, 0)], -1)
    table[(rng.random(table.shape) < holes) & (np.arange(width)[None] < (ctx // page)[:, None])] = -1
    table = np.where(np.arange(width)[None] < -(-ctx // page)[:, None], table, rng.integers(-9, 9, table.shape))
    head = int(rng.integers(0, max(pages, 1)))
    pool = np.full(max(pages, 1), -7)
    pool[(head + np.arange(free)) % max(pages, 1)] = ids[used:used + free]
    return dict(ctx=ctx, table=table, pool=pool, state=[head, free], pages=max(pages, 1), page=page)


def _branches(rng, s, kind):
    R = len(s["ctx"])
    parent = np.arange(R)
    if kind == "any":
        parent = rng.integers(-1, R, R)
    elif kind == "few":
        parent = np.where(rng.random(R) < 0.2, rng.integers(-1, R, R), parent)
    elif kind == "one":
        parent[:] = int(np.argmax(s["ctx"]))
    have = np.where(parent >= 0, s["ctx"][parent], 0)
    keep = np.where(rng.random(R) < 0.5, have, rng.integers(-2, have + 3))
    return parent, keep


def _shape(s, KV=2):
    R, width = s["table"].shape
    return M.make_paged_shape(R, 1, KV, KV, s["page"], s["pages"], width)


def _workspace(shape):
    return torch.randint(0, 256, (M.moe_paged_pages_workspace_size(shape),), dtype=torch.uint8, device=DEV)


def _run_fork(s, parent, keep, window=0, sinks=0, in_place=True, stream=None):
    R, width = s["table"].shape
    shape = _shape(s)
    g = dict(block_table=_i32(s["table"]), pool=_i32(s["pool"]), next_ctx=_i32(s["ctx"]), pool_state=_i32(s["state"]),
             copies=torch.full((R, 4), -77, dtype=torch.int32, device=DEV), info=_i32([-77] * 4))
    ins = g if in_place else {k: v.clone() for k, v in g.items()}
    args = [None if v is None else _i32(v) for v in (parent, keep)]
    ws = _workspace(shape)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())

    def call():
        M.moe_paged_fork(shape, *args, window, sinks, ins["next_ctx"], ins["block_table"], g["block_table"], g["pool"],
                         ins["pool_state"], g["pool_state"], g["next_ctx"], g["copies"], g["info"], ws, stream=stream)

    call()
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy() for k, v in g.items()}
    if not in_place:  # repeated on the same inputs
        call()
        torch.cuda.synchronize()
        assert all(np.array_equal(got[k], v.cpu().numpy()) for k, v in g.items())
    return got


def _equal(got, ref):
    n = len(ref["copies"]) if "copies" in ref else 0
    for k, v in ref.items():
        assert np.array_equal(got[k][:n] if k == "copies" else got[k], v), f"{k}: {got[k]} != {v}"
    if "copies" in ref:
        assert (got["copies"][n:] == -77).all()


def _check_fork(s, parent, keep, window=0, sinks=0, **kw):
    got = _run_fork(s, parent, keep, window, sinks, **kw)
    ref = P.fork(parent, keep, s["ctx"], s["table"], s["pool"], s["state"], s["pages"], s["page"], window, sinks)
    _equal(got, ref)
    return ref


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind", ["any", "few", "one", "self"])
@pytest.mark.parametrize("R,page,width", [(1, 16, 1), (2, 128, 3), (9, 16, 140), (33, 32, 20), (300, 64, 7), (1021, 16, 30),
                                          (1025, 16, 3), (4096, 16, 5), (3, 16, 5000)])
def test_fork_matches_oracle(R, page, width, kind, in_place):
    rng = np.random.default_rng(R + width)
    s = _state(rng, R, page, width, free=R + 3)
    parent, keep = _branches(rng, s, kind)
    ref = _check_fork(s, parent, keep, in_place=in_place)
    assert ref["info"][2] == 0
    _check_fork(s, parent, None, in_place=in_place)
    _check_fork(s, None, keep, in_place=in_place)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (40, 17), (100, 4), (5000, 0), (2 ** 31 - 1, 3), (1, 2 ** 31 - 1)])
def test_fork_gives_up_pages_behind_a_window(window, sinks, in_place):
    rng = np.random.default_rng(window % 1000 + sinks % 1000)
    for R, page, width in ((40, 16, 30), (500, 32, 12)):
        s = _state(rng, R, page, width, free=R, holes=0.2)
        for kind in ("any", "self"):
            _check_fork(s, *_branches(rng, s, kind), window, sinks, in_place=in_place)


@pytest.mark.parametrize("free", [0, 1, 2, 7, 30])
def test_fork_cuts_rows_short_when_the_pool_has_no_page(free):
    """Forty empty rows go on from rows that stay: more copies than pages are free."""
    cut = 0
    for seed in range(8):
        rng = np.random.default_rng(seed)
        s = _state(rng, 64, 16, 6, free=free, share=0.9, extra=int(rng.integers(0, 3)))
        s["ctx"] = np.where(np.arange(64) < 40, 0, s["ctx"])
        cut += _check_fork(s, np.where(np.arange(64) < 40, 40 + np.arange(64) % 24, np.arange(64)), None)["info"][2]
    assert cut > 0 or free >= 30
    assert M.moe_device_status() == 0  # a short pool is no error


@pytest.mark.parametrize("seed", range(30))
def test_fork_at_random(seed):
    rng = np.random.default_rng(3000 + seed)
    R, page = int(np.exp(rng.uniform(0, np.log(700)))), int(rng.choice([16, 32, 64, 128]))
    s = _state(rng, R, page, int(rng.integers(1, 40)), free=int(rng.integers(0, R + 2)), share=rng.random(),
               holes=rng.choice([0, 0.1]), extra=int(rng.integers(0, 50)))
    window = int(rng.choice([0, 0, rng.integers(1, 300)]))
    _check_fork(s, *_branches(rng, s, rng.choice(["any", "few", "one", "self"])), window, int(rng.integers(0, 60)),
                in_place=bool(rng.integers(2)))


def test_fork_of_a_large_cache():
    """Two million pages, most of them nobody's."""
    rng = np.random.default_rng(5)
    s = _state(rng, 50, 16, 40, free=2_000_000)
    _check_fork(s, *_branches(rng, s, "any"))
    _check_fork(s, *_branches(rng, s, "few"), in_place=False)


def _check_release(s, new, window=0, sinks=0):
    shape = _shape(s)
    g = dict(next_ctx=_i32(s["ctx"]), block_table=_i32(s["table"]), pool=_i32(s["pool"]), pool_state=_i32(s["state"]),
             info=_i32([-77] * 4))
    M.moe_paged_release(shape, _i32(new), window, sinks, g["next_ctx"], g["block_table"], g["pool"], g["pool_state"],
                        g["info"], _workspace(shape))
    torch.cuda.synchronize()
    ref = P.release(new, s["ctx"], s["table"], s["pool"], s["state"], s["pages"], s["page"], window, sinks)
    _equal({k: v.cpu().numpy() for k, v in g.items()}, ref)
    return ref


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (50, 17)])
@pytest.mark.parametrize("R,page,width", [(1, 16, 1), (33, 32, 20), (1021, 16, 30), (4096, 16, 3)])
def test_release_matches_oracle(R, page, width, window, sinks):
    rng = np.random.default_rng(R)
    s = _state(rng, R, page, width, free=3, holes=0.1 if window else 0)
    for p in (0.0, 0.2, 1.0):
        ref = _check_release(s, np.where(rng.random(R) < p, -1, rng.integers(0, 5, R)), window, sinks)
        assert p < 1 or ref["info"][3] == 0


def _check_compact(s, in_place):
    shape = _shape(s)
    table, ctx = _i32(s["table"]), _i32(s["ctx"])
    g = dict(block_table=table if in_place else table.clone(), pool=_i32(s["pool"]), pool_state=_i32([-77] * 2),
             copies=torch.full((max(1, s["pages"] // 2), 4), -77, dtype=torch.int32, device=DEV), info=_i32([-77] * 4))
    M.moe_paged_compact(shape, ctx, table, g["block_table"], g["pool"], g["pool_state"], g["copies"], g["info"],
                        _workspace(shape))
    torch.cuda.synchronize()
    ref = P.compact(s["ctx"], s["table"], s["pool"], s["pages"], s["page"])
    _equal({k: v.cpu().numpy() for k, v in g.items()}, ref)
    return ref


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("R,page,width,free", [(1, 16, 1, 0), (1, 16, 1, 1), (2, 128, 3, 40), (33, 32, 20, 3),
                                               (300, 64, 7, 9000), (1021, 16, 30, 20000), (4096, 16, 3, 5), (9, 16, 140, 0),
                                               (20, 16, 40, 1000000)])
def test_compact_matches_oracle(R, page, width, free, in_place):
    rng = np.random.default_rng(R + free)
    for holes in (0, 0.2):
        s = _state(rng, R, page, width, free=free, holes=holes, extra=int(rng.integers(0, 3)))
        _check_compact(s, in_place)
    s["ctx"][:] = 0  # nothing in use
    assert _check_compact(s, in_place)["info"].tolist() == [0, 0, 0, 0]


def test_compact_of_a_full_cache_moves_nothing():
    rng = np.random.default_rng(2)
    s = _state(rng, 7, 16, 9, free=0, share=0)
    assert _check_compact(s, True)["info"][0] == 0


# ------------------------------------------------------------------------------ copies

@pytest.mark.parametrize("KV,page,caches,n", [(2, 16, 2, 1), (2, 16, 2, 300), (1, 128, 3, 20), (4, 64, 70, 5), (3, 32, 130, 9),
                                              (2, 16, 1, 0)])
def test_copies(KV, page, caches, n):
    rng = np.random.default_rng(KV * page)
    pages = 2 * n + 5
    ids = rng.permutation(pages)
    tokens = rng.integers(0, page + 1, n)
    tokens[:2] = [page, 0][:min(n, 2)]
    jobs = np.full((n + 3, 4), 10 ** 9)  # past the count: not looked at
    jobs[:n] = np.stack([ids[:n], ids[n:2 * n], tokens, np.zeros(n)], 1)
    mem = [torch.randint(-2 ** 15, 2 ** 15, (pages, KV, page, 128), dtype=torch.int16, device=DEV).view(torch.bfloat16)
           for _ in range(caches)]
    want = [m.clone().view(torch.int16) for m in mem]
    for src, dst, t, _ in jobs[:n]:
        for w in want:
            w[dst, :, :t] = w[src, :, :t]
    shape = M.make_paged_shape(1, 1, KV, KV, page, pages, 1)
    M.moe_paged_copy(shape, _i32(jobs), _i32([n, 0, 0, 0]), mem)
    torch.cuda.synchronize()
    for m, w in zip(mem, want):
        assert torch.equal(m.view(torch.int16), w)
    M.moe_paged_copy(shape, _i32(jobs), _i32([-3, 0, 0, 0]), mem)  # a count below none is none
    M.moe_paged_copy(shape, _i32(jobs), _i32([n, 0, 0, 0]), [])
    if n:
        M.moe_paged_copy(shape, _i32(jobs[:1]), _i32([n, 0, 0, 0]), mem)  # no more than there is room for
    torch.cuda.synchronize()
    for m, w in zip(mem, want):
        assert torch.equal(m.view(torch.int16), w)


def test_copies_far_into_a_large_cache():
    """Elements past 2^32."""
    KV, page, pages = 2, 128, 140000
    cache = torch.empty(pages, KV, page, 128, dtype=torch.bfloat16, device=DEV)
    far = [pages - 1, 65536, 131072, 3]
    for i, f in enumerate(far):
        cache[f] = torch.randn(KV, page, 128, device=DEV).to(torch.bfloat16) if i % 2 == 0 else 0
    src, dst = far[0::2], far[1::2]
    want = [cache[f].clone() for f in src]
    M.moe_paged_copy(M.make_paged_shape(1, 1, KV, KV, page, pages, 1), _i32([[s, d, page, 0] for s, d in zip(src, dst)]),
                     _i32([2, 0, 0, 0]), [cache])
    torch.cuda.synchronize()
    for d, w in zip(dst, want):
        assert torch.equal(cache[d], w)


@pytest.mark.parametrize("bad", [(-1, 2, 16), (8, 2, 16), (1, -1, 16), (1, 8, 16), (1, 2, 17), (1, 2, -1)])
def test_copies_out_of_range_are_reported_and_left_out(bad):
    cache = torch.randn(8, 2, 16, 128, device=DEV).to(torch.bfloat16)
    want = cache.clone()
    want[4] = want[3]
    assert M.moe_device_status() == 0
    M.moe_paged_copy(M.make_paged_shape(1, 1, 2, 2, 16, 8, 1), _i32([[*bad, 0], [3, 4, 16, 0]]), _i32([2, 0, 0, 0]), [cache])
    assert M.moe_device_status() == 6
    assert torch.equal(cache, want)


# ------------------------------------------------------------------------- other calls

def _lengths(r, c):
    return lambda t: t["ctx"].__setitem__(r, c)


def _entry(v):
    return lambda t: t["table"].__setitem__((3, 0), v)


def _parent(v):
    return lambda t: t["parent"].__setitem__(4, v)


def _pool(*v):
    return lambda t: t.update(state=list(v))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("change,meant", [(_lengths(3, 97), _lengths(3, 0)), (_lengths(3, -1), _lengths(3, 0)),
                                          (_entry(100), _entry(-1)), (_entry(-2), _entry(-1)),
                                          (_parent(12), _parent(-1)), (_parent(-2), _parent(-1)),
                                          (_pool(100, 3), _pool(0, 0)), (_pool(-1, 3), _pool(0, 0)),
                                          (_pool(0, 101), _pool(0, 0)), (_pool(0, -1), _pool(0, 0))])
def test_what_is_out_of_range_is_reported(change, meant, in_place):
    """MOE_ERR_DEVICE, and the results of a call in which it is what the documentation puts in its place."""
    rng = np.random.default_rng(7)
    s = dict(ctx=rng.integers(20, 96, 12), table=np.arange(72).reshape(12, 6), pages=100, page=16, state=[0, 28],
             pool=np.r_[np.arange(72, 100), np.full(72, -7)], parent=np.array([0, 0, 2, 3, 3, 5, 6, 7, -1, 9, 10, 11]))
    a, b = ({k: v.copy() if isinstance(v, np.ndarray) else v for k, v in s.items()} for _ in range(2))
    change(a)
    meant(b)
    assert M.moe_device_status() == 0
    got = _run_fork(a, a["parent"], None, in_place=in_place)
    assert M.moe_device_status() == 6
    ref = P.fork(b["parent"], None, b["ctx"], b["table"], b["pool"], b["state"], 100, 16)
    for k in ("next_ctx", "info", "pool_state"):
        assert np.array_equal(got[k], ref[k]), k
    rows = P.pages_in_use(ref["next_ctx"], ref["block_table"], 16)
    assert P.pages_in_use(got["next_ctx"], got["block_table"], 16) == rows


def test_more_free_pages_than_there_are_is_reported():
    s = dict(ctx=np.array([20, 80, 33, 64]), table=np.arange(20).reshape(4, 5), pages=20, page=16, pool=np.full(20, 3),
             state=[2, 19])
    assert M.moe_device_status() == 0
    got = _run_fork(s, [-1] * 4, None)
    assert M.moe_device_status() == 6
    assert got["pool_state"][1] == 20 and (got["next_ctx"] == 0).all()


def test_calls_on_other_streams_and_in_a_graph():
    rng = np.random.default_rng(9)
    states = [_state(rng, 200, 16, 30, free=300), _state(rng, 40, 32, 100, free=70)]
    jobs = [(s, *_branches(rng, s, "any")) for s in states]
    for stream in (torch.cuda.Stream(), torch.cuda.Stream()):
        for s, parent, keep in jobs:
            _check_fork(s, parent, keep, stream=stream)
    # Captured in place: every replay goes on from the last.
    s, parent, keep = jobs[0]
    shape, R, width = _shape(s), 200, 30
    ctx, table, pool, state = (_i32(s[k]) for k in ("ctx", "table", "pool", "state"))
    par, kp, new = _i32(parent), _i32(keep), _i32([0] * R)
    copies, info = torch.zeros(max(R, s["pages"] // 2), 4, dtype=torch.int32, device=DEV), _i32([0] * 4)
    cache = torch.randn(s["pages"], 2, 16, 128, device=DEV).to(torch.bfloat16)
    ws = _workspace(shape)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        M.moe_paged_release(shape, new, 0, 0, ctx, table, pool, state, info, ws, stream=side)
        M.moe_paged_fork(shape, par, kp, 0, 0, ctx, table, table, pool, state, state, ctx, copies, info, ws, stream=side)
        M.moe_paged_copy(shape, copies, info, [cache], stream=side)
        M.moe_paged_compact(shape, ctx, table, table, pool, state, copies, info, ws, stream=side)
        M.moe_paged_copy(shape, copies, info, [cache], stream=side)
    now = dict(s)

    def tokens(ctx_, table_, mem):  # of every row, what it finds in the cache
        return [[mem[p, :, :min(16, int(c) - 16 * j)].float().cpu().numpy() for j, p in enumerate(row)]
                for c, row in zip(ctx_, P.pages_in_use(ctx_, table_, 16))]

    for turn in range(4):
        ended = np.where(rng.random(R) < 0.1, -1, 1)
        par_np = np.where(rng.random(R) < 0.3, rng.integers(-1, R, R), np.arange(R))
        keep_np = rng.integers(0, 500, R)
        new.copy_(_i32(ended))
        par.copy_(_i32(par_np))
        kp.copy_(_i32(keep_np))
        before = tokens(now["ctx"], now["table"], cache)
        graph.replay()
        torch.cuda.synchronize()
        r1 = P.release(ended, now["ctx"], now["table"], now["pool"], now["state"], s["pages"], 16)
        r2 = P.fork(par_np, keep_np, r1["next_ctx"], r1["block_table"], r1["pool"], r1["pool_state"], s["pages"], 16)
        r3 = P.compact(r2["next_ctx"], r2["block_table"], r2["pool"], s["pages"], 16)
        now.update(ctx=r2["next_ctx"], table=r3["block_table"], pool=r3["pool"], state=r3["pool_state"])
        for got, want in ((ctx, now["ctx"]), (table, now["table"]), (pool, now["pool"]), (state, now["state"]),
                          (info, r3["info"])):
            assert np.array_equal(got.cpu().numpy(), want)
        after = tokens(now["ctx"], now["table"], cache)
        for r in range(R):
            q, n = par_np[r], int(now["ctx"][r])
            if n == 0:
                continue
            was = np.concatenate(before[q], axis=1)[:, :n]
            assert np.array_equal(np.concatenate(after[r], axis=1), was)


def test_calls_on_two_streams_at_once():
    """Forks, compactions and copies of two caches queued again and again without a wait between the streams."""
    rng = np.random.default_rng(10)
    queues = []
    for R, page, width in ((300, 16, 30), (60, 64, 200)):
        s = _state(rng, R, page, width, free=R)
        parent, keep = _branches(rng, s, "any")
        shape, stream = _shape(s), torch.cuda.Stream()
        ins = [_i32(v) for v in (parent, keep, s["ctx"], s["table"], s["pool"], s["state"])]
        outs = dict(block_table=ins[3].clone(), pool_state=_i32([-7] * 2), next_ctx=_i32([-7] * R),
                    copies=torch.full((R, 4), -77, dtype=torch.int32, device=DEV), info=_i32([-7] * 4))
        moved = dict(block_table=ins[3].clone(), pool=ins[4].clone(), pool_state=_i32([-7] * 2),
                     copies=torch.full((s["pages"] // 2, 4), -77, dtype=torch.int32, device=DEV), info=_i32([-7] * 4))
        cache = torch.randn(s["pages"], 2, page, 128, device=DEV).to(torch.bfloat16)
        queues.append((s, parent, keep, shape, stream, ins, outs, moved, cache, _workspace(shape), cache.clone()))
    torch.cuda.synchronize()
    for _ in range(30):
        for s, _, _, shape, stream, i, o, m, cache, ws, _ in queues:
            M.moe_paged_fork(shape, i[0], i[1], 0, 0, i[2], i[3], o["block_table"], i[4], i[5], o["pool_state"],
                             o["next_ctx"], o["copies"], o["info"], ws, stream=stream)
            M.moe_paged_copy(shape, o["copies"], o["info"], [cache], stream=stream)
            M.moe_paged_compact(shape, i[2], i[3], m["block_table"], m["pool"], m["pool_state"], m["copies"], m["info"],
                                ws, stream=stream)
    torch.cuda.synchronize()
    for s, parent, keep, _, _, ins, o, m, cache, _, was in queues:
        ref = P.fork(parent, keep, s["ctx"], s["table"], s["pool"], s["state"], s["pages"], s["page"])
        _equal({**{k: v.cpu().numpy() for k, v in o.items()}, "pool": ins[4].cpu().numpy()}, ref)
        _equal({k: v.cpu().numpy() for k, v in m.items()}, P.compact(s["ctx"], s["table"], s["pool"], s["pages"], s["page"]))
        for src, dst, t, _ in ref["copies"]:
            was[dst, :, :t] = was[src, :, :t]
        assert torch.equal(cache.view(torch.int16), was.view(torch.int16))
    assert M.moe_device_status() == 0


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("free", [0, 1, 2])
@pytest.mark.parametrize("page,window,sinks", [(16, 24, 0), (16, 1, 0), (16, 17, 33), (64, 40, 4), (128, 300, 0)])
def test_rows_cut_short_behind_a_window_find_what_they_see(page, window, sinks, free, in_place):
    """Releases and forks that are given window + page_size - 1 for a window: in every row, cut short or not, the page of
    every key that its next token sees is the parent's, or the copy of the parent's."""
    cut = 0
    for seed in range(4):
        rng = np.random.default_rng(100 * seed + page + window)
        R, width = 20, 12
        s = _state(rng, R, page, width, free=free, share=0.0)
        s["ctx"][:12] = 0  # rows that will branch off the others
        new = np.where(rng.random(R) < 0.1, -1, 1)
        kept = window + page - 1
        ref = _check_release(s, new, kept, sinks)
        s.update(ctx=ref["next_ctx"].astype(np.int64), table=ref["block_table"], pool=ref["pool"],
                 state=[int(ref["pool_state"][0]), free])  # what came back is somebody else's
        parent = np.r_[rng.integers(12, R, 12), np.arange(12, R)]
        got = _run_fork(s, parent, None, kept, sinks, in_place=in_place)
        copied = {int(d): int(a) for a, d, _, _ in got["copies"][:got["info"][0]]}
        for r, q in enumerate(parent):
            length, had = int(got["next_ctx"][r]), int(s["ctx"][q])
            assert length == had or length == had // page * page
            cut += length < had
            keys = np.arange(length)
            for j in np.unique(keys[(keys > length - window) | (keys < sinks)] // page):
                id = int(got["block_table"][r, j])
                assert 0 <= id < s["pages"], f"row {r}, {length} tokens: page {j} is {id}"
                if id != s["table"][q, j]:
                    assert copied[id] == s["table"][q, j] and (j + 1) * page > length
    assert cut > 0 and M.moe_device_status() == 0


@pytest.mark.parametrize("free", [0, 1, 2, 7, 30])
def test_as_many_rows_are_cut_short_as_copies_find_no_page(free):
    """Forty rows go on, two from each of twenty that stay and end inside a page of their own; nothing comes back."""
    for seed in range(4):
        rng = np.random.default_rng(900 + seed)
        ctx = np.r_[np.zeros(40, int), rng.integers(0, 6, 20) * 16 + rng.integers(1, 16, 20)]
        held = -(-ctx // 16)
        used = int(held.sum())
        table = np.full((60, 6), -1)
        ids = rng.permutation(used + free)
        for r in range(60):
            table[r, :held[r]] = ids[held[:r].sum():held[:r + 1].sum()]
        pool = np.full(used + free, -7)
        pool[:free] = ids[used:]
        s = dict(ctx=ctx, table=table, pool=pool, state=[0, free], pages=used + free, page=16)
        got = _run_fork(s, np.r_[40 + np.arange(40) % 20, 40 + np.arange(20)], None)
        # Of three rows that end in a page the lowest keeps it: 40 copies are wanted.
        assert got["info"][:3].tolist() == [free, 0, 40 - free]
        assert (got["next_ctx"] < np.r_[ctx[40:], ctx[40:], ctx[40:]]).sum() == 40 - free
    assert M.moe_device_status() == 0


@pytest.mark.parametrize("pages", [1 << 17, (1 << 17) + 1, 1 << 18, (1 << 18) + 1])
def test_caches_around_the_most_pages_with_marks_in_shared_memory(pages):
    """A block's share of the pages doubles behind 2^17; behind 2^18 the marks are in the workspace.  Pages of both ends
    of the cache are in use."""
    rng = np.random.default_rng(pages % 1000)
    s = _state(rng, 100, 16, 40, free=0)
    used = s["pages"]
    spread = np.sort(rng.choice(pages - 2, used - 2, replace=False)) + 1
    ids = rng.permutation(np.r_[0, spread, pages - 1])
    inside = np.arange(40)[None] < -(-s["ctx"] // 16)[:, None]
    s["table"] = np.where(inside & (s["table"] >= 0), ids[np.clip(s["table"], 0, used - 1)], s["table"])
    free = np.setdiff1d(np.arange(pages), ids)
    pool = np.full(pages, -7)
    pool[(pages - 5 + np.arange(len(free))) % pages] = rng.permutation(free)
    s.update(pages=pages, pool=pool, state=[pages - 5, len(free)])
    for in_place in (True, False):
        _check_fork(s, *_branches(rng, s, "few"), in_place=in_place)
        assert _check_compact(s, in_place)["info"][3] == used
    _check_release(s, np.where(rng.random(100) < 0.3, -1, 1), 100, 4)
    assert M.moe_device_status() == 0
