"""GPU tests of attention over a paged key/value cache against oracle/paged_oracle.py (plain
loops in 64 bits), through the C ABI.

Tolerances, from the arithmetic alone:
* plan: whole numbers, equal;
* append: one rounding to bf16 (2^-8 relative) of a value with a few fp32 roundings (2^-20
  covers them); values are copied, equal;
* attention: a score is a sum of 128 products whose absolute values add up to at most
  sqrt(128) rms(q) rms(k) (Cauchy-Schwarz), each fp32 addition within 2^-23 of that (rounded or
  cut off): ds = 128 2^-23 sqrt(128) scale^2, scale = the rms of q and of k.  out is rounded
  once to bf16 (2^-8 |out|), each softmax weight once to bf16 before it multiplies V, and is
  off by 2 ds from its score and its row's sum (both times the weighted sum of |v|, the
  oracle's `weight`); fp32 sums and the exponential take 2^-12 weight.  lse: ds, the sum of
  `keys` exponentials within keys 2^-24 relatively, 2^-20 (1 + |lse|) for exp and log.
"""
import numpy as np
import pytest
import torch

import aux_loss_free_gb300 as M
from gpu_util import assert_close_bf16, bf16_to_np, bf64
from oracle import attention_oracle as A
from oracle import paged_oracle as P
from synth import ATTN_CONFIGS, make_attention
from aux_loss_free_gb300.layer import to_device_bf16
from aux_loss_free_gb300.paged import PagedAttention, PagedStep

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


# ------------------------------------------------------------------------------- plan

def _random_step(rng, R, page, max_pages, new, free, pad=0):
    """Inputs of a step: ctx of every request within its table, its pages at random ids; the
    pool's ring starts at a random place."""
    new = np.asarray(new)
    room = max_pages * page - np.maximum(new, 0)
    ctx = np.array([rng.integers(0, max(1, m + 1)) for m in room])
    held = -(-ctx // page)
    pages = int(held.sum()) + free + 1
    ids = rng.permutation(pages)
    table = np.full((R, max_pages), -1)
    at = 0
    for r in range(R):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    head = int(rng.integers(0, pages))
    pool = np.full(pages, -1)
    pool[(head + np.arange(free)) % pages] = ids[at:at + free]
    return dict(ctx=ctx, new=new, table=table, pool=pool, state=[head, free], pages=pages,
                tokens=max(1, int(np.maximum(new, 0).sum()) + pad))


def _run_plan(s, page, stream=None):
    R, max_pages = s["table"].shape
    shape = M.make_paged_shape(R, s["tokens"], 8, 2, page, s["pages"], max_pages)
    g = {"block_table": _i32(s["table"]), "pool": _i32(s["pool"])}
    sizes = dict(pool_state=2, row_start=R + 1, slot_map=s["tokens"], kv_len=R, next_ctx=R, info=4)
    g.update({k: torch.full((n,), -77, dtype=torch.int32, device=DEV) for k, n in sizes.items()})
    ins = [_i32(s["ctx"]), _i32(s["new"]), _i32(s["state"])]
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())

    def call():
        M.moe_paged_plan(shape, ins[0], ins[1], g["block_table"], g["pool"], ins[2], g["pool_state"], g["row_start"],
                         g["slot_map"], g["kv_len"], g["next_ctx"], g["info"], stream=stream)

    call()
    torch.cuda.synchronize()
    first = {k: v.cpu().numpy().copy() for k, v in g.items()}
    call()  # the same inputs again: the same outputs
    torch.cuda.synchronize()
    for k, v in g.items():
        assert np.array_equal(v.cpu().numpy(), first[k]), k
    return first


def _check_plan(s, page, stream=None):
    got = _run_plan(s, page, stream)
    ref = P.step_plan(s["ctx"], s["new"], s["table"], s["pool"], s["state"], s["tokens"], s["pages"], page)
    for k, v in ref.items():
        assert np.array_equal(got[k], v), f"{k}: {got[k]} != {v}"


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("R", [1, 2, 31, 256, 257, 4096])
def test_plan_matches_oracle(R, page):
    rng = np.random.default_rng(R * 1000 + page)
    new = rng.choice([-1, 0, 1, 1, 1, 5, 16, 17, 130], size=R)
    _check_plan(_random_step(rng, R, page, 12 if R > 300 else 40, new, free=int(R * 12 + 12), pad=R % 3), page)


@pytest.mark.parametrize("free", [0, 1, 3, 10, 25])
def test_plan_denies_what_the_pool_cannot_give(free):
    rng = np.random.default_rng(free)
    _check_plan(_random_step(rng, 64, 16, 20, rng.choice([-1, 0, 1, 1, 40], size=64), free=free, pad=5), 16)
    assert M.moe_device_status() == 0  # a short pool is no error


def test_plan_all_ended_all_idle_and_one_long_prompt():
    rng = np.random.default_rng(3)
    _check_plan(_random_step(rng, 40, 32, 30, [-1] * 40, free=2), 32)
    _check_plan(_random_step(rng, 40, 32, 30, [0] * 40, free=0), 32)
    s = _random_step(rng, 3, 16, 700, [1, 10000, 2], free=700)
    s["ctx"] = np.array([0, 0, 0])
    s["table"][:] = -1
    _check_plan(s, 16)


def test_plan_reports_requests_that_do_not_fit():
    """Longer than the table's row, rows past the batch, a negative context: denied, the
    others served as if those asked for nothing; MOE_ERR_DEVICE in the status word."""
    rng = np.random.default_rng(9)
    for change in ("long", "rows", "negative"):
        s = _random_step(rng, 6, 16, 8, [1, 1, 20, 1, 3, 1], free=20)
        if change == "long":
            s["ctx"][2] = 8 * 16 - 19
        elif change == "rows":
            s["tokens"] = 23
        else:
            s["ctx"][2] = -1
        assert M.moe_device_status() == 0
        _check_plan(s, 16)
        assert M.moe_device_status() == 6
    assert M.moe_device_status() == 0


def test_plan_reports_bad_pool_states_and_pages():
    rng = np.random.default_rng(10)
    for state in ([-1, 2], [1000000, 2], [0, 1000000], [0, -3]):
        s = _random_step(rng, 3, 16, 8, [40, 1, 0], free=9)
        s["state"] = state
        got = _run_plan(s, 16)
        assert got["info"][1] == 0 and got["kv_len"][0] == 0  # nothing is taken
        assert M.moe_device_status() == 6
    s = _random_step(rng, 2, 16, 8, [1, 1], free=9)
    s["ctx"] = np.array([5, 5])
    s["table"][:, 0] = [s["pages"], 0]  # no such page
    got = _run_plan(s, 16)
    assert got["slot_map"].tolist() == [-1, 5]
    assert M.moe_device_status() == 6


def test_plan_on_another_stream():
    rng = np.random.default_rng(11)
    _check_plan(_random_step(rng, 100, 64, 10, rng.choice([-1, 0, 1, 30], size=100), free=300), 64,
                stream=torch.cuda.Stream())


# ----------------------------------------------------------------------------- append

APPEND = [(1, 8, 2, 16, 0), (5, 6, 2, 32, 2), (64, 8, 8, 16, 0), (257, 16, 2, 128, 31), (1000, 4, 1, 64, 0),
          (33, 64, 1, 16, 1), (40, 1, 1, 64, 0)]


def _rows(rng, *shape, scale=1.0):
    return torch.tensor(rng.standard_normal(shape) * scale, dtype=torch.float32, device=DEV).to(torch.bfloat16)


@pytest.mark.parametrize("T,H,KV,page,pad", APPEND)
@pytest.mark.parametrize("form", ["dense", "strided", "in_place"])
def test_append_matches_oracle(T, H, KV, page, pad, form):
    rng = np.random.default_rng(T)
    pages = T // page + 4
    slots = np.full(T + pad, -1)
    slots[:T] = rng.permutation(pages * page)[:T]
    slots = rng.permutation(slots)
    qkv = _rows(rng, T + pad, (H + 2 * KV) * 128, scale=3.0)
    qkv[T // 2] = 0  # a row of zeros: 0 / sqrt(eps)
    k0, v0 = _rows(rng, pages, KV, page, 128), _rows(rng, pages, KV, page, 128)
    rq, rk, rv = P.append(bf16_to_np(qkv), slots, H, KV, page, bf16_to_np(k0), bf16_to_np(v0))
    stride = {"dense": 0, "strided": H * 128 + 24, "in_place": (H + 2 * KV) * 128}[form]
    shape = M.make_paged_shape(1, T + pad, H, KV, page, pages, 1, q_stride=stride)
    q = qkv if form == "in_place" else _rows(rng, T + pad, stride or H * 128)
    was = q.clone()
    M.moe_paged_append(shape, qkv, _i32(slots), q, k0, v0)
    torch.cuda.synchronize()

    def near(got, ref):
        assert (np.abs(got - ref) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(ref)).all()

    near(bf16_to_np(q)[:, :H * 128], rq)
    assert torch.equal(q[:, H * 128:], was[:, H * 128:])  # nothing beside the query heads is written
    near(bf16_to_np(k0), rk)
    assert np.array_equal(bf16_to_np(v0), rv)


def test_append_ignores_slots_outside_the_cache():
    rng = np.random.default_rng(1)
    shape = M.make_paged_shape(1, 3, 8, 2, 16, 4, 1)
    k0, v0 = _rows(rng, 4, 2, 16, 128), _rows(rng, 4, 2, 16, 128)
    k1, v1 = k0.clone(), v0.clone()
    q = torch.empty(3, 1024, dtype=torch.bfloat16, device=DEV)
    M.moe_paged_append(shape, _rows(rng, 3, 12 * 128), _i32([64, -5, 2 ** 31 - 1]), q, k0, v0)
    torch.cuda.synchronize()
    assert torch.equal(k0, k1) and torch.equal(v0, v1)


# -------------------------------------------------------------------------- attention

def _attn_inputs(rng, ctx, new, H, KV, page, pad=0, extra_cols=1, stale=float("nan"), scale=1.0):
    """A step's tensors; what the pages hold past the requests' keys, and the pages of nobody,
    is `stale`."""
    R = len(ctx)
    kv = np.array(ctx) + np.array(new)
    held = -(-kv // page)
    pages = int(held.sum()) + 3
    ids = rng.permutation(pages)
    table = np.full((R, int(held.max()) + extra_cols), -1)
    kc = torch.full((pages, KV, page, 128), stale, dtype=torch.bfloat16, device=DEV)
    vc = torch.full_like(kc, stale)
    at = 0
    for r in range(R):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
        pos = np.arange(kv[r])
        slot_page, off = torch.tensor(table[r][pos // page], device=DEV), torch.tensor(pos % page, device=DEV)
        k = rng.standard_normal((kv[r], KV, 128)) * scale
        kc[slot_page, :, off] = torch.tensor(k / np.sqrt((k * k).mean(-1, keepdims=True)) * scale,
                                             dtype=torch.float32, device=DEV).to(torch.bfloat16)
        vc[slot_page, :, off] = _rows(rng, kv[r], KV, 128)
    T = int(np.sum(new)) + pad
    q = rng.standard_normal((max(T, 1), H, 128))
    q = torch.tensor(q / np.sqrt((q * q).mean(-1, keepdims=True)) * scale, dtype=torch.float32,
                     device=DEV).to(torch.bfloat16).reshape(max(T, 1), H * 128)
    return dict(q=q, k=kc, v=vc, table=table, row_start=np.concatenate([[0], np.cumsum(new)]), kv=kv, H=H, KV=KV,
                page=page, pages=pages)


def _attend(a, stream=None, lse=True, q_stride=0, calls=1):
    T = a["q"].shape[0]
    shape = M.make_paged_shape(len(a["kv"]), T, a["H"], a["KV"], a["page"], a["pages"], a["table"].shape[1],
                               q_stride=q_stride)
    n = M.moe_paged_attention_workspace_size(shape)
    ws = torch.randint(0, 256, (n,), dtype=torch.uint8, device=DEV)  # the workspace needs no clearing
    dev = [_i32(a["table"]), _i32(a["row_start"]), _i32(a["kv"])]
    outs = []
    for _ in range(calls):
        out = torch.full((T, a["H"] * 128), 7.0, dtype=torch.bfloat16, device=DEV)
        ls = torch.full((T, a["H"]), 7.0, dtype=torch.float32, device=DEV) if lse else None
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        M.moe_paged_attention(shape, a["q"], a["k"], a["v"], *dev, out, ls, ws, stream=stream)
        torch.cuda.synchronize()
        outs.append((out, ls))
    for o, ls in outs[1:]:
        assert torch.equal(o.view(torch.int16), outs[0][0].view(torch.int16))
        assert ls is None or torch.equal(ls, outs[0][1])
    return outs[0]


def _check_attention(a, scale=1.0, **kw):
    T = a["q"].shape[0]
    out, lse = _attend(a, **kw)
    q = bf16_to_np(a["q"])[:, :a["H"] * 128]
    ref = P.paged_attention(q, bf16_to_np(a["k"]), bf16_to_np(a["v"]), a["table"], a["row_start"], a["kv"], a["H"],
                            a["KV"])
    got = bf16_to_np(out)
    ds = 128 * 2.0 ** -23 * np.sqrt(128) * 1.02 * scale * scale  # 1.02: the rms after rounding to bf16
    bound = 2.0 ** -8 * np.abs(ref["out"]) + (2.0 ** -8 + 2.0 ** -12 + 2 * ds) * ref["weight"]
    off = np.abs(got - ref["out"])
    assert np.isfinite(got).all()
    assert (off <= bound).all(), f"{(off / np.maximum(bound, 1e-30)).max()} times the bound, first row " \
                                 f"{np.argwhere(off > bound)[0]}"
    if lse is not None:
        ls = lse.cpu().numpy().astype(np.float64)
        empty = np.isneginf(ref["lse"])
        assert np.array_equal(np.isneginf(ls), empty)
        keys = int(a["kv"].max())
        tol = ds + 2.0 ** -24 * keys + 2.0 ** -20 * (1 + np.abs(ref["lse"]))
        assert (np.abs(ls[~empty] - ref["lse"][~empty]) <= tol[~empty]).all()
    # Rows without keys are exactly zero.
    assert (got.reshape(T, a["H"], 128)[np.isneginf(ref["lse"])] == 0).all()


# (ctx, new, n_head, n_kv_head, page, padding rows)
ATTN = {
    "one-token-no-context": ([0], [1], 8, 2, 16, 0),
    "one-token-one-key-before": ([1], [1], 8, 2, 16, 0),
    "decode-page-and-tile-edges": ([14, 15, 16, 126, 127, 128, 129, 255, 256], [1] * 9, 8, 2, 16, 0),
    "decode-ragged-64": ([int(x) for x in np.random.default_rng(0).integers(0, 900, 64)], [1] * 64, 8, 2, 32, 3),
    "decode-long": ([20011], [1], 8, 2, 128, 0),
    "decode-long-beside-short": ([9000, 3, 0, 700], [1] * 4, 4, 1, 64, 0),
    "verify-5-groups-of-3": ([0, 7, 123, 1000], [5] * 4, 6, 2, 32, 7),
    "prompt-one-tile": ([0], [128], 8, 2, 64, 0),
    "prompt-odd": ([0], [333], 8, 2, 16, 1),
    "prompts-ragged": ([0, 0, 0], [1, 130, 70], 8, 2, 128, 0),
    "chunk-over-context": ([1000], [200], 8, 2, 32, 0),
    "chunk-many-rows": ([77, 513], [257, 64], 4, 1, 16, 5),
    "no-grouping": ([40, 300], [100, 1], 4, 4, 16, 0),
    "no-grouping-long-chunk": ([5], [400], 2, 2, 64, 0),
    "groups-of-5": ([200, 3], [70, 1], 5, 1, 64, 0),
    "groups-of-7": ([64], [39], 14, 2, 16, 0),
    "one-shared-head-of-16": ([100, 600], [33, 1], 16, 1, 32, 0),
    "one-shared-head-of-64": ([50, 10], [9, 1], 64, 1, 16, 0),
    "one-head": ([300], [150], 1, 1, 128, 2),
    "mixed-step": ([700, 0, 64, 1, 2000, 0], [1, 180, 1, 40, 1, 1], 8, 2, 16, 40),
    "idle-requests-between": ([100, 50, 7, 0, 90], [1, 0, 3, 0, 1], 8, 2, 16, 2),
    # Work tiles in one, two, three and many parts over the CTAs, pairs and single ones.
    "prompt-2048": ([0], [2048], 8, 2, 64, 0),
    "chunk-in-many-parts": ([20000], [64], 8, 2, 32, 1),
    "chunks-in-three-parts": ([6000, 5000], [700, 27], 4, 1, 128, 0),
    "few-rows-in-many-parts": ([9000, 9100], [3, 5], 8, 2, 64, 0),
    # More requests than the kernel has threads.
    "decode-700": ([int(x) for x in np.random.default_rng(1).integers(0, 70, 700)], [1] * 700, 4, 1, 16, 0),
    "decode-1300-some-idle": ([int(x) for x in np.random.default_rng(2).integers(0, 40, 1300)],
                              [int(x) for x in np.random.default_rng(3).integers(0, 3, 1300)], 2, 2, 16, 50),
}


@pytest.mark.parametrize("name", ATTN)
def test_attention_matches_oracle(name):
    ctx, new, H, KV, page, pad = ATTN[name]
    _check_attention(_attn_inputs(np.random.default_rng(len(name)), ctx, new, H, KV, page, pad), calls=2)


@pytest.mark.parametrize("stale", [float("inf"), -float("inf"), 3e38])
def test_attention_never_uses_what_lies_past_the_keys(stale):
    rng = np.random.default_rng(2)
    _check_attention(_attn_inputs(rng, [130, 9, 0], [1, 40, 1], 8, 2, 64, 1, stale=stale))


# (ctx, new, positions of request 0 whose keys of key/value head 0 are NaN)
NAN_KEYS = {
    "decode": ([300], [1], (17, 18)),
    "decode-every-key": ([300], [1], (0, 301)),
    "decode-in-parts": ([9000, 40], [1, 1], (5000, 5001)),
    "decode-whole-parts": ([9000, 40], [1, 1], (0, 4000)),
    "few-rows-in-parts": ([9000, 9100], [3, 5], (9001, 9002)),
    "chunk": ([100], [200], (230, 231)),
    "chunk-in-many-parts": ([20000], [64], (0, 15000)),
    "chunks-in-three-parts": ([6000, 5000], [700, 27], (6300, 6301)),
}


@pytest.mark.parametrize("name", NAN_KEYS)
def test_attention_rows_that_see_a_nan_are_nan_and_no_others(name):
    ctx, new, (first, last) = NAN_KEYS[name]
    a = _attn_inputs(np.random.default_rng(21), ctx, new, 8, 2, 16, pad=1)
    ref_out, ref_lse = _attend(a)
    pos = np.arange(first, last)
    b = dict(a, k=a["k"].clone())
    b["k"][torch.tensor(a["table"][0][pos // 16], device=DEV), 0, torch.tensor(pos % 16, device=DEV)] = float("nan")
    out, lse = _attend(b)
    sees = torch.zeros(out.shape[0], 8, dtype=torch.bool, device=DEV)
    sees[:new[0], :4] = (torch.arange(ctx[0], ctx[0] + new[0], device=DEV) >= first)[:, None]
    assert torch.isnan(lse[sees]).all() and torch.equal(lse[~sees], ref_lse[~sees])
    out, ref_out = out.reshape(-1, 8, 128), ref_out.reshape(-1, 8, 128)
    assert torch.isnan(out[sees]).all()
    assert torch.equal(out[~sees].view(torch.int16), ref_out[~sees].view(torch.int16))


def test_attention_of_denied_requests_and_padding_is_zero():
    a = _attn_inputs(np.random.default_rng(4), [50, 300, 20, 10], [1, 70, 2, 1], 8, 2, 16, pad=300)
    a["kv"][[1, 3]] = 0  # denied: no keys, whatever the rows
    _check_attention(a)
    a["kv"][:] = 0  # no row of the batch has keys
    _check_attention(a)


def test_attention_with_large_scores():
    """Rows whose softmax is a near one-hot, and running maxima that keep growing: scores up
    to 16 x 16 x sqrt(128)."""
    rng = np.random.default_rng(6)
    a = _attn_inputs(rng, [900, 0], [1, 300], 8, 2, 16, scale=16.0)
    _check_attention(a, scale=16.0)
    # Keys that grow along the sequence: every tile raises the maximum.
    a = _attn_inputs(rng, [1500], [40], 4, 1, 64)
    pos = np.arange(1540)
    ids, off = torch.tensor(a["table"][0][pos // 64], device=DEV), torch.tensor(pos % 64, device=DEV)
    a["k"][ids, :, off] = (a["q"][-1, :128][None, None] * torch.linspace(0.01, 4, 1540, device=DEV)[:, None, None]
                           ).to(torch.bfloat16)
    _check_attention(a, scale=4.0)


def test_attention_reads_strided_queries_and_skips_lse():
    rng = np.random.default_rng(7)
    a = _attn_inputs(rng, [40, 200], [70, 1], 8, 2, 16, 2)
    wide = _rows(rng, a["q"].shape[0], 12 * 128)
    wide[:, :8 * 128] = a["q"]
    a["q"] = wide
    _check_attention(a, q_stride=12 * 128, lse=False)


def test_attention_on_another_stream():
    a = _attn_inputs(np.random.default_rng(8), [40, 2000], [70, 1], 8, 2, 16, 2)
    _check_attention(a, stream=torch.cuda.Stream(), calls=3)


def test_attention_far_into_a_large_cache():
    """Pages whose elements lie past 2^31 and 2^32: 32-bit element offsets would wrap."""
    KV, page, pages = 2, 128, 140000  # 2 x 9.2 GB, 4.6e9 elements each
    k = torch.empty(pages, KV, page, 128, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    a = _attn_inputs(np.random.default_rng(12), [300, 100], [40, 1], 8, 2, page)
    small_k, small_v = a["k"], a["v"]
    far = np.array([pages - 1, 70000, 139000, 65536, 131072, 3, 100000, 99999])[:a["pages"]]
    for i, f in enumerate(far):
        k[f], v[f] = small_k[i], small_v[i]
    T = a["q"].shape[0]
    ref_out, ref_lse = _attend(a)
    table = np.where(a["table"] >= 0, far[a["table"]], -1)
    big = dict(a, k=k, v=v, table=table, pages=pages)
    out, lse = _attend(big)
    assert torch.equal(out.view(torch.int16), ref_out.view(torch.int16)) and torch.equal(lse, ref_lse)
    # The write side at the same places.
    shape = M.make_paged_shape(1, T, 8, KV, page, pages, 1)
    slots = far[np.arange(T) % len(far)].astype(np.int64) * page + np.arange(T) // len(far)
    qkv = _rows(np.random.default_rng(13), T, 12 * 128)
    M.moe_paged_append(shape, qkv, _i32(slots), torch.empty(T, 1024, dtype=torch.bfloat16, device=DEV), k, v)
    torch.cuda.synchronize()
    st = torch.tensor(slots, device=DEV)
    assert torch.equal(v[st // page, :, st % page].reshape(T, -1), qkv[:, 10 * 128:])


def test_attention_through_one_workspace_and_a_captured_graph():
    """Calls of other lengths through one workspace, directly and as replays of one captured
    call whose lengths change: equal bits.  What a call leaves in the workspace, and where its
    work tiles are cut, differ from call to call."""
    rng = np.random.default_rng(16)
    H, KV, page, T = 8, 2, 16, 1300
    steps = [([0, 3000, 700, 1], [1200, 1, 60, 39]), ([9000, 10, 10, 10], [64, 1, 1, 1]), ([0, 0, 0, 0], [1, 1, 1, 1]),
             ([100, 200, 5000, 300], [300, 500, 400, 100]), ([2500, 2600, 2700, 2800], [325, 325, 325, 325])]
    ins = [_attn_inputs(rng, c, n, H, KV, page, pad=T - sum(n)) for c, n in steps]
    pages, width = max(a["pages"] for a in ins), max(a["table"].shape[1] for a in ins)
    shape = M.make_paged_shape(4, T, H, KV, page, pages, width)
    ws = torch.randint(0, 256, (M.moe_paged_attention_workspace_size(shape),), dtype=torch.uint8, device=DEV)
    k = torch.empty(pages, KV, page, 128, dtype=torch.bfloat16, device=DEV)
    v, q = torch.empty_like(k), torch.empty(T, H * 128, dtype=torch.bfloat16, device=DEV)
    table, rs, kv = torch.empty(4, width, dtype=torch.int32, device=DEV), _i32([0] * 5), _i32([0] * 4)
    out, lse = torch.empty_like(q), torch.empty(T, H, dtype=torch.float32, device=DEV)

    def load(a):
        k[:a["pages"]], v[:a["pages"]] = a["k"], a["v"]
        q.copy_(a["q"])
        table.fill_(-1)
        table[:, :a["table"].shape[1]] = _i32(a["table"])
        rs.copy_(_i32(a["row_start"]))
        kv.copy_(_i32(a["kv"]))

    def call(stream=None):
        M.moe_paged_attention(shape, q, k, v, table, rs, kv, out, lse, ws, stream=stream)

    direct = []
    for a in ins:
        load(a)
        call()
        torch.cuda.synchronize()
        direct.append((out.clone(), lse.clone()))
        ref, ref_lse = _attend(a)  # a workspace of its own
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16)) and torch.equal(lse, ref_lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(side)
    for i in (0, 1, 3, 0, 4, 2, 4, 1, 0):
        load(ins[i])
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), direct[i][0].view(torch.int16)) and torch.equal(lse, direct[i][1])


def test_attention_reports_tables_and_lengths_out_of_range():
    """A table entry that is no page, lengths past the table: status MOE_ERR_DEVICE, the other
    requests' rows as they should be."""
    rng = np.random.default_rng(14)
    a = _attn_inputs(rng, [100, 40], [1, 3], 8, 2, 16)
    ref, _ = _attend(a)
    for change in ("page", "negative", "kv"):
        b = dict(a, table=a["table"].copy(), kv=a["kv"].copy())
        if change == "kv":
            b["kv"][0] = 16 * b["table"].shape[1] + 1
        else:
            b["table"][0, 2] = a["pages"] if change == "page" else -1
        assert M.moe_device_status() == 0
        out, _ = _attend(b)
        assert M.moe_device_status() == 6
        assert torch.equal(out[1:].view(torch.int16), ref[1:].view(torch.int16))


def test_plan_append_attention_in_a_captured_graph():
    """One step captured once and replayed with other lengths and rows in the same buffers."""
    rng = np.random.default_rng(15)
    H, KV, page, R, T, pages, width = 8, 2, 16, 4, 96, 64, 12
    shape = M.make_paged_shape(R, T, H, KV, page, pages, width)
    k = torch.full((pages, KV, page, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    v = torch.full_like(k, float("nan"))
    ctx, new = _i32([0] * R), _i32([1] * R)
    table, pool = torch.full((R, width), -1, dtype=torch.int32, device=DEV), _i32(rng.permutation(pages))
    state, nxt, info = _i32([0, pages]), torch.empty(R, dtype=torch.int32, device=DEV), _i32([0] * 4)
    state_out, rs, slot, kv = _i32([0, 0]), _i32([0] * (R + 1)), _i32([0] * T), _i32([0] * R)
    qkv, q = _rows(rng, T, (H + 2 * KV) * 128), torch.empty(T, H * 128, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q)
    ws = torch.empty(M.moe_paged_attention_workspace_size(shape), dtype=torch.uint8, device=DEV)

    def step(stream):
        M.moe_paged_plan(shape, ctx, new, table, pool, state, state_out, rs, slot, kv, nxt, info, stream=stream)
        M.moe_paged_append(shape, qkv, slot, q, k, v, stream=stream)
        M.moe_paged_attention(shape, q, k, v, table, rs, kv, out, None, ws, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(side)  # warm, outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    table.fill_(-1)
    hist = {r: [] for r in range(R)}
    for lens in ([60, 0, 3, 33], [1, 17, 1, 1], [1, 1, 50, 1], [1, 1, 1, 20]):
        rows = _rows(rng, T, (H + 2 * KV) * 128)
        qkv.copy_(rows)
        new.copy_(_i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        u = bf16_to_np(rows).reshape(T, H + 2 * KV, 128)
        at = 0
        for r, n in enumerate(lens):
            hist[r] += list(u[at:at + n])
            if n:
                seq = np.stack(hist[r])
                qn, kn, vn = P.append(seq.reshape(len(seq), -1), np.arange(len(seq)), H, KV, len(seq),
                                      np.zeros((1, KV, len(seq), 128)), np.zeros((1, KV, len(seq), 128)))
                ref = P.paged_attention(qn[-n:], kn, vn, np.array([[0]]), np.array([0, n]), np.array([len(seq)]), H, KV)
                got = bf16_to_np(out)[at:at + n]
                # q and k are rounded to bf16 here and not in the reference: scores move by at
                # most 2 x 2^-8 x sqrt(128) < 0.09 each, the weights by that share.
                assert (np.abs(got - ref["out"]) <= 2.0 ** -8 * np.abs(ref["out"]) + 0.2 * ref["weight"]).all()
                rel = np.linalg.norm(got - ref["out"]) / np.linalg.norm(ref["out"])
                assert rel <= 2e-2
            at += n
        ctx.copy_(nxt)
        state.copy_(state_out)
        assert (bf16_to_np(out)[at:] == 0).all()


@pytest.mark.parametrize("residual", [True, False])
def test_block_in_steps_matches_the_dense_oracle(residual):
    """Three sequences through the whole block in uneven steps, one of them in a row of the
    block table that another request has left, against the dense oracle on each sequence (the
    block tests' tolerance); padding rows come out as x (or zero)."""
    a = ATTN_CONFIGS["attn_tiny"].replace(batch=1, seq=150, n_head=8, n_kv_head=2, d=512)
    H = make_attention(a, "attn_tiny")
    w_qkv = to_device_bf16(np.concatenate([H["w_q"], H["w_k"], H["w_v"]], axis=0), DEV)
    step = PagedStep(requests=3, pages=20, page_size=16, max_pages=10, max_tokens=160)
    block = PagedAttention(step, a.d, 8, 2, w_qkv, to_device_bf16(H["w_o"], DEV), a.eps)
    rng = np.random.default_rng(21)
    script = [([40, 0, 7], 3), ([1, 90, 1], 0), ([50, 1, 0], 5), ([-1, 1, 30], 0), ([0, 3, 1], 1), ([60, 1, -1], 0),
              ([1, 1, 0], 6)]
    seqs, rows_of, got = {}, {0: "a", 1: "b", 2: "c"}, {}
    for lens, pad in script:
        T = sum(max(n, 0) for n in lens) + pad
        x = _rows(rng, max(T, 1), a.d)
        out = torch.full_like(x, 9.0)
        block.forward(x, step.plan(_i32(lens), x.shape[0]) and out, residual=residual)
        torch.cuda.synchronize()
        at = 0
        for r, n in enumerate(lens):
            if n < 0:
                rows_of[r] += "'"
            elif n:
                seqs.setdefault(rows_of[r], []).append(bf16_to_np(x)[at:at + n])
                got.setdefault(rows_of[r], []).append(bf16_to_np(out)[at:at + n])
                at += n
        assert np.array_equal(bf16_to_np(out)[at:], bf16_to_np(x)[at:] if residual else np.zeros((x.shape[0] - at, a.d)))
        assert step.info.tolist()[3] == 0
    w = [bf64(H[n]) for n in ("w_q", "w_k", "w_v", "w_o")]
    assert sorted(seqs) == ["a", "a'", "b", "c"]
    for name, parts in seqs.items():
        xs = np.concatenate(parts)
        ref = A.gqa_attention(xs, *w, 1, len(xs), 8, 2, 128, a.eps, residual=residual, round_stored=True)
        assert_close_bf16(np.concatenate(got[name]), ref["out"], f"sequence {name}")
    assert step.free_pages.item() == 20 - -(-61 // 16) - -(-98 // 16)


def test_step_refuses_more_rows_than_it_was_made_for():
    step = PagedStep(requests=2, pages=4, page_size=16, max_pages=2, max_tokens=8)
    with pytest.raises(ValueError):
        step.plan(_i32([9, 0]), 9)


def _dense(xs, w, a, residual=True):
    return A.gqa_attention(xs, *w, 1, len(xs), a.n_head, a.n_kv_head, 128, a.eps, residual=residual,
                           round_stored=True)["out"]


def test_a_captured_step_goes_on_where_the_last_one_ended():
    """PagedStep.plan and PagedAttention.forward captured once and replayed with other new_len,
    an eager step between two replays, against the dense oracle on each sequence.  Capturing
    itself moves nothing."""
    a = ATTN_CONFIGS["attn_tiny"].replace(batch=1, seq=150, n_head=8, n_kv_head=2, d=512)
    H = make_attention(a, "attn_tiny")
    w_qkv = to_device_bf16(np.concatenate([H["w_q"], H["w_k"], H["w_v"]], axis=0), DEV)
    T, R = 48, 3
    step = PagedStep(requests=R, pages=24, page_size=16, max_pages=10, max_tokens=T)
    block = PagedAttention(step, a.d, 8, 2, w_qkv, to_device_bf16(H["w_o"], DEV), a.eps)
    x = torch.zeros(T, a.d, dtype=torch.bfloat16, device=DEV)
    out, new = torch.empty_like(x), _i32([0] * R)
    rng = np.random.default_rng(31)

    def call():
        block.forward(x, step.plan(new, T) and out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()  # warm: a step without tokens
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    assert step.ctx_len.tolist() == [0] * R and step.free_pages.item() == 24
    seqs, got, rows_of = {}, {}, {0: "a", 1: "b", 2: "c"}
    script = [([20, 17, 5], "replay"), ([1, 30, 16], "replay"), ([1, 1, 1], "replay"), ([16, 1, 1], "eager"),
              ([1, -1, 40], "replay"), ([1, 19, 1], "replay"), ([2, 1, 1], "eager"), ([1, 1, 1], "replay")]
    ctx = [0] * R
    for lens, how in script:
        rows = _rows(rng, T, a.d)
        x.copy_(rows)
        new.copy_(_i32(lens))
        out.fill_(9.0)
        if how == "replay":
            graph.replay()
        else:
            call()
        torch.cuda.synchronize()
        ctx = [0 if n < 0 else c + n for c, n in zip(ctx, lens)]
        assert step.ctx_len.tolist() == ctx
        assert step.free_pages.item() == 24 - sum(-(-c // 16) for c in ctx)
        at = 0
        for r, n in enumerate(lens):
            if n < 0:
                rows_of[r] += "'"
            elif n:
                seqs.setdefault(rows_of[r], []).append(bf16_to_np(rows)[at:at + n])
                got.setdefault(rows_of[r], []).append(bf16_to_np(out)[at:at + n])
                at += n
    w = [bf64(H[n]) for n in ("w_q", "w_k", "w_v", "w_o")]
    assert sorted(seqs) == ["a", "b", "b'", "c"]
    for name, parts in seqs.items():
        assert_close_bf16(np.concatenate(got[name]), _dense(np.concatenate(parts), w, a), f"sequence {name}")


def test_rows_past_the_planned_step_write_no_cache():
    """A large step, then a small one: the slot map still holds the large step's slots behind
    the small one's rows.  The class refuses a batch of another size; the C call takes the rows
    past the plan as padding and leaves every other token's keys and values as they are."""
    a = ATTN_CONFIGS["attn_tiny"].replace(batch=1, seq=64, n_head=8, n_kv_head=2, d=512)
    H = make_attention(a, "attn_tiny")
    w_qkv = to_device_bf16(np.concatenate([H["w_q"], H["w_k"], H["w_v"]], axis=0), DEV)
    step = PagedStep(requests=2, pages=12, page_size=16, max_pages=6, max_tokens=64)
    block = PagedAttention(step, a.d, 8, 2, w_qkv, to_device_bf16(H["w_o"], DEV), a.eps)
    block.k_cache.zero_()
    block.v_cache.zero_()
    rng = np.random.default_rng(33)
    x = _rows(rng, 60, a.d)
    out = torch.empty_like(x)
    with pytest.raises(ValueError):
        block.forward(x, out)  # nothing is planned yet
    step.plan(_i32([40, 20]), 60)
    block.forward(x, out)
    step.plan(_i32([1, 1]), 2)
    y = _rows(rng, 60, a.d)
    for rows, to in ((y, out), (y[:2], out), (y, out[:2]), (y[:1], out[:1])):
        with pytest.raises(ValueError):
            block.forward(rows, to)
    slots = step.slot_map[:2].tolist()
    k, v = block.k_cache.clone(), block.v_cache.clone()
    M.moe_attention_paged_fwd(step.shape(60, 8, 2, a.eps), a.d, y, block.w_qkv, block.w_o, True, block.k_cache,
                              block.v_cache, step.block_table, step.row_start, step.slot_map, step.kv_len, out,
                              block.workspace)
    torch.cuda.synchronize()
    assert torch.equal(out[2:], y[2:])  # padding rows
    for cache, was in ((block.k_cache, k), (block.v_cache, v)):
        changed = (cache != was).any(dim=3).any(dim=1).flatten().nonzero().flatten().tolist()
        assert changed == sorted(slots)


@pytest.mark.parametrize("R,max_pages,pad", [(1, 4, 0), (8, 20, 2), (40, 30, 3), (700, 12, 1), (4096, 6, 0)])
@pytest.mark.parametrize("which", ["both", "ctx", "pool"])
def test_plan_in_place(R, max_pages, pad, which):
    """next_ctx over ctx_len and pool_state_out over pool_state_in, with one CTA and with many:
    the oracle's outputs, step after step from the lengths that the last one left."""
    rng = np.random.default_rng(R + pad)
    choices = [-1, 0, 1, 1, 5, 17, 40]
    s = _random_step(rng, R, 16, max_pages, rng.choice(choices, size=R), free=R // 20 + 1)
    T = s["tokens"] = max(s["tokens"], 4 * R) + pad
    shape = M.make_paged_shape(R, T, 8, 2, 16, s["pages"], max_pages)
    ctx, state, table, pool = _i32(s["ctx"]), _i32(s["state"]), _i32(s["table"]), _i32(s["pool"])
    nxt, after = (ctx if which != "pool" else torch.empty_like(ctx)), (state if which != "ctx" else _i32([7, 7]))
    rs, slot, kv, info = _i32([0] * (R + 1)), _i32([0] * T), _i32([0] * R), _i32([0] * 4)
    denied = 0
    for _ in range(4):
        ref = P.step_plan(s["ctx"], s["new"], s["table"], s["pool"], s["state"], T, s["pages"], 16)
        M.moe_paged_plan(shape, ctx, _i32(s["new"]), table, pool, state, after, rs, slot, kv, nxt, info)
        torch.cuda.synchronize()
        got = dict(block_table=table, pool=pool, row_start=rs, slot_map=slot, kv_len=kv, next_ctx=nxt,
                   pool_state=after, info=info)
        for k, v in ref.items():
            assert np.array_equal(got[k].cpu().numpy(), v), k
        denied += ref["info"][3]
        ctx.copy_(nxt)
        state.copy_(after)
        s.update(ctx=ref["next_ctx"], table=ref["block_table"], pool=ref["pool"], state=ref["pool_state"])
        room = np.minimum(rng.choice(choices, size=R), max_pages * 16 - s["ctx"])
        s["new"] = np.where(np.cumsum(np.maximum(room, 0)) <= T, room, 0)
    assert denied or R < 700  # the pool runs short in the larger ones
    assert M.moe_device_status() == 0


# (ctx, new, n_head, n_kv_head, page): work tiles of 256 tokens (no grouping) down to 16, whole and
# cut, their first tokens at a key tile's beginning and inside one.
LATE_VALUES = {
    "no-grouping-prompt": ([0], [256], 2, 2, 16),
    "no-grouping-odd": ([64, 5], [300, 1], 4, 4, 16),
    "no-grouping-long": ([5000], [520], 1, 1, 64),
    "groups-of-2": ([40], [200], 4, 2, 32),
    "groups-of-3": ([100, 2], [70, 9], 6, 2, 64),
    "groups-of-4": ([100, 700], [200, 1], 8, 2, 16),
    "groups-of-4-prompt": ([0, 0], [129, 40], 8, 2, 128),
    "groups-of-16": ([30], [40], 16, 1, 16),
    "verification": ([9000, 300], [7, 5], 8, 2, 64),
    "chunk-in-many-parts": ([20000], [64], 8, 2, 32),
    "chunks-in-three-parts": ([6000, 5000], [700, 27], 4, 1, 128),
}


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("name", LATE_VALUES)
def test_attention_values_reach_no_earlier_row(name, value):
    """NaN and infinities in the values of a request's new tokens: the rows from that position on
    have them in that column, every other output has equal bits, and so has every lse."""
    ctx, new, H, KV, page = LATE_VALUES[name]
    a = _attn_inputs(np.random.default_rng(41), ctx, new, H, KV, page, pad=3)
    ref_out, ref_lse = _attend(a)
    n, G, inf = new[0], H // KV, float("inf")
    put = [(0, 0, value), (1, 9, value), (n // 3, 63, value), (n // 2, 64, value), (n - 2, 100, value),
           (n - 1, 127, value), (n // 3, 37, inf), (2 * n // 3, 37, -inf), (n // 4, 90, value), (n // 2, 90, value)]
    b = dict(a, v=a["v"].clone())
    want = ref_out.clone().reshape(-1, H, 128)
    for i, col, x in put:
        pos = ctx[0] + i
        b["v"][int(a["table"][0][pos // page]), 0, pos % page, col] = x
        want[i:n, :G, col] += x  # inf - inf gives NaN
    out, lse = _attend(b, calls=2)
    out = out.reshape(-1, H, 128)
    assert torch.equal(lse, ref_lse)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(out[keep].view(torch.int16), want[keep].view(torch.int16))
    # A whole row of values.
    b = dict(a, v=a["v"].clone())
    pos = ctx[0] + n - 1
    b["v"][int(a["table"][0][pos // page]), :, pos % page] = value
    out, lse = _attend(b)
    want = ref_out.clone()
    want[n - 1] += value
    assert torch.equal(lse, ref_lse) and torch.equal(out.isnan(), want.isnan())
    keep = ~want.isnan()
    assert torch.equal(out[keep].view(torch.int16), want[keep].view(torch.int16))


@pytest.mark.parametrize("entry", [-1, "pages"])
def test_plan_reports_a_returned_page_that_is_none(entry):
    """An ended request's table holds no page where its context says that one is: reported in
    the step that puts it back, not when another request is given it."""
    s = _random_step(np.random.default_rng(17), 3, 16, 8, [-1, 1, -1], free=2)
    s["ctx"] = np.array([40, 5, 17])
    s["pages"] = 12
    s["table"] = np.full((3, 8), -1)
    s["table"][0, :3], s["table"][1, 0], s["table"][2, :2] = [1, 2, 3], 4, [5, 6]
    s["pool"] = np.array([7, 8] + [-1] * 10)
    s["state"] = [0, 2]
    _check_plan(s, 16)
    assert M.moe_device_status() == 0
    s["table"][2, 1] = s["pages"] if entry == "pages" else entry
    got = _run_plan(s, 16)
    assert M.moe_device_status() == 6
    assert got["slot_map"].tolist() == [4 * 16 + 5] and got["info"].tolist() == [1, 0, 5, 0]


def _prepared(a, stream):
    """A call on `a` in buffers of its own; returns it with its outputs."""
    T = a["q"].shape[0]
    shape = M.make_paged_shape(len(a["kv"]), T, a["H"], a["KV"], a["page"], a["pages"], a["table"].shape[1])
    ws = torch.randint(0, 256, (M.moe_paged_attention_workspace_size(shape),), dtype=torch.uint8, device=DEV)
    dev = [_i32(a["table"]), _i32(a["row_start"]), _i32(a["kv"])]
    out = torch.empty(T, a["H"] * 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(T, a["H"], dtype=torch.float32, device=DEV)
    return lambda: M.moe_paged_attention(shape, a["q"], a["k"], a["v"], *dev, out, lse, ws, stream=stream), out, lse


# Pairs of calls: work tiles that are joined by the CTA of their first part, tiles in many parts,
# decode steps.
TWO_STREAMS = [(([3000, 100, 5000], [400, 700, 1], 8, 2, 16), ([9000, 10], [64, 1300], 8, 2, 32)),
               (([0], [2048], 8, 2, 64), ([20000, 3], [5, 1], 4, 1, 128)),
               (([600, 0], [900, 300], 2, 2, 64), ([500] * 40, [1] * 40, 8, 2, 16))]


@pytest.mark.parametrize("pair", range(len(TWO_STREAMS)))
def test_attention_on_two_streams_at_once(pair):
    """Two calls with workspaces of their own, queued on two streams again and again without a
    wait between them: the bits of the calls alone, and a clear status word.  Parts of a call wait
    for other parts of it while the other call holds SMs."""
    rng = np.random.default_rng(60 + pair)
    ins = [_attn_inputs(rng, *c[:2], *c[2:], pad=2) for c in TWO_STREAMS[pair]]
    alone = [_attend(a) for a in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    calls = [_prepared(a, s) for a, s in zip(ins, streams)]
    torch.cuda.synchronize()
    for _ in range(40):
        for call, _, _ in calls:
            call()
    torch.cuda.synchronize()
    for (_, out, lse), (ref, ref_lse) in zip(calls, alone):
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16)) and torch.equal(lse, ref_lse)
    assert M.moe_device_status() == 0


@pytest.mark.parametrize("seed", range(24))
def test_attention_at_random_shapes(seed):
    """Lengths, groups (powers of two and others), pages and padding drawn from the seed."""
    rng = np.random.default_rng(1000 + seed)
    KV, G = int(rng.choice([1, 2, 4])), int(rng.choice([1, 2, 3, 4, 5, 7, 8, 16]))
    R, page = int(rng.integers(1, 9)), int(rng.choice([16, 32, 64, 128]))
    ctx = [int(np.exp(rng.uniform(0, np.log(6000)))) - 1 for _ in range(R)]
    new = [int(rng.choice([0, 1, 1, 5, rng.integers(1, 300), rng.integers(1, 1200)])) for _ in range(R)]
    new[0] = max(new[0], 1)
    _check_attention(_attn_inputs(rng, ctx, new, KV * G, KV, page, int(rng.choice([0, 1, 40]))), calls=2)


def test_attention_reports_rows_before_the_first_request():
    """row_start[0] is 0: rows before it would belong to no request and stay unwritten."""
    a = _attn_inputs(np.random.default_rng(18), [100, 40], [3, 3], 8, 2, 16)
    ref, _ = _attend(a)
    assert M.moe_device_status() == 0
    out, _ = _attend(dict(a, row_start=np.array([1, 3, 6])))
    assert M.moe_device_status() == 6
    assert torch.equal(out[3:].view(torch.int16), ref[3:].view(torch.int16))
