"""The paged cache's calls refuse what they cannot serve, before any launch (no GPU), and
the oracle's step plan and paged attention agree with hand-worked values and the dense
oracle."""
import ctypes
import types

import numpy as np
import pytest
import torch

import aux_loss_free_gb300 as M
from aux_loss_free_gb300 import build as B
from aux_loss_free_gb300 import paged
from oracle import attention_oracle as A
from oracle import paged_oracle as P

GOOD = dict(requests=3, tokens=20, n_head=8, n_kv_head=2, page_size=16, pages=10, max_pages=4)


@pytest.fixture(scope="module")
def lib():
    return M.load_library(B.build())


def _calls(lib, shape, p, ws=1 << 30):
    """The status of every call on `shape`, its pointers all p."""
    s = ctypes.byref(shape)
    return [lib.moe_paged_plan(s, *[p] * 11, None), lib.moe_paged_append(s, *[p] * 5, None),
            lib.moe_paged_attention(s, *[p] * 8, p, ws, None),
            lib.moe_attention_paged_fwd(s, 1024, p, p, p, 1, *[p] * 7, p, ws, None)]


BAD_SHAPES = [(dict(requests=0), 1), (dict(tokens=0), 1), (dict(n_head=0), 1), (dict(n_kv_head=0), 1),
              (dict(page_size=0), 1), (dict(pages=0), 1), (dict(max_pages=0), 1), (dict(eps=0.0), 1),
              (dict(eps=float("nan")), 1), (dict(q_stride=-8), 1), (dict(q_stride=1016), 1), (dict(q_stride=1028), 1),
              (dict(requests=4097), 2), (dict(tokens=(1 << 20) + 1), 2), (dict(head_dim=64), 2), (dict(n_head=9), 2),
              (dict(n_head=66), 2), (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=256), 2),
              (dict(pages=1 << 26), 2), (dict(max_pages=(1 << 20) + 1), 2)]


@pytest.mark.parametrize("change,code", BAD_SHAPES, ids=[str(c[0]) for c in BAD_SHAPES])
def test_bad_shapes_are_refused(lib, change, code):
    shape = M.make_paged_shape(**{**GOOD, **change})
    assert M.moe_paged_attention_workspace_size(shape) == 0
    assert M.moe_attention_paged_workspace_size(shape, 1024) == 0
    assert _calls(lib, shape, ctypes.c_void_p(16)) == [code] * 4


def test_bad_pointers_widths_and_workspaces_are_refused(lib):
    shape = M.make_paged_shape(**GOOD)
    assert _calls(lib, shape, None) == [1] * 4
    assert _calls(lib, shape, ctypes.c_void_p(24)) == [1] * 4  # not 16-byte aligned
    assert lib.moe_paged_plan(None, *[ctypes.c_void_p(16)] * 11, None) == 1
    p, s = ctypes.c_void_p(16), ctypes.byref(shape)
    need = M.moe_paged_attention_workspace_size(shape)
    assert need > 0
    assert lib.moe_paged_attention(s, *[p] * 8, p, need - 1, None) == 3
    block = M.moe_attention_paged_workspace_size(shape, 1024)
    assert block >= need + 2 * 20 * 12 * 128 + 2 * 20 * 8 * 128
    assert lib.moe_attention_paged_fwd(s, 1024, p, p, p, 1, *[p] * 7, p, block - 1, None) == 3
    for d, code in ((0, 1), (-64, 1), (1000, 2), (8256, 2)):
        assert M.moe_attention_paged_workspace_size(shape, d) == 0
        assert lib.moe_attention_paged_fwd(s, d, p, p, p, 1, *[p] * 7, p, block, None) == code
    # In place the query rows are the projection's, (8 + 2 * 2) * 128 apart.
    assert lib.moe_paged_append(s, p, p, p, p, p, None) == 1


def test_step_plan_oracle_on_a_worked_step():
    """Pages of 16, five requests: 0 decodes into its half-full page, 1 begins a page, 2 has
    ended (two pages back), 3 is idle, 4 starts with 20 tokens (two pages)."""
    table = [[7, -1], [5, -1], [3, 2], [6, -1], [-1, -1]]
    pool = [1, 4, -1, -1, -1, -1, -1, 0]  # pages 0, 1, 4 free, from place 7 on
    r = P.step_plan([3, 16, 20, 9, 0], [1, 1, -1, 0, 20], table, pool, [7, 3], tokens=24, pages=8, page_size=16)
    assert r["row_start"].tolist() == [0, 1, 2, 2, 2, 22]
    assert r["block_table"].tolist() == [[7, -1], [5, 0], [3, 2], [6, -1], [1, 4]]
    assert r["slot_map"].tolist() == [7 * 16 + 3, 0] + list(range(16, 32)) + list(range(64, 68)) + [-1, -1]
    assert r["kv_len"].tolist() == [4, 17, 0, 9, 20]
    assert r["next_ctx"].tolist() == [4, 17, 0, 9, 20]
    assert r["pool"].tolist() == [1, 4, 3, 2, -1, -1, -1, 0]
    assert r["pool_state"].tolist() == [2, 2]
    assert r["info"].tolist() == [22, 3, 2, 0]


def test_step_plan_oracle_denies_in_order():
    """One free page: request 0 wants two and is denied, 1 wants one and is denied after it, 2
    needs none and is served."""
    r = P.step_plan([0, 0, 5], [20, 3, 1], [[-1, -1]] * 2 + [[1, -1]], [0, -1], [0, 1], tokens=24, pages=2,
                    page_size=16)
    assert r["kv_len"].tolist() == [0, 0, 6] and r["next_ctx"].tolist() == [0, 0, 6]
    assert r["slot_map"].tolist() == [-1] * 23 + [21]
    assert r["info"].tolist() == [24, 0, 0, 2] and r["pool_state"].tolist() == [0, 1]


def test_paged_attention_oracle_equals_the_dense_oracle():
    """A prompt and a second chunk of one sequence, through pages placed at random, against
    the dense causal oracle over the whole sequence."""
    rng = np.random.default_rng(5)
    d, H, KV, S, page = 64, 4, 2, 45, 16
    x = rng.standard_normal((S, d))
    w = [rng.standard_normal((n * 128, d)) * 0.1 for n in (H, KV, KV)]
    r = A.gqa_attention(x, *w, np.zeros((d, H * 128)), 1, S, H, KV, residual=False, round_stored=False)
    ids = np.array([4, 0, 2])
    kc, vc = rng.standard_normal((2, 5, KV, page, 128))
    slots = ids[np.arange(S) // page] * page + np.arange(S) % page
    qkv = np.concatenate([x @ m.T for m in w], axis=1)
    q, kc, vc = P.append(qkv, slots, H, KV, page, kc, vc)
    np.testing.assert_allclose(q, r["q"].reshape(S, -1), rtol=1e-12)
    for a, b in ((0, 30), (30, 45)):
        got = P.paged_attention(q[a:b], kc, vc, ids[None], np.array([0, b - a]), np.array([b]), H, KV)
        np.testing.assert_allclose(got["out"], r["o"][a:b], rtol=1e-10, atol=1e-12)



@pytest.fixture
def step(lib, monkeypatch):
    """A step of two requests whose tensors lie on the host; a call that gets past the checks
    fails the test instead of passing host addresses on."""
    def reached(*_, **__):
        raise AssertionError("the library was called")

    monkeypatch.setattr(paged.L, "moe_paged_plan", reached)
    monkeypatch.setattr(paged.L, "moe_attention_paged_fwd", reached)
    return paged.PagedStep(requests=2, pages=4, page_size=16, max_pages=2, max_tokens=8, device="cpu")


NEW_LEN = {  # of two requests, and what the refusal says
    "int64": (lambda: torch.tensor([1, 1]), "type"),
    "float": (lambda: torch.tensor([1.0, 1.0]), "type"),
    "too-few": (lambda: torch.tensor([1], dtype=torch.int32), "size"),
    "too-many": (lambda: torch.tensor([1, 1, 1], dtype=torch.int32), "size"),
    "two-dims": (lambda: torch.tensor([[1, 1]], dtype=torch.int32), "size"),
    "strided": (lambda: torch.tensor([1, 7, 1, 7], dtype=torch.int32)[::2], "contiguous"),
    "elsewhere": (lambda: torch.empty(2, dtype=torch.int32, device="meta"), "device"),
    "on-the-host": (lambda: torch.tensor([1, 1], dtype=torch.int32), "CUDA device"),
}


@pytest.mark.parametrize("name", NEW_LEN)
def test_plan_refuses_other_tensors(step, name):
    make, why = NEW_LEN[name]
    with pytest.raises(ValueError, match=why):
        step.plan(make(), 2)
    assert step.tokens == 0


def _block(step, w_qkv=(512, 64), w_o=(64, 256), dtype=torch.bfloat16):
    return paged.PagedAttention(step, 64, 2, 1, torch.zeros(w_qkv, dtype=dtype), torch.zeros(w_o, dtype=dtype))


@pytest.mark.parametrize("change,why", [(dict(w_qkv=(511, 64)), "w_qkv: size"), (dict(w_qkv=(512, 128)), "w_qkv: size"),
                                        (dict(w_o=(256, 64)), "w_o: size"), (dict(w_o=(64, 128)), "w_o: size"),
                                        (dict(dtype=torch.float32), "w_qkv: type")], ids=str)
def test_the_block_refuses_other_weights(step, change, why):
    with pytest.raises(ValueError, match=why):
        _block(step, **change)


ROWS = {  # of a step of 4 rows, width 64
    "float32": (lambda: torch.zeros(4, 64), "type"),
    "too-few": (lambda: torch.zeros(3, 64, dtype=torch.bfloat16), "size"),
    "too-many": (lambda: torch.zeros(5, 64, dtype=torch.bfloat16), "size"),
    "wide": (lambda: torch.zeros(4, 128, dtype=torch.bfloat16), "size"),
    "three-dims": (lambda: torch.zeros(1, 4, 64, dtype=torch.bfloat16), "size"),
    "columns-of-wider-rows": (lambda: torch.zeros(4, 128, dtype=torch.bfloat16)[:, :64], "contiguous"),
    "transposed": (lambda: torch.zeros(64, 4, dtype=torch.bfloat16).t(), "contiguous"),
    "elsewhere": (lambda: torch.empty(4, 64, dtype=torch.bfloat16, device="meta"), "device"),
}


@pytest.mark.parametrize("name", ROWS)
@pytest.mark.parametrize("which", ["x", "out"])
def test_the_block_refuses_other_rows(step, name, which):
    block, good = _block(step), torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x: size"):  # nothing is planned yet
        block.forward(good, good)
    step.tokens = 4
    make, why = ROWS[name]
    with pytest.raises(ValueError, match=f"{which}: .*{why}"):
        block.forward(*((make(), good) if which == "x" else (good, make())))
    with pytest.raises(ValueError, match="CUDA device"):
        block.forward(good, good)


@pytest.mark.parametrize("missing", [None, "_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_the_current_stream_without_pytorchs_own_calls(monkeypatch, missing):
    """The calls that read the handle directly are not public: without one of them it comes from
    the public Stream object."""
    for name, value in (("_cuda_getCurrentRawStream", lambda d: 100 + d), ("_cuda_getDevice", lambda: 3)):
        if name == missing:
            monkeypatch.delattr(torch._C, name, raising=False)
        else:
            monkeypatch.setattr(torch._C, name, value, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=7))
    monkeypatch.setattr(M._lib, "_current", None, raising=False)
    assert M._lib._stream(None) == (7 if missing else 103)
    assert M._lib._stream(types.SimpleNamespace(cuda_stream=9)) == 9
