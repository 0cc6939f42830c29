"""Paged attention with a window refuses what it cannot serve, before any launch (no GPU), and the oracle
agrees with hand-worked values."""
import ctypes
from types import SimpleNamespace

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
    s = ctypes.byref(shape)
    return [lib.moe_paged_window_attention(s, window, sinks, *[p] * 8, p, ws, None),
            lib.moe_attention_paged_window_fwd(s, 1024, None, window, sinks, p, p, p, 1, *[p] * 7, p, ws, None)]


BAD_SHAPES = [(dict(requests=0), 1), (dict(tokens=0), 1), (dict(n_kv_head=0), 1), (dict(page_size=0), 1),
              (dict(pages=0), 1), (dict(max_pages=0), 1), (dict(eps=0.0), 1), (dict(q_stride=1016), 1),
              (dict(requests=4097), 2), (dict(head_dim=64), 2), (dict(n_head=9), 2), (dict(page_size=48), 2),
              (dict(pages=1 << 26), 2), (dict(max_pages=(1 << 20) + 1), 2)]


@pytest.mark.parametrize("change,code", BAD_SHAPES, ids=[str(c[0]) for c in BAD_SHAPES])
def test_bad_shapes_are_refused(lib, change, code):
    assert _calls(lib, M.make_paged_shape(**{**GOOD, **change}), ctypes.c_void_p(16)) == [code] * 2


def test_bad_pointers_windows_and_workspaces_are_refused(lib):
    shape, p = M.make_paged_shape(**GOOD), ctypes.c_void_p(16)
    assert _calls(lib, shape, None) == [1] * 2
    assert _calls(lib, shape, ctypes.c_void_p(24)) == [1] * 2  # not 16-byte aligned
    assert _calls(lib, shape, p, window=-1) == [1] * 2
    assert _calls(lib, shape, p, sinks=-1) == [1] * 2
    assert _calls(lib, shape, p, window=0, sinks=-1) == [1] * 2
    assert _calls(lib, shape, p, ws=M.moe_paged_attention_workspace_size(shape) - 1) == [3] * 2
    bad = M.MoERope()  # a rotation that was never made
    assert lib.moe_attention_paged_window_fwd(ctypes.byref(shape), 1024, ctypes.byref(bad), 0, 0, p, p, p, 1, *[p] * 7,
                                              p, 1 << 30, None) == 2
    assert lib.moe_attention_paged_window_fwd(ctypes.byref(shape), 1000, None, 0, 0, p, p, p, 1, *[p] * 7, p, 1 << 30,
                                              None) == 2


def test_the_block_refuses_windows_below_none():
    step = paged.PagedStep(requests=2, pages=4, page_size=16, max_pages=2, max_tokens=8, device="cpu")
    w = [torch.zeros(512, 64, dtype=torch.bfloat16), torch.zeros(64, 256, dtype=torch.bfloat16)]
    for kw in (dict(window=-1), dict(window=4, sinks=-1)):
        with pytest.raises(ValueError, match="window"):
            paged.PagedAttention(step, 64, 2, 1, *w, **kw)


def test_window_oracle():
    """Scores of zero: a row is the mean of the values that it sees; a window past the context is none."""
    rng = np.random.default_rng(1)
    v = rng.standard_normal((3, 1, 16, 128))
    flat = v[[2, 0, 1], 0].reshape(-1, 128)
    args = (np.zeros((5, 128)), np.zeros_like(v), v, np.array([[2, 0, 1]]), np.array([0, 5]), np.array([44]), 1, 1)
    got = P.paged_attention(*args, window=4, sinks=2)
    for i, p in enumerate(range(39, 44)):
        np.testing.assert_allclose(got["out"][i], flat[[0, 1, p - 3, p - 2, p - 1, p]].mean(0), rtol=1e-12)
    np.testing.assert_allclose(got["lse"], np.log(6), rtol=1e-12)
    whole = P.paged_attention(*args)
    np.testing.assert_array_equal(P.paged_attention(*args, window=44)["out"], whole["out"])
    np.testing.assert_array_equal(P.paged_attention(*args, window=1, sinks=44)["out"], whole["out"])


@pytest.mark.parametrize("window,sinks", [(1 << 32, 0), ((1 << 32) + 5, 0), (1 << 31, 0), (9, 1 << 32), (-(1 << 32), 0)])
def test_the_calls_refuse_windows_beyond_32_bits(lib, window, sinks):
    """They would arrive as other numbers: 2^32 as no window at all."""
    shape, none, on = M.make_paged_shape(**GOOD), torch.empty(0, dtype=torch.uint8), SimpleNamespace(cuda_stream=None)
    for call in (lambda w, s: M.moe_paged_window_attention(shape, w, s, *[None] * 8, none, stream=on),
                 lambda w, s: M.moe_attention_paged_window_fwd(shape, 1024, None, w, s, None, None, None, True,
                                                               *[None] * 7, none, stream=on),
                 lambda w, s: M.moe_paged_fork(shape, None, None, w, s, *[None] * 9, none, stream=on),
                 lambda w, s: M.moe_paged_release(shape, None, w, s, *[None] * 5, none, stream=on)):
        with pytest.raises(ValueError, match="32 bits"):
            call(window, sinks)
        with pytest.raises(M.MoEError):  # these reach the library, which has no addresses
            call((1 << 31) - 1, (1 << 31) - 1)
