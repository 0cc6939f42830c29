"""QK-norm with rotary positions refuses what it cannot serve, before any launch (no GPU); the rotation's
frequencies; and the oracle agrees with hand-worked values and finite differences."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import aux_loss_free_gb300 as M
from aux_loss_free_gb300 import build as B
from oracle import rope_oracle as R

GOOD = dict(requests=3, tokens=20, n_head=8, n_kv_head=2, page_size=16, pages=10, max_pages=4)


@pytest.fixture(scope="module")
def lib():
    return M.load_library(B.build())


def _rope(**change):
    r = M.make_rope(64)
    for k, v in change.items():
        setattr(r, k, v)
    return r


BAD_SHAPES = [(dict(requests=0), 1), (dict(tokens=0), 1), (dict(n_kv_head=0), 1), (dict(page_size=0), 1),
              (dict(pages=0), 1), (dict(max_pages=0), 1), (dict(eps=0.0), 1), (dict(requests=4097), 2),
              (dict(head_dim=64), 2), (dict(n_head=9), 2), (dict(page_size=48), 2), (dict(pages=1 << 26), 2),
              (dict(max_pages=(1 << 20) + 1), 2)]


@pytest.mark.parametrize("change,code", BAD_SHAPES, ids=[str(c[0]) for c in BAD_SHAPES])
def test_the_append_refuses_bad_shapes(lib, change, code):
    shape, p = M.make_paged_shape(**{**GOOD, **change}), ctypes.c_void_p(16)
    assert lib.moe_paged_append_rope(ctypes.byref(shape), ctypes.byref(_rope()), *[p] * 7, None) == code


def test_the_append_refuses_bad_pointers(lib):
    s, rope = ctypes.byref(M.make_paged_shape(**GOOD)), ctypes.byref(_rope())
    good = [ctypes.c_void_p(16 * (i + 1)) for i in range(7)]
    for i in range(7):
        for bad in (None, ctypes.c_void_p(24)):  # null; not 16-byte aligned
            assert lib.moe_paged_append_rope(s, rope, *[bad if j == i else g for j, g in enumerate(good)], None) == 1
    # In place the query rows are the projection's, (8 + 2 * 2) * 128 apart.
    good[4] = good[0]
    assert lib.moe_paged_append_rope(s, None, *good, None) == 1


BAD_ROPES = [(dict(rotary_dim=0), 2), (dict(rotary_dim=8), 2), (dict(rotary_dim=72), 2), (dict(rotary_dim=144), 2),
             (dict(rotary_dim=-16), 2), (dict(layout=2), 1), (dict(layout=-1), 1), (dict(magnitude=0.0), 1),
             (dict(magnitude=-1.0), 1), (dict(magnitude=float("nan")), 1), (dict(magnitude=float("inf")), 1)]


@pytest.mark.parametrize("change,code", BAD_ROPES, ids=[str(c[0]) for c in BAD_ROPES])
def test_bad_rotations_are_refused(lib, change, code):
    rope, p = ctypes.byref(_rope(**change)), ctypes.c_void_p(16)
    s, a = ctypes.byref(M.make_paged_shape(**GOOD)), ctypes.byref(M.make_attn_shape(1, 20, 1024, 8, 2))
    assert lib.moe_paged_append_rope(s, rope, *[p] * 7, None) == code
    assert lib.moe_qk_norm_rope(a, rope, p, p, p, None) == code
    assert lib.moe_qk_norm_rope_bwd(a, rope, p, p, p, p, None) == code
    assert lib.moe_attention_rope_fwd(a, rope, p, p, p, p, 1, p, p, 1 << 30, None) == code


def test_the_dense_calls_refuse_bad_shapes_and_pointers(lib):
    p, rope = ctypes.c_void_p(16), ctypes.byref(_rope())
    for bad, code in ((M.make_attn_shape(4, 2048, 1024, 8, 2, head_dim=64), 2), (M.make_attn_shape(4, 20, 1024, 8, 3), 2),
                      (M.make_attn_shape(0, 20, 1024, 8, 2), 1), (M.make_attn_shape(4, 20, 1024, 8, 2, eps=0.0), 1)):
        s = ctypes.byref(bad)
        assert lib.moe_qk_norm_rope(s, rope, None, p, p, None) == code
        assert lib.moe_qk_norm_rope_bwd(s, rope, None, p, p, p, None) == code
        assert lib.moe_attention_rope_fwd(s, rope, None, p, p, p, 1, p, p, 1 << 30, None) == code
    good, off = ctypes.byref(M.make_attn_shape(1, 20, 1024, 8, 2)), ctypes.c_void_p(24)
    for i in range(2):
        for bad in (None, off):
            q = [bad if j == i else p for j in range(2)]
            assert lib.moe_qk_norm_rope(good, rope, None, *q, None) == 1
    for i in range(3):
        for bad in (None, off):
            q = [bad if j == i else p for j in range(3)]
            assert lib.moe_qk_norm_rope_bwd(good, rope, None, *q, None) == 1
    assert lib.moe_qk_norm_rope(good, rope, off, p, p, None) == 1  # positions
    assert lib.moe_qk_norm_rope_bwd(good, rope, off, p, p, p, None) == 1
    assert lib.moe_attention_rope_fwd(good, rope, off, p, p, p, 1, p, p, 1 << 30, None) == 1
    assert lib.moe_attention_rope_fwd(good, rope, None, p, p, p, 1, p, p, 16, None) == 3


INIT = [(dict(base=0.5), 1), (dict(base=float("inf")), 1), (dict(base=float("nan")), 1), (dict(factor=0.9), 1),
        (dict(factor=float("nan")), 1), (dict(factor=float("inf")), 1), (dict(trained_len=-1), 1),
        (dict(trained_len=10, slow_turns=-1.0), 1), (dict(trained_len=10, slow_turns=2.0, fast_turns=2.0), 1),
        (dict(trained_len=10, fast_turns=float("inf")), 1), (dict(trained_len=10, fast_turns=float("nan")), 1),
        (dict(magnitude=0.0), 1), (dict(rotary_dim=12), 2), (dict(rotary_dim=256), 2)]


@pytest.mark.parametrize("change,code", INIT, ids=[str(c[0]) for c in INIT])
def test_bad_rotation_settings_are_refused(lib, change, code):
    with pytest.raises(M.MoEError) as e:
        M.make_rope(**change)
    assert e.value.code == code
    assert lib.moe_rope_init(None, 128, 0, 1e4, 1.0, 0, 1.0, 32.0, 1.0) == 1


FREQ = [dict(rotary_dim=128), dict(rotary_dim=16, base=1.0), dict(rotary_dim=96, base=5e5, factor=4.0),
        dict(rotary_dim=64, factor=32.0, trained_len=4096),
        dict(rotary_dim=128, factor=8.0, trained_len=8192, slow_turns=1.0, fast_turns=4.0)]


@pytest.mark.parametrize("kw", FREQ, ids=str)
def test_frequencies_in_turns(lib, kw):
    """turns[i] is the oracle's frequency / 2 pi in units of 2^-64, both in 64-bit arithmetic: a few
    roundings of 2^-53 each, and of the powers' exponent, at most ln(5e5) < 14 of them."""
    rope = M.make_rope(**kw)
    n = kw["rotary_dim"] // 2
    want = R.frequencies(**kw) / (2 * np.pi)
    for i in range(n):
        got = float(Fraction(rope.turns[i], 1 << 64))
        assert abs(got - want[i]) <= 40 * 2.0 ** -53 * want[i] + 2.0 ** -64
    assert all(t == 0 for t in list(rope.turns)[n:])
    assert (rope.rotary_dim, rope.layout, rope.magnitude) == (kw["rotary_dim"], M.MOE_ROPE_HALVES, 1.0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_oracle(interleaved):
    """One pair by hand; scores depend on the distance of the positions alone; back undoes it."""
    x = np.zeros((1, 1, 128))
    a, b = (2, 3) if interleaved else (1, 9)
    x[0, 0, a], x[0, 0, b], x[0, 0, 100] = 3.0, 4.0, 5.0
    f = R.frequencies(16, base=10000.0)
    y = R.rotate(x, [7], f, interleaved, magnitude=2.0)
    t = 7 * 10000.0 ** (-2 / 16)
    np.testing.assert_allclose([y[0, 0, a], y[0, 0, b], y[0, 0, 100]],
                               [2 * (3 * np.cos(t) - 4 * np.sin(t)), 2 * (4 * np.cos(t) + 3 * np.sin(t)), 5.0], rtol=1e-14)
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 128))
    f = R.frequencies(128)
    dots = [np.sum(R.rotate(q, [p + 13], f, interleaved) * R.rotate(k, [p], f, interleaved)) for p in (0, 5, 1000)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-9)
    z = R.rotate(R.rotate(q, [77], f, interleaved), [77], f, interleaved, back=True)
    np.testing.assert_allclose(z, q, rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("interleaved,rot", [(False, 128), (True, 64), (False, 32)])
def test_gradient_oracle_against_differences(interleaved, rot):
    rng = np.random.default_rng(rot)
    u, dy = rng.standard_normal((2, 3, 4 * 128))
    f, pos = R.frequencies(rot), [0, 5, 4000]
    args = (pos, 2, 1, f, interleaved, 1.3)
    got, bound = R.norm_rope_bwd(u, dy, *args)
    assert (np.abs(got) <= bound * (1 + 1e-12)).all()
    h = 1e-6
    for _ in range(40):
        r, c = rng.integers(3), rng.integers(4 * 128)
        e = np.zeros_like(u)
        e[r, c] = h
        diff = np.sum(dy * (R.norm_rope(u + e, *args) - R.norm_rope(u - e, *args))) / (2 * h)
        assert abs(diff - got[r, c]) <= 1e-7 * (1 + abs(got[r, c]))


@pytest.mark.parametrize("kw", [dict(rotary_dim=(1 << 32) + 64), dict(trained_len=1 << 32), dict(trained_len=1 << 31)])
def test_sizes_beyond_32_bits_are_refused(lib, kw):
    """They would arrive as other numbers: a trained length of 2^32 as none."""
    with pytest.raises(ValueError, match="32 bits"):
        M.make_rope(factor=8.0, **kw)
    M.make_rope(factor=8.0, trained_len=(1 << 31) - 1)


@pytest.mark.parametrize("n_head", [65, 1 << 24, 1 << 25, (1 << 25) + 8, (1 << 31) - 8])
def test_more_heads_than_the_block_has_are_refused(lib, n_head):
    """Values of a row past 8192, counted without a product that passes 32 bits."""
    p, s = ctypes.c_void_p(16), ctypes.byref(M.make_attn_shape(1, 20, 1024, n_head, n_head // 4 if n_head % 4 == 0 else 1))
    assert lib.moe_attention_workspace_size(s) == 0
    assert lib.moe_attention_core(s, p, p, None) == 2
    assert lib.moe_attention_fwd(s, p, p, p, 1, p, p, 1 << 30, None) == 2
    assert lib.moe_qk_norm_rope(s, None, None, p, p, None) == 2
    assert lib.moe_qk_norm_rope_bwd(s, None, None, p, p, p, None) == 2
    assert lib.moe_attention_rope_fwd(s, None, None, p, p, p, 1, p, p, 1 << 30, None) == 2
