"""Rotary positions, windows, branches and pages given up, together, as a serving program uses them
(PagedStep, PagedAttention): two layers, prompts, decoding, drafts that are rejected, a search that branches,
requests that end and start, a cache moved together; every row of every step against the dense
computation of its sequence in 64 bits, rounded where the library stores (the block tests' tolerance)."""
import numpy as np
import pytest
import torch

import aux_loss_free_gb300 as M
from aux_loss_free_gb300.layer import to_device_bf16
from aux_loss_free_gb300.paged import PagedAttention, PagedStep
from gpu_util import assert_close_bf16, bf16_to_np, bf64
from oracle import paged_oracle as P
from oracle import rope_oracle as R
from oracle.moe_oracle import round_to_bf16
from synth import ATTN_CONFIGS, make_attention

pytestmark = pytest.mark.gpu

DEV = "cuda"
H, KV, D = 8, 2, 512


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    M.load_library()
    yield
    assert M.moe_device_status() == 0


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


class Layer:
    """A layer's weights, its block, and the sequences of rows that it has been given."""

    def __init__(self, step, seed, rope_kw, window, sinks):
        a = ATTN_CONFIGS["attn_tiny"].replace(batch=1, seq=8, n_head=H, n_kv_head=KV, d=D, eps=1e-6)
        w = make_attention(a, "attn_tiny")
        rng = np.random.default_rng(seed)
        self.w = {n: np.asarray(v)[rng.permutation(len(v))] for n, v in w.items() if n != "x"}
        w_qkv = to_device_bf16(np.concatenate([self.w["w_q"], self.w["w_k"], self.w["w_v"]], axis=0), DEV)
        rope = None if rope_kw is None else M.make_rope(**rope_kw)
        self.block = PagedAttention(step, D, H, KV, w_qkv, to_device_bf16(self.w["w_o"], DEV), 1e-6, rope=rope,
                                    window=window, sinks=sinks)
        self.block.k_cache.fill_(float("nan"))
        self.block.v_cache.fill_(float("nan"))
        kw = dict(rope_kw or {})
        self.inter = kw.pop("interleaved", False)
        self.freq = np.zeros(0) if rope_kw is None else R.frequencies(kw.pop("rotary_dim", 128), **kw)
        self.window, self.sinks = window, sinks
        self.rows = [np.zeros((0, D)) for _ in range(step.requests)]

    def want(self, r, n):
        """The last n rows of sequence r."""
        x = self.rows[r]
        S = len(x)
        qkv = round_to_bf16(np.concatenate([x @ bf64(self.w[k]).T for k in ("w_q", "w_k", "w_v")], axis=1))
        t = round_to_bf16(R.norm_rope(qkv, np.arange(S), H, KV, self.freq, self.inter)).reshape(S, H + 2 * KV, 128)
        kc, vc = (t[:, i:i + KV].transpose(1, 0, 2)[None] for i in (H, H + KV))
        o = P.paged_attention(t[S - n:, :H].reshape(n, -1), kc, vc, np.array([[0]]), np.array([0, n]), np.array([S]), H,
                              KV, self.window, self.sinks)["out"]
        return round_to_bf16(o) @ bf64(self.w["w_o"]).T + x[S - n:]


def _serve(script, layers, step, graph=False):
    rng = np.random.default_rng(11)
    T = step.max_tokens
    x, h, y = (torch.zeros(T, D, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    new = _i32([0] * step.requests)
    free = []

    def run(stream=None):
        step.plan(new, T, stream=stream)
        layers[0].block.forward(x, h, stream=stream)
        layers[1].block.forward(h, y, stream=stream)

    captured = None
    if graph:
        captured, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(captured, stream=side):
            run(side)
    for kind, arg in script:
        if kind == "compact":
            step.compact()
            continue
        if kind == "fork":
            parent, keep = arg
            step.fork(_i32(parent), None if keep is None else _i32(keep))
            for layer in layers:
                old = layer.rows
                layer.rows = [np.zeros((0, D)) if q < 0 else old[q][:len(old[q]) if keep is None else keep[r]]
                              for r, q in enumerate(parent)]
            torch.cuda.synchronize()
            assert step.ctx_len.tolist() == [len(s) for s in layers[0].rows]
            assert step.pages_info.tolist()[2] == 0
            continue
        lens = arg
        new.copy_(_i32(lens))
        n = sum(max(v, 0) for v in lens)
        x.copy_(torch.tensor(rng.standard_normal((T, D)), dtype=torch.float32).to(DEV).to(torch.bfloat16))
        captured.replay() if captured else run()
        torch.cuda.synchronize()
        assert step.info.tolist()[0] == n and step.info.tolist()[3] == 0
        free.append(step.free_pages.item())
        for layer, src, out in ((layers[0], x, h), (layers[1], h, y)):
            src, out, at = bf16_to_np(src), bf16_to_np(out), 0
            for r, v in enumerate(lens):
                if v < 0:
                    layer.rows[r] = np.zeros((0, D))
                elif v > 0:
                    layer.rows[r] = np.concatenate([layer.rows[r], src[at:at + v]])
                    assert_close_bf16(out[at:at + v], layer.want(r, v), f"{kind} {lens}, row {r}")
                    at += v
            assert np.array_equal(out[n:], src[n:])  # padding rows
    assert step.ctx_len.tolist() == [len(s) for s in layers[0].rows]
    return free


SCRIPT = [
    ("step", [70, 33, 0, 0, 0]), ("step", [1, 1, 20, 0, 0]),
    ("fork", ([0, 1, 2, 0, 0], None)),                       # two more branches of row 0 (71 tokens: a page with room left)
    ("step", [1, 1, 1, 1, 1]),
    ("step", [5, 5, 1, 1, 1]),                               # drafts
    ("fork", ([0, 1, 2, 3, 4], [74, 35, 22, 73, 73])),       # some rejected
    ("step", [1, 30, 1, 1, 1]),
    ("fork", ([3, 1, 2, 0, -1], [74, 65, 22, 64, 0])),       # rows change places, one goes, one goes on from whole pages
    ("step", [1, 1, -1, 1, 40]),
    ("compact", None),
    ("step", [1, 1, 17, 1, 1]),
    ("step", [-1, 1, 1, 1, 1]),
    ("fork", ([1, 1, 1, 1, 4], None)),                       # four branches of one
    ("step", [3, 2, 1, 4, 1]), ("step", [1, 1, 1, -1, 1]), ("compact", None), ("step", [1, 1, 1, 9, 1]),
    ("step", [-1, -1, -1, -1, -1]),
]


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("rope", [dict(), dict(rotary_dim=64, interleaved=True, factor=4.0, trained_len=32), None])
def test_serving_with_branches(rope, graph):
    step = PagedStep(requests=5, pages=40, page_size=16, max_pages=10, max_tokens=128, sharing=True)
    layers = [Layer(step, 1, rope, 0, 0), Layer(step, 2, rope, 48, 4)]
    free = _serve(SCRIPT, layers, step, graph)
    assert free[-1] == 40  # every page is back


# Behind a window of 40 and 4 first tokens: rows that are long since past it, cut back by drafts alone.
# Forks give (parent, rejected tokens).
LONG = [("step", [100, 20, 0]), ("step", [60, 1, 90])] + [("step", [1, 25, 1])] * 4 + [
    ("fork", ([0, 0, 2], [0, 0, 0])), ("step", [6, 6, 1]), ("fork", ([0, 1, 2], [4, 0, 0])), ("step", [1, 1, 1]),
    ("compact", None), ("step", [30, 1, -1]), ("step", [1, 1, 50]), ("step", [1, 1, 50])] + [
    ("step", [20, 0, 1])] * 5 + [("step", [-1, 0, 0]), ("step", [0, -1, -1])]


@pytest.mark.parametrize("graph", [False, True])
def test_serving_behind_a_window(graph):
    """Pages behind the window come back as the rows grow: 24 pages of 16 tokens, where rows that kept all
    of theirs would need 30."""
    step = PagedStep(requests=3, pages=24, page_size=16, max_pages=30, max_tokens=160, sharing=True, window=40, sinks=4)
    layers = [Layer(step, 3, dict(), 40, 4), Layer(step, 4, dict(interleaved=True), 17, 1)]
    script, ctx, most = [], [0, 0, 0], 0
    for kind, arg in LONG:  # what is kept follows from the lengths
        if kind == "step":
            ctx = [0 if n < 0 else c + n for c, n in zip(ctx, arg)]
        elif kind == "fork":
            ctx = [ctx[q] - d for q, d in zip(*arg)]
            arg = (arg[0], ctx)
        most = max(most, sum(-(-c // 16) for c in ctx))
        script.append((kind, arg))
    assert most > 24
    free = _serve(script, layers, step, graph)
    assert free[-1] == 24


def test_rows_cut_short_behind_a_window_serve_on():
    """A search behind a window in a full pool: branches without a page for their copy go on from whole pages, and their
    next tokens see all that they should, the 40 keys behind them reaching into the first page."""
    step = PagedStep(requests=5, pages=7, page_size=16, max_pages=10, max_tokens=112, sharing=True, window=40)
    layers = [Layer(step, 5, dict(), 40, 0), Layer(step, 6, None, 17, 0)]
    rng = np.random.default_rng(12)
    x, h, y = (torch.zeros(112, D, dtype=torch.bfloat16, device=DEV) for _ in range(3))

    def run(lens):
        x.copy_(torch.tensor(rng.standard_normal((112, D)), dtype=torch.float32).to(DEV).to(torch.bfloat16))
        step.plan(_i32(lens), 112)
        layers[0].block.forward(x, h)
        layers[1].block.forward(h, y)
        torch.cuda.synchronize()
        assert M.moe_device_status() == 0 and step.info.tolist()[3] == 0
        for layer, src, out in ((layers[0], x, h), (layers[1], h, y)):
            src, out, at = bf16_to_np(src), bf16_to_np(out), 0
            for r, v in enumerate(lens):
                layer.rows[r] = np.concatenate([layer.rows[r], src[at:at + v]]) if v >= 0 else np.zeros((0, D))
                if v > 0:
                    assert_close_bf16(out[at:at + v], layer.want(r, v), f"{lens}, row {r}")
                    at += v

    run([59, 0, 0, 0, 48])
    run([1, 0, 0, 0, 0])
    assert step.free_pages.item() == 0
    step.fork(_i32([0, 0, 0, 0, 4]))
    torch.cuda.synchronize()
    assert step.ctx_len.tolist() == [60, 48, 48, 48, 48] and step.pages_info.tolist() == [0, 0, 3, 7]
    for layer in layers:
        layer.rows[1:4] = [layer.rows[0][:48]] * 3
    run([1, 1, 5, 9, -1])
    run([3, 1, 1, 1, 0])
    run([0, 14, 10, 6, 0])
    run([-1, -1, -1, -1, 0])
    assert step.free_pages.item() == 7
