"""A paged key/value cache for serving: the step's tables, shared by all layers, and one
attention block's cache and weights.

PyTorch provides the device memory; every computation runs in the library
(moe_paged_plan, moe_attention_paged_fwd).  `PagedStep.plan` is one moe_paged_plan call,
`PagedAttention.forward` one moe_attention_paged_fwd call; neither waits for the GPU, and
both can be captured and replayed with other lengths.
"""
from __future__ import annotations

import torch

from . import _lib as L


def _check(name: str, t: torch.Tensor, dtype: torch.dtype, shape: tuple, device: torch.device):
    """The library gets addresses alone: what it finds there is checked here."""
    if t.dtype != dtype:
        raise ValueError(f"{name}: type {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: size {list(t.shape)}, not {list(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous (strides {list(t.stride())})")
    if t.device != device:
        raise ValueError(f"{name}: on device {t.device}, not {device}")


def _check_cuda(device: torch.device):
    if device.type != "cuda":
        raise ValueError(f"the calls run on a CUDA device, not on {device}")


class PagedStep:
    """Block tables, page pool and lengths of up to `requests` requests at a time.

    A request is a row of the block table.  It starts with its first tokens (its context
    length is 0 then), grows with every step, and gives its pages back in the step that
    passes -1 for it; its row can start another request from the next step on.  `info`
    (rows in use, pages taken, pages returned, requests denied) tells what a step did; a
    denied request keeps its context and can be tried again.

    A plan replaces the lengths that the last one left, on the stream that it is given: plans and
    the calls that use their tables belong to one stream, or to streams that wait for each other."""

    def __init__(self, requests: int, pages: int, page_size: int, max_pages: int, max_tokens: int, device="cuda"):
        dev = torch.device(device)
        self.requests, self.pages, self.page_size, self.max_pages = requests, pages, page_size, max_pages
        self.max_tokens = max_tokens
        self.tokens = 0  # rows of the step that was planned (or captured) last

        def i32(*shape):
            return torch.zeros(*shape, dtype=torch.int32, device=dev)

        self.block_table = torch.full((requests, max_pages), -1, dtype=torch.int32, device=dev)
        self.pool = torch.arange(pages, dtype=torch.int32, device=dev)
        # Every plan takes these in place, so that a captured one goes on from where the last step
        # or replay ended.
        self._ctx, self._state = i32(requests), torch.tensor([0, pages], dtype=torch.int32, device=dev)
        self.row_start, self.slot_map, self.kv_len, self.info = i32(requests + 1), i32(max_tokens), i32(requests), i32(4)

    @property
    def ctx_len(self) -> torch.Tensor:
        """[requests] int32: the tokens that every request has in the cache."""
        return self._ctx

    @property
    def free_pages(self) -> torch.Tensor:
        """[1] int32: pages in the pool."""
        return self._state[1:]

    def shape(self, tokens: int, n_head: int = 1, n_kv_head: int = 1, eps: float = 1e-6):
        if tokens > self.max_tokens:
            raise ValueError(f"{tokens} rows in a step made for at most {self.max_tokens}")
        return L.make_paged_shape(self.requests, tokens, n_head, n_kv_head, self.page_size, self.pages, self.max_pages,
                                  eps=eps)

    def plan(self, new_len: torch.Tensor, tokens: int, stream=None) -> "PagedStep":
        """One step of `tokens` rows: new_len [requests] int32 (device): new tokens per request,
        0 = none, -1 = ended.  Rows past their sum are padding."""
        ctx, state = self._ctx, self._state
        _check("new_len", new_len, torch.int32, (self.requests,), ctx.device)
        _check_cuda(ctx.device)
        L.moe_paged_plan(self.shape(tokens), ctx, new_len, self.block_table, self.pool, state, state, self.row_start,
                         self.slot_map, self.kv_len, ctx, self.info, stream=stream)
        self.tokens = tokens
        return self


class PagedAttention:
    """One layer's attention block over a paged cache (weights as for moe_attention_fwd)."""

    def __init__(self, step: PagedStep, d: int, n_head: int, n_kv_head: int, w_qkv: torch.Tensor, w_o: torch.Tensor,
                 eps: float = 1e-6):
        self.step, self.d, self.n_head, self.n_kv_head, self.eps = step, d, n_head, n_kv_head, eps
        dev = step.block_table.device
        _check("w_qkv", w_qkv, torch.bfloat16, ((n_head + 2 * n_kv_head) * 128, d), dev)
        _check("w_o", w_o, torch.bfloat16, (d, n_head * 128), dev)
        self.w_qkv, self.w_o = w_qkv, w_o
        cache = (step.pages, n_kv_head, step.page_size, 128)
        self.k_cache = torch.empty(cache, dtype=torch.bfloat16, device=dev)
        self.v_cache = torch.empty(cache, dtype=torch.bfloat16, device=dev)
        n = L.moe_attention_paged_workspace_size(step.shape(step.max_tokens, n_head, n_kv_head, eps), d)
        if n == 0:
            raise L.MoEError("moe_attention_paged_workspace_size", 2)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=dev)

    def forward(self, x: torch.Tensor, out: torch.Tensor, residual: bool = True, stream=None) -> torch.Tensor:
        """x, out [tokens][d] bf16: the rows of the step that was planned last, all of them."""
        st = self.step
        rows = (st.tokens, self.d)
        _check("x", x, torch.bfloat16, rows, self.w_qkv.device)
        _check("out", out, torch.bfloat16, rows, self.w_qkv.device)
        _check_cuda(self.w_qkv.device)
        L.moe_attention_paged_fwd(st.shape(x.shape[0], self.n_head, self.n_kv_head, self.eps), self.d, x, self.w_qkv,
                                  self.w_o, residual, self.k_cache, self.v_cache, st.block_table, st.row_start,
                                  st.slot_map, st.kv_len, out, self.workspace, stream=stream)
        return out
