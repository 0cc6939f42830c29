"""A paged key/value cache for serving: the step's tables, shared by all layers, and one
attention block's cache and weights.

PyTorch provides the device memory; every computation runs in the library
(moe_paged_plan, moe_attention_paged_fwd).  `PagedStep.plan` is one moe_paged_plan call,
`PagedAttention.forward` one moe_attention_paged_fwd call; neither waits for the GPU.
"""
from __future__ import annotations

import torch

from . import _lib as L


class PagedStep:
    """Block tables, page pool and lengths of up to `requests` requests at a time.

    A request is a row of the block table.  It starts with its first tokens (its context
    length is 0 then), grows with every step, and gives its pages back in the step that
    passes -1 for it; its row can start another request from the next step on.  `info`
    (rows in use, pages taken, pages returned, requests denied) tells what a step did; a
    denied request keeps its context and can be tried again."""

    def __init__(self, requests: int, pages: int, page_size: int, max_pages: int, max_tokens: int, device="cuda"):
        dev = torch.device(device)
        self.requests, self.pages, self.page_size, self.max_pages = requests, pages, page_size, max_pages
        self.max_tokens = max_tokens

        def i32(*shape):
            return torch.zeros(*shape, dtype=torch.int32, device=dev)

        self.block_table = torch.full((requests, max_pages), -1, dtype=torch.int32, device=dev)
        self.pool = torch.arange(pages, dtype=torch.int32, device=dev)
        # Context lengths and the pool's state before and after a step, by turns.
        self._ctx = [i32(requests), i32(requests)]
        self._state = [torch.tensor([0, pages], dtype=torch.int32, device=dev), i32(2)]
        self._now = 0
        self.row_start, self.slot_map, self.kv_len, self.info = i32(requests + 1), i32(max_tokens), i32(requests), i32(4)

    @property
    def ctx_len(self) -> torch.Tensor:
        """[requests] int32: the tokens that every request has in the cache."""
        return self._ctx[self._now]

    @property
    def free_pages(self) -> torch.Tensor:
        """[1] int32: pages in the pool."""
        return self._state[self._now][1:]

    def shape(self, tokens: int, n_head: int = 1, n_kv_head: int = 1, eps: float = 1e-6):
        if tokens > self.max_tokens:
            raise ValueError(f"{tokens} rows in a step planned for at most {self.max_tokens}")
        return L.make_paged_shape(self.requests, tokens, n_head, n_kv_head, self.page_size, self.pages, self.max_pages,
                                  eps=eps)

    def plan(self, new_len: torch.Tensor, tokens: int, stream=None) -> "PagedStep":
        """One step of `tokens` rows: new_len [requests] int32 (device): new tokens per request,
        0 = none, -1 = ended.  Rows past their sum are padding."""
        a, b = self._now, 1 - self._now
        L.moe_paged_plan(self.shape(tokens), self._ctx[a], new_len, self.block_table, self.pool, self._state[a],
                         self._state[b], self.row_start, self.slot_map, self.kv_len, self._ctx[b], self.info,
                         stream=stream)
        self._now = b
        return self


class PagedAttention:
    """One layer's attention block over a paged cache (weights as for moe_attention_fwd)."""

    def __init__(self, step: PagedStep, d: int, n_head: int, n_kv_head: int, w_qkv: torch.Tensor, w_o: torch.Tensor,
                 eps: float = 1e-6):
        self.step, self.d, self.n_head, self.n_kv_head, self.eps = step, d, n_head, n_kv_head, eps
        self.w_qkv, self.w_o = w_qkv, w_o
        cache = (step.pages, n_kv_head, step.page_size, 128)
        self.k_cache = torch.empty(cache, dtype=torch.bfloat16, device=w_qkv.device)
        self.v_cache = torch.empty(cache, dtype=torch.bfloat16, device=w_qkv.device)
        n = L.moe_attention_paged_workspace_size(step.shape(step.max_tokens, n_head, n_kv_head, eps), d)
        if n == 0:
            raise L.MoEError("moe_attention_paged_workspace_size", 2)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=w_qkv.device)

    def forward(self, x: torch.Tensor, out: torch.Tensor, residual: bool = True, stream=None) -> torch.Tensor:
        """x, out [tokens][d] bf16: the rows of the step that was planned last."""
        st = self.step
        L.moe_attention_paged_fwd(st.shape(x.shape[0], self.n_head, self.n_kv_head, self.eps), self.d, x, self.w_qkv,
                                  self.w_o, residual, self.k_cache, self.v_cache, st.block_table, st.row_start,
                                  st.slot_map, st.kv_len, out, self.workspace, stream=stream)
        return out
