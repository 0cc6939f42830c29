"""A paged key/value cache for serving: the step's tables, shared by all layers, and one
attention block's cache and weights.

PyTorch provides the device memory; every computation runs in the library
(moe_paged_plan, moe_attention_paged_fwd and their relatives).  `PagedStep.plan` is one
moe_paged_plan call (with `sharing` a moe_paged_release in front of it), `fork` and `compact`
one call and the page copies that it asks for, `PagedAttention.forward` one
moe_attention_paged_fwd or moe_attention_paged_window_fwd call; none waits for the GPU, and all
can be captured and replayed with other lengths.
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
    the calls that use their tables belong to one stream, or to streams that wait for each other.

    With `sharing`, rows can branch off others, be cut back (fork) and be moved together (compact) between
    two plans; requests that end give back the pages that no other row holds, and `pages_info`
    (copies, pages given back, rows cut short, pages in use) tells what the last of these calls did.
    With `window` (and `sinks`) too, every plan also gives back the pages that no later token sees, but for one
    page of a row at most: every layer's attention then has a window of at most this one and at most these sinks, and a row can be cut
    back or branched off no further back than it stood when it was last planned or forked (what its next token
    should see is gone then: the attention reports MOE_ERR_DEVICE).  A row that fork cuts short, because
    the pool has no page for its copy, goes on from the whole pages that it kept."""

    def __init__(self, requests: int, pages: int, page_size: int, max_pages: int, max_tokens: int, device="cuda",
                 sharing: bool = False, window: int = 0, sinks: int = 0):
        if not (0 <= window < 1 << 31 and 0 <= sinks < 1 << 31):
            raise ValueError(f"a window of {window} tokens and {sinks} first ones")
        if window and not sharing:
            raise ValueError("pages are given back behind a window with sharing=True alone")
        dev = torch.device(device)
        self.sharing, self.window, self.sinks = sharing, window, sinks
        # A row that is cut short later loses up to page_size - 1 tokens, and its window moves back by as
        # many: what it sees then is kept from the start, at most one page of a row.
        self._kept = min(window + page_size - 1, (1 << 31) - 1) if window else 0
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
        self._caches = {}  # key/value heads -> the layers' caches with so many
        if sharing:
            self.pages_info, self._copies = i32(4), i32(max(requests, pages // 2), 4)
            n = L.moe_paged_pages_workspace_size(self.shape(1))
            if n == 0:
                raise L.MoEError("moe_paged_pages_workspace_size", 2)
            self._workspace = torch.empty(n, dtype=torch.uint8, device=dev)

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
        shape = self.shape(tokens)
        if self.sharing:
            L.moe_paged_release(shape, new_len, self._kept, self.sinks, ctx, self.block_table, self.pool, state,
                                self.pages_info, self._workspace, stream=stream)
        L.moe_paged_plan(shape, ctx, new_len, self.block_table, self.pool, state, state, self.row_start,
                         self.slot_map, self.kv_len, ctx, self.info, stream=stream)
        self.tokens = tokens
        return self

    def add_caches(self, n_kv_head: int, *caches: torch.Tensor):
        """Caches [pages][n_kv_head][page_size][128] whose pages fork and compact copy, and which the step
        keeps (PagedAttention adds its own to a step with sharing)."""
        for cache in caches:
            _check("cache", cache, torch.bfloat16, (self.pages, n_kv_head, self.page_size, 128), self._ctx.device)
        self._caches.setdefault(n_kv_head, []).extend(caches)

    def _between_steps(self):
        if not self.sharing:
            raise ValueError("rows branch and pages move with sharing=True alone")
        _check_cuda(self._ctx.device)

    def _copy(self, stream):
        for n_kv_head, caches in self._caches.items():
            L.moe_paged_copy(self.shape(1, n_kv_head, n_kv_head), self._copies, self.pages_info, caches, stream=stream)

    def fork(self, parent: torch.Tensor | None = None, keep: torch.Tensor | None = None, stream=None) -> "PagedStep":
        """Every row goes on from the first `keep` tokens of row `parent` ([requests] int32, device; None: each row
        itself, all tokens; parent -1: none), in every layer: branches of a search, a prefix that several requests
        have in common, rejected tokens.  Takes place between the layers' last step and the next plan."""
        ctx, state = self._ctx, self._state
        for name, t in (("parent", parent), ("keep", keep)):
            if t is not None:
                _check(name, t, torch.int32, (self.requests,), ctx.device)
        self._between_steps()
        L.moe_paged_fork(self.shape(1), parent, keep, self._kept, self.sinks, ctx, self.block_table, self.block_table,
                         self.pool, state, state, ctx, self._copies, self.pages_info, self._workspace, stream=stream)
        self._copy(stream)
        return self

    def compact(self, stream=None) -> "PagedStep":
        """The pages in use to the front of every layer's cache, between two steps; the pages behind
        them (pages_info[3] tells how many are in use) hold nothing then."""
        self._between_steps()
        L.moe_paged_compact(self.shape(1), self._ctx, self.block_table, self.block_table, self.pool, self._state,
                            self._copies, self.pages_info, self._workspace, stream=stream)
        self._copy(stream)
        return self


class PagedAttention:
    """One layer's attention block over a paged cache (weights as for moe_attention_fwd).

    rope: a rotation (make_rope) of queries and keys by their positions; window: a token sees the last so
    many tokens, itself among them, and the first `sinks` (0: all)."""

    def __init__(self, step: PagedStep, d: int, n_head: int, n_kv_head: int, w_qkv: torch.Tensor, w_o: torch.Tensor,
                 eps: float = 1e-6, rope=None, window: int = 0, sinks: int = 0):
        if not (0 <= window < 1 << 31 and 0 <= sinks < 1 << 31):
            raise ValueError(f"a window of {window} tokens and {sinks} first ones")
        if step.window and not (0 < window <= step.window and sinks <= step.sinks):
            raise ValueError(f"a window of {window} tokens and {sinks} first ones in a step that keeps the last "
                             f"{step.window} and the first {step.sinks}")
        self.step, self.d, self.n_head, self.n_kv_head, self.eps = step, d, n_head, n_kv_head, eps
        self.rope, self.window, self.sinks = rope, window, sinks
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
        if step.sharing:
            step.add_caches(n_kv_head, self.k_cache, self.v_cache)

    def forward(self, x: torch.Tensor, out: torch.Tensor, residual: bool = True, stream=None) -> torch.Tensor:
        """x, out [tokens][d] bf16: the rows of the step that was planned last, all of them."""
        st = self.step
        rows = (st.tokens, self.d)
        _check("x", x, torch.bfloat16, rows, self.w_qkv.device)
        _check("out", out, torch.bfloat16, rows, self.w_qkv.device)
        _check_cuda(self.w_qkv.device)
        shape = st.shape(x.shape[0], self.n_head, self.n_kv_head, self.eps)
        rest = (x, self.w_qkv, self.w_o, residual, self.k_cache, self.v_cache, st.block_table, st.row_start,
                st.slot_map, st.kv_len, out, self.workspace)
        if self.rope is None and self.window == 0:
            L.moe_attention_paged_fwd(shape, self.d, *rest, stream=stream)
        else:
            L.moe_attention_paged_window_fwd(shape, self.d, self.rope, self.window, self.sinks, *rest, stream=stream)
        return out
