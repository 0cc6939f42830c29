"""Serving through a paged key/value cache: requests come, decode and go, step by step.

Every step plans its tables on the GPU from the requests' lengths, runs the attention block
over the pages (projections, QK-norm, cache write, paged attention, output projection) and
then the top-1 int4 MoE layer on the same rows, with no host round trip in between.  Weights
and token embeddings are random; the model's shapes are the Nano ones (hidden 1024, 8 query
heads on 2 key/value heads, 64 experts of width 512, a shared expert of width 2048).

    python examples/paged_serving.py [--steps 12]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import aux_loss_free_gb300 as M  # noqa: E402
from aux_loss_free_gb300.layer import LayerOnDevice  # noqa: E402
from aux_loss_free_gb300.paged import PagedAttention, PagedStep  # noqa: E402
from synth import ATTN_CONFIGS, CONFIGS, make_attention, make_layer  # noqa: E402


def bf16(bits, dev):
    return torch.from_numpy(bits.view("int16")).to(dev).view(torch.bfloat16)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=12)
    args = ap.parse_args()
    dev = "cuda"
    a, s = ATTN_CONFIGS["attn"].replace(batch=1, seq=1), CONFIGS["decode"].replace(T=64)
    host = make_attention(a, "attn")
    w_qkv = torch.cat([bf16(host[n], dev) for n in ("w_q", "w_k", "w_v")])
    step = PagedStep(requests=4, pages=64, page_size=64, max_pages=16, max_tokens=64, device=dev)
    attention = PagedAttention(step, a.d, a.n_head, a.n_kv_head, w_qkv, bf16(host["w_o"], dev), a.eps)
    moe = LayerOnDevice(s, make_layer(s, "decode", with_tokens=False), dev)

    g = torch.Generator(device=dev).manual_seed(0)
    # New tokens per request and step: prompts in chunks, decoding, one request ends, another starts.
    script = [[48, 0, 0, 0], [30, 20, 0, 0], [1, 40, 10, 0], [1, 1, 1, 40], [1, 1, 1, 1], [1, -1, 1, 1], [1, 33, 1, 1]]
    for i in range(args.steps):
        lens = script[i] if i < len(script) else [1, 1, 1, 1]
        rows = sum(max(n, 0) for n in lens)
        tokens = rows + (-rows) % 8  # a serving loop pads its batch to sizes that it has captured
        x = torch.randn(tokens, a.d, generator=g, device=dev).to(torch.bfloat16)
        h, y = torch.empty_like(x), torch.empty_like(x)
        new_len = torch.tensor(lens, dtype=torch.int32, device=dev)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        step.plan(new_len, tokens)
        attention.forward(x, h)
        shape = M.make_shape(tokens, s.d, s.E, s.f, s.F, 1, renorm=False, w_format=M.MOE_W_INT4_G32)
        M.moe_layer_fwd(shape, h, moe.w_router, moe.logit_offset, moe.bias, moe.gamma, False, moe.weights, h, y,
                        moe.workspace)
        torch.cuda.synchronize()
        us = (time.perf_counter() - t0) * 1e6
        rows_used, taken, returned, denied = step.info.tolist()
        print(f"step {i}: new tokens {lens}, rows {rows_used} of {tokens}, pages taken {taken}, returned {returned}, "
              f"denied {denied}, free {step.free_pages.item()}; contexts {step.ctx_len.tolist()}; "
              f"|y| {y[:rows_used].float().norm().item():.1f}; {us:.0f} us")
    if M.moe_device_status() != 0:
        raise SystemExit("the device status word is set")


if __name__ == "__main__":
    main()
