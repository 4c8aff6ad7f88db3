"""One rank's share of an attention layer's decode step, from the residual stream to its partial sum.

    python -m allgather_gemm_persistent_amd.attn_layer [--sequences N] [--context N] [--dtype bf16|fp8] [--cache bf16|fp8]

rms_norm -> the query, key and value projection with its bias (linear) -> kv_write (rotation, and the new rows into the
paged cache) -> paged_attn -> the output projection (linear). With fp8 weights the normalised rows and the attention's rows
are quantised with a scale per row (rms_norm's output, quant_rows). A rank holds whole heads: its part of the query heads and
the cache heads that they read. The ranks' partial sums meet in a ReduceScatter or AllReduce of the caller's.

Roundings between the steps: the normalised rows, the projected rows, the rotated queries and the attention's rows are
bf16 (or e4m3 over a row's scale where an fp8 product takes them); the cache is bf16 or e4m3 over a scale for each token
and head. The sums inside every step and the layer's output are fp32.

PyTorch provides device memory and streams only; every step runs in libagg.
"""

from __future__ import annotations

import argparse
import time

import torch

from . import binding as B


class AttnLayer:
    """Weights, cache and buffers of one rank, and the calls in order.

    norm: bf16[hidden]; w_qkv: hidden x (q_heads + 2 kv_heads) head_dim (queries, keys, values side by side); w_out:
    q_heads head_dim x hidden, both bf16, or float8_e4m3fn with qkv_scale and out_scale (fp32, per column). bias: bf16 per
    column of w_qkv, or None. rope: fp32, positions x rope_dim (cosines, then sines), or None. The cache: `pages` pages of
    page_size tokens, made here ("bf16" or "fp8"). `tokens` is the most a call takes. ctx: the caller's, which outlives the
    layer (layers that share one share its workspaces: one of paged_attn's for a stream or a graph, whatever the number
    of layers), or None: one of the layer's own.
    """

    def __init__(self, tokens, q_heads, kv_heads, head_dim, norm, w_qkv, w_out, pages, page_size=64, cache="bf16",
                 qkv_scale=None, out_scale=None, bias=None, rope=None, rope_pairs=False, window=0, scale=None, eps=1e-6,
                 device="cuda", ctx=None):
        self.device = B.cuda_device(device)
        to = lambda t: None if t is None else t.to(self.device).contiguous()  # noqa: E731
        self.norm, self.w_qkv, self.w_out, self.bias = to(norm), to(w_qkv), to(w_out), to(bias)
        self.qkv_scale, self.out_scale, self.rope = to(qkv_scale), to(out_scale), to(rope)
        self.hidden = w_qkv.shape[0]
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.q_cols, self.kv_cols = q_heads * head_dim, kv_heads * head_dim
        self.dtype = "fp8" if w_qkv.dtype == torch.float8_e4m3fn else "bf16"
        self.tokens, self.rope_pairs, self.window, self.eps = tokens, rope_pairs, window, eps
        self.scale = head_dim ** -0.5 if scale is None else scale
        bf16, fp8, f32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32
        new = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device=self.device)  # noqa: E731
        cols = self.q_cols + 2 * self.kv_cols
        self.x = new(tokens, self.hidden, dtype=bf16)           # normalised rows
        self.qkv = new(tokens, cols, dtype=bf16)
        # (a token without a place in the cache leaves its row of queries as it is: zeros, or an earlier call's)
        self.q = torch.zeros(tokens, self.q_cols, dtype=bf16, device=self.device)
        self.y = new(tokens, self.q_cols, dtype=bf16)
        self.out = new(tokens, self.hidden, dtype=f32)
        if self.dtype == "fp8":
            self.x8, self.x_scale = new(tokens, self.hidden, dtype=fp8), new(tokens, dtype=f32)
            self.y8, self.y_scale = new(tokens, self.q_cols, dtype=fp8), new(tokens, dtype=f32)
        pool = lambda: new(pages, page_size, kv_heads, head_dim, dtype=fp8 if cache == "fp8" else bf16)  # noqa: E731
        scales = lambda: new(pages, kv_heads, page_size, dtype=f32) if cache == "fp8" else None  # noqa: E731
        self.cache = B.KvCache(pool(), pool(), scales(), scales())
        self.owns_ctx = ctx is None
        self.ctx = B.agg_ctx_create(self.device.index) if ctx is None else ctx

    def run(self, x, positions, lens, table, seq=None, residual=None, stream=None):
        """x: tokens x hidden, bf16 or fp32 (what gemm_ar or gemm_rs left); residual: bf16 or None, then overwritten
        with x + residual. Token t belongs to sequence seq[t] (None: t) at positions[t] and attends to the first lens[t]
        tokens of it, its own among them; table: the sequences' pages (int32). Returns this rank's partial sum, fp32 (a
        buffer of the layer)."""
        t, s = x.shape[0], stream or torch.cuda.current_stream(self.device)
        if t > self.tokens:
            raise B.AggError(B.AGG_E_ARG, "AttnLayer.run", f"{t} tokens, the layer was made for {self.tokens}")
        if t == 0:
            return self.out[:0]
        h, qc, kc, fp8 = self.hidden, self.q_cols, self.kv_cols, self.dtype == "fp8"
        a, a_scale = (self.x8, self.x_scale) if fp8 else (self.x, None)
        B.rms_norm(self.ctx, t, h, x, self.norm, a, residual=residual, residual_out=residual, eps=self.eps, scales=a_scale,
                   stream=s)
        B.linear(self.ctx, t, qc + 2 * kc, h, self.dtype, a, self.w_qkv, self.qkv, a_scale=a_scale, b_scale=self.qkv_scale,
                 bias=self.bias, stream=s)
        q, k, v = self.qkv[:, :qc], self.qkv[:, qc:qc + kc], self.qkv[:, qc + kc:]
        B.kv_write(self.ctx, self.cache, t, k, v, positions, table, token_seq=seq, q=q, q_out=self.q, rope=self.rope,
                   rope_pairs=self.rope_pairs, stream=s)
        B.paged_attn(self.ctx, self.cache, t, self.q, lens, table, self.y, scale=self.scale, row_seq=seq,
                     window=self.window, stream=s)
        a, a_scale = self.y, None
        if fp8:
            B.quant_rows(self.ctx, t, qc, self.y, self.y8, scales=self.y_scale, stream=s)
            a, a_scale = self.y8, self.y_scale
        B.linear(self.ctx, t, h, qc, self.dtype, a, self.w_out, self.out, a_scale=a_scale, b_scale=self.out_scale, stream=s)
        return self.out[:t]

    def close(self):
        if self.ctx is not None and self.owns_ctx:
            B.agg_ctx_destroy(self.ctx)
        self.ctx = None


def rotations(positions, dim, base=10000.0):
    """Cosines and then sines of every position's dim / 2 angles, position * base^(-2i / dim), fp32 from 64 bits."""
    rate = base ** (-torch.arange(dim // 2, dtype=torch.float64) / (dim // 2))
    turn = torch.arange(positions, dtype=torch.float64)[:, None] * rate
    return torch.cat([turn.cos(), turn.sin()], 1).float()


def random_layer(tokens, hidden, q_heads, kv_heads, head_dim, pages, dtype="bf16", seed=0, device="cuda", positions=None,
                 **kw):
    """A layer with seeded random weights of usual sizes (standard deviation 1 / sqrt(rows)), a bias, and the rotations
    of `positions` positions (None: no rotation)."""
    g = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=g, device=device)  # noqa: E731
    cols = (q_heads + 2 * kv_heads) * head_dim
    norm, bias = (1 + 0.1 * rand(hidden)).bfloat16(), (0.1 * rand(cols)).bfloat16()
    weights, scales = [], []
    for rows, n in ((hidden, cols), (q_heads * head_dim, hidden)):
        w = rand(rows, n) / rows ** 0.5
        scale = w.abs().amax(0) / 448
        weights.append((w / scale).to(torch.float8_e4m3fn) if dtype == "fp8" else w.bfloat16())
        scales.append(scale if dtype == "fp8" else None)
    rope = None if positions is None else rotations(positions, head_dim)
    return AttnLayer(tokens, q_heads, kv_heads, head_dim, norm, *weights, pages, qkv_scale=scales[0], out_scale=scales[1],
                     bias=bias, rope=rope, device=device, **kw)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--sequences", type=int, default=16)
    ap.add_argument("--context", type=int, default=8192)
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--q-heads", type=int, default=64)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--head-dim", type=int, default=128)
    ap.add_argument("--page", type=int, default=64)
    ap.add_argument("--dtype", choices=("bf16", "fp8"), default="bf16")
    ap.add_argument("--cache", choices=("bf16", "fp8"), default="bf16")
    ap.add_argument("--steps", type=int, default=50)
    a = ap.parse_args()
    n, each = a.sequences, -(-a.context // a.page)
    layer = random_layer(n, a.hidden, a.q_heads, a.kv_heads, a.head_dim, n * each, a.dtype, positions=a.context,
                         page_size=a.page, cache=a.cache)
    try:
        for x in (layer.cache.k, layer.cache.v):
            x.view(torch.uint8).zero_()
        for x in (layer.cache.k_scale, layer.cache.v_scale):
            if x is not None:
                x.fill_(1.0)
        i32 = dict(dtype=torch.int32, device="cuda")
        table = torch.randperm(n * each, device="cuda").int().reshape(n, each)
        lens = torch.full((n,), a.context, **i32)
        x = torch.randn(n, a.hidden, device="cuda")
        for _ in range(3):
            layer.run(x, lens - 1, lens, table)
        positions = lens - 1
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for _ in range(a.steps):
            layer.run(x, positions, lens, table)
        torch.cuda.synchronize()
        us = (time.perf_counter() - t0) / a.steps * 1e6
        el = 1 if a.cache == "fp8" else 2
        held = n * a.context * a.kv_heads * 2 * (a.head_dim * el + (4 if el == 1 else 0))
        weights = layer.w_qkv.numel() * layer.w_qkv.element_size() + layer.w_out.numel() * layer.w_out.element_size()
        print(f"{n} sequences of {a.context} tokens, {a.q_heads} heads on {a.kv_heads} of {a.head_dim}, hidden {a.hidden}, "
              f"{a.dtype}, {a.cache} cache: {us:.1f} us a step, {(held + weights) / us / 1e6:.2f} TB/s of cache and weights",
              flush=True)
    finally:
        layer.close()


if __name__ == "__main__":
    main()
