"""One rank's share of a mixture-of-experts layer, from the residual stream to its partial sum.

    python -m allgather_gemm_persistent_amd.moe_layer [--tokens N] [--dtype bf16|fp8]

rms_norm -> the router's logits (ag_gemm of one rank) -> moe_route -> moe_plan -> moe_gemm (gated) ->
moe_gemm -> moe_combine. With fp8 experts the normalised rows and the rows between the two products
are quantised with a scale per row (quant_rows). A rank that holds a part of the experts gets the sum
over its own; the ranks' sums meet in a ReduceScatter or AllReduce of the caller's.

Roundings between the steps: the normalised rows, the router's logits and the rows after each product are
bf16, what the operators between them read and write (the weights of a choice are fp32, and so are the sums
inside every step and the layer's output). With fp8 experts the normalised rows are quantised from their
bf16 form, which the router takes, since rms_norm has one output.

PyTorch provides device memory and streams only; every step runs in libagg.
"""

from __future__ import annotations

import argparse
import time

import torch

from . import binding as B


class MoeLayer:
    """Weights and buffers of one rank, and the calls in order.

    norm: bf16[hidden]; router: bf16 hidden x experts; w_up: n_local x hidden x 2 inner (gate columns,
    then up columns); w_down: n_local x inner x hidden, both bf16, or float8_e4m3fn with up_scale
    (n_local x 2 inner) and down_scale (n_local x hidden), fp32. Experts [first, first + n_local) are
    this rank's. score, bias, groups, top_groups, renorm and scale are moe_route's. `tokens` is the most
    a call takes.
    """

    def __init__(self, tokens, top_k, norm, router, w_up, w_down, up_scale=None, down_scale=None, first=0,
                 score="softmax", bias=None, groups=1, top_groups=1, scale=1.0, eps=1e-6, device="cuda", renorm=True):
        self.device = B.cuda_device(device)
        to = lambda t: None if t is None else t.to(self.device).contiguous()  # noqa: E731
        self.norm, self.router, self.w_up, self.w_down = to(norm), to(router), to(w_up), to(w_down)
        self.up_scale, self.down_scale, self.bias = to(up_scale), to(down_scale), to(bias)
        self.hidden, self.experts = router.shape
        self.n_local, self.inner = w_down.shape[0], w_down.shape[1]
        self.dtype = "fp8" if w_up.dtype == torch.float8_e4m3fn else "bf16"
        self.tokens, self.top_k, self.first, self.eps = tokens, top_k, first, eps
        self.routing = dict(score=score, groups=groups, top_groups=top_groups, renorm=renorm, scale=scale)
        pairs, h = tokens * top_k, self.hidden
        bf16, fp8, f32, i32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32
        new = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device=self.device)  # noqa: E731
        self.x = new(tokens, h, dtype=bf16)                     # normalised rows
        # (the product wants rows of whole 16 bytes: experts that are no multiple of 8 are padded)
        pad = -self.experts % 8
        self.router_b = torch.nn.functional.pad(self.router, (0, pad)).contiguous() if pad else self.router
        self.logits_c = new(tokens, self.experts + pad, dtype=bf16)
        self.logits = self.logits_c[:, :self.experts] if pad else self.logits_c
        self.ids, self.weights = new(tokens, top_k, dtype=i32), new(tokens, top_k, dtype=f32)
        self.offsets = new(self.n_local + 1, dtype=i32)
        self.slot_token, self.token_slot = new(pairs, dtype=i32), new(tokens, top_k, dtype=i32)
        self.work = new(B.moe_plan_words(tokens, top_k, self.n_local), dtype=i32)
        # (rows of a last slot that no expert holds are never written by the first product, but read, as
        # whole rows, by the quantisation)
        self.mid = torch.zeros(pairs, self.inner, dtype=bf16, device=self.device)
        self.y = new(pairs, h, dtype=bf16)
        self.out = new(tokens, h, dtype=f32)
        if self.dtype == "fp8":
            self.x8, self.x_scale = new(tokens, h, dtype=fp8), new(tokens, dtype=f32)
            self.mid8, self.mid_scale = new(pairs, self.inner, dtype=fp8), new(pairs, dtype=f32)
        self.ctx = B.agg_ctx_create(self.device.index)

    def run(self, x, residual=None, stream=None):
        """x: tokens x hidden, bf16 or fp32 (what gemm_ar or gemm_rs left); residual: bf16 or None, then
        overwritten with x + residual. Returns this rank's partial sum, fp32 (a buffer of the layer)."""
        t, h, k, s = x.shape[0], self.hidden, self.top_k, stream or torch.cuda.current_stream(self.device)
        if t > self.tokens:
            raise B.AggError(B.AGG_E_ARG, "MoeLayer.run", f"{t} tokens, the layer was made for {self.tokens}")
        if t == 0:
            return self.out[:0]
        pairs, fp8 = t * k, self.dtype == "fp8"
        B.rms_norm(self.ctx, t, h, x, self.norm, self.x, residual=residual, residual_out=residual, eps=self.eps,
                   stream=s)
        B.ag_gemm(self.ctx, 1, 0, t, self.router_b.shape[1], h, t, "bf16", 1.0, 1.0, None, self.x, None,
                  self.router_b, self.logits_c, stream=s)
        B.moe_route(self.ctx, t, self.experts, k, self.logits, self.ids, self.weights, bias=self.bias, stream=s,
                    **self.routing)
        B.moe_plan(self.ctx, t, k, self.ids, self.first, self.n_local, self.offsets, self.slot_token,
                   self.token_slot, self.work, stream=s)
        a, a_scale = self.x, None
        if fp8:
            B.quant_rows(self.ctx, t, h, self.x, self.x8, scales=self.x_scale, stream=s)
            a, a_scale = self.x8, self.x_scale
        B.moe_gemm(self.ctx, pairs, self.n_local, self.inner, h, self.dtype, a, self.w_up, self.offsets, self.mid,
                   gated=True, slot_token=self.slot_token, a_scale=a_scale, b_scale=self.up_scale, stream=s)
        a, a_scale = self.mid, None
        if fp8:
            B.quant_rows(self.ctx, pairs, self.inner, self.mid, self.mid8, scales=self.mid_scale, stream=s)
            a, a_scale = self.mid8, self.mid_scale
        B.moe_gemm(self.ctx, pairs, self.n_local, h, self.inner, self.dtype, a, self.w_down, self.offsets, self.y,
                   a_scale=a_scale, b_scale=self.down_scale, stream=s)
        B.moe_combine(self.ctx, t, k, h, pairs, self.y, self.token_slot, self.weights, self.out, stream=s)
        return self.out[:t]

    def close(self):
        if self.ctx is not None:
            B.agg_ctx_destroy(self.ctx)
            self.ctx = None


def random_layer(tokens, hidden, inner, experts, top_k, dtype="bf16", n_local=None, first=0, seed=0, device="cuda",
                 **kw):
    """A layer with seeded random weights of usual sizes (standard deviation 1 / sqrt(rows))."""
    g = torch.Generator(device=device).manual_seed(seed)
    n_local = n_local or experts
    rand = lambda *shape: torch.randn(*shape, generator=g, device=device)  # noqa: E731
    norm = (1 + 0.1 * rand(hidden)).bfloat16()
    router = (rand(hidden, experts) / hidden ** 0.5).bfloat16()
    up, down, scales = [], [], {}
    for _ in range(n_local):
        up.append(rand(hidden, 2 * inner) / hidden ** 0.5)
        down.append(rand(inner, hidden) / inner ** 0.5)
        if dtype == "fp8":
            for name, w in (("up_scale", up), ("down_scale", down)):
                scale = w[-1].abs().amax(0) / 448
                w[-1] = (w[-1] / scale).to(torch.float8_e4m3fn)
                scales.setdefault(name, []).append(scale)
        else:
            up[-1], down[-1] = up[-1].bfloat16(), down[-1].bfloat16()
    scales = {name: torch.stack(s) for name, s in scales.items()}
    return MoeLayer(tokens, top_k, norm, router, torch.stack(up), torch.stack(down), first=first, device=device,
                    **scales, **kw)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--inner", type=int, default=3584)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--top-k", type=int, default=2)
    ap.add_argument("--dtype", choices=("bf16", "fp8"), default="bf16")
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    layer = random_layer(a.tokens, a.hidden, a.inner, a.experts, a.top_k, a.dtype)
    try:
        x = torch.randn(a.tokens, a.hidden, device="cuda")
        for _ in range(3):
            layer.run(x)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for _ in range(a.steps):
            layer.run(x)
        torch.cuda.synchronize()
        us = (time.perf_counter() - t0) / a.steps * 1e6
        flops = 6.0 * a.tokens * a.top_k * a.hidden * a.inner
        print(f"{a.tokens} tokens, {a.experts} experts of {a.hidden} x {a.inner}, top {a.top_k}, {a.dtype}: "
              f"{us:.1f} us a layer, {flops / us / 1e6:.0f} TFLOP/s of experts' products", flush=True)
    finally:
        layer.close()


if __name__ == "__main__":
    main()
