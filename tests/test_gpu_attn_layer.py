"""An attention layer's decode steps as they are run: norm, projection, write, attention and output projection, each step
from the rows that entered it, and the routed layer after it.

Tolerances: a bfloat16 row is within 2^-8 of its value; e4m3 rows within 2^-4 of theirs, which a product of n of them
averages to about 2^-4 of the sums' root mean square at most."""

import math

import pytest
import torch

from allgather_gemm_persistent_amd import binding as B
from allgather_gemm_persistent_amd import attn_layer, moe_layer

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8


def _near(got, want, rel, what):
    got, want = got.double().cpu(), want.double().cpu()
    assert bool(got.isfinite().all()), what
    off = float((got - want).norm() / want.norm())
    assert off <= rel, f"{what}: {off:.3g} of the norm, not {rel:.3g}"


def _rotated(x, angles):
    r = angles.shape[1] // 2
    c, s = angles[:, None, :r].double(), angles[:, None, r:].double()
    a, b = x[..., :r], x[..., r:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


class _Reference:
    """The layer's steps in 64 bits over the tokens seen so far, from the layer's own rows at each step's entry."""

    def __init__(self, layer, sequences):
        self.l = layer
        self.k, self.v = [[] for _ in range(sequences)], [[] for _ in range(sequences)]

    def step(self, x, residual, seq, positions, lens):
        layer, t = self.l, x.shape[0]
        w_qkv, w_out = layer.w_qkv.double().cpu(), layer.w_out.double().cpu()
        if layer.dtype == "fp8":
            w_qkv, w_out = w_qkv * layer.qkv_scale.double().cpu(), w_out * layer.out_scale.double().cpu()
        s = x.double().cpu() + (0 if residual is None else residual.double().cpu())
        rows = s * torch.rsqrt((s * s).mean(1, keepdim=True) + layer.eps) * layer.norm.double().cpu()
        qkv = rows @ w_qkv + layer.bias.double().cpu()
        d, qc, kc = layer.head_dim, layer.q_cols, layer.kv_cols
        q = _rotated(qkv[:, :qc].reshape(t, -1, d), layer.rope.cpu()[positions])
        k = _rotated(qkv[:, qc:qc + kc].reshape(t, -1, d), layer.rope.cpu()[positions])
        v = qkv[:, qc + kc:].reshape(t, -1, d)
        for i, n in enumerate(seq):
            assert len(self.k[n]) == positions[i]
            self.k[n].append(k[i])
            self.v[n].append(v[i])
        y = torch.zeros(t, layer.q_heads, d, dtype=torch.float64)
        for i, n in enumerate(seq):
            kk, vv = (torch.stack(z[n][:lens[i]]).transpose(0, 1) for z in (self.k, self.v))
            group = layer.q_heads // layer.kv_heads
            x2 = layer.scale * (q[i].reshape(-1, group, d) @ kk.transpose(1, 2).contiguous())
            y[i] = (torch.softmax(x2, -1) @ vv).reshape(-1, d)
        return y.reshape(t, -1) @ w_out


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "fp8"), ("fp8", "fp8")])
@pytest.mark.parametrize("sequences", [1, 5])
def test_decode_steps(gpu, dtype, cache, sequences):
    """A prompt of several tokens a sequence (each attends to those before it and itself), then single new tokens."""
    hidden, q_heads, kv_heads, d, page, context = 256, 8, 2, 64, 16, 48
    each = context // page
    layer = attn_layer.random_layer(4 * sequences, hidden, q_heads, kv_heads, d, sequences * each, dtype, positions=context,
                                    page_size=page, cache=cache, seed=sequences)
    ref = _Reference(layer, sequences)
    g = torch.Generator().manual_seed(7)
    table = torch.randperm(sequences * each, generator=g).int().reshape(sequences, each).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    # bf16: each of the few roundings between the steps is at most 2^-8 of a value; 8 bits: the weights are the
    # reference's too, the rows and the cache are rounded to 2^-4 of a value at most, 2^-5.4 in the mean, at four places
    rel = 4 * HALF_BF16 if dtype == "bf16" and cache == "bf16" else 0.08
    try:
        at = 0
        for step, count in enumerate([4, 3, 1, 1, 1]):
            seq = [s for s in range(sequences) for _ in range(count)]
            pos = [at + j for _ in range(sequences) for j in range(count)]
            lens = [p + 1 for p in pos]
            x = torch.randn(len(seq), hidden, generator=g)
            x = x if step % 2 else x.bfloat16()
            r = torch.randn(len(seq), hidden, generator=g).bfloat16() if step % 2 else None
            rr = None if r is None else r.cuda()
            got = layer.run(x.cuda(), torch.tensor(pos, **i32), torch.tensor(lens, **i32), table,
                            seq=torch.tensor(seq, **i32), residual=rr)
            _near(got, ref.step(x, r, seq, pos, lens), rel, f"step {step}")
            if r is not None:
                assert torch.equal(rr.cpu(), (x.float() + r.float()).bfloat16())
            at += count
        # the cache holds what was written
        back = [torch.empty(at, kv_heads * d, device="cuda") for _ in range(2)]
        B.kv_read(layer.ctx, layer.cache, at, torch.arange(at, **i32), table, *back, token_seq=torch.zeros(at, **i32),
                  stream=torch.cuda.current_stream())
        for b, z in zip(back, (ref.k, ref.v)):
            _near(b.reshape(at, kv_heads, d), torch.stack(z[0]), 4 * HALF_BF16 if rel < 0.05 else 0.06, "cache")
        assert layer.run(x.cuda()[:0], torch.zeros(0, **i32), torch.zeros(0, **i32), table).shape == (0, hidden)
        with pytest.raises(B.AggError):
            layer.run(torch.zeros(4 * sequences + 1, hidden, device="cuda"), torch.zeros(4 * sequences + 1, **i32),
                      torch.zeros(4 * sequences + 1, **i32), table, seq=torch.zeros(4 * sequences + 1, **i32))
    finally:
        layer.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_a_decoder_layer_in_a_replayed_graph(gpu, dtype):
    """Attention and routed experts of a layer, captured once and replayed as the sequences grow, each replay against the
    eager step on a layer of its own."""
    hidden, n, page, context = 256, 3, 16, 400
    each = context // page
    make = lambda: attn_layer.random_layer(n, hidden, 8, 2, 64, n * each, dtype, positions=context, page_size=page,  # noqa: E731
                                           cache=dtype, seed=1)
    attn, twin = make(), make()
    moe, moe_twin = (moe_layer.random_layer(n, hidden, 128, 8, 2, dtype, seed=2) for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.arange(n * each, **i32).reshape(n, each)
    x, r = torch.zeros(n, hidden, device="cuda"), torch.zeros(n, hidden, dtype=torch.bfloat16, device="cuda")
    pos, lens = torch.zeros(n, **i32), torch.zeros(n, **i32)
    rr = [torch.zeros_like(r) for _ in range(2)]

    def step(a, m, res):
        res.copy_(r)
        return m.run(a.run(x, pos, lens, table, residual=res), residual=res)

    try:
        for z in (attn, twin):
            for c in (z.cache.k, z.cache.v):
                c.view(torch.uint8).zero_()
            for c in (z.cache.k_scale, z.cache.v_scale):
                if c is not None:
                    c.fill_(1.0)
        step(twin, moe_twin, rr[1])                        # (writes position 0 of every sequence: of both caches)
        step(attn, moe, rr[0])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(attn, moe, rr[0])
        g = torch.Generator().manual_seed(3)
        for i in range(6):
            x.copy_(torch.randn(n, hidden, generator=g))
            r.copy_(torch.randn(n, hidden, generator=g).bfloat16())
            p = torch.tensor([i, 100 + 40 * i, 399 - i], dtype=torch.int32)
            pos.copy_(p)
            lens.copy_(p + 1)
            want = step(twin, moe_twin, rr[1]).clone()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(rr[0], rr[1]), i
            assert bool(want.isfinite().all()) and float(want.abs().max()) > 0
    finally:
        for z in (attn, twin, moe, moe_twin):
            z.close()


def test_layers_on_streams_at_once(gpu):
    """Two layers' steps on streams of their own give what they give one after another."""
    layers = [attn_layer.random_layer(4, 256, 8, 2, 64, 4 * 20, positions=320, seed=i, page_size=16) for i in range(2)]
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.arange(80, **i32).reshape(4, 20)
    lens = torch.tensor([1, 320, 17, 200], **i32)
    x = torch.randn(4, 256, device="cuda")
    try:
        for z in layers:
            for c in (z.cache.k, z.cache.v):
                c.normal_()
        want = [z.run(x, lens - 1, lens, table).clone() for z in layers]
        streams = [torch.cuda.Stream() for _ in layers]
        pos = lens - 1
        torch.cuda.synchronize()
        for _ in range(10):
            got = [z.run(x, pos, lens, table, stream=s) for z, s in zip(layers, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert math.isfinite(float(want[0].sum()))
    finally:
        for z in layers:
            z.close()


def test_layers_that_share_a_ctx(gpu):
    """Layers of several sizes on one ctx, eager, in two graphs replayed in turn, and after one of them is closed: what
    they give on their own."""
    ctx = B.agg_ctx_create(0)
    sizes = [(8, 2, 64), (12, 1, 128), (4, 4, 64)]
    i32 = dict(dtype=torch.int32, device="cuda")
    make = lambda i, **kw: attn_layer.random_layer(4, 256, *sizes[i], 4 * 60, positions=960, seed=i, page_size=16, **kw)  # noqa: E731
    shared, own = [make(i, ctx=ctx) for i in range(3)], [make(i) for i in range(3)]
    table = torch.arange(240, **i32).reshape(4, 60)
    x = torch.randn(4, 256, device="cuda")
    lens, pos = torch.zeros(4, **i32), torch.zeros(4, **i32)

    def set_lens(*n):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        pos.copy_(lens - 1)

    try:
        for a, b in zip(shared, own):
            for c in ("k", "v"):
                getattr(a.cache, c).normal_()
                getattr(b.cache, c).copy_(getattr(a.cache, c))
        set_lens(1, 960, 17, 300)
        run = lambda layers: [z.run(x, pos, lens, table).clone() for z in layers]  # noqa: E731
        for a, b in zip(run(shared), run(own)):
            assert torch.equal(a, b)
        graphs, outs = [], []
        for part in (shared, shared[1:]):
            torch.cuda.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                outs.append([z.run(x, pos, lens, table) for z in part])
        for i, n in enumerate([(5, 700, 18, 301), (6, 701, 19, 960), (7, 2, 20, 303), (960, 960, 959, 958)]):
            set_lens(*n)
            x.normal_()
            want = run(own)
            torch.cuda.synchronize()
            graphs[i % 2].replay()
            torch.cuda.synchronize()
            for a, b in zip(outs[i % 2], want[i % 2:]):
                assert torch.equal(a, b), i
            if i % 2:                                     # (the first layer's cache did not get the row: it runs alone)
                assert torch.equal(shared[0].run(x, pos, lens, table), want[0])
        shared[0].close()
        assert shared[0].ctx is None
        assert torch.equal(shared[1].run(x, pos, lens, table), own[1].run(x, pos, lens, table))
    finally:
        for z in shared + own:
            z.close()
        B.agg_ctx_destroy(ctx)
