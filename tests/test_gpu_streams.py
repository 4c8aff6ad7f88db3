"""Calls of one ctx on several streams: a call starts after the last one, whichever stream that was on,
and calls that are only captured in between change nothing about it; the experts' products with a split K
do not meet and give the same bits everywhere."""

import ctypes

import pytest
import torch

from allgather_gemm_persistent_amd import binding as B

pytestmark = pytest.mark.gpu

M, N, K = 256, 512, 1024


def _gemm(ctx, a, b, c, stream):
    B.ag_gemm(ctx, 1, 0, M, N, K, M, "bf16", 1.0, 1.0, None, a, None, b, c, mode="gemm_only", stream=stream)


@pytest.mark.parametrize("captured", [False, True])
def test_a_call_on_another_stream_starts_after_the_last_one(gpu, captured):
    """A call on one stream, held back by other work there; then, captured or not, a call on a second
    one; then a call on a third, which must not end before the first."""
    g = torch.Generator().manual_seed(1)
    a = [torch.randn(M, K, generator=g).bfloat16().cuda() for _ in range(3)]
    b = torch.randn(K, N, generator=g).bfloat16().cuda()
    ctx = B.agg_ctx_create(0)
    try:
        want = [torch.zeros(M, N, dtype=torch.bfloat16, device="cuda") for _ in a]
        for x, c in zip(a, want):
            _gemm(ctx, x, b, c, torch.cuda.current_stream())
        torch.testing.assert_close(want[0].float(), a[0].float() @ b.float(), rtol=2e-2, atol=0.5)
        got = [torch.zeros_like(c) for c in want]
        first, second, third = (torch.cuda.Stream() for _ in range(3))
        big = torch.randn(8192, 8192, device="cuda").bfloat16()
        out = torch.empty_like(big)
        torch.mm(big, big, out=out)
        torch.cuda.synchronize()
        with torch.cuda.stream(first):
            for _ in range(200):
                torch.mm(big, big, out=out)
        _gemm(ctx, a[0], b, got[0], first)
        ends = [torch.cuda.Event(), torch.cuda.Event()]
        ends[0].record(first)
        graph = torch.cuda.CUDAGraph()
        if captured:
            with torch.cuda.stream(second):
                graph.capture_begin()
                _gemm(ctx, a[1], b, got[1], second)
                graph.capture_end()
        assert not ends[0].query()              # the first call has not ended yet
        _gemm(ctx, a[2], b, got[2], third)
        ends[1].record(third)
        ends[1].synchronize()
        assert ends[0].query()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
        # what was captured runs when it is replayed, not before
        assert (got[1] == 0).all()
        if captured:
            for _ in range(3):
                got[1].zero_()
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(got[1], want[1])
                _gemm(ctx, a[0], b, got[0], torch.cuda.current_stream())
                torch.cuda.synchronize()
                assert torch.equal(got[0], want[0])
        assert B.agg_ctx_status(ctx, torch.cuda.current_stream()) == (0, -1)
    finally:
        torch.cuda.synchronize()
        B.agg_ctx_destroy(ctx)


class _Stream:
    """A stream that is destroyed at the end (torch keeps its own for good)."""

    def __enter__(self):
        self.hip = ctypes.CDLL("libamdhip64.so")
        handle = ctypes.c_void_p()
        assert self.hip.hipStreamCreateWithFlags(ctypes.byref(handle), 1) == 0       # non-blocking
        self.handle = handle
        return handle.value

    def __exit__(self, *_):
        assert self.hip.hipStreamDestroy(self.handle) == 0


def test_a_call_after_the_last_ones_stream_is_gone(gpu):
    """The last call's stream may be destroyed before the next call."""
    g = torch.Generator().manual_seed(2)
    a, b = torch.randn(M, K, generator=g).bfloat16().cuda(), torch.randn(K, N, generator=g).bfloat16().cuda()
    ctx = B.agg_ctx_create(0)
    try:
        want, got = (torch.zeros(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        _gemm(ctx, a, b, want, torch.cuda.current_stream())
        for _ in range(3):
            torch.cuda.synchronize()
            with _Stream() as s:
                _gemm(ctx, a, b, got, s)
            _gemm(ctx, a, b, got, torch.cuda.current_stream())
            torch.cuda.synchronize()
            assert torch.equal(got, want)
    finally:
        B.agg_ctx_destroy(ctx)


def test_calls_that_take_turns_between_streams(gpu):
    """Calls on three streams in turn, each on what the one before it wrote, with other work between
    them; then many on one stream and a change again."""
    g = torch.Generator().manual_seed(3)
    w = (torch.randn(K, K, generator=g) / 32).bfloat16().cuda()
    x = [torch.randn(M, K, generator=g).bfloat16().cuda()] + [torch.zeros(M, K, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    first = x[0].clone()
    ctx = B.agg_ctx_create(0)

    def step(i, s):
        B.ag_gemm(ctx, 1, 0, M, K, K, M, "bf16", 1.0, 1.0, None, x[i % 3], None, w, x[(i + 1) % 3], mode="gemm_only", stream=s)

    def run(streams):
        x[0].copy_(first)
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            step(i, s)
        torch.cuda.synchronize()
        return x[len(streams) % 3].clone()

    try:
        here = torch.cuda.current_stream()
        want = run([here] * 90)
        assert torch.isfinite(want.float()).all() and want.float().abs().max() > 0
        some = [torch.cuda.Stream() for _ in range(3)]
        for streams in (some * 30, [some[0]] * 40 + [some[1]] * 25 + [here] * 2 + [some[2]] * 23, some[:2] * 20 + [here] * 50):
            assert torch.equal(run(streams), want)
        assert B.agg_ctx_status(ctx, here) == (0, -1)
    finally:
        B.agg_ctx_destroy(ctx)


def test_calls_beside_a_capture_in_progress(gpu):
    """While a stream is being captured, work of others: many calls on one stream, then one on another,
    which waits for them; the capture goes on."""
    g = torch.Generator().manual_seed(4)
    a = [torch.randn(M, K, generator=g).bfloat16().cuda() for _ in range(2)]
    b = torch.randn(K, N, generator=g).bfloat16().cuda()
    ctx = B.agg_ctx_create(0)
    try:
        want = [torch.zeros(M, N, dtype=torch.bfloat16, device="cuda") for _ in a]
        for x, c in zip(a, want):
            _gemm(ctx, x, b, c, torch.cuda.current_stream())
        got, count = [torch.zeros_like(c) for c in want], torch.zeros(1, device="cuda")
        captured, first, second = (torch.cuda.Stream() for _ in range(3))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(captured):
            graph.capture_begin()
            count.add_(1)
            for _ in range(30):
                _gemm(ctx, a[0], b, got[0], first)
            _gemm(ctx, a[1], b, got[1], second)
            count.add_(1)
            graph.capture_end()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for i in range(3):
            graph.replay()
            torch.cuda.synchronize()
            assert count.item() == 2 * (i + 1)
        assert B.agg_ctx_status(ctx, torch.cuda.current_stream()) == (0, -1)
    finally:
        B.agg_ctx_destroy(ctx)


@pytest.mark.parametrize("producer", ["cu", "kernel", "sdma"])
@pytest.mark.parametrize("timing", [0, 1])
def test_the_order_of_calls_with_every_producer(gpu, producer, timing):
    """Gathers of two ranks on changing streams, with and without timing events: every result is whole."""
    from allgather_gemm_persistent_amd.workload import AgWorkload
    g = torch.Generator().manual_seed(5)
    shards = [torch.randn(128, 256, generator=g).bfloat16() for _ in range(2)]
    b = torch.randn(256, 256, generator=g).bfloat16()
    w = AgWorkload(2, 0, shards, b, 64, producer=producer)
    try:
        B.agg_ctx_set_timing(w.ctx, timing)
        w.run("overlap")
        torch.cuda.synchronize()
        want = w.c.clone()
        ref = torch.cat(shards).double() @ b.double()
        assert ((want.double().cpu() - ref).abs() <= ref.abs() * 2.0 ** -8 + 256 * 2.0 ** -23 * 16 * 256).all()
        streams = [torch.cuda.Stream() for _ in range(3)]
        for i in range(24):
            s = streams[i * i % 3]
            w.run(("overlap", "serial", "gemm_only")[i % 3], stream=s)
            if i % 8 == 7:
                torch.cuda.synchronize()
                assert torch.equal(w.c, want) and w.status() == (0, -1)
                w.c.zero_()
                torch.cuda.synchronize()
    finally:
        w.close()


# ------------------------------------------------------------------------------ a split K

class _Split:
    """A call whose K is split over workgroups."""
    ROWS, E, COLS, DEPTH = 3, 2, 1024, 4096

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        assert B.agg_moe_gemm_shape("bf16", self.ROWS, self.E, self.COLS, self.DEPTH)[1] > 1
        self.a = torch.randn(self.ROWS, self.DEPTH, generator=g).bfloat16().cuda()
        self.b = (torch.randn(self.E, self.DEPTH, self.COLS, generator=g) / 64).bfloat16().cuda()
        self.off = torch.tensor([0, 1 + seed % 2, self.ROWS], dtype=torch.int32, device="cuda")
        self.out = torch.zeros(self.ROWS, self.COLS, dtype=torch.bfloat16, device="cuda")
        self.want = None

    def run(self, ctx, stream):
        B.moe_gemm(ctx, self.ROWS, self.E, self.COLS, self.DEPTH, "bf16", self.a, self.b, self.off, self.out,
                   stream=stream)

    def check(self):
        """The bits of the first run, which is compared with 64 bits."""
        torch.cuda.synchronize()
        if self.want is None:
            a, b, cut = self.a.double().cpu(), self.b.double().cpu(), int(self.off[1])
            ref = torch.cat([a[:cut] @ b[0], a[cut:] @ b[1]])
            size = torch.cat([a[:cut].abs() @ b[0].abs(), a[cut:].abs() @ b[1].abs()])
            # (half a unit of bfloat16, and 4096 fp32 products and sums)
            assert ((self.out.double().cpu() - ref).abs() <= ref.abs() * 2.0 ** -8 + size * self.DEPTH * 2.0 ** -23).all()
            self.want = self.out.clone()
        assert torch.equal(self.out, self.want)
        self.out.zero_()
        torch.cuda.synchronize()


def test_split_k_gives_the_same_bits_on_every_stream(gpu):
    """One call after another, each on a stream that the ctx has not seen, short-lived ones among them."""
    ctx, x = B.agg_ctx_create(0), _Split(1)
    try:
        streams = [torch.cuda.current_stream()] + [torch.cuda.Stream() for _ in range(7)]
        for s in streams + streams[::-1]:
            x.run(ctx, s)
            x.check()
        for _ in range(6):
            with _Stream() as one, _Stream() as two:
                for s in (one, two, one):
                    x.run(ctx, s)
                    x.check()
    finally:
        B.agg_ctx_destroy(ctx)


def test_split_k_on_many_streams_at_once(gpu):
    """Calls on eight streams, none of which waits for another, over and over."""
    ctx, xs = B.agg_ctx_create(0), [_Split(i) for i in range(8)]
    try:
        for x in xs:
            x.run(ctx, torch.cuda.current_stream())
            x.check()
        streams = [torch.cuda.Stream() for _ in xs]
        for _ in range(5):
            for _ in range(20):
                for x, s in zip(xs, streams):
                    x.run(ctx, s)
            for x in xs:
                x.check()
    finally:
        torch.cuda.synchronize()
        B.agg_ctx_destroy(ctx)


def test_split_k_in_graphs_replayed_at_once(gpu):
    """Two graphs from torch's one capture stream, replayed on two streams while eager calls run on a
    third, and after a reset."""
    ctx, xs = B.agg_ctx_create(0), [_Split(i) for i in range(3)]
    try:
        for x in xs:
            x.run(ctx, torch.cuda.current_stream())
            x.check()
        graphs = []
        for x in xs[:2]:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                for _ in range(4):
                    x.run(ctx, torch.cuda.current_stream())
            graphs.append(graph)
        streams = [torch.cuda.Stream() for _ in xs]
        for turn in range(6):
            for _ in range(10):
                for graph, s in zip(graphs, streams):
                    with torch.cuda.stream(s):
                        graph.replay()
                xs[2].run(ctx, streams[2])
            for x in xs:
                x.check()
            if turn == 3:
                B.agg_ctx_reset(ctx, torch.cuda.current_stream())
                torch.cuda.synchronize()
    finally:
        torch.cuda.synchronize()
        B.agg_ctx_destroy(ctx)
