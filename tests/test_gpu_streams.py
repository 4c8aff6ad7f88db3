"""Calls of one ctx on several streams: a call starts after the last one, whichever stream that was on,
and calls that are only captured in between change nothing about it."""

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
