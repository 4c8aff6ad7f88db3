"""Calls of one ctx on several streams: a call starts after the last one, whichever stream that was on,
and calls that are only captured in between change nothing about it."""

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
