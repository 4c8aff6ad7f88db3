"""The mixture-of-experts operators' host side, without a GPU: the argument checks' codes, the choice
of the experts' kernel, and the binding's own checks."""

import pytest
import torch

from allgather_gemm_persistent_amd import binding as B

FAKE = 1 << 20          # an aligned non-NULL address (never dereferenced by the checks)


@pytest.fixture(scope="module")
def lib():
    return B.load()


def _norm(lib, **kw):
    d = dict(rows=16, cols=64, xd=B.AGG_BF16, x=FAKE, lx=64, r=FAKE, lr=64, ro=FAKE, lro=64, w=FAKE, eps=1e-6,
             od=B.AGG_BF16, out=FAKE, lo=64, scales=None, scale=1.0)
    d.update(kw)
    return lib.agg_check_norm_args(*d.values())


@pytest.mark.parametrize("kw", [
    dict(), dict(rows=0, x=None, out=None), dict(cols=0, lx=0), dict(r=None, ro=None), dict(ro=None),
    dict(xd=B.AGG_FP32), dict(od=B.AGG_FP8_E4M3), dict(od=B.AGG_FP8_E4M3, scales=FAKE, scale=0.0), dict(eps=0.0),
    dict(lx=72, lr=80, lro=88, lo=96), dict(od=B.AGG_FP8_E4M3, lo=72), dict(cols=32768, lx=32768, lr=32768, lro=32768, lo=32768)])
def test_norm_args_ok(lib, kw):
    assert _norm(lib, **kw) == B.AGG_OK


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), B.AGG_E_ARG), (dict(cols=-8), B.AGG_E_ARG), (dict(cols=60), B.AGG_E_ARG),
    (dict(xd=B.AGG_FP8_E4M3), B.AGG_E_ARG), (dict(od=B.AGG_FP32), B.AGG_E_ARG), (dict(eps=-1.0), B.AGG_E_ARG),
    (dict(eps=float("nan")), B.AGG_E_ARG), (dict(od=B.AGG_FP8_E4M3, scale=0.0), B.AGG_E_ARG),
    (dict(od=B.AGG_FP8_E4M3, scale=float("inf")), B.AGG_E_ARG), (dict(r=None), B.AGG_E_ARG), (dict(x=None), B.AGG_E_ARG),
    (dict(out=None), B.AGG_E_ARG), (dict(x=FAKE + 2), B.AGG_E_ARG), (dict(w=FAKE + 8), B.AGG_E_ARG),
    (dict(r=FAKE + 4), B.AGG_E_ARG), (dict(ro=FAKE + 4), B.AGG_E_ARG), (dict(lx=63), B.AGG_E_ARG),
    (dict(lx=68), B.AGG_E_ARG), (dict(lr=56), B.AGG_E_ARG), (dict(lro=65), B.AGG_E_ARG), (dict(lo=60), B.AGG_E_ARG),
    (dict(cols=32776, lx=32776), B.AGG_E_UNSUPPORTED), (dict(rows=(1 << 30) + 1), B.AGG_E_UNSUPPORTED),
    (dict(lx=1 << 32), B.AGG_E_UNSUPPORTED), (dict(lr=1 << 62), B.AGG_E_UNSUPPORTED),
    (dict(lro=1 << 62), B.AGG_E_UNSUPPORTED), (dict(lo=1 << 62), B.AGG_E_UNSUPPORTED)])
def test_norm_args_rejected(lib, kw, code):
    assert _norm(lib, **kw) == code
    assert B.last_error()


def _route(lib, **kw):
    d = dict(tokens=4, experts=64, k=2, ld=B.AGG_FP32, logits=FAKE, stride=64, score=0, groups=1, top_groups=1,
             scale=1.0, ids=FAKE, weights=FAKE)
    d.update(kw)
    return lib.agg_check_route_args(*d.values())


def test_route_args_ok(lib):
    for kw in (dict(), dict(tokens=0, logits=None), dict(experts=1, k=1), dict(experts=1024, k=16, stride=1024),
               dict(groups=64, top_groups=2), dict(groups=8, top_groups=2, k=16), dict(score=1, ld=B.AGG_BF16), dict(scale=-2.5)):
        assert _route(lib, **kw) == B.AGG_OK, kw


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), B.AGG_E_ARG), (dict(experts=0), B.AGG_E_ARG), (dict(experts=1025, stride=1025), B.AGG_E_ARG),
    (dict(k=0), B.AGG_E_ARG), (dict(k=17), B.AGG_E_ARG), (dict(experts=4, k=5), B.AGG_E_ARG),
    (dict(groups=8, top_groups=1, k=9), B.AGG_E_ARG), (dict(groups=0), B.AGG_E_ARG), (dict(groups=3), B.AGG_E_ARG),
    (dict(experts=1024, stride=1024, groups=128), B.AGG_E_ARG), (dict(groups=4, top_groups=5), B.AGG_E_ARG),
    (dict(top_groups=0), B.AGG_E_ARG), (dict(score=2), B.AGG_E_ARG), (dict(ld=B.AGG_FP8_E4M3), B.AGG_E_ARG),
    (dict(scale=float("nan")), B.AGG_E_ARG), (dict(stride=63), B.AGG_E_ARG), (dict(logits=None), B.AGG_E_ARG),
    (dict(ids=None), B.AGG_E_ARG), (dict(weights=None), B.AGG_E_ARG), (dict(tokens=(1 << 30) + 1), B.AGG_E_UNSUPPORTED),
    (dict(stride=1 << 62), B.AGG_E_UNSUPPORTED)])
def test_route_args_rejected(lib, kw, code):
    assert _route(lib, **kw) == code
    assert B.last_error()


def _plan(lib, **kw):
    d = dict(tokens=10, k=2, ids=FAKE, first=0, n=8, offsets=FAKE, st=FAKE, ts=FAKE, work=FAKE)
    d.update(kw)
    return lib.agg_check_plan_args(*d.values())


def test_plan_args(lib):
    for kw in (dict(), dict(tokens=0, ids=None, st=None, ts=None, work=None), dict(first=100), dict(n=1024, k=16)):
        assert _plan(lib, **kw) == B.AGG_OK, kw
    for kw in (dict(tokens=-1), dict(k=0), dict(k=17), dict(first=-1), dict(n=0), dict(n=1025), dict(offsets=None),
               dict(ids=None), dict(st=None), dict(ts=None), dict(work=None)):
        assert _plan(lib, **kw) == B.AGG_E_ARG, kw
    assert _plan(lib, tokens=1 << 30) == B.AGG_E_UNSUPPORTED
    assert _plan(lib, tokens=1 << 62, k=16) == B.AGG_E_UNSUPPORTED   # (the product of the two wraps to 0)


def _gemm(lib, **kw):
    d = dict(slots=32, e=8, n=64, k=128, dt=B.AGG_BF16, gated=0, rows=32, a=FAKE, la=128, sa=None, st=FAKE, b=FAKE,
             sb=None, off=FAKE, out=FAKE)
    d.update(kw)
    return lib.agg_check_moe_gemm_args(*d.values())


def test_gemm_args_ok(lib):
    for kw in (dict(), dict(slots=0, a=None, b=None), dict(n=0), dict(gated=1), dict(st=None), dict(rows=1),
               dict(la=136), dict(dt=B.AGG_FP8_E4M3, sa=FAKE, sb=FAKE), dict(e=1024),
               dict(st=None, rows=1 << 20, slots=1 << 20, k=8192, la=8192)):
        assert _gemm(lib, **kw) == B.AGG_OK, kw


@pytest.mark.parametrize("kw,code", [
    (dict(slots=-1), B.AGG_E_ARG), (dict(n=-8), B.AGG_E_ARG), (dict(k=-8), B.AGG_E_ARG), (dict(rows=-1), B.AGG_E_ARG),
    (dict(e=0), B.AGG_E_ARG), (dict(e=1025), B.AGG_E_ARG), (dict(dt=B.AGG_FP32), B.AGG_E_ARG), (dict(k=124), B.AGG_E_ARG),
    (dict(n=60), B.AGG_E_ARG), (dict(k=0, la=0), B.AGG_E_ARG),
    (dict(dt=B.AGG_FP8_E4M3, sa=FAKE, sb=FAKE, k=136, la=144), B.AGG_E_ARG),
    (dict(dt=B.AGG_FP8_E4M3, sa=FAKE, sb=FAKE, n=72), B.AGG_E_ARG), (dict(dt=B.AGG_FP8_E4M3, sb=FAKE), B.AGG_E_ARG),
    (dict(dt=B.AGG_FP8_E4M3, sa=FAKE), B.AGG_E_ARG), (dict(la=120), B.AGG_E_ARG), (dict(la=130), B.AGG_E_ARG),
    (dict(rows=0), B.AGG_E_ARG), (dict(st=None, rows=31), B.AGG_E_ARG), (dict(a=None), B.AGG_E_ARG),
    (dict(b=None), B.AGG_E_ARG), (dict(off=None), B.AGG_E_ARG), (dict(out=None), B.AGG_E_ARG),
    (dict(a=FAKE + 8), B.AGG_E_ARG), (dict(b=FAKE + 2), B.AGG_E_ARG), (dict(out=FAKE + 2), B.AGG_E_ARG),
    (dict(rows=1 << 20, k=8192, la=8192), B.AGG_E_UNSUPPORTED), (dict(rows=16, la=1 << 60), B.AGG_E_UNSUPPORTED),
    (dict(n=1 << 16, k=1 << 14, la=1 << 14), B.AGG_E_UNSUPPORTED),
    (dict(n=1 << 15, k=1 << 14, la=1 << 14, gated=1), B.AGG_E_UNSUPPORTED)])
def test_gemm_args_rejected(lib, kw, code):
    assert _gemm(lib, **kw) == code
    assert B.last_error()


def test_combine_args(lib):
    def call(**kw):
        d = dict(tokens=4, k=2, n=64, slots=8, y=FAKE, ts=FAKE, w=FAKE, od=B.AGG_BF16, out=FAKE)
        d.update(kw)
        return lib.agg_check_combine_args(*d.values())
    for kw in (dict(), dict(tokens=0, ts=None), dict(slots=0, y=None), dict(od=B.AGG_FP32), dict(k=16)):
        assert call(**kw) == B.AGG_OK, kw
    for kw in (dict(tokens=-1), dict(n=-8), dict(slots=-1), dict(k=0), dict(k=17), dict(n=60), dict(od=B.AGG_FP8_E4M3),
               dict(y=None), dict(y=FAKE + 4), dict(ts=None), dict(w=None), dict(out=None), dict(out=FAKE + 8)):
        assert call(**kw) == B.AGG_E_ARG, kw
    assert call(tokens=(1 << 30) + 1) == B.AGG_E_UNSUPPORTED


def test_a_call_without_a_ctx_or_weight_is_refused(lib):
    assert lib.moe_plan(None, 10, 2, FAKE, 0, 8, FAKE, FAKE, FAKE, FAKE, None) == B.AGG_E_ARG
    assert "ctx" in B.last_error()
    assert lib.rms_norm(None, 1, 8, B.AGG_BF16, FAKE, 8, None, 0, None, 0, None, 1e-6, B.AGG_BF16, FAKE, 8, None, 1.0,
                        None) == B.AGG_E_ARG
    assert "weight" in B.last_error()


def test_kernel_choice(lib):
    """Few rows an expert over a long K stream the weights, K split while the strips of the busy
    experts leave compute units idle; many rows take tiles as high as the rows call for."""
    kind, parts = B.agg_moe_gemm_shape("bf16", 1, 8, 3584, 8192)
    assert kind == "stream" and 28 * parts <= 256 < 28 * (parts + 1)
    assert B.agg_moe_gemm_shape("bf16", 32, 8, 3584, 8192, gated=True) == ("stream", 1)
    assert B.agg_moe_gemm_shape("fp8", 32, 8, 3584, 8192, gated=True) == ("stream", 2)
    assert B.agg_moe_gemm_shape("bf16", 8 * 11, 8, 3584, 8192)[0] == "stream"
    assert B.agg_moe_gemm_shape("bf16", 8 * 16, 8, 3584, 8192)[0] == "tiles"
    # a second wave of strips with few blocks of K each
    assert B.agg_moe_gemm_shape("bf16", 30 * 16, 30, 1032, 1000) == ("tiles", (64, 64))
    # partial sums that would not fit the workspace, more strips than counters: fewer parts
    assert B.agg_moe_gemm_shape("bf16", 16, 1, 8192, 1 << 15) == ("stream", 4)
    assert B.agg_moe_gemm_shape("bf16", 1, 1024, 1024, 8192) == ("stream", 1)
    for dtype, slots in (("bf16", 10240), ("fp8", 16384)):
        kind, shape = B.agg_moe_gemm_shape(dtype, slots, 8, 3584, 8192, gated=True)
        assert kind == "tiles" and shape[0] == 256
    # sizes without work still name a kernel
    assert B.agg_moe_gemm_shape("fp8", 0, 1, 16, 16)[0] in ("tiles", "stream")
    with pytest.raises(B.AggError):
        B._call("agg_moe_gemm_shape", 0, 1, 1, 8, 8, 0, None, None, None)


def test_binding_refuses_what_the_call_would_read_wrongly(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(B.AggError, match="device tensor"):
        B.rms_norm(None, 4, 64, x, w, x)
    with pytest.raises(B.AggError, match="shape"):
        B.rms_norm(None, 5, 64, x, w, x)
    with pytest.raises(B.AggError, match="contiguous columns"):
        B.rms_norm(None, 64, 4, x.t(), w, x)
    with pytest.raises(B.AggError, match="float16"):
        B.quant_rows(None, 0, 64, x[:0].half(), x[:0].to(torch.float8_e4m3fn))
    with pytest.raises(B.AggError, match="int32"):
        B.moe_plan(None, 4, 2, torch.zeros(8, dtype=torch.int64), 0, 8, None, None, None, None)
    with pytest.raises(B.AggError, match="contiguous and hold"):
        B.moe_plan(None, 4, 2, torch.zeros(7, dtype=torch.int32), 0, 8, None, None, None, None)
    assert B.moe_plan_words(512, 2, 7) == 16


@pytest.mark.parametrize("kw,code", [
    (dict(n=-64), B.AGG_E_ARG),
    (dict(k=-64), B.AGG_E_ARG), (dict(slots=-4), B.AGG_E_ARG), (dict(n_experts=0), B.AGG_E_ARG),
    (dict(n_experts=-2), B.AGG_E_ARG), (dict(n_experts=1025), B.AGG_E_ARG), (dict(dtype=5), B.AGG_E_ARG),
    (dict(n=60), B.AGG_E_ARG), (dict(k=60), B.AGG_E_ARG), (dict(slots=1 << 62), B.AGG_E_UNSUPPORTED),
    (dict(n=1 << 62, k=1 << 62), B.AGG_E_UNSUPPORTED), (dict(n=1 << 20, k=1 << 20), B.AGG_E_UNSUPPORTED)])
def test_moe_gemm_shape_refuses_what_the_product_does(kw, code):
    """Sizes of no product are an error, and sizes without work are not, rather than the end of the
    process (no columns, and sizes whose products wrap, were a division by zero)."""
    args = dict(dtype="bf16", slots=4, n_experts=2, n=64, k=64)
    for empty in (dict(), dict(n=0), dict(slots=0), dict(k=0), dict(n=0, slots=0, k=0)):
        assert B.agg_moe_gemm_shape(**{**args, **empty})[0] in ("stream", "tiles")
    with pytest.raises(B.AggError) as e:
        B.agg_moe_gemm_shape(**{**args, **kw})
    assert e.value.code == code


# ------------------------------------------------------------------------------ the layer

class _Weight:
    """A tensor that lies wherever it was sent."""

    def __init__(self, *shape, places):
        self.shape, self.dtype, self.places = shape, torch.bfloat16, places

    def to(self, device):
        self.places.append(torch.device(device))
        return self

    def contiguous(self):
        return self


@pytest.mark.parametrize("device,current,want", [("cuda", 3, 3), ("cuda", 0, 0), ("cuda:2", 3, 2),
                                                 (torch.device("cuda", 1), 0, 1)])
def test_layer_and_its_ctx_on_one_device(monkeypatch, device, current, want):
    """Without an index a layer lies on torch's current device, its ctx and every buffer with it."""
    from allgather_gemm_persistent_amd import moe_layer
    places, ctxs = [], []
    new = lambda *shape, dtype, device: places.append(torch.device(device))  # noqa: E731
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    monkeypatch.setattr(torch, "empty", new)
    monkeypatch.setattr(torch, "zeros", new)
    monkeypatch.setattr(B, "agg_ctx_create", lambda index=0: ctxs.append(index))
    w = lambda *shape: _Weight(*shape, places=places)  # noqa: E731
    moe_layer.MoeLayer(4, 2, w(64), w(64, 8), w(8, 64, 64), w(8, 32, 64), bias=w(8), device=device)
    assert ctxs == [want] and len(places) > 10 and set(places) == {torch.device("cuda", want)}
