"""The product with an epilogue, its host side without a GPU: the argument checks' codes, the choice of the kernel, and
the binding's own checks."""

import pytest
import torch

from allgather_gemm_persistent_amd import binding as B

FAKE = 1 << 20          # an aligned non-NULL address (never dereferenced by the checks)


@pytest.fixture(scope="module")
def lib():
    return B.load()


def _linear(lib, **kw):
    d = dict(m=4, n=64, k=128, dtype=B.AGG_BF16, a=FAKE, la=128, a_scale=None, b=FAKE, b_scale=None, bias=FAKE, act=0,
             rd=B.AGG_BF16, r=FAKE, lr=64, od=B.AGG_BF16, out=2 * FAKE, lo=64)
    d.update(kw)
    return lib.agg_check_linear_args(*d.values())


FP8 = dict(dtype=B.AGG_FP8_E4M3, a_scale=FAKE, b_scale=FAKE)


@pytest.mark.parametrize("kw", [
    dict(), FP8, dict(FP8, a_scale=FAKE + 4), dict(m=0, a=None, b=None, out=None), dict(n=0, a=None, b=None, out=None),
    dict(bias=None, r=None), dict(r=None, rd=77), dict(act=4), dict(rd=B.AGG_FP32), dict(od=B.AGG_FP32),
    dict(od=B.AGG_FP32, lo=68), dict(la=136, lr=72, lo=80), dict(out=FAKE), dict(out=FAKE, rd=B.AGG_FP32, od=B.AGG_FP32),
    dict(out=FAKE, lo=72, m=1), dict(m=1 << 30), dict(k=1 << 20, la=1 << 20, n=1016, lr=1016, lo=1016)])
def test_args_ok(lib, kw):
    assert _linear(lib, **kw) == B.AGG_OK, B.last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(m=-1), B.AGG_E_ARG), (dict(n=-8), B.AGG_E_ARG), (dict(k=-8), B.AGG_E_ARG), (dict(k=0), B.AGG_E_ARG),
    (dict(dtype=B.AGG_FP32), B.AGG_E_ARG), (dict(n=60), B.AGG_E_ARG), (dict(FP8, n=72), B.AGG_E_ARG), (dict(k=124), B.AGG_E_ARG),
    (dict(FP8, k=120), B.AGG_E_ARG), (dict(act=5), B.AGG_E_ARG), (dict(act=-1), B.AGG_E_ARG), (dict(rd=B.AGG_FP8_E4M3), B.AGG_E_ARG),
    (dict(od=B.AGG_FP8_E4M3), B.AGG_E_ARG), (dict(od=9), B.AGG_E_ARG), (dict(a=None), B.AGG_E_ARG), (dict(b=None), B.AGG_E_ARG),
    (dict(out=None), B.AGG_E_ARG), (dict(a=FAKE + 8), B.AGG_E_ARG), (dict(b=FAKE + 4), B.AGG_E_ARG), (dict(bias=FAKE + 2), B.AGG_E_ARG),
    (dict(r=FAKE + 8), B.AGG_E_ARG), (dict(out=FAKE + 2), B.AGG_E_ARG), (dict(la=120), B.AGG_E_ARG), (dict(la=132), B.AGG_E_ARG),
    (dict(lr=56), B.AGG_E_ARG), (dict(lr=68), B.AGG_E_ARG), (dict(lo=63), B.AGG_E_ARG), (dict(lo=66), B.AGG_E_ARG),
    (dict(FP8, a_scale=None), B.AGG_E_ARG), (dict(FP8, b_scale=None), B.AGG_E_ARG), (dict(FP8, b_scale=FAKE + 4), B.AGG_E_ARG),
    (dict(out=FAKE, od=B.AGG_FP32), B.AGG_E_ARG), (dict(out=FAKE, lo=72), B.AGG_E_ARG), (dict(m=(1 << 30) + 1), B.AGG_E_UNSUPPORTED),
    (dict(n=1 << 62), B.AGG_E_UNSUPPORTED), (dict(k=1 << 62, la=1 << 62), B.AGG_E_UNSUPPORTED),
    (dict(n=1 << 20, k=1 << 10, la=1 << 10, lr=1 << 20, lo=1 << 20), B.AGG_E_UNSUPPORTED), (dict(la=1 << 23), B.AGG_E_UNSUPPORTED),
    (dict(lo=1 << 33), B.AGG_E_UNSUPPORTED), (dict(lr=1 << 33), B.AGG_E_UNSUPPORTED)])
def test_args_rejected(lib, kw, code):
    assert _linear(lib, **kw) == code
    assert B.last_error()


def test_a_call_without_a_ctx_is_refused(lib):
    assert lib.linear(None, 4, 64, 128, B.AGG_BF16, FAKE, 128, None, FAKE, None, None, 0, 0, None, 0, B.AGG_BF16, FAKE, 64,
                      None) == B.AGG_E_ARG


def test_kernel_choice():
    """Few rows stream the weight, many take tiles; every size names a kernel, and sizes that are refused none."""
    for dtype in ("bf16", "fp8"):
        assert B.agg_linear_shape(dtype, 1, 8192, 8192)[0] == "stream"
        assert B.agg_linear_shape(dtype, 16, 1024, 8192)[1] > 1
        assert B.agg_linear_shape(dtype, 8192, 8192, 8192) == ((256, 256), 1)
        for m in (0, 1, 33, 500, 1 << 30):
            for n in (0, 16, 1008, 10240):
                for k in (16, 1008, 8192):
                    how, parts = B.agg_linear_shape(dtype, m, n, k)
                    assert 1 <= parts <= 16 and how in ["stream", (256, 256), (256, 224), (128, 128), (128, 64), (64, 64)]
                    assert parts == 1 or how in ["stream", (128, 128), (128, 64), (64, 64)]
                    assert parts * 32 <= max(k, 32)
    for bad in ((0, 1, -1, 8), (0, 1, 8, 4), (3, 1, 8, 8), (0, 1, 1 << 20, 1 << 11)):
        with pytest.raises(B.AggError):
            B.agg_linear_shape(*bad)


def test_binding_refuses_what_the_call_would_read_wrongly():
    a, b, y = (torch.zeros(*s, dtype=torch.bfloat16) for s in ((4, 64), (64, 32), (4, 32)))
    for call in (lambda: B.linear(None, 4, 32, 64, "bf16", a, b, y),                        # host tensors
                 lambda: B.linear(None, 0, 32, 64, "bf16", a.float(), b, y),
                 lambda: B.linear(None, 0, 32, 64, "fp8", a, b, y),
                 lambda: B.linear(None, 0, 24, 64, "bf16", a, b, y),
                 lambda: B.linear(None, 0, 32, 0, "bf16", a[:, :0], b, y.half()),
                 lambda: B.linear(None, 5, 32, 64, "bf16", a, b, y),
                 lambda: B.linear(None, 0, 32, 0, "bf16", a[:, :0], b[:0], y, bias=torch.zeros(31, dtype=torch.bfloat16)),
                 lambda: B.linear(None, 0, 32, 0, "bf16", a[:, :0], b[:0], y, residual=y.half())):
        with pytest.raises(B.AggError) as e:
            call()
        assert e.value.code == B.AGG_E_ARG
    with pytest.raises(KeyError):
        B.linear(None, 0, 0, 0, "bf16", a[:, :0], b[:0], y[:, :0], act="tanh")
