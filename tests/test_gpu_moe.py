"""The mixture-of-experts operators on the GPU against plain implementations in 64 bits.

Tolerances, derived from the formats: a bfloat16 output is within half a unit, 2^-8 of its value, of
the fp32 result it rounds; a sum of n fp32 terms is within n * 2^-23 of the sum of their sizes (each
of n additions and products rounds by at most 2^-24, both may); e4m3 has three fraction bits, half a
unit is 2^-4 of the value and 2^-10 below its normal range; exp and rsqrt are within 2^-21. The fp8
matrix instructions (16x16x32 and 32x32x64, probed with products of known sizes) add 8 products of
consecutive K after cutting each to multiples of 2^-13 of the largest of them, so a sum of them is
within 8 * 2^-13 of the sum of the sizes; what they add to the accumulator is fp32. Choices and places are compared exactly, on logits whose keys are either equal or clearly apart."""

import math

import numpy as np
import pytest
import torch

from allgather_gemm_persistent_amd import binding as B

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8
EPS32 = 2.0 ** -23
FINE = 2.0 ** -20            # a few elementary functions and products in fp32
FP8_SUM = 2.0 ** -10         # the fp8 matrix instructions' cut, of the sum of the products' sizes


@pytest.fixture(scope="module")
def ctx(gpu):
    c = B.agg_ctx_create(0)
    yield c
    B.agg_ctx_destroy(c)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _within(got, ref, bound, what):
    got, ref = got.double().cpu(), ref.double()
    err = (got - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds; worst error over bound "
                           f"{float((err / bound).nan_to_num(math.inf).max()):.3g}")


# ------------------------------------------------------------------------------ norm

def _strided(t, extra):
    """The same values in a tensor whose rows are `extra` elements further apart."""
    wide = torch.zeros(t.shape[0], t.shape[1] + extra, dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t.cuda()
    return wide[:, :t.shape[1]]


def _norm_ref(x, r, w, eps):
    s = x.double() + (r.double() if r is not None else 0)
    return s, s * torch.rsqrt((s * s).mean(1, keepdim=True) + eps) * w.double()


def _check_fp8(q, scale, y, cols):
    """q is a nearest e4m3 of y / scale, up to the fp32 steps before the rounding."""
    want = (y / scale[:, None].double()).clamp(-448, 448)
    slack = cols * EPS32 + FINE
    _within(q.float(), want, torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10)) + want.abs() * slack, "fp8")


NORM_SHAPES = [(1, 8), (3, 64), (1, 520), (5, 1024), (17, 1032), (2, 2048), (33, 4096), (1, 8192), (300, 8192),
               (7, 7168), (2, 16384), (3, 32768), (4, 16392)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("xd", ["bf16", "fp32"])
@pytest.mark.parametrize("out", ["bf16", "fp8", "fp8_static"])
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm(ctx, rows, cols, xd, out, residual):
    g = _gen(rows * 7 + cols)
    x = torch.randn(rows, cols, generator=g) * 3
    x = x if xd == "fp32" else x.bfloat16()
    r = torch.randn(rows, cols, generator=g).bfloat16() if residual else None
    w = (1 + 0.2 * torch.randn(cols, generator=g)).bfloat16()
    s, y = _norm_ref(x, r, w, 1e-5)
    extra = 8 * (rows % 3)
    dx = _strided(x, extra)
    dr = _strided(r, 2 * extra) if residual else None
    dro = _strided(torch.zeros(rows, cols, dtype=torch.bfloat16), 16) if residual else None
    od = torch.bfloat16 if out == "bf16" else torch.float8_e4m3fn
    do = _strided(torch.zeros(rows, cols, dtype=od), 16)
    scales = torch.full((rows,), -1.0, device="cuda") if out == "fp8" else None
    B.rms_norm(ctx, rows, cols, dx, w.cuda(), do, residual=dr, residual_out=dro, eps=1e-5, scales=scales, scale=1 / 64,
               stream=torch.cuda.current_stream())
    slack = cols * EPS32 + FINE
    if out == "bf16":
        _within(do, y, y.abs() * (HALF_BF16 + slack) + 1e-30, "y")
    else:
        scale = scales.cpu() if out == "fp8" else torch.full((rows,), 1 / 64)
        if out == "fp8":
            want = y.abs().amax(1) / 448
            _within(scale, want, want * slack, "scales")
        _check_fp8(do.cpu(), scale, y, cols)
    if residual:
        _within(dro, s, s.abs() * (HALF_BF16 + EPS32), "residual_out")


def test_rms_norm_in_place_and_zero_rows(ctx):
    """residual_out over residual, out over x; a row of zeros stays zeros in every output."""
    rows, cols = 6, 512
    g = _gen(3)
    x, r = torch.randn(rows, cols, generator=g).bfloat16(), torch.randn(rows, cols, generator=g).bfloat16()
    x[2] = 0
    r[2] = 0
    w = torch.ones(cols).bfloat16()
    s, y = _norm_ref(x, r, w, 1e-6)
    dx, dr = x.cuda(), r.cuda()
    B.rms_norm(ctx, rows, cols, dx, w.cuda(), dx, residual=dr, residual_out=dr, stream=torch.cuda.current_stream())
    _within(dx, y, y.abs() * (HALF_BF16 + cols * EPS32 + FINE) + 1e-30, "y over x")
    _within(dr, s, s.abs() * (HALF_BF16 + EPS32), "s over residual")
    q = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(rows, device="cuda")
    B.rms_norm(ctx, rows, cols, x.cuda(), w.cuda(), q, residual=r.cuda(), scales=scales, eps=0.0,
               stream=torch.cuda.current_stream())
    # (with eps 0 the zero row is 0 * inf: not a number, and its scale is 1)
    assert scales[2].item() == 1 and torch.isnan(q[2].float()).all()
    B.quant_rows(ctx, rows, cols, x.cuda(), q, scales=scales, stream=torch.cuda.current_stream())
    assert scales[2].item() == 1 and (q[2].float() == 0).all()


def test_rows_that_are_not_numbers(ctx):
    """A NaN stays in its row and place; an infinity makes its row's norm zeros and itself a NaN; the
    other rows do not notice."""
    rows, cols = 5, 264
    x = torch.randn(rows, cols, generator=_gen(5))
    x[1, 7] = math.nan
    x[3, 100] = math.inf
    w = torch.ones(cols).bfloat16()
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    B.rms_norm(ctx, rows, cols, x.cuda(), w.cuda(), out, stream=torch.cuda.current_stream())
    got = out.cpu().float()
    assert torch.isnan(got[1]).all()
    assert torch.isnan(got[3, 100]) and (got[3, :100] == 0).all() and (got[3, 101:] == 0).all()
    _, y = _norm_ref(x[[0, 2, 4]], None, w, 1e-6)
    _within(got[[0, 2, 4]], y, y.abs() * (HALF_BF16 + cols * EPS32 + FINE) + 1e-30, "other rows")
    q, scales = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, device="cuda")
    B.quant_rows(ctx, rows, cols, x.cuda(), q, scales=scales, stream=torch.cuda.current_stream())
    q = q.cpu().float()
    assert scales[1].item() == 1 and torch.isnan(q[1, 7]) and not torch.isnan(q[1, :7]).any()
    assert math.isinf(scales[3].item()) and torch.isnan(q[3, 100])


@pytest.mark.parametrize("rows,cols", [(1, 64), (40, 3584), (9, 1000)])
def test_quant_rows(ctx, rows, cols):
    x = (torch.randn(rows, cols, generator=_gen(cols)) * 0.01).bfloat16()
    q, scales = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, device="cuda")
    B.quant_rows(ctx, rows, cols, x.cuda(), q, scales=scales, stream=torch.cuda.current_stream())
    want = x.double().abs().amax(1) / 448
    _within(scales, want, want * EPS32, "scales")
    _check_fp8(q.cpu(), scales.cpu(), x.double(), 1)
    # a given scale saturates
    B.quant_rows(ctx, rows, cols, x.cuda(), q, scale=1e-6, stream=torch.cuda.current_stream())
    _check_fp8(q.cpu(), torch.full((rows,), 1e-6), x.double(), 1)
    assert q.float().abs().max().item() == 448


def test_quant_rows_of_the_smallest_and_largest_numbers(ctx):
    """Row scales whose reciprocal overflows, and rows near fp32's largest number."""
    x = torch.randn(4, 512, generator=_gen(1))
    x = x / x.abs().amax(1, keepdim=True)
    x[0] *= 1e-40
    x[1] *= 3e-36
    x[2] *= 3e38
    q, scales = torch.empty(4, 512, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(4, device="cuda")
    B.quant_rows(ctx, 4, 512, x.cuda(), q, scales=scales, stream=torch.cuda.current_stream())
    want = x.double().abs().amax(1) / 448
    # (a subnormal scale is rounded to a multiple of 2^-149)
    _within(scales, want, want * EPS32 + 2.0 ** -149, "scales")
    _check_fp8(q.cpu(), scales.cpu(), x.double(), 1)


@pytest.mark.parametrize("xd", ["bf16", "fp32"])
def test_quant_rows_beside_a_nan_saturates(ctx, xd):
    """The scale of a row with a NaN is 1: its other elements are rounded to e4m3 as they are, those
    beyond +-448 to +-448, infinities among them."""
    x = torch.randn(3, 1032, generator=_gen(6)) * 300
    x[1, 5], x[1, 6], x[1, 7], x[1, 8], x[1, 9] = math.nan, 1000.0, -464.5, math.inf, -math.inf
    x = x if xd == "fp32" else x.bfloat16()
    q, scales = torch.empty(3, 1032, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(3, device="cuda")
    B.quant_rows(ctx, 3, 1032, x.cuda(), q, scales=scales, stream=torch.cuda.current_stream())
    q, want = q.cpu(), x[1].float()
    assert scales[1].item() == 1 and torch.isnan(q[1, 5].float())
    assert q[1, 6:10].float().tolist() == [448, -448, 448, -448]
    keep = torch.arange(1032) != 5
    want = want[keep].clamp(-448, 448).to(torch.float8_e4m3fn)
    assert (want.float().abs() == 448).sum() > 100 and torch.equal(q[1, keep].float(), want.float())
    _check_fp8(q[[0, 2]], scales.cpu()[[0, 2]], x[[0, 2]].double(), 1)


@pytest.mark.parametrize("units", [1, 200, 225, 448, 600, 671, 700, 1000, 6000, 448 * 8388608, 500 * 8388608])
def test_fp8_rows_of_subnormal_scales(ctx, units):
    """A largest element of `units` times 2^-149, whose scale is rounded to a multiple of 2^-149 (or to
    none: then it is 1): every element is its quotient by that scale, kept inside +-448."""
    tiny = 2.0 ** -149
    x = torch.linspace(-1, 1, 520, dtype=torch.float64) * units
    x = (x.round() * tiny).float()[None].repeat(2, 1)
    q, scales = torch.empty(2, 520, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(2, device="cuda")
    B.quant_rows(ctx, 2, 520, x.cuda(), q, scales=scales, stream=torch.cuda.current_stream())
    scale = scales.cpu().double()
    want = units * tiny / 448
    # (the quotient is rounded to 24 bits, or to a multiple of 2^-149)
    assert (scale == 1).all() if units <= 224 else ((scale - want).abs() <= max(want * EPS32, tiny / 2)).all()
    # the kernel's quotient is rounded to fp32 before the conversion
    exact = (x.double() / scale[:, None]).clamp(-448, 448)
    _within(q.float(), exact, torch.maximum(exact.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10)) + exact.abs() * FINE, "fp8")


@pytest.mark.parametrize("extra", [1, 5, 36])
def test_a_single_row_of_any_stride(ctx, extra):
    """Where there is one row no stride is taken, so one that no other row could have is no error."""
    cols, s = 64, torch.cuda.current_stream()
    wide = lambda t: _strided(t, extra)  # noqa: E731
    x, r, w = torch.randn(1, cols, generator=_gen(extra)), torch.randn(1, cols, generator=_gen(1)).bfloat16(), torch.ones(cols).bfloat16()
    out, ro = wide(torch.zeros(1, cols).bfloat16()), wide(torch.zeros(1, cols).bfloat16())
    B.rms_norm(ctx, 1, cols, wide(x), w.cuda(), out, residual=wide(r), residual_out=ro, stream=s)
    ref, y = _norm_ref(x, r, w, 1e-6)
    _within(out, y, y.abs() * (HALF_BF16 + cols * EPS32 + FINE) + 1e-30, "y")
    _within(ro, ref, ref.abs() * (HALF_BF16 + EPS32), "residual_out")
    q, scales = wide(torch.zeros(1, cols).to(torch.float8_e4m3fn)), torch.zeros(1, device="cuda")
    B.quant_rows(ctx, 1, cols, wide(x), q, scales=scales, stream=s)
    _check_fp8(q.cpu(), scales.cpu(), x.double(), 1)
    a, b = wide(r), torch.randn(1, cols, 16, generator=_gen(2)).bfloat16()
    c = torch.zeros(1, 16, dtype=torch.bfloat16, device="cuda")
    B.moe_gemm(ctx, 1, 1, 16, cols, "bf16", a, b.cuda(), torch.tensor([0, 1], dtype=torch.int32, device="cuda"), c, stream=s)
    ref, size = r.double() @ b[0].double(), r.double().abs() @ b[0].double().abs()
    _within(c, ref, ref.abs() * HALF_BF16 + size * (cols * EPS32 + FINE), "product")
    # two rows of such a stride are still refused
    with pytest.raises(B.AggError) as e:
        B.quant_rows(ctx, 2, cols, _strided(torch.zeros(2, cols).bfloat16(), 4), torch.zeros(2, cols, dtype=torch.float8_e4m3fn, device="cuda"),
                     scales=torch.zeros(2, device="cuda"), stream=s)
    assert e.value.code == B.AGG_E_ARG


# ------------------------------------------------------------------------------ routing

def _route_ref(x, bias, score, groups, top_groups, k, renorm, scale):
    """ids, weights in 64 bits, token by token, from the definition."""
    T, E = x.shape
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        cand = [e for e in range(E) if x[t, e] > -np.inf]
        if not cand:
            continue
        if score == "softmax":
            m = max(x[t, e] for e in cand)
            ex = {e: math.exp(x[t, e] - m) for e in cand}
            tot = sum(ex.values())
            p = {e: ex[e] / tot for e in cand}
        else:
            p = {e: 1 / (1 + math.exp(-x[t, e])) for e in cand}
        key = {e: p[e] + (bias[e] if bias is not None else 0) for e in cand}
        if groups > 1:
            size = E // groups
            gs = []
            for g in range(groups):
                best = sorted((key[e] for e in cand if e // size == g), reverse=True)
                gs.append(-np.inf if not best else best[0] if score == "softmax" else sum(best[:2]))
            kept = sorted(range(groups), key=lambda g: (-gs[g], g))[:top_groups]
            cand = [e for e in cand if e // size in kept]
        pick = sorted(cand, key=lambda e: (-key[e], e))[:k]
        tot = sum(p[e] for e in pick) if renorm else 1.0
        for j, e in enumerate(pick):
            ids[t, j], w[t, j] = e, p[e] / tot * scale
    return ids, w


def _run_route(ctx, x, k, **kw):
    T, E = x.shape
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    B.moe_route(ctx, T, E, k, x, ids, w, stream=torch.cuda.current_stream(), **kw)
    return ids.cpu().numpy(), w.cpu().double().numpy()


def _grid_logits(T, E, seed, dtype):
    """Logits on a coarse grid: many exact ties, every other difference large. The grid does not
    hold -v beside v, whose sigmoids would sum to one in every such pair."""
    x = torch.randint(-24, 25, (T, E), generator=_gen(seed)).float() / 8 + 1 / 32
    return x if dtype == "fp32" else x.bfloat16()


ROUTES = [  # tokens, experts, k, groups, top_groups
    (1, 1, 1, 1, 1), (1, 64, 2, 1, 1), (33, 7, 7, 1, 1), (64, 60, 4, 1, 1), (5, 64, 16, 1, 1), (40, 65, 8, 1, 1),
    (17, 128, 6, 4, 2), (130, 256, 8, 8, 4), (3, 200, 5, 10, 3), (9, 300, 16, 2, 1), (50, 512, 8, 64, 8),
    (12, 1000, 3, 1, 1), (6, 1024, 16, 32, 4), (21, 64, 3, 64, 5), (10, 96, 16, 3, 1)]


@pytest.mark.parametrize("T,E,k,groups,top_groups", ROUTES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(ctx, T, E, k, groups, top_groups, dtype, score, renorm):
    x = _grid_logits(T, E, T + E, dtype)
    x[0, E // 2:] = -math.inf                       # disabled experts
    if T > 2:
        x[2] = -math.inf                            # a padded token
        x[1, 0] = math.nan
    ref = x.double().numpy().copy()
    ref[np.isnan(ref)] = -np.inf
    want_ids, want_w = _route_ref(ref, None, score, groups, top_groups, k, renorm, 2.5)
    ids, w = _run_route(ctx, x.cuda(), k, score=score, groups=groups, top_groups=top_groups, renorm=renorm, scale=2.5)
    np.testing.assert_array_equal(ids, want_ids)
    assert (np.abs(w - want_w) <= want_w * (E * EPS32 + FINE)).all(), np.abs(w - want_w).max()


@pytest.mark.parametrize("E", [64, 128, 256, 512, 1024])
@pytest.mark.parametrize("groups", [2, 4, 8, 16, 32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups(ctx, E, groups, score):
    """Few candidates, so that groups hold none, one or several: 16 values of logits, whose sigmoids'
    sums of two are equal or far apart, most experts disabled, whole groups and the last experts among
    them."""
    T, k, top_groups = 37, 6, max(1, groups // 3)
    values = torch.randn(16, generator=_gen(groups)).sort().values
    sums = torch.sort((values.double().sigmoid()[:, None] + values.double().sigmoid()[None, :]).reshape(-1)).values
    gap = sums.diff()
    assert gap[gap > 1e-12].min() > 1e-6
    x = values[torch.randint(0, 16, (T, E), generator=_gen(E))]
    x[torch.rand(T, E, generator=_gen(E + 1)) < 0.9] = -math.inf
    x[5, E // groups:] = -math.inf
    x[6, :E - E // groups] = -math.inf
    x[7] = -math.inf
    x[7, E - 1] = 0.5
    want_ids, want_w = _route_ref(x.double().numpy(), None, score, groups, top_groups, k, True, 1.0)
    ids, w = _run_route(ctx, x.cuda(), k, score=score, groups=groups, top_groups=top_groups)
    np.testing.assert_array_equal(ids, want_ids)
    assert (np.abs(w - want_w) <= want_w * (E * EPS32 + FINE)).all(), np.abs(w - want_w).max()


@pytest.mark.parametrize("T,E,k,groups,top_groups", [(70, 64, 4, 1, 1), (33, 256, 8, 8, 4), (9, 1024, 8, 16, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_bias(ctx, T, E, k, groups, top_groups, score):
    """The bias moves the choice and not the weight. The keys that decide are at least 1e-6 apart or
    equal by construction (equal logits and equal biases)."""
    x = _grid_logits(T, E, 11, "fp32")
    bias = torch.randint(-3, 4, (E,), generator=_gen(12)).float() / 16
    p = x.double().softmax(1) if score == "softmax" else x.double().sigmoid()
    key = np.sort((p + bias.double()).numpy(), axis=1)
    gap = np.diff(key, axis=1)
    if score == "sigmoid" and groups == 1:
        assert gap[(gap > 1e-12)].min() > 1e-6
    want_ids, want_w = _route_ref(x.double().numpy(), bias.double().numpy(), score, groups, top_groups, k, True, 1.0)
    strided = _strided(x, 3)
    ids, w = _run_route(ctx, strided, k, score=score, bias=bias.cuda(), groups=groups, top_groups=top_groups)
    if score == "softmax":      # keys of tiny probabilities may lie closer than fp32 tells apart: compare what matters
        same = (ids == want_ids).all(1)
        for t in np.flatnonzero(~same):
            kp = p[t] + bias.double()
            assert np.allclose(np.sort(kp[ids[t]]), np.sort(kp[want_ids[t]]), rtol=0, atol=1e-6)
        assert same.mean() > 0.5
    else:
        same = np.ones(T, bool)
        np.testing.assert_array_equal(ids, want_ids)
    assert (np.abs(w - want_w)[same] <= want_w[same] * (E * EPS32 + FINE) + 1e-9).all()


@pytest.mark.parametrize("T,E,k,groups,top_groups", [
    (9, 7, 7, 1, 1), (70, 64, 4, 1, 1), (33, 60, 2, 1, 1), (40, 256, 8, 8, 4), (17, 256, 8, 1, 1), (5, 1000, 16, 1, 1),
    (9, 1024, 16, 16, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("low,high", [(-300, -95), (-100, -80), (-110, -60), (-86, -69)])
def test_route_renormalises_scores_that_underflow(ctx, T, E, k, groups, top_groups, score, low, high):
    """A bias chooses experts whose scores are below fp32's numbers, or just above: the weights are their
    scores' shares all the same. Logits and biases are multiples of 1/8 and 1/16, so differences of
    logits are exact, and a key is its bias wherever a choice depends on it."""
    g = _gen(T + E)
    x = torch.randint(low * 8, high * 8 + 1, (T, E), generator=g).float() / 8
    bias = (torch.randperm(E, generator=g).float() + 1) / 16
    if score == "softmax":          # experts that take all the probability, never chosen unless all are
        x[:, ::5] = 0
        bias[::5] -= 1000
    if T > 5:
        x[3] = -math.inf
        x[4, 1:] = -math.inf
    want_ids, want_w = _route_ref(x.double().numpy(), bias.double().numpy(), score, groups, top_groups, k, True, 2.5)
    ids, w = _run_route(ctx, x.cuda(), k, score=score, bias=bias.cuda(), groups=groups, top_groups=top_groups, scale=2.5)
    np.testing.assert_array_equal(ids, want_ids)
    held = (want_ids >= 0).any(1)
    np.testing.assert_allclose(w.sum(1)[held], 2.5, rtol=(k + 2) * EPS32)
    # (beside fp32's roundings: 2^-49 of the sum for what lies below its numbers)
    assert (np.abs(w - want_w) <= want_w * (E * EPS32 + FINE) + k * 2.5 * 2.0 ** -49).all(), np.abs(w - want_w).max()


def test_route_many_tokens_distinct_logits(ctx):
    """Every token's logits are a permutation of distinct values: the order is known without a sort."""
    T, E, k = 3001, 256, 8
    order = torch.argsort(torch.rand(T, E, generator=_gen(9)), dim=1)
    x = torch.empty(T, E)
    x.scatter_(1, order, -torch.arange(E).float().repeat(T, 1) / 16)
    ids, w = _run_route(ctx, x.cuda(), k, renorm=False)
    np.testing.assert_array_equal(ids, order[:, :k].int().numpy())
    want = torch.softmax(-torch.arange(E).double() / 16, 0)[:k].numpy()
    assert (np.abs(w - want) <= want * (E * EPS32 + FINE)).all()


def test_more_rows_than_a_launch_holds(ctx):
    """Rows and tokens beyond 2^32 threads (64 and 8 of them a row): equal rows, so equal results, to the
    last."""
    rows = (1 << 26) + 5
    x = torch.tensor([1.0, -2.0, 3.0, 0.5, -0.25, 4.0, -6.0, 7.0], device="cuda").bfloat16().repeat(rows, 1)
    out = torch.zeros(rows, 8, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.zeros(rows, device="cuda")
    B.quant_rows(ctx, rows, 8, x, out, scales=scales, stream=torch.cuda.current_stream())
    assert bool((scales == scales[0]).all()) and abs(float(scales[0]) * 448 / 7 - 1) < 1e-6
    bits = out.view(torch.uint8).view(torch.int64).reshape(-1)
    assert bool((bits == bits[0]).all())
    np.testing.assert_allclose(out[-1].float().cpu().numpy() * float(scales[0]), x[-1].float().cpu().numpy(), rtol=2.0 ** -4)
    del x, out, scales, bits
    tokens = (1 << 29) + 7
    ids = torch.full((tokens, 1), -7, dtype=torch.int32, device="cuda")
    w = torch.zeros(tokens, 1, device="cuda")
    B.moe_route(ctx, tokens, 1, 1, torch.ones(tokens, 1, dtype=torch.bfloat16, device="cuda"), ids, w,
                stream=torch.cuda.current_stream())
    assert bool((ids == 0).all()) and bool((w == 1).all())
    torch.cuda.empty_cache()


# ------------------------------------------------------------------------------ the plan

def _plan_ref(ids, first, n):
    T, k = ids.shape
    flat = ids.reshape(-1).astype(np.int64)
    local = np.where((flat >= 0) & (flat >= first) & (flat < first + n), flat - first, n)
    order = np.argsort(local, kind="stable")
    held = int((local < n).sum())
    slot_token = np.full(T * k, -1, np.int32)
    slot_token[:held] = order[:held] // k
    token_slot = np.full(T * k, -1, np.int32)
    token_slot[order[:held]] = np.arange(held)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(local, minlength=n + 1)[:n])]).astype(np.int32)
    return offsets, slot_token, token_slot.reshape(T, k)


@pytest.mark.parametrize("T,k,n,first,total", [
    (0, 2, 8, 0, 8), (1, 1, 1, 0, 1), (1, 16, 64, 0, 64), (16, 2, 64, 0, 64), (63, 1, 5, 0, 5), (1023, 1, 8, 0, 8),
    (1024, 1, 8, 0, 8), (1025, 1, 8, 4, 16), (512, 2, 32, 96, 256), (4951, 4, 60, 0, 60), (5000, 8, 1024, 0, 1024),
    (32768, 8, 32, 128, 256), (3000, 3, 255, 1, 256), (700, 4, 256, 0, 300), (12288, 1, 64, 0, 64),
    (12289, 1, 64, 3, 70), (30001, 1, 900, 0, 1000), (40007, 8, 128, 0, 128), (1048579, 1, 20, 0, 30),
    (150001, 9, 77, 5, 90)])
def test_plan(ctx, T, k, n, first, total):
    rng = np.random.default_rng(T + n)
    ids = rng.integers(-1, total, (T, k)).astype(np.int32)
    _check_plan(ctx, ids, first, n)


def _check_plan(ctx, ids, first, n):
    T, k = ids.shape
    want = _plan_ref(ids, first, n)
    dev = [torch.full((m,), -9, dtype=torch.int32, device="cuda") for m in (n + 1, T * k, T * k)]
    work = torch.full((B.moe_plan_words(T, k, n),), 12345, dtype=torch.int32, device="cuda")
    B.moe_plan(ctx, T, k, torch.from_numpy(ids).cuda(), first, n, *dev, work, stream=torch.cuda.current_stream())
    for got, ref, what in zip(dev, want, ("offsets", "slot_token", "token_slot")):
        np.testing.assert_array_equal(got.cpu().numpy(), ref.reshape(-1), err_msg=what)


def test_plan_one_expert_takes_all_and_none_held(ctx):
    _check_plan(ctx, np.full((900, 3), 5, np.int32), 0, 8)
    _check_plan(ctx, np.full((900, 3), 5, np.int32), 6, 8)
    _check_plan(ctx, np.full((40, 2), -1, np.int32), 0, 8)


# ------------------------------------------------------------------------------ the experts' products

class _Experts:
    """One call's data: counts per expert, rows taken through slot_token (or in place), and the
    result and its error bound in 64 bits."""

    def __init__(self, counts, n, k, dtype, gated, gather, seed=0, a_rows=None, extra=0, spare=0):
        g = _gen(seed + n + k + sum(counts))
        self.counts, self.n, self.k, self.dtype, self.gated = counts, n, k, dtype, gated
        self.E, self.slots = len(counts), sum(counts) + spare
        cols = 2 * n if gated else n
        self.a_rows = a_rows or (max(1, self.slots // 2) if gather else max(1, self.slots))
        a = torch.randn(self.a_rows, k, generator=g)
        b = torch.randn(self.E, k, cols, generator=g) / math.sqrt(k)
        self.offsets = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
        self.tok = torch.randint(0, self.a_rows, (self.slots,), generator=g).int() if gather else None
        if dtype == "fp8":
            self.a, self.b = (a * 100).clamp(-448, 448).to(torch.float8_e4m3fn), (b * 50).clamp(-448, 448).to(torch.float8_e4m3fn)
            self.sa, self.sb = torch.rand(self.a_rows, generator=g) / 100 + 1e-3, torch.rand(self.E, cols, generator=g) / 50 + 1e-3
        else:
            self.a, self.b, self.sa, self.sb = a.bfloat16(), b.bfloat16(), None, None
        self.extra = extra

    def run(self, ctx, stream=None, tok=None):
        out = torch.full((max(1, self.slots), self.n), 77.0, dtype=torch.bfloat16, device="cuda")
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731
        a = _strided(self.a, self.extra) if self.extra else self.a.cuda()
        self.held = [a, dev(self.b), dev(self.offsets), dev(self.tok if tok is None else tok), dev(self.sa), dev(self.sb)]
        a, b, off, tok, sa, sb = self.held
        B.moe_gemm(ctx, self.slots, self.E, self.n, self.k, self.dtype, a, b, off, out, gated=self.gated, slot_token=tok,
                   a_scale=sa, b_scale=sb, stream=stream or torch.cuda.current_stream())
        return out

    def check(self, out, tok=None):
        tok = self.tok if tok is None else tok
        for e, c in enumerate(self.counts):
            lo = int(self.offsets[e])
            if c == 0:
                continue
            row = tok[lo:lo + c].long() if tok is not None else torch.arange(lo, lo + c)
            bad = (row < 0) | (row >= self.a_rows)
            row = torch.where(bad, 0, row)
            a, b = self.a[row].double(), self.b[e].double()
            a[bad] = 0
            if self.sa is not None:
                a, b = a * self.sa[row].double()[:, None], b * self.sb[e].double()
            y, size = a @ b, a.abs() @ b.abs()
            err = size * (self.k * EPS32 + FINE + (FP8_SUM if self.sa is not None else 0))
            if self.gated:
                gate, up = y[:, :self.n], y[:, self.n:]
                ge, ue = err[:, :self.n], err[:, self.n:]
                act = gate * torch.sigmoid(gate)
                # |silu'| <= 1.1
                y, err = act * up, 1.1 * ge * (up.abs() + ue) + act.abs() * ue + (act * up).abs() * FINE
            _within(out[lo:lo + c].float(), y, y.abs() * HALF_BF16 + err * 1.01 + 1e-30, f"expert {e}")
        # rows past the last offset are left alone
        assert (out[int(self.offsets[-1]):self.slots].float() == 77).all()


COUNTS = {
    "one row": [1], "single tokens": [1, 0, 1, 0, 0, 1, 1, 0], "few": [3, 16, 0, 17, 5, 1, 9, 2],
    "one holds most": [0, 75, 0, 2, 0], "tens": [40, 31, 64, 3], "hundreds": [200, 0, 131, 64, 257, 1],
    "none": [0, 0, 0]}


@pytest.mark.parametrize("which", list(COUNTS))
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("n,k", [(16, 16), (272, 208), (128, 1024), (1040, 80)])
def test_moe_gemm(ctx, which, dtype, gated, gather, n, k):
    x = _Experts(COUNTS[which], n, k, dtype, gated, gather, extra=16 if which == "tens" else 0, spare=5)
    x.check(x.run(ctx))


@pytest.mark.parametrize("tile", [(64, 64), (128, 64), (128, 128), (256, 224), (256, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("gated", [False, True])
def test_moe_gemm_every_tile(ctx, tile, dtype, gated):
    """Every tile shape, at counts below, at and above its rows, and widths that end inside it."""
    B.agg_ctx_set_tile(ctx, *tile)
    try:
        for counts, n, k, gather in (([1, 0, 63, 65], 64, 64, True), ([255, 256, 257, 0, 2], 464, 160, False),
                                     ([300, 5], 1104, 1168, True), ([130] * 9, 96, 32, False)):
            x = _Experts(counts, n, k, dtype, gated, gather, spare=3)
            x.check(x.run(ctx))
    finally:
        B.agg_ctx_set_tile(ctx, 0, 0)


@pytest.mark.parametrize("tile", [(256, 224), (256, 256), (128, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_moe_gemm_more_tiles_than_workgroups(ctx, tile, dtype):
    """Several whole and low tiles a workgroup: each row tile is computed, whatever the experts' last
    rows are (none, one, half a tile, one more than half)."""
    B.agg_ctx_set_tile(ctx, *tile)
    try:
        rng = np.random.default_rng(3)
        counts = [int(c) for c in rng.integers(0, 700, 40)] + [0, 1, 128, 129, 256, 257, 384, 385]
        x = _Experts(counts, 2064, 32, dtype, False, True, spare=2)
        x.check(x.run(ctx))
        x = _Experts([1, 128, 3, 0, 77], 4112, 48, dtype, True, False)   # low tiles alone
        x.check(x.run(ctx))
    finally:
        B.agg_ctx_set_tile(ctx, 0, 0)


@pytest.mark.parametrize("per,experts", [(1, 2), (12, 3), (30, 3), (60, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("gated", [False, True])
def test_moe_gemm_long_k_few_rows(ctx, per, experts, dtype, gated):
    """Few rows over K of 8192 and odd block counts: every wave's share of K, and their sum."""
    for k in (8192, 32 * 24 + 16, 32 * 9):
        x = _Experts([per] * experts, 144, k, dtype, gated, True)
        x.check(x.run(ctx))


def test_moe_gemm_many_experts(ctx):
    rng = np.random.default_rng(4)
    counts = [int(c) for c in rng.integers(0, 4, 1024)]
    x = _Experts(counts, 16, 32, "bf16", False, True)
    x.check(x.run(ctx))
    B.agg_ctx_set_tile(ctx, 64, 64)
    try:
        x.check(x.run(ctx))
    finally:
        B.agg_ctx_set_tile(ctx, 0, 0)


@pytest.mark.parametrize("tile", [(0, 0), (64, 64), (256, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_moe_gemm_rows_outside_a_are_zeros(ctx, tile, dtype):
    B.agg_ctx_set_tile(ctx, *tile)
    try:
        x = _Experts([7, 9, 4], 48, 96, dtype, False, True)
        tok = x.tok.clone()
        tok[3], tok[8], tok[19] = -1, x.a_rows, 1 << 30
        x.check(x.run(ctx, tok=tok), tok=tok)
    finally:
        B.agg_ctx_set_tile(ctx, 0, 0)


@pytest.mark.parametrize("counts", [[5, 9, 3], [200, 140, 90]])
def test_moe_gemm_repeats_its_bits_and_order_of_rows_does_not_matter(ctx, counts):
    x = _Experts(counts, 272, 512, "bf16", True, True)
    first = x.run(ctx)
    assert torch.equal(first, x.run(ctx))
    # the rows of one expert in another order: the same rows of the result
    perm = torch.cat([int(x.offsets[e]) + torch.randperm(c, generator=_gen(1)) for e, c in enumerate(counts)])
    assert torch.equal(first[perm.cuda()], x.run(ctx, tok=x.tok[perm]))


def test_moe_gemm_output_past_4_gib(ctx):
    """Row offsets of the output beyond 32 bits: the last rows of a 5 GB result."""
    slots, n, k, E = 300_000, 8192, 32, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    a = torch.randn(slots, k, generator=g, device="cuda").bfloat16()
    b = torch.randn(E, k, n, generator=g, device="cuda").bfloat16()
    off = torch.tensor([0, 150_001, slots], dtype=torch.int32, device="cuda")
    out = torch.empty(slots, n, dtype=torch.bfloat16, device="cuda")
    B.moe_gemm(ctx, slots, E, n, k, "bf16", a, b, off, out, stream=torch.cuda.current_stream())
    for lo, hi, e in ((0, 300, 0), (149_900, 150_001, 0), (150_001, 150_300, 1), (slots - 300, slots, 1)):
        ref = a[lo:hi].double().cpu() @ b[e].double().cpu()
        size = a[lo:hi].double().cpu().abs() @ b[e].double().cpu().abs()
        _within(out[lo:hi].float(), ref, ref.abs() * HALF_BF16 + size * (k * EPS32), f"rows {lo}..{hi}")


# ------------------------------------------------------------------------------ the combine

@pytest.mark.parametrize("T,k,n", [(1, 1, 8), (1, 2, 8192), (5, 16, 72), (300, 3, 2056), (70, 5, 4096)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_moe_combine(ctx, T, k, n, out):
    g = _gen(T + n)
    slots = max(1, T * k - 2)
    y = torch.randn(slots, n, generator=g).bfloat16()
    at = torch.randint(-1, slots + 2, (T, k), generator=g).int()     # past the end: no slot either
    if T > 3:
        at[1] = -1
        y[0] = math.nan
        at[at == 0] = -1                                             # a row no token takes may hold anything
    w = torch.rand(T, k, generator=g)
    has = (at >= 0) & (at < slots)
    terms = torch.where(has[:, :, None], y.double()[at.long().clamp(0, slots - 1)], 0) * w.double()[:, :, None]
    ref, size = terms.sum(1), terms.abs().sum(1)
    got = torch.full((T, n), 9.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    B.moe_combine(ctx, T, k, n, slots, y.cuda(), at.cuda(), w.cuda(), got, stream=torch.cuda.current_stream())
    _within(got, ref, size * (k + 1) * EPS32 + (ref.abs() * HALF_BF16 if out == "bf16" else 0) + 1e-30, "combine")
    if T > 3:
        assert (got[1] == 0).all()


def test_moe_combine_beyond_65535_tokens(ctx):
    T, k, n = 70_001, 2, 8
    g = _gen(8)
    y = torch.randn(1000, n, generator=g).bfloat16()
    at = torch.randint(0, 1000, (T, k), generator=g).int()
    w = torch.rand(T, k, generator=g)
    got = torch.empty(T, n, device="cuda")
    B.moe_combine(ctx, T, k, n, 1000, y.cuda(), at.cuda(), w.cuda(), got, stream=torch.cuda.current_stream())
    terms = y.double()[at.long()] * w.double()[:, :, None]
    _within(got, terms.sum(1), terms.abs().sum(1) * 3 * EPS32 + 1e-30, "combine")


# ------------------------------------------------------------------------------ together

def _layer(ctx, x, logits, w1, w2, out, bufs, stream):
    T, E, k = logits.shape[0], logits.shape[1], bufs["ids"].shape[1]
    H, F = w1.shape[1], w2.shape[1]
    B.moe_route(ctx, T, E, k, logits, bufs["ids"], bufs["w"], stream=stream)
    B.moe_plan(ctx, T, k, bufs["ids"], 0, E, bufs["off"], bufs["st"], bufs["ts"], bufs["work"], stream=stream)
    B.moe_gemm(ctx, T * k, E, F, H, "bf16", x, w1, bufs["off"], bufs["h"], gated=True, slot_token=bufs["st"], stream=stream)
    B.moe_gemm(ctx, T * k, E, H, F, "bf16", bufs["h"], w2, bufs["off"], bufs["y"], stream=stream)
    B.moe_combine(ctx, T, k, H, T * k, bufs["y"], bufs["ts"], bufs["w"], out, stream=stream)


def _layer_data(T, E=6, k=2, H=256, F=144):
    g = _gen(T)
    bf, i32 = torch.bfloat16, torch.int32
    w1 = (torch.randn(E, H, 2 * F, generator=g) / 16).bfloat16().cuda()
    w2 = (torch.randn(E, F, H, generator=g) / 12).bfloat16().cuda()
    mk = lambda *s, d: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    bufs = dict(ids=mk(T, k, d=i32), w=mk(T, k, d=torch.float32), off=mk(E + 1, d=i32), st=mk(T * k, d=i32), ts=mk(T, k, d=i32),
                work=mk(B.moe_plan_words(T, k, E), d=i32), h=mk(T * k, F, d=bf), y=mk(T * k, H, d=bf))
    return w1, w2, bufs, g


def _layer_ref(x, logits, w1, w2, k):
    p = torch.softmax(logits.double().cpu(), 1)
    w, ids = torch.topk(p, k, 1)
    w = w / w.sum(1, keepdim=True)
    x, w1, w2 = (t.double().cpu() for t in (x, w1, w2))
    F = w2.shape[1]
    out = torch.zeros(x.shape, dtype=torch.float64)
    for t in range(x.shape[0]):
        for j in range(k):
            y = x[t] @ w1[ids[t, j]]
            out[t] += w[t, j] * ((y[:F] * torch.sigmoid(y[:F]) * y[F:]) @ w2[ids[t, j]])
    return out


@pytest.mark.parametrize("T", [1, 8, 150])
def test_layer_on_a_side_stream_and_in_a_replayed_graph(ctx, T):
    """The whole path on another stream than torch's, then captured and replayed on new inputs, each
    replay against the eager result."""
    w1, w2, bufs, g = _layer_data(T)
    H, E = w1.shape[1], w1.shape[0]
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    logits = torch.empty(T, E, device="cuda")
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")

    def fill(seed):
        gg = _gen(seed)
        x.copy_(torch.randn(T, H, generator=gg).bfloat16())
        logits.copy_(torch.randn(T, E, generator=gg))

    side = torch.cuda.Stream()
    fill(1)
    side.wait_stream(torch.cuda.current_stream())
    _layer(ctx, x, logits, w1, w2, out, bufs, side)
    torch.cuda.current_stream().wait_stream(side)
    ref = _layer_ref(x, logits, w1, w2, 2)
    # h, y and out are rounded to bf16: three half units, the first two of terms up to a few times the sum
    tol = 8 * HALF_BF16 * ref.abs() + 4 * HALF_BF16 * ref.abs().mean()
    _within(out, ref, tol, "side stream")

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        _layer(ctx, x, logits, w1, w2, out, bufs, torch.cuda.current_stream())
    for seed in range(2, 7):
        fill(seed)
        _layer(ctx, x, logits, w1, w2, out, bufs, torch.cuda.current_stream())
        torch.cuda.synchronize()
        eager = out.clone()
        out.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), seed


def test_split_k_on_more_streams_than_workspaces(ctx):
    """Calls of few rows and experts, K split over workgroups, at once on six streams (two of them go
    without a workspace) and over and over: every result is its own."""
    xs = [_Experts([1, 2], 256, 4096, "bf16", i % 2 == 0, True, seed=i) for i in range(6)]
    assert B.agg_moe_gemm_shape("bf16", 3, 2, 256, 4096, True)[1] > 1
    streams = [torch.cuda.Stream() for _ in xs]
    outs = []
    for x in xs:
        x.run(ctx)                                   # lays the data out on the device
        outs.append(torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    for _ in range(20):
        for x, s, out in zip(xs, streams, outs):
            a, b, off, tok, sa, sb = x.held
            B.moe_gemm(ctx, 3, 2, 256, 4096, "bf16", a, b, off, out, gated=x.gated, slot_token=tok, stream=s)
    torch.cuda.synchronize()
    for x, out in zip(xs, outs):
        x.check(out)


@pytest.mark.parametrize("T", [1, 9, 200])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("held", [8, 4])
def test_moe_layer(gpu, T, dtype, held):
    """The layer from the residual stream to the rank's partial sum. The steps between the operators
    round to bf16 or e4m3, so each is compared from the rows that entered it."""
    from allgather_gemm_persistent_amd.moe_layer import random_layer
    H, F, E, k = 256, 128, 8, 2
    layer = random_layer(T + 3, H, F, E, k, dtype, n_local=held, first=E - held, seed=T, score="sigmoid",
                         bias=torch.linspace(-0.1, 0.1, E))
    try:
        g = _gen(T)
        x, r = torch.randn(T, H, generator=g), torch.randn(T, H, generator=g).bfloat16()
        residual = r.cuda()
        out = layer.run(x.cuda(), residual).cpu()
        s, y = _norm_ref(x, r, layer.norm.cpu(), 1e-6)
        _within(residual, s, s.abs() * (HALF_BF16 + EPS32), "residual")
        xn = layer.x[:T].cpu()
        _within(xn, y, y.abs() * (HALF_BF16 + H * EPS32 + FINE) + 1e-30, "norm")
        logits = layer.logits[:T].cpu()
        ref = xn.double() @ layer.router.double().cpu()
        size = xn.double().abs() @ layer.router.double().cpu().abs()
        _within(logits, ref, ref.abs() * HALF_BF16 + size * H * EPS32 + 1e-30, "logits")
        ids, w = layer.ids[:T].cpu(), layer.weights[:T].cpu().double()
        want_ids, want_w = _route_ref(logits.double().numpy(), np.linspace(-0.1, 0.1, E, dtype=np.float32).astype(np.float64),
                                      "sigmoid", 1, 1, k, True, 1.0)
        assert (ids.numpy() == want_ids).all()
        assert (np.abs(w.numpy() - want_w) <= want_w * (E * EPS32 + FINE)).all()
        # the products from what the layer itself quantised or rounded before them
        ref, size = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
        slot = layer.token_slot[:T].cpu() if T == layer.tokens else layer.token_slot.view(-1)[:T * k].view(T, k).cpu()
        for t in range(T):
            for j in range(k):
                e = int(ids[t, j]) - (E - held)
                if e < 0:
                    assert slot[t, j] == -1
                    continue
                m = int(slot[t, j])
                if dtype == "fp8":
                    a = layer.x8[t].cpu().double() * float(layer.x_scale[t])
                    up = layer.w_up[e].cpu().double() * layer.up_scale[e].cpu().double()
                    down = layer.w_down[e].cpu().double() * layer.down_scale[e].cpu().double()
                    mid = layer.mid8[m].cpu().double() * float(layer.mid_scale[m])
                else:
                    a, up, down = xn[t].double(), layer.w_up[e].cpu().double(), layer.w_down[e].cpu().double()
                    mid = layer.mid[m].cpu().double()
                z, zs = a @ up, a.abs() @ up.abs()
                act = z[:F] * torch.sigmoid(z[:F])
                cut = FP8_SUM if dtype == "fp8" else 0
                err = zs * (H * EPS32 + FINE + cut)
                bound = 1.1 * err[:F] * (z[F:].abs() + err[F:]) + act.abs() * err[F:] + (act * z[F:]).abs() * (FINE + HALF_BF16)
                _within(layer.mid[m].cpu(), act * z[F:], 1.01 * bound + 1e-30, "between the products")
                y = mid @ down
                ref[t] += w[t, j] * y
                size[t] += w[t, j] * (y.abs() * HALF_BF16 + (mid.abs() @ down.abs()) * (F * EPS32 + FINE + cut))
        _within(out, ref, 1.01 * size + ref.abs() * 4 * EPS32 + 1e-30, "the layer")
        assert layer.run(x[:0].cuda()).shape == (0, H)
        with pytest.raises(B.AggError):
            layer.run(torch.zeros(T + 4, H, device="cuda"))
    finally:
        layer.close()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_moe_layer_weights(gpu, score, renorm):
    """A layer whose weights are the chosen probabilities themselves, times a scale, or their shares."""
    from allgather_gemm_persistent_amd.moe_layer import random_layer
    T, H, F, E, k = 21, 128, 64, 16, 4
    layer = random_layer(T, H, F, E, k, seed=3, score=score, renorm=renorm, scale=1.5)
    try:
        out = layer.run(torch.randn(T, H, generator=_gen(4)).cuda()).cpu()
        ids, w = layer.ids.cpu(), layer.weights.cpu().double()
        want_ids, want_w = _route_ref(layer.logits.cpu().double().numpy(), None, score, 1, 1, k, renorm, 1.5)
        assert (ids.numpy() == want_ids).all()
        assert (np.abs(w.numpy() - want_w) <= want_w * (E * EPS32 + FINE)).all()
        terms = layer.y.cpu().double()[layer.token_slot.cpu().long()] * w[:, :, None]
        _within(out, terms.sum(1), terms.abs().sum(1) * (k + 1) * EPS32 + 1e-30, "combine")
    finally:
        layer.close()


@pytest.mark.parametrize("T,E,k", [(1, 60, 4), (33, 60, 4), (300, 7, 2), (20, 1, 1)])
def test_moe_layer_of_any_number_of_experts(gpu, T, E, k):
    """Expert counts whose router has no rows of whole 16 bytes."""
    from allgather_gemm_persistent_amd.moe_layer import random_layer
    H, F = 128, 64
    layer = random_layer(T, H, F, E, k, seed=E)
    try:
        out = layer.run(torch.randn(T, H, generator=_gen(T)).cuda()).cpu()
        xn, logits = layer.x.cpu(), layer.logits.cpu()
        assert logits.shape == (T, E)
        ref = xn.double() @ layer.router.double().cpu()
        size = xn.double().abs() @ layer.router.double().cpu().abs()
        _within(logits, ref, ref.abs() * HALF_BF16 + size * H * EPS32 + 1e-30, "logits")
        want_ids, want_w = _route_ref(logits.double().numpy(), None, "softmax", 1, 1, k, True, 1.0)
        assert (layer.ids.cpu().numpy() == want_ids).all()
        w = layer.weights.cpu().double()
        assert (np.abs(w.numpy() - want_w) <= want_w * (E * EPS32 + FINE)).all()
        terms = layer.y.cpu().double()[layer.token_slot.cpu().long()] * w[:, :, None]
        _within(out, terms.sum(1), terms.abs().sum(1) * (k + 1) * EPS32 + 1e-30, "combine")
    finally:
        layer.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_split_k_in_a_replayed_graph_and_after_reset(ctx, dtype):
    """K in parts, captured and replayed between eager calls of other rows; then after a reset."""
    x = _Experts([1, 3], 256, 4096, dtype, True, True, seed=5)
    assert B.agg_moe_gemm_shape(dtype, 4, 2, 256, 4096, True)[1] > 1
    want = x.run(ctx)
    x.check(want)
    a, b, off, tok, sa, sb = x.held
    out = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_gemm(ctx, 4, 2, 256, 4096, dtype, a, b, off, out, gated=True, slot_token=tok, a_scale=sa, b_scale=sb,
                   stream=torch.cuda.current_stream())
    first = tok.clone()
    for i in range(5):
        perm = torch.tensor([0, 1 + (1 + i) % 3, 1 + (2 + i) % 3, 1 + i % 3], device="cuda")
        tok.copy_(first[perm])
        out.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[perm]), i
        x.check(x.run(ctx))
    B.agg_ctx_reset(ctx, torch.cuda.current_stream())
    assert torch.equal(x.run(ctx), want)
