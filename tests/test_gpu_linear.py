"""The product with an epilogue on the GPU against a plain implementation in 64 bits.

Tolerances, derived from the formats: a bfloat16 output is within half a unit, 2^-8 of its value, of the fp32 result
it rounds; a sum of k fp32 products is within k * 2^-23 of the sum of their sizes; the fp8 matrix instructions cut each
of 8 products to multiples of 2^-13 of the largest of them: within 2^-10 of the sum of the sizes. An activation's slope
is at most 1.13, so it passes on the product's error hardly enlarged; its own steps are within 2^-20 of 1 + its value's
size."""

import math

import pytest
import torch

from allgather_gemm_persistent_amd import binding as B

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8
EPS32 = 2.0 ** -23
FINE = 2.0 ** -20
FP8_SUM = 2.0 ** -10
BF16, FP8, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32
ACTS = {"none": lambda x: x, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
        "gelu_tanh": lambda x: torch.nn.functional.gelu(x, approximate="tanh")}


@pytest.fixture(scope="module")
def ctx(gpu):
    c = B.agg_ctx_create(0)
    yield c
    B.agg_ctx_set_tile(c)
    B.agg_ctx_destroy(c)


class _Product:
    """Operands, what the epilogue adds, and the result in 64 bits with its bound."""

    def __init__(self, m, n, k, dtype="bf16", bias=True, residual="bf16", out="bf16", act="none", seed=0, extra=0):
        g = torch.Generator().manual_seed(seed + m + n + k)
        self.m, self.n, self.k, self.dtype, self.act = m, n, k, dtype, act
        rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        kinds = {"bf16": BF16, "fp32": F32}
        a, b = rand(m, k), rand(k, n) / k ** 0.5
        self.a_scale = self.b_scale = None
        if dtype == "fp8":
            self.a_scale, self.b_scale = a.abs().amax(1) / 448 + 1e-6, b.abs().amax(0) / 448 + 1e-6
            a, b = (a / self.a_scale[:, None]).to(FP8), (b / self.b_scale).to(FP8)
        else:
            a, b = a.bfloat16(), b.bfloat16()
        self.bias = rand(n).bfloat16() if bias else None
        self.r = rand(m, n).to(kinds[residual]) if residual else None
        self.out = kinds[out]
        x, y = a.double(), b.double()
        z, size = x @ y, x.abs() @ y.abs()
        if dtype == "fp8":
            s = self.a_scale.double()[:, None] * self.b_scale.double()
            z, size = z * s, size * s
        err = size * (k * EPS32 + (FP8_SUM if dtype == "fp8" else 0) + FINE)
        if bias:
            z = z + self.bias.double()
            err = err + z.abs() * EPS32
        self.want = ACTS[act](z)
        if act != "none":
            err = 1.2 * err + FINE * (1 + z.abs())
        if self.r is not None:
            self.want = self.want + self.r.double()
        err = err + self.want.abs() * EPS32
        self.bound = err + (HALF_BF16 * (self.want.abs() + err) if out == "bf16" else 0)
        # rows `extra` elements further apart than they have to be, on the device
        self.a, self.b = self._wide(a, extra), b.cuda()
        self.r = None if self.r is None else self._wide(self.r, extra)
        for name in ("a_scale", "b_scale", "bias"):
            x = getattr(self, name)
            setattr(self, name, None if x is None else x.cuda())
        self.extra = extra

    @staticmethod
    def _wide(x, extra):
        w = torch.zeros(x.shape[0], x.shape[1] + extra, dtype=x.dtype, device="cuda")
        w[:, :x.shape[1]] = x.cuda()
        return w[:, :x.shape[1]]

    def run(self, ctx, out=None, stream=None, residual=None):
        y = out if out is not None else torch.full((self.m + 1, self.n + self.extra), 7.0, dtype=self.out, device="cuda")
        B.linear(ctx, self.m, self.n, self.k, self.dtype, self.a, self.b, y[:self.m, :self.n], a_scale=self.a_scale,
                 b_scale=self.b_scale, bias=self.bias, act=self.act, residual=self.r if residual is None else residual,
                 stream=stream or torch.cuda.current_stream())
        return y

    def check(self, y):
        torch.cuda.synchronize()
        if y.shape[0] > self.m:
            assert bool((y[self.m:] == 7).all()) and bool((y[:, self.n:] == 7).all()), "what surrounds the result"
        err = (y[:self.m, :self.n].double().cpu() - self.want).abs()
        bad = ~(err <= self.bound)
        assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} out of bounds; worst "
                               f"{float((err / self.bound).nan_to_num(math.inf).max()):.3g}")


SHAPES = [(1, 8, 8), (1, 16, 16), (1, 256, 4096), (2, 1000, 64), (3, 128, 1032), (7, 520, 256), (16, 2048, 2048), (17, 136, 40),
          (31, 264, 512), (32, 1024, 8192), (33, 384, 1000), (64, 640, 320), (65, 72, 72), (100, 1032, 1000), (128, 2048, 512),
          (129, 256, 96), (200, 224, 1024), (256, 512, 128), (257, 1000, 48), (300, 1808, 264), (777, 1000, 1032), (1024, 1024, 512)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_sizes(ctx, m, n, k, dtype, out):
    if dtype == "fp8":
        n, k = -(-n // 16) * 16, -(-k // 16) * 16
    p = _Product(m, n, k, dtype, out=out, act="silu", extra=16)
    p.check(p.run(ctx))


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [None, "bf16", "fp32"])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("m", [5, 300])
def test_epilogues(ctx, act, bias, residual, out, m):
    p = _Product(m, 264, 512, "bf16" if bias else "fp8" if m == 5 else "bf16", bias, residual, out, act) if m != 5 or bias \
        else _Product(m, 272, 512, "fp8", bias, residual, out, act)
    p.check(p.run(ctx))


@pytest.mark.parametrize("tile", [(256, 256), (256, 224), (128, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("m,n,k", [(1, 16, 16), (63, 208, 80), (64, 256, 128), (129, 464, 320), (192, 240, 528), (300, 672, 1040),
                                   (321, 512, 256)])
def test_every_tile(ctx, tile, dtype, m, n, k):
    p = _Product(m, n, k, dtype, residual="fp32", act="gelu_tanh", extra=16)
    B.agg_ctx_set_tile(ctx, *tile)
    try:
        p.check(p.run(ctx))
    finally:
        B.agg_ctx_set_tile(ctx)


@pytest.mark.parametrize("tile", [(256, 256), (64, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_more_tiles_than_workgroups(ctx, tile, dtype):
    m, n = (3000, 8208) if tile[0] == 256 else (1000, 2576)
    p = _Product(m, n, 64, dtype, residual="bf16", act="relu", extra=16)
    B.agg_ctx_set_tile(ctx, *tile)
    try:
        p.check(p.run(ctx))
    finally:
        B.agg_ctx_set_tile(ctx)


@pytest.mark.parametrize("tile", [(128, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("parts", [2, 3, 5, 16])
@pytest.mark.parametrize("m,n,k", [(1, 16, 128), (65, 208, 1040), (200, 336, 4096)])
def test_split_tiles(ctx, tile, dtype, parts, m, n, k):
    """K of tiles in parts (as many as it has slice pairs at most), called again and on another stream: the same bits."""
    p = _Product(m, n, k, dtype, residual="bf16", out="fp32", act="silu", extra=16)
    B.agg_ctx_set_tile(ctx, *tile)
    B.agg_ctx_set_split(ctx, parts)
    try:
        first = p.run(ctx)
        p.check(first)
        side = torch.cuda.Stream()
        for s in (None, side, side, None):
            again = torch.zeros_like(first)
            torch.cuda.synchronize()
            p.run(ctx, out=again, stream=s)
            torch.cuda.synchronize()
            assert torch.equal(again[:m, :n], first[:m, :n])
    finally:
        B.agg_ctx_set_tile(ctx)
        B.agg_ctx_set_split(ctx)


def test_split_tiles_in_replayed_graphs(ctx):
    """Two captures of a call whose tiles' K is split, replayed between eager calls of other rows."""
    ps = [_Product(100, 512, 8192, "bf16", seed=i) for i in range(3)]
    how, parts = B.agg_linear_shape("bf16", 100, 512, 8192)
    assert how != "stream" and parts > 1
    graphs = []
    for p in ps[:2]:
        y = torch.zeros(100, 512, dtype=BF16, device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            p.run(ctx, out=y, stream=torch.cuda.current_stream())
        graphs.append((p, g, y))
    for i in range(6):
        p, g, y = graphs[i % 2]
        p.a.copy_(p.a.roll(1, 0))
        want = p.run(ctx)[:100].clone()
        ps[2].check(ps[2].run(ctx))
        y.fill_(5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("m", [1, 32, 40])
def test_split_k(ctx, dtype, m):
    p = _Product(m, 256, 8192, dtype, residual="fp32", out="fp32", act="silu")
    if m <= 32:
        assert B.agg_linear_shape(dtype, m, 256, 8192)[1] > 1
    first = p.run(ctx)
    p.check(first)
    for _ in range(5):
        assert torch.equal(p.run(ctx), first)


@pytest.mark.parametrize("m,n,k,dtype", [(9, 512, 4096, "bf16"), (300, 512, 256, "bf16"), (9, 512, 4096, "fp8"), (300, 512, 256, "fp8")])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_into_the_residual(ctx, m, n, k, dtype, kind):
    p = _Product(m, n, k, dtype, residual=kind, out=kind)
    r = p.r.clone()
    p.run(ctx, out=r, residual=r)
    p.check(r)


def test_values_that_are_not_finite(ctx):
    """A NaN or an infinity of A reaches its row alone, one of the residual its element; a NaN passes every activation."""
    for act in ACTS:
        for m in (4, 200):
            p = _Product(m, 64, 64, act=act, residual="fp32", out="fp32")
            p.a[1, 3] = math.nan
            p.a[2, 5] = math.inf
            p.r[3, 7] = -math.inf
            y = p.run(ctx)[:m]
            z = p.a.float() @ p.b.float() + p.bias.float()
            want = ACTS[act](z.double()) + p.r.double()
            assert bool(y[1].isnan().all()) and torch.equal(y.isnan(), want.isnan()), act
            assert torch.equal(y == math.inf, want == math.inf) and torch.equal(y == -math.inf, want == -math.inf)


def test_activations_of_large_values(ctx):
    p = _Product(8, 64, 64, residual=None, out="fp32")
    for act in ACTS:
        p.act = act
        for scale in (1e4, 1e18, 1e30):
            p.bias = (torch.linspace(-1, 1, 64) * scale).bfloat16().cuda()
            y = p.run(ctx)[:8].double().cpu()
            want = ACTS[act]((p.a.double() @ p.b.double() + p.bias.double()).cpu())
            assert bool(((y - want).abs() <= 2.0 ** -18 * want.abs() + 1e-3).all()), (act, scale)


def test_rows_past_4_gib(ctx):
    """An output whose last rows lie past 2^32 bytes."""
    m, n, k = 1 << 21, 1048, 16
    a = torch.zeros(m, k, dtype=BF16, device="cuda")
    a[-5:] = 1
    b = torch.eye(k, n, dtype=BF16, device="cuda")
    y = torch.full((m, n), 7.0, dtype=BF16, device="cuda")
    B.linear(ctx, m, n, k, "bf16", a, b, y, residual=y, stream=torch.cuda.current_stream())
    assert bool((y[-5:, :16] == 8).all()) and bool((y[-5:, 16:] == 7).all()) and bool((y[-600:-5] == 7).all())
    assert bool((y[:600] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_streams_and_replayed_graphs(ctx, dtype):
    """Calls with K in parts on several streams at once, and two graphs replayed between eager calls of other operands."""
    ps = [_Product(4, 256, 4096, dtype, seed=i, act="gelu") for i in range(4)]
    assert B.agg_linear_shape(dtype, 4, 256, 4096)[1] > 1
    streams = [torch.cuda.Stream() for _ in ps]
    outs = [p.run(ctx) for p in ps]
    torch.cuda.synchronize()
    for _ in range(10):
        for p, s, y in zip(ps, streams, outs):
            p.run(ctx, out=y, stream=s)
    for p, y in zip(ps, outs):
        p.check(y)
    graphs, caught = [], []
    for p in ps[:2]:
        y = torch.zeros(4, 256, dtype=BF16, device="cuda")
        graphs.append(torch.cuda.CUDAGraph())
        torch.cuda.synchronize()
        with torch.cuda.graph(graphs[-1]):
            p.run(ctx, out=y, stream=torch.cuda.current_stream())
        caught.append(y)
    for i in range(6):
        p, y, g = ps[i % 2], caught[i % 2], graphs[i % 2]
        p.a.copy_(ps[2 + i % 2].a if i % 4 < 2 else p.a.flip(0))
        want = p.run(ctx)[:4].clone()
        y.fill_(5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("m,dtype", [(5, "bf16"), (300, "bf16"), (5, "fp8"), (300, "fp8")])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_activations_keep_their_small_values(ctx, act, m, dtype, out):
    """A product of zeros, so that the bias is the activation's argument to the bit, from -10 to 10: each value within
    some units of itself, the tails' too. The steps' errors in units of 2^-24 of the result, each rounding half a unit in
    the last place (1), v_exp and v_rcp a whole one (2); an exponent's relative error counts as often as the exponent is large:
      SiLU       the exponent's constant and product 1.5 |x|, then v_exp 2, the sum 1, v_rcp 2, the product 1
      GELU       the exponent x^2 / 2: the square, its constant and the product 3 x^2 / 2; t: 5 steps, which Q t passes on 2.9
                 times; Q: 1.6e-7, 2.6, and its sums, of terms 1.4 times it in all, 8; v_exp 2, three products 3
      GELU tanh  the exponent 2 u of eight roundings; then as SiLU
    A reciprocal below 2^-126, which may come out as zero, adds |x| 2^-126."""
    n, k = 2048, 16
    x = torch.cat([torch.linspace(-10, 10, n - 64), torch.logspace(-30, 0, 32), -torch.logspace(-30, 0, 32)]).bfloat16()
    z = x.double()
    u2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    want, units = {"silu": (z / (1 + torch.exp(-z)), 6 + 1.5 * z.abs()),
                   "gelu": (0.5 * z * torch.special.erfc(-z / math.sqrt(2)), 31 + 1.5 * z * z),
                   "gelu_tanh": (z / (1 + torch.exp(-u2)), 6 + 9.5 * u2.abs())}[act]
    err = want.abs() * units * 2.0 ** -24 + z.abs() * 2.0 ** -126
    bound = err + (HALF_BF16 * (want.abs() + err) if out == "bf16" else 0)
    el, to = (FP8, BF16)[dtype == "bf16"], {"bf16": BF16, "fp32": F32}[out]
    ones = (torch.ones(m, device="cuda"), torch.ones(n, device="cuda")) if dtype == "fp8" else (None, None)
    y = torch.empty(m, n, dtype=to, device="cuda")
    B.linear(ctx, m, n, k, dtype, torch.zeros(m, k, device="cuda").to(el), torch.zeros(k, n, device="cuda").to(el), y,
             a_scale=ones[0], b_scale=ones[1], bias=x.cuda(), act=act, stream=torch.cuda.current_stream())
    got = y.double().cpu()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()}; worst error over bound "
                           f"{float(((got - want).abs() / bound).nan_to_num(0).max()):.3g} at x = "
                           f"{float(z[((got - want).abs() / bound).nan_to_num(0).amax(0).argmax()])}")


def _exact_product(m, n, k, dtype, seed):
    """Operands of which every product and sum is a multiple of 1/4 below 2^17, so fp32 (and the fp8 instruction, which cuts
    products to 2^-13 of the largest of eight: 4) holds them exactly; none is zero, so that none can be lost unseen."""
    g = torch.Generator().manual_seed(seed)
    values = torch.tensor([0.5, 1.0, 2.0, -0.5, -1.0, -2.0])
    pick = lambda *s: values[torch.randint(0, 6, s, generator=g)]  # noqa: E731
    a, b = pick(m, k), pick(k, n)
    want = (a.cuda().double() @ b.cuda().double()).cpu()
    if dtype == "bf16":
        return a.bfloat16().cuda(), b.bfloat16().cuda(), None, None, want
    sa, sb = (2.0 ** torch.randint(-3, 4, (x,), generator=g) for x in (m, n))
    return a.to(FP8).cuda(), b.to(FP8).cuda(), sa.cuda(), sb.cuda(), want * sa.double()[:, None] * sb.double()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("m,n,k", [(1, 256, 4096), (3, 128, 1040), (16, 2048, 2048), (32, 1024, 8192), (33, 384, 1008), (64, 2048, 8192),
                                   (100, 1040, 1008), (128, 512, 8192), (257, 1008, 4096), (300, 1808, 1040), (1024, 1024, 2048),
                                   (2100, 2064, 1040)])
def test_no_product_is_lost(ctx, dtype, m, n, k):
    a, b, sa, sb, want = _exact_product(m, n, k, dtype, m + n + k)
    y = torch.empty(m, n, device="cuda")
    B.linear(ctx, m, n, k, dtype, a, b, y, a_scale=sa, b_scale=sb, stream=torch.cuda.current_stream())
    assert torch.equal(y.double().cpu(), want)


@pytest.mark.parametrize("tile", [(256, 256), (256, 224), (128, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("parts", [1, 3, 16])
def test_no_product_is_lost_in_a_tile(ctx, dtype, tile, parts):
    m, n, k = 321, 528, 2064
    a, b, sa, sb, want = _exact_product(m, n, k, dtype, parts)
    y = torch.empty(m, n, device="cuda")
    B.agg_ctx_set_tile(ctx, *tile)
    B.agg_ctx_set_split(ctx, parts)
    try:
        B.linear(ctx, m, n, k, dtype, a, b, y, a_scale=sa, b_scale=sb, stream=torch.cuda.current_stream())
        assert torch.equal(y.double().cpu(), want)
    finally:
        B.agg_ctx_set_tile(ctx)
        B.agg_ctx_set_split(ctx)
