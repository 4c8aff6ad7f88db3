"""The paged cache and the attention over it on the GPU against plain implementations in 64 bits.

Tolerances, derived from the formats: a bfloat16 output is within half a unit, 2^-8 of its value, of the fp32
result it rounds; a sum of n fp32 terms is within n * 2^-23 of the sum of their sizes; e4m3 has three
fraction bits, half a unit is 2^-4 of the value and 2^-10 below its normal range; the exponential, the logarithm and
a few products are within 2^-20. The weights of the attention enter the matrix units as two bf16 parts: within 2^-16
of themselves."""

import math

import pytest
import torch

from allgather_gemm_persistent_amd import binding as B

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8
EPS32 = 2.0 ** -23
FINE = 2.0 ** -20
BF16, FP8, F32, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32


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
    same = (got == ref) | (got.isnan() & ref.isnan())      # (infinities, and what is no number on both sides)
    bad = ~((err <= bound) | same)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds; worst error over bound "
                           f"{float((err / bound)[~same].nan_to_num(math.inf).max()):.3g}")


class _Paged:
    """Caches of sequences of given lengths, on the host in 64 bits and on the device. What no sequence holds is NaN."""

    def __init__(self, lengths, kv_heads, dim, page=16, dtype="bf16", heads_first=False, seed=0, spare=3, room=None):
        g = self.g = _gen(seed)
        self.lengths, self.h, self.d, self.page, self.dtype = lengths, kv_heads, dim, page, dtype
        held = [-(-n // page) for n in lengths]
        self.width = max(max(held), 1) if room is None else room
        self.pages = sum(held) + spare
        order = torch.randperm(self.pages, generator=g)
        self.table = torch.full((len(lengths), self.width), -1, dtype=I32)
        at = 0
        for i, n in enumerate(held):
            self.table[i, :n] = order[at:at + n].int()
            at += n
        used = torch.zeros(self.pages, page, dtype=torch.bool)
        for i, n in enumerate(lengths):
            t = torch.arange(n)
            used[self.table[i].long()[t // page], t % page] = True
        self.k, self.k_scale = self._pool(used, heads_first)
        self.v, self.v_scale = self._pool(used, heads_first)
        self.cache = B.KvCache(self.k, self.v, self.k_scale, self.v_scale)
        self.dev_table = self.table.cuda()

    def _pool(self, used, heads_first):
        x = torch.randn(self.pages, self.page, self.h, self.d, generator=self.g)
        scale = None
        if self.dtype == "fp8":
            x = (x * 100).clamp(-448, 448).to(FP8)
            x.view(torch.uint8)[~used] = 0x7F
            scale = 0.01 * (0.5 + torch.rand(self.pages, self.h, self.page, generator=self.g))
            scale.transpose(1, 2)[~used] = math.nan
            scale = scale.cuda()
        else:
            x = x.bfloat16()
            x[~used] = math.nan
        x = x.cuda()
        if heads_first:
            x = x.transpose(1, 2).contiguous().transpose(1, 2)
        return x, scale

    def rows(self, name, seq, n=None):
        """The first n rows of a sequence in 64 bits: n x heads x dim."""
        n = self.lengths[seq] if n is None else n
        p = self.table[seq, :-(-n // self.page)].long().cuda()
        x = getattr(self, name)[p].double()
        s = getattr(self, name + "_scale")
        if s is not None:
            x = x * s[p].double().transpose(1, 2)[..., None]
        return x.reshape(-1, self.h, self.d)[:n].cpu()


def _attention(q, k, v, scale, first=0):
    """q: heads x d, k, v: n x kv heads x d, 64 bits: out, lse, and the error that fp32 steps may bring."""
    n, h, d = k.shape
    group = q.shape[0] // h
    if n <= first:
        return torch.zeros(q.shape, dtype=torch.float64), torch.full((q.shape[0],), -math.inf, dtype=torch.float64), \
            torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape[0], dtype=torch.float64)
    k, v = k[first:].transpose(0, 1), v[first:].transpose(0, 1)
    qq = q.reshape(h, group, d)
    x = scale * (qq @ k.transpose(1, 2).contiguous())
    size = abs(scale) * (qq.abs() @ k.abs().transpose(1, 2).contiguous())
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    p = p / total
    out = p @ v
    # an error of x moves the weights by as much of themselves, and so their sum; then the weights' two parts and
    # the sums over the tokens
    dx = (d * EPS32 * size).amax(-1) + FINE * (1 + x.abs().amax(-1))
    err = (p @ v.abs()) * (2 * dx + 2.0 ** -15 + 2 * (n - first) * EPS32 + FINE)[..., None]
    lse = (top + torch.log(total))[..., 0]
    return (out.reshape(q.shape), lse.reshape(-1), err.reshape(q.shape),
            (dx + (n - first) * EPS32 + FINE * (1 + lse.abs())).reshape(-1))


def _check(p, ctx, q_heads, lens=None, row_seq=None, window=0, out="bf16", lse=True, scale=None, q=None, stream=None,
           table=None):
    lens = list(p.lengths) if lens is None else lens
    seqs = list(range(len(lens))) if row_seq is None else row_seq
    rows, d = len(lens), p.d
    scale = d ** -0.5 if scale is None else scale
    q = (1.5 * torch.randn(rows, q_heads * d, generator=p.g)).bfloat16() if q is None else q
    y = torch.full((rows, q_heads * d), 7.0, dtype=BF16 if out == "bf16" else F32, device="cuda")
    sums = torch.full((rows, q_heads), 7.0, device="cuda") if lse else None
    B.paged_attn(ctx, p.cache, rows, q.cuda(), torch.tensor(lens, dtype=I32, device="cuda"),
                 p.dev_table if table is None else table, y, scale=scale,
                 row_seq=None if row_seq is None else torch.tensor(row_seq, dtype=I32, device="cuda"), window=window,
                 lse=sums, stream=stream or torch.cuda.current_stream())
    torch.cuda.synchronize()
    for r in range(rows):
        n, s = lens[r], seqs[r]
        n = 0 if not 0 <= s < len(p.lengths) else max(0, min(n, p.width * p.page))
        k, v = (p.rows(x, s, n) if n else torch.zeros(0, p.h, d, dtype=torch.float64) for x in "kv")
        want, want_lse, err, err_lse = _attention(q[r].double().reshape(q_heads, d), k, v, scale,
                                                  max(0, n - window) if window else 0)
        bound = err + (HALF_BF16 * (want.abs() + err) if out == "bf16" else EPS32 * want.abs())
        _within(y[r].reshape(q_heads, d), want, bound, f"row {r} of {n} tokens")
        if lse:
            _within(sums[r], want_lse, err_lse, f"lse of row {r} of {n} tokens")
    return y, sums


# ------------------------------------------------------------------------------ attention

LENGTHS = [17, 0, 1, 2, 15, 16, 31, 32, 33, 48, 100, 257, 700]


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 240, 256])
@pytest.mark.parametrize("heads", [(1, 1), (4, 2), (24, 3)])
def test_attn_widths(ctx, dtype, dim, heads):
    p = _Paged(LENGTHS, heads[1], dim, 16, dtype, dim % 32 == 0, seed=dim + heads[0])
    _check(p, ctx, heads[0], out="fp32" if dim % 64 else "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("dim", [64, 128, 192])
@pytest.mark.parametrize("group", [2, 3, 7, 8, 15, 16, 17, 31, 32, 33, 48, 64, 65, 100, 130])
def test_attn_groups(ctx, dtype, dim, group):
    p = _Paged([5, 300, 64], 2, dim, 32, dtype, group % 2 == 0, seed=group)
    _check(p, ctx, 2 * group, out="fp32")


@pytest.mark.parametrize("page", [16, 32, 48, 64, 112, 256, 4096])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("heads_first", [False, True])
def test_attn_pages(ctx, page, dtype, heads_first):
    p = _Paged([1, 47, 48, 49, 500, 1025, 63], 2, 64, page, dtype, heads_first, seed=page)
    _check(p, ctx, 8)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 32, 33, 100, 256, 1000, 1 << 40])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_attn_window(ctx, window, dtype):
    """What lies before the window is NaN, as is what follows the sequences."""
    p = _Paged([0, 1, 16, 17, 40, 333, 1000], 2, 128, 32, dtype, seed=window % 97)
    for i, n in enumerate(p.lengths):
        t = torch.arange(max(0, n - window))
        at = p.table[i].long()[t // p.page].cuda(), (t % p.page).cuda()
        for x, s in ((p.k, p.k_scale), (p.v, p.v_scale)):
            if dtype == "fp8":
                x.view(torch.uint8)[at] = 0x7F
                s.transpose(1, 2)[at] = math.nan
            else:
                x[at] = math.nan
    rows = p.rows
    p.rows = lambda *a: rows(*a).nan_to_num(0.0)           # (the reference leaves them out by their place)
    _check(p, ctx, 8, window=window, out="fp32")


@pytest.mark.parametrize("n", [4097, 20000, 70001])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("rows", [1, 3])
def test_attn_long(ctx, n, dtype, rows):
    p = _Paged([n, 5, 900][:rows], 2, 64, 64, dtype, seed=n)
    _check(p, ctx, 6, out="fp32")


@pytest.mark.parametrize("n", [3, 64, 1000, 40000])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_attn_takes_every_token_once(ctx, n, dtype):
    """Equal weights; channel c of the values is 1 at one token and 0 elsewhere: out is 1 / n, or 0 if the token is lost."""
    p = _Paged([n], 1, 128, 48, dtype, seed=n)
    p.v.copy_(torch.zeros(p.v.shape).to(p.v.dtype))
    if dtype == "fp8":
        p.k_scale.fill_(1)
        p.v_scale.fill_(1)
    marked = torch.unique(torch.cat([torch.linspace(0, n - 1, 100).long(), torch.tensor([0, 1, n - 1, n - 2]).clamp(0, n - 1)]))[:128]
    for c, t in enumerate(marked.tolist()):
        p.v[int(p.table[0, t // p.page]), t % p.page, 0, c] = 1.0
    q = torch.zeros(1, 4 * 128, dtype=BF16)
    y, lse = _check(p, ctx, 4, q=q, out="fp32")
    want = torch.zeros(128)
    want[:len(marked)] = 1.0 / n
    _within(y.reshape(4, 128), want.expand(4, 128), want * FINE * 8, "marked tokens")
    _within(lse, torch.full((1, 4), math.log(n)), torch.tensor(FINE * 16), "lse")


def test_attn_many_rows(ctx):
    """More rows than a workgroup has threads, most of them short, one long; and rows in another order."""
    g = _gen(3)
    lengths = [int(x) for x in torch.randint(0, 40, (700,), generator=g)]
    lengths[123] = 5000
    p = _Paged(lengths, 2, 64, 16, "bf16", seed=4)
    order = torch.randperm(700, generator=g).tolist()
    _check(p, ctx, 4, lens=[lengths[s] for s in order], row_seq=order)
    _check(p, ctx, 4)


@pytest.mark.parametrize("rows", [63, 64, 65, 255, 256, 257, 513])
def test_attn_row_counts(ctx, rows):
    """Row counts around those at which the work is divided in other ways; a few long rows among them."""
    g = _gen(rows)
    lengths = [int(x) for x in torch.randint(0, 20, (rows,), generator=g)]
    for i in (0, rows // 2, rows - 1):
        lengths[i] = 1500
    p = _Paged(lengths, 1, 64, 16, "bf16", seed=rows)
    _check(p, ctx, 2)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("lengths,heads,dim", [([256] * 8, 8, 64), ([256] * 7 + [257], 8, 64), ([16384], 1, 64), ([16385], 1, 64),
                                               ([4096, 1], 4, 64), ([4064, 0], 4, 64), ([1025, 3], 1, 128), ([256, 31, 0], 2, 128),
                                               ([257, 31, 0], 2, 128), ([8192], 1, 256), ([8193], 1, 256), ([0] * 64, 2, 64)])
def test_attn_few_tiles(ctx, dtype, lengths, heads, dim):
    """As many tiles of 32 tokens as there are workgroups (two a compute unit up to 128 channels, one beyond), one more, and
    rows around those that are not split."""
    p = _Paged(lengths, heads, dim, 64, dtype, seed=sum(lengths))
    _check(p, ctx, 2 * heads)


def test_attn_more_rows_than_a_launch(ctx):
    """A table so wide that its rows go in several launches, sequences by the rows' numbers."""
    p = _Paged([20] * 4 + [5000], 1, 16, 4096, "bf16", seed=6)
    rows, width = 600, 65536
    table = torch.full((rows, width), -1, dtype=I32, device="cuda")
    seqs = [i % 4 for i in range(rows)]
    seqs[400] = 4
    table[:, :2] = p.dev_table[torch.tensor(seqs)]
    lens = torch.tensor([1 + i % 20 for i in range(rows)], dtype=I32)
    lens[400] = 4999
    q = torch.randn(rows, 32, generator=p.g).bfloat16()
    y, lse = torch.full((rows, 32), 7.0, device="cuda"), torch.full((rows, 2), 7.0, device="cuda")
    B.paged_attn(ctx, p.cache, rows, q.cuda(), lens.cuda(), table, y, scale=0.25, lse=lse, stream=torch.cuda.current_stream())
    for r in range(rows):
        n = int(lens[r])
        want, want_lse, err, err_lse = _attention(q[r].double().reshape(2, 16), p.rows("k", seqs[r], n), p.rows("v", seqs[r], n), 0.25)
        _within(y[r].reshape(2, 16), want, err + EPS32 * want.abs(), f"row {r}")
        _within(lse[r], want_lse, err_lse, f"lse {r}")


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("rows,n", [(1, 300), (1, 3000), (1, 40000), (30, 900), (200, 300)])
def test_attn_called_again_and_again(ctx, dtype, rows, n):
    """Calls behind each other on one stream, of other lengths each time, leave the workspace's counters as they found
    them: the first call's result comes back to the bit."""
    p = _Paged([max(1, n - 7 * i) for i in range(rows)], 2, 64, 16, dtype, seed=rows)
    q = torch.randn(rows, 8 * 64, generator=p.g).bfloat16().cuda()
    st = torch.cuda.current_stream()
    y = [torch.zeros(rows, 8 * 64, device="cuda") for _ in range(8)]
    for i, out in enumerate(y):
        lens = torch.tensor([max(0, x - (37 * i if 0 < i < 7 else 0)) for x in p.lengths], dtype=I32, device="cuda")
        B.paged_attn(ctx, p.cache, rows, q, lens, p.dev_table, out, scale=0.125, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(y[0], y[7]) and not torch.equal(y[0], y[3])


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("heads_first,dim", [(True, 128), (False, 128), (True, 64), (False, 256)])
def test_attn_of_a_large_cache(ctx, dtype, heads_first, dim):
    """A pool beyond the size from which its lines are read past the last level, most of it free."""
    p = _Paged([700, 1, 0, 333], 2, dim, 64, dtype, heads_first, seed=dim, spare=(600000 if dtype == "bf16" else 1200000) // dim)
    _check(p, ctx, 8, out="fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_attn_rows_of_one_sequence(ctx, dtype):
    """Several new tokens of a sequence, each up to its own place."""
    p = _Paged([130, 70], 2, 128, 16, dtype, seed=9)
    _check(p, ctx, 8, lens=[127, 128, 129, 130, 1, 0, 70, 69], row_seq=[0, 0, 0, 0, 0, 1, 1, 1])


def test_attn_refused_places(ctx):
    """Lengths past the table's room are cut, negative ones and unknown sequences are empty rows; the tokens of a page
    that is none are left out."""
    p = _Paged([64, 64, 64, 64], 2, 64, 16, "bf16", seed=1)
    _check(p, ctx, 4, lens=[1000, -1, -(1 << 31), 64, 5, (1 << 31) - 1], row_seq=[0, 1, 2, -1, 4, 3])
    rows = p.rows
    table = p.table.clone()
    table[0, 1], table[1, 0], table[2] = -1, p.pages, torch.tensor([-(1 << 31), (1 << 31) - 1, -5, p.pages + 3])
    keep = {0: [t for t in range(64) if t // 16 != 1], 1: list(range(16, 64)), 2: [], 3: list(range(64))}
    q = torch.randn(4, 256, generator=p.g).bfloat16()
    y, lse = torch.full((4, 256), 7.0, device="cuda"), torch.full((4, 4), 7.0, device="cuda")
    B.paged_attn(ctx, p.cache, 4, q.cuda(), torch.full((4,), 64, dtype=I32, device="cuda"), table.cuda(), y, scale=0.125,
                 lse=lse, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    for r in range(4):
        k, v = rows("k", r)[keep[r]], rows("v", r)[keep[r]]
        want, want_lse, err, err_lse = _attention(q[r].double().reshape(4, 64), k, v, 0.125)
        _within(y[r].reshape(4, 64), want, err + EPS32 * want.abs(), f"row {r}")
        _within(lse[r], want_lse, err_lse, f"lse {r}")


def test_attn_without_anything(ctx):
    """No rows, no sequences, no pages."""
    st = torch.cuda.current_stream()
    p = _Paged([20], 1, 64, 16, "bf16")
    empty = torch.zeros(0, 128, dtype=BF16, device="cuda")
    lens = torch.full((3,), 20, dtype=I32, device="cuda")
    B.paged_attn(ctx, p.cache, 0, empty, lens, p.dev_table, empty, scale=1.0, stream=st)
    q = torch.ones(3, 128, dtype=BF16, device="cuda")
    none = B.KvCache(p.k[:0], p.v[:0])
    for cache, table in ((p.cache, p.dev_table[:0]), (p.cache, p.dev_table[:, :0]), (none, p.dev_table)):
        y, lse = torch.full((3, 128), 7.0, dtype=BF16, device="cuda"), torch.zeros(3, 2, device="cuda")
        B.paged_attn(ctx, cache, 3, q, lens, table, y, scale=1.0, lse=lse, row_seq=torch.zeros(3, dtype=I32, device="cuda"),
                     stream=st)
        assert bool((y == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("scale", [0.0, -0.3, 8.0, 1e30])
def test_attn_scales(ctx, scale):
    """Equal weights, turned signs, weights of one token almost alone, and scores far beyond the exponential's range."""
    p = _Paged([50, 400, 1], 2, 64, 16, "bf16", seed=2)
    if scale < 1e6:
        _check(p, ctx, 4, scale=scale, out="fp32")
        return
    q = torch.zeros(3, 4 * 64).bfloat16()
    q[:, ::64] = 1.0                                       # the score is channel 0: the largest takes all
    y = torch.zeros(3, 256, device="cuda")
    B.paged_attn(ctx, p.cache, 3, q.cuda(), torch.tensor([50, 400, 1], dtype=I32, device="cuda"), p.dev_table, y,
                 scale=scale, stream=torch.cuda.current_stream())
    for r in range(3):
        k, v = p.rows("k", r), p.rows("v", r)
        x = k[:, :, 0]
        best = x == x.amax(0, keepdim=True)                # (several where bf16 makes them equal)
        want = (best[..., None] * v).sum(0) / best.sum(0)[:, None]
        _within(y[r].reshape(2, 2, 64), want[:, None].expand(2, 2, 64), want.abs()[:, None] * 2.0 ** -15 + 1e-6, f"row {r}")


def test_attn_keys_that_are_not_finite(ctx):
    """A score of -inf leaves its token out; a NaN in a key that counts, or an infinite score, makes its row NaN; rows of
    other sequences are untouched."""
    p = _Paged([40, 40, 40, 40], 1, 64, 16, "bf16", seed=6)
    q = torch.zeros(4, 64)
    q[:, 0] = 1.0
    for s, x in ((0, -math.inf), (1, math.nan), (2, math.inf)):
        p.k[int(p.table[s, 1]), 3, 0, 0] = x
    y, lse = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 1, device="cuda")
    B.paged_attn(ctx, p.cache, 4, q.bfloat16().cuda(), torch.full((4,), 40, dtype=I32, device="cuda"), p.dev_table, y,
                 scale=1.0, lse=lse, stream=torch.cuda.current_stream())
    y, lse = y.cpu(), lse.cpu()
    assert y[1].isnan().all() and y[2].isnan().all() and y[0].isfinite().all() and y[3].isfinite().all()
    for s in (0, 3):
        keep = [t for t in range(40) if not (s == 0 and t == 19)]
        want, want_lse, err, err_lse = _attention(q[s:s + 1].double(), p.rows("k", s)[keep], p.rows("v", s)[keep], 1.0)
        _within(y[s:s + 1], want, err + EPS32 * want.abs(), f"sequence {s}")
        _within(lse[s], want_lse, err_lse, f"lse {s}")


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_attn_parts_join(ctx, dtype):
    """Parts of a sequence, joined by their lse, are the whole."""
    p = _Paged([640], 2, 128, 16, dtype, seed=12)
    q = torch.randn(1, 8 * 128, generator=p.g).bfloat16()
    whole, lse = _check(p, ctx, 8, q=q, out="fp32")
    parts = []
    for first, count in ((0, 10), (10, 13), (23, 17)):     # pages
        y, s = torch.zeros(1, 1024, device="cuda"), torch.zeros(1, 8, device="cuda")
        B.paged_attn(ctx, p.cache, 1, q.cuda(), torch.tensor([count * 16], dtype=I32, device="cuda"),
                     p.dev_table[:, first:first + count], y, scale=128 ** -0.5, lse=s, stream=torch.cuda.current_stream())
        parts.append((y.double().cpu().reshape(8, 128), s.double().cpu().reshape(8, 1)))
    w = torch.softmax(torch.cat([s for _, s in parts], 1), 1)
    joined = sum(w[:, i:i + 1] * y for i, (y, _) in enumerate(parts))
    _within(whole.reshape(8, 128), joined, joined.abs().amax() * 2.0 ** -12, "joined")


def test_attn_strides(ctx):
    """Queries and results inside wider rows, a table inside a wider one; what surrounds them stays."""
    p = _Paged([33, 100, 7], 2, 64, 16, "bf16", seed=8)
    wide_q = torch.randn(3, 256 + 64, generator=p.g).bfloat16().cuda()
    wide_y = torch.full((3, 256 + 96), 7.0, dtype=BF16, device="cuda")
    wide_t = torch.full((3, p.width + 5), 1 << 30, dtype=I32, device="cuda")
    wide_t[:, 2:2 + p.width] = p.dev_table
    lens = torch.tensor(p.lengths, dtype=I32, device="cuda")
    y = torch.zeros(3, 256, dtype=BF16, device="cuda")
    st = torch.cuda.current_stream()
    B.paged_attn(ctx, p.cache, 3, wide_q[:, 8:264], lens, wide_t[:, 2:2 + p.width], wide_y[:, 32:288], scale=0.125, stream=st)
    B.paged_attn(ctx, p.cache, 3, wide_q[:, 8:264].contiguous(), lens, p.dev_table, y, scale=0.125, stream=st)
    assert torch.equal(wide_y[:, 32:288], y)
    assert bool((wide_y[:, :32] == 7).all()) and bool((wide_y[:, 288:] == 7).all())
    _check(p, ctx, 4)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_attn_and_write_past_32_bits(ctx, dtype):
    """Pages whose elements' numbers pass 2^32."""
    pages, h, d = 270000, 8, 128
    t = BF16 if dtype == "bf16" else FP8
    k, v = (torch.empty(pages, 16, h, d, dtype=t, device="cuda") for _ in range(2))
    scales = [torch.empty(pages, h, 16, device="cuda") for _ in range(2)] if dtype == "fp8" else [None, None]
    cache = B.KvCache(k, v, *scales)
    far = [pages - 1, 5, pages - 7, 262144 + 11]
    table = torch.tensor([far], dtype=I32, device="cuda")
    g = _gen(5)
    rows = [torch.randn(60, h * d, generator=g).bfloat16().cuda() for _ in range(2)]
    pos = torch.arange(60, dtype=I32, device="cuda")
    seq = torch.zeros(60, dtype=I32, device="cuda")
    st = torch.cuda.current_stream()
    B.kv_write(ctx, cache, 60, *rows, pos, table, token_seq=seq, stream=st)
    back = [torch.empty(60, h * d, device="cuda") for _ in range(2)]
    B.kv_read(ctx, cache, 60, pos, table, *back, token_seq=seq, stream=st)
    held = [x[far].reshape(64, h, d)[:60].double().cpu() for x in (k, v)]
    if dtype == "fp8":
        held = [x * s[far].transpose(1, 2).reshape(64, h)[:60].double().cpu()[..., None] for x, s in zip(held, scales)]
    for got, want, first in zip(back, held, rows):
        _within(got.reshape(60, h, d), want, want.abs() * EPS32, "read")
        _within(got, first.double().cpu(), first.double().cpu().abs() * 2.0 ** -4 + (1e-2 if dtype == "fp8" else 0), "written")
    q = torch.randn(1, 8 * 128, generator=g).bfloat16()
    y = torch.zeros(1, 8 * 128, device="cuda")
    B.paged_attn(ctx, cache, 1, q.cuda(), torch.tensor([60], dtype=I32, device="cuda"), table, y, scale=d ** -0.5, stream=st)
    want, _, err, _ = _attention(q.double().reshape(8, 128), *held, d ** -0.5)
    _within(y.reshape(8, 128), want, err + EPS32 * want.abs(), "attention")


# ------------------------------------------------------------------------------ write and read

def _angles(rows, dim, g):
    a = torch.rand(rows, dim // 2, generator=g, dtype=torch.float64) * 6.28
    return torch.cat([a.cos(), a.sin()], 1).float()


def _rotate(x, table, pairs):
    """x: tokens x heads x d in 64 bits, table: tokens x rope_dim."""
    r = table.shape[1]
    cs, sn = table[:, None, :r // 2].double(), table[:, None, r // 2:].double()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if pairs else (x[..., :r // 2], x[..., r // 2:r])
    y = x.clone()
    size = x.abs()
    u, w = a * cs - b * sn, b * cs + a * sn
    if pairs:
        y[..., 0:r:2], y[..., 1:r:2] = u, w
        size[..., 0:r:2] = size[..., 1:r:2] = a.abs() + b.abs()
    else:
        y[..., :r // 2], y[..., r // 2:r] = u, w
        size[..., :r // 2] = size[..., r // 2:r] = a.abs() + b.abs()
    return y, size * 4 * EPS32


def _check_row8(q, scale, y, err):
    """q (fp8) is a nearest e4m3 of y / scale, up to fp32 steps; scale is the rows' max / 448."""
    top = y.abs().amax(-1) / 448
    want_scale = torch.where(top > 0, top, 1.0)
    _within(scale, want_scale, want_scale * FINE + err.amax(-1) / 448, "scales")
    s = scale.double().cpu()[..., None]
    want = (y / s).clamp(-448, 448)
    _within(q.float(), want, torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10)) + want.abs() * FINE + err / s, "fp8")


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("dim,rope", [(16, 16), (32, 16), (64, 64), (64, 0), (80, 80), (96, 32), (112, 112), (128, 128), (128, 64),
                                      (144, 144), (192, 64), (256, 256)])
@pytest.mark.parametrize("pairs", [False, True])
def test_write_and_read(ctx, dtype, dim, rope, pairs):
    """Tokens of several sequences, some without a place: the cache is right where one is and untouched elsewhere."""
    q_heads, h, page = 6, 3, 32
    p = _Paged([70, 0, 33, 160], h, dim, page, dtype, dim % 32 == 0, seed=dim + rope)
    g = p.g
    tokens = 41
    seq, pos = [], []
    for t in range(tokens):
        s = [0, 2, 3][t % 3]
        seq.append(s)
        pos.append((t // 3) * 2 + (1 if s == 2 else 40 if s == 3 else 0))
    for t, (s, x) in enumerate([(0, -1), (-1, 3), (4, 3), (0, p.width * page), (1, 0), (0, 96), (2, -(1 << 31)), (3, (1 << 31) - 1)]):
        seq[5 * t], pos[5 * t] = s, x                      # (sequence 1, and 0 past its third page, have no page there)
    left_out = {5 * t for t in range(8)}
    rows_limit = 125
    angles = _angles(rows_limit, rope, g) if rope else None
    wide = torch.randn(tokens, (q_heads + 2 * h) * dim + 8, generator=g)
    wide[3, q_heads * dim:(q_heads + 1) * dim] = 0.0       # a key of zeros
    wide = wide.bfloat16().cuda()
    q, k, v = wide[:, :q_heads * dim], wide[:, q_heads * dim:(q_heads + h) * dim], wide[:, (q_heads + h) * dim:-8]
    q_out = torch.full((tokens, q_heads * dim + 16), 7.0, dtype=BF16, device="cuda")
    before = [x.clone() if x is not None else None for x in (p.k, p.v, p.k_scale, p.v_scale)]
    st = torch.cuda.current_stream()
    dseq, dpos = torch.tensor(seq, dtype=I32, device="cuda"), torch.tensor(pos, dtype=I32, device="cuda")
    B.kv_write(ctx, p.cache, tokens, k, v, dpos, p.dev_table, token_seq=dseq, q=q, q_out=q_out[:, :q_heads * dim],
               rope=None if angles is None else angles.cuda(), rope_pairs=pairs, stream=st)
    torch.cuda.synchronize()
    good = [t for t in range(tokens) if t not in left_out and not (rope and pos[t] >= rows_limit)]
    assert len({(seq[t], pos[t]) for t in good}) == len(good) and len(good) > 25
    at = [int(p.table[seq[t], pos[t] // page]) for t in good], [pos[t] % page for t in good]
    turn = angles[[pos[t] for t in good]] if rope else torch.zeros(len(good), 0)
    # queries
    x = q.double().cpu()[good].reshape(len(good), q_heads, dim)
    want, err = _rotate(x, turn, pairs)
    _within(q_out[good][:, :q_heads * dim].reshape(want.shape), want, err + HALF_BF16 * (want.abs() + err), "queries")
    rest = torch.ones(tokens, dtype=torch.bool)
    rest[good] = False
    assert bool((q_out[rest.cuda()] == 7).all()) and bool((q_out[:, q_heads * dim:] == 7).all())
    # the cache
    for name, src, turns in (("k", k, turn), ("v", v, turn[:, :0])):
        want, err = _rotate(src.double().cpu()[good].reshape(len(good), h, dim), turns, pairs)
        pool, scale = getattr(p, name), getattr(p, name + "_scale")
        if dtype == "bf16":
            _within(pool[at], want, err + HALF_BF16 * (want.abs() + err), name)
        else:
            _check_row8(pool[at], scale.transpose(1, 2)[at], want, err)
    written = torch.zeros(p.pages, page, dtype=torch.bool, device="cuda")
    written[at] = True
    bits = torch.int16 if dtype == "bf16" else torch.uint8
    for now, was in zip((p.k, p.v), before):
        assert torch.equal(now.view(bits)[~written], was.view(bits)[~written])
    for now, was in zip((p.k_scale, p.v_scale), before[2:]):
        if now is not None:
            assert torch.equal(now.transpose(1, 2)[~written].view(I32), was.transpose(1, 2)[~written].view(I32))
    # and back, tokens without a place as zeros, some twice, in both types
    for out in (BF16, F32):
        back = [torch.full((tokens + 2, h * dim + 8), 7.0, dtype=out, device="cuda") for _ in range(2)]
        B.kv_read(ctx, p.cache, tokens, dpos, p.dev_table, *(b[:tokens, :h * dim] for b in back), token_seq=dseq, stream=st)
        for b, pool, scale in zip(back, (p.k, p.v), (p.k_scale, p.v_scale)):
            x = pool[at].float()
            x = x if scale is None else x * scale.transpose(1, 2)[at][..., None]
            assert torch.equal(b[good, :h * dim], x.to(out).reshape(len(good), -1))
            assert bool((b[tokens:] == 7).all()) and bool((b[:, h * dim:] == 7).all())
            zero = [t for t in sorted(left_out)]
            assert bool((b[zero][:, :h * dim] == 0).all())


def test_write_in_place_and_without_queries(ctx):
    p = _Paged([64, 64], 2, 64, 16, "bf16", seed=21)
    angles = _angles(64, 64, p.g).cuda()
    rows = torch.randn(2, 8 * 64, generator=p.g).bfloat16().cuda()
    q, k, v = rows[:, :256], rows[:, 256:384], rows[:, 384:]
    pos = torch.tensor([5, 63], dtype=I32, device="cuda")
    out = torch.zeros(2, 256, dtype=BF16, device="cuda")
    st = torch.cuda.current_stream()
    B.kv_write(ctx, p.cache, 2, k, v, pos, p.dev_table, q=q, q_out=out, rope=angles, stream=st)
    kept = p.k.clone()
    B.kv_write(ctx, p.cache, 2, k, v, pos, p.dev_table, rope=angles, stream=st)
    assert torch.equal(p.k.view(torch.int16), kept.view(torch.int16))
    B.kv_write(ctx, p.cache, 2, k, v, pos, p.dev_table, q=q, q_out=q, rope=angles, stream=st)
    assert torch.equal(q, out)


def test_write_rows_that_are_not_numbers(ctx):
    """In 8 bits: a row with a NaN keeps it and has scale 1 (the others saturate), an infinite row is 0 and NaN over
    an infinite scale; subnormal and zero rows come back within their format."""
    p = _Paged([16], 4, 64, 16, "fp8", seed=30)
    k = torch.randn(4, 4 * 64)
    v = torch.zeros(4, 4 * 64)
    k[0, 3], k[0, 5] = math.nan, 1000.0
    k[1, 7] = math.inf
    k[2] *= 1e-38
    k[3] = 0.0
    k = k.bfloat16()
    B.kv_write(ctx, p.cache, 4, k.cuda(), v.bfloat16().cuda(), torch.arange(4, dtype=I32, device="cuda"), p.dev_table,
               token_seq=torch.zeros(4, dtype=I32, device="cuda"), stream=torch.cuda.current_stream())
    page = int(p.table[0, 0])
    got, scale = p.k[page].float().cpu(), p.k_scale[page].cpu()
    assert scale[0, 0] == 1 and got[0, 0, 3].isnan() and got[0, 0, 5] == 448 and int(got[0, 0].isnan().sum()) == 1
    assert scale[0, 1] == math.inf and got[1, 0, 7].isnan() and bool((got[1, 0, :7] == 0).all())
    assert bool((scale[:, 3] == 1).all()) and bool((got[3] == 0).all())
    x = k[2].double().reshape(4, 64)
    back = got[2].double() * scale[:, 2].double()[:, None]
    # (a scale that is a multiple m of 2^-149 is off by up to 1 / 2m of itself, which clamps or shrinks the row)
    _within(back, x, x.abs() * 2.0 ** -4 + scale[:, 2].double()[:, None] * 2.0 ** -10 + 448 * 2.0 ** -150, "subnormal")
    assert bool((p.v[page].float()[:4] == 0).all()) and bool((p.v_scale[page][:, :4] == 1).all())


def test_write_rows_as_the_division_has_them(ctx):
    """In 8 bits the elements are the nearest e4m3 of x / scale, the scale of max|x| / 448, both fp32 divisions: to the bit (a
    product with the reciprocal puts some of half a million on the other side of a tie)."""
    p = _Paged([512], 8, 128, 16, "fp8", seed=33)
    x = (torch.randn(512, 8, 128, generator=p.g) * torch.logspace(-30, 30, 512)[:, None, None]).bfloat16()
    rows = x.reshape(512, -1).cuda()
    B.kv_write(ctx, p.cache, 512, rows, rows, torch.arange(512, dtype=I32, device="cuda"), p.dev_table,
               token_seq=torch.zeros(512, dtype=I32, device="cuda"), stream=torch.cuda.current_stream())
    at = p.table[0].long().cuda()
    want_scale = x.float().abs().amax(-1) / torch.tensor(448.0)
    want = (x.float() / want_scale[..., None]).to(FP8)
    for pool, scale in ((p.k, p.k_scale), (p.v, p.v_scale)):
        assert torch.equal(scale[at].cpu().transpose(1, 2).reshape(512, 8), want_scale)
        assert torch.equal(pool[at].view(torch.uint8).cpu().reshape(512, 8, 128), want.view(torch.uint8))


def test_write_and_read_beyond_a_launch(ctx):
    """More rows than one launch counts: tokens of 1024 heads."""
    tokens, h, d = (1 << 19) + 9, 1024, 16
    p = _Paged([64], h, d, 16, "bf16", seed=31)
    pos = torch.full((tokens,), -1, dtype=I32, device="cuda")
    pos[-20:] = torch.arange(20, dtype=I32, device="cuda")
    pos[3] = 40
    seq = torch.zeros(tokens, dtype=I32, device="cuda")
    x = torch.full((tokens, h * d), 3.0, dtype=BF16, device="cuda")
    last = torch.randn(20, h * d, generator=p.g).bfloat16().cuda()
    x[-20:] = last
    st = torch.cuda.current_stream()
    B.kv_write(ctx, p.cache, tokens, x, x, pos, p.dev_table, token_seq=seq, stream=st)
    t = torch.cat([torch.arange(20), torch.tensor([40])])
    at = p.table[0].long()[t // 16].tolist(), (t % 16).tolist()
    for pool in (p.k, p.v):
        assert torch.equal(pool[at].reshape(21, -1), torch.cat([last, x[3:4]]))
    y = torch.full((tokens, h * d), 7.0, dtype=BF16, device="cuda")
    B.kv_read(ctx, p.cache, tokens, pos, p.dev_table, x, y, token_seq=seq, stream=st)
    for out in (x, y):
        assert torch.equal(out[-20:], last) and bool((out[3] == 3).all())
        assert bool((out[4:-20] == 0).all()) and bool((out[:3] == 0).all())


def test_write_and_read_more_tokens_than_a_launch(ctx):
    tokens, d = (1 << 23) + 9, 16
    p = _Paged([64, 64], 1, d, 16, "fp8", seed=32)
    pos = torch.full((tokens,), -1, dtype=I32, device="cuda")
    pos[-20:] = torch.arange(20, dtype=I32, device="cuda")
    pos[3] = 40
    seq = torch.ones(tokens, dtype=I32, device="cuda")
    x = torch.full((tokens, d), 7.0, dtype=BF16, device="cuda")
    x[-20:] = torch.randint(-7, 8, (20, d), generator=p.g).bfloat16().cuda()
    x[-20:, 3] = 7.0                                       # (whole numbers below 8 over 7 / 448 = 2^-6: exact in 8 bits)
    st = torch.cuda.current_stream()
    B.kv_write(ctx, p.cache, tokens, x, x, pos, p.dev_table, token_seq=seq, stream=st)
    back = [torch.full((tokens, d), 5.0, dtype=BF16, device="cuda") for _ in range(2)]
    B.kv_read(ctx, p.cache, tokens, pos, p.dev_table, *back, token_seq=seq, stream=st)
    for y in back:
        assert torch.equal(y[-20:], x[-20:]) and torch.equal(y[3], x[3])
        assert bool((y[4:-20] == 0).all()) and bool((y[:3] == 0).all())
    # a token is a sequence of its own: those past the table have no place
    B.kv_read(ctx, p.cache, 2, pos[3:].contiguous(), p.dev_table, *back, stream=st)
    assert bool((back[0][1] == 0).all())


# ------------------------------------------------------------------------------ streams and graphs

def test_attn_repeats_its_bits_on_any_stream(ctx):
    p = _Paged([9000, 3, 1200], 2, 128, 16, "bf16", seed=40)
    q = torch.randn(3, 8 * 128, generator=p.g).bfloat16().cuda()
    lens = torch.tensor(p.lengths, dtype=I32, device="cuda")
    outs = []
    streams = [torch.cuda.Stream() for _ in range(5)]
    torch.cuda.synchronize()
    for s in [torch.cuda.current_stream()] + streams * 4:
        y = torch.zeros(3, 8 * 128, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        B.paged_attn(ctx, p.cache, 3, q, lens, p.dev_table, y, scale=0.1, stream=s)
        outs.append(y)
    torch.cuda.synchronize()
    for y in outs[1:]:
        assert torch.equal(y, outs[0])
    _check(p, ctx, 8)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_decode_steps_in_replayed_graphs(ctx, dtype):
    """A step of write and attention captured twice, replayed in turn with eager steps and other lengths between; every
    replay against the eager result on its own cache."""
    h, d, heads, rows = 2, 64, 8, 3
    p = _Paged([3000, 3000, 3000], h, d, 16, dtype, seed=50)
    twin = _Paged([3000, 3000, 3000], h, d, 16, dtype, seed=50)
    for mine in (p, twin):
        for x, s in ((mine.k, mine.k_scale), (mine.v, mine.v_scale)):
            x.view(torch.int16 if dtype == "bf16" else torch.uint8)[:] = 0
            if s is not None:
                s.fill_(1)
    x = torch.zeros(rows, (heads + 2 * h) * d, dtype=BF16, device="cuda")
    lens, pos = torch.zeros(rows, dtype=I32, device="cuda"), torch.zeros(rows, dtype=I32, device="cuda")
    angles = _angles(3000, d, p.g).cuda()
    bufs = {n: (torch.zeros(rows, heads * d, dtype=BF16, device="cuda"), torch.zeros(rows, heads * d, device="cuda")) for n in "abe"}

    def step(mine, name):
        st = torch.cuda.current_stream()
        turned, y = bufs[name]
        B.kv_write(ctx, mine.cache, rows, x[:, heads * d:(heads + h) * d], x[:, (heads + h) * d:], pos, mine.dev_table,
                   q=x[:, :heads * d], q_out=turned, rope=angles, stream=st)
        B.paged_attn(ctx, mine.cache, rows, turned, lens, mine.dev_table, y, scale=0.2, stream=st)
        return y

    def fill(i):
        g = _gen(i)
        x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        n = torch.tensor([1 + i, 1500 + 37 * i, 3000 - i], dtype=I32)
        lens.copy_(n)
        pos.copy_(n - 1)

    fill(0)
    step(twin, "e")
    torch.cuda.synchronize()
    graphs = {}
    for name in "ab":
        graphs[name] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[name]):
            step(p, name)
    for i in range(8):
        fill(i)
        name = "ab"[i % 2]
        want = step(twin, "e").clone()
        torch.cuda.synchronize()
        graphs[name].replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs[name][1], want), i
        assert bool(want.isfinite().all()) and float(want.abs().max()) > 0


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("fp8", 128), ("bf16", 64)])
def test_attn_of_all_of_a_large_cache(ctx, dtype, dim):
    """A pool beyond the last level's size read whole, its sequences read by two rows each, and only one of them: the kernel
    tells them apart by the lengths, and reads them with other cache policies."""
    heads = 2
    n = int(270e6 / (2 * heads * dim * (2 if dtype == "bf16" else 1))) // 6
    p = _Paged([n] * 5 + [n + 21], heads, dim, 64, dtype, heads_first=True, seed=dim)
    _check(p, ctx, 8)
    _check(p, ctx, 8, lens=[n] * 10, row_seq=[0, 1, 2, 3, 4] * 2)
    _check(p, ctx, 8, lens=[n + 20, 100], row_seq=[5, 1])


@pytest.mark.parametrize("rows", [2047, 2048, 2049, 5000])
@pytest.mark.parametrize("named", [False, True])
def test_attn_rows_around_a_launch(ctx, rows, named):
    """More rows than a launch takes: every row's own length and sequence, by its number or by name, one of them long."""
    g = _gen(rows)
    lengths = [int(x) for x in torch.randint(0, 24, (rows,), generator=g)]
    lengths[rows - 2] = 3000
    p = _Paged(lengths, 1, 16, 16, "bf16", seed=rows)
    order = torch.randperm(rows, generator=g).tolist() if named else list(range(rows))
    _check(p, ctx, 2, lens=[lengths[s] for s in order], row_seq=order if named else None, out="fp32")


def _in_parts(w, parts):
    """w as the sum of so many bfloat16 numbers, each the nearest to what the ones before leave."""
    total = torch.zeros_like(w)
    for _ in range(parts):
        total = total + (w - total).bfloat16().double()
    return total


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("group,dim", [(1, 64), (8, 128), (24, 128), (48, 64), (16, 256), (32, 256)])
def test_attn_fp32_results_have_the_whole_weights(ctx, dtype, group, dim):
    """Two tokens, the second with weight w = e^x, -2 <= x < 0, and the values 0 and 1: out = w / (1 + w). The products are
    exact, and the steps' errors, in units of 2^-24 of the result (half a unit of a float): the score's scale and two
    products 3 |x| <= 6, v_exp 2, the weight's three parts 1, their sum in the matrix unit 6, 1 + w and the division and the
    product with it 3. In two parts a weight is up to 2^-17 of itself off, 128 units, which is seen."""
    rows, heads = 64, group
    p = _Paged([2] * rows, 1, dim, 16, dtype, seed=group)
    for x, second in ((p.k, -1.0), (p.v, 1.0)):
        x.copy_(torch.zeros(x.shape).to(x.dtype))
        at = p.table[:, 0].long().cuda()
        if x is p.k:
            x[at, 1, 0, 0] = second
        else:
            x[at, 1, 0] = torch.ones(dim, device="cuda").to(x.dtype)
    if dtype == "fp8":
        p.k_scale.fill_(1)
        p.v_scale.fill_(1)
    q = torch.zeros(rows, heads, dim)
    q[..., 0] = 0.01 + 1.98 * torch.rand(rows, heads, generator=p.g)
    q = q.bfloat16()
    y = torch.zeros(rows, heads * dim, device="cuda")
    B.paged_attn(ctx, p.cache, rows, q.reshape(rows, -1).cuda(), torch.full((rows,), 2, dtype=I32, device="cuda"), p.dev_table, y,
                 scale=1.0, stream=torch.cuda.current_stream())
    w = torch.exp(-q[..., 0].double())
    want = w / (1 + w)
    bound = want * 18 * 2.0 ** -24
    two = _in_parts(w, 2) / (1 + w)
    assert bool(((two - want).abs() > bound).any()), "weights in two parts would pass"
    _within(y.reshape(rows, heads, dim), want[..., None].expand(rows, heads, dim), bound[..., None], "weights")
