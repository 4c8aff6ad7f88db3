"""The attention operators' host side, without a GPU: the argument checks' codes and the binding's own checks."""

import ctypes

import pytest
import torch

from allgather_gemm_persistent_amd import binding as B

FAKE = 1 << 20          # an aligned non-NULL address (never dereferenced by the checks)


@pytest.fixture(scope="module")
def lib():
    return B.load()


def _cache(**kw):
    d = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, pages=10, ld_page=2048, ld_token=128, ld_head=64,
             dtype=B.AGG_BF16, page_size=16, kv_heads=2, head_dim=64)
    d.update(kw)
    return B._CacheStruct(*d.values())


def _ref(c):
    return None if c is None else ctypes.addressof(c)


CACHE_KEYS = ("k", "v", "k_scale", "v_scale", "pages", "ld_page", "ld_token", "ld_head", "dtype", "page_size", "kv_heads",
              "head_dim")


def _split(kw):
    return _cache(**{x: y for x, y in kw.items() if x in CACHE_KEYS}), {x: y for x, y in kw.items() if x not in CACHE_KEYS}


def _write(lib, **kw):
    c, kw = _split(kw)
    d = dict(cache=_ref(c), tokens=4, q_heads=4, q=FAKE, lq=256, qo=FAKE, lqo=256, k_in=FAKE, lk=128, v_in=FAKE, lv=128,
             rope=FAKE, rope_rows=100, rope_dim=64, pairs=0, positions=FAKE, table=FAKE, seqs=4, seq_pages=8, lt=8)
    d.update(kw)
    return lib.agg_check_kv_write_args(*d.values())


def _read(lib, **kw):
    c, kw = _split(kw)
    d = dict(cache=_ref(c), tokens=4, positions=FAKE, table=FAKE, seqs=4, seq_pages=8, lt=8, od=B.AGG_BF16, ko=FAKE,
             lk=128, vo=FAKE, lv=128)
    d.update(kw)
    return lib.agg_check_kv_read_args(*d.values())


def _attn(lib, **kw):
    c, kw = _split(kw)
    d = dict(cache=_ref(c), rows=4, q_heads=4, q=FAKE, lq=256, scale=0.125, lens=FAKE, table=FAKE, seqs=4, seq_pages=8,
             lt=8, window=0, od=B.AGG_BF16, out=FAKE, lo=256)
    d.update(kw)
    return lib.agg_check_paged_attn_args(*d.values())


@pytest.mark.parametrize("call", [_write, _read, _attn])
@pytest.mark.parametrize("kw", [
    dict(), dict(dtype=B.AGG_FP8_E4M3), dict(k_scale=None, v_scale=None), dict(page_size=48), dict(page_size=4096),
    dict(ld_page=1 << 20), dict(ld_token=64, ld_head=1024), dict(pages=1, ld_page=-5), dict(pages=0, k=None, v=None),
    dict(seqs=0, table=None), dict(seq_pages=0, table=None, lt=0), dict(seqs=1, lt=0)])
def test_caches_and_tables_ok(lib, call, kw):
    assert call(lib, **kw) == B.AGG_OK, B.last_error()


@pytest.mark.parametrize("call", [_write, _read, _attn])
@pytest.mark.parametrize("kw,code", [
    (dict(cache=None), B.AGG_E_ARG), (dict(dtype=B.AGG_FP32), B.AGG_E_ARG), (dict(dtype=7), B.AGG_E_ARG),
    (dict(page_size=8), B.AGG_E_ARG), (dict(page_size=24), B.AGG_E_ARG), (dict(page_size=4112), B.AGG_E_ARG),
    (dict(page_size=0), B.AGG_E_ARG), (dict(page_size=-16), B.AGG_E_ARG), (dict(head_dim=0), B.AGG_E_ARG),
    (dict(head_dim=72), B.AGG_E_ARG), (dict(head_dim=272), B.AGG_E_ARG), (dict(kv_heads=0), B.AGG_E_ARG),
    (dict(kv_heads=1025), B.AGG_E_ARG), (dict(pages=-1), B.AGG_E_ARG), (dict(pages=(1 << 30) + 1), B.AGG_E_UNSUPPORTED),
    (dict(k=None), B.AGG_E_ARG), (dict(v=None), B.AGG_E_ARG), (dict(k=FAKE + 8), B.AGG_E_ARG), (dict(v=FAKE + 2), B.AGG_E_ARG),
    (dict(dtype=B.AGG_FP8_E4M3, k_scale=None), B.AGG_E_ARG), (dict(dtype=B.AGG_FP8_E4M3, v_scale=FAKE + 4), B.AGG_E_ARG),
    (dict(ld_page=63), B.AGG_E_ARG), (dict(ld_token=32), B.AGG_E_ARG), (dict(ld_head=0), B.AGG_E_ARG),
    (dict(ld_head=-64), B.AGG_E_ARG), (dict(ld_token=132), B.AGG_E_ARG), (dict(ld_page=2052), B.AGG_E_ARG),
    (dict(dtype=B.AGG_FP8_E4M3, ld_head=72), B.AGG_E_ARG), (dict(ld_page=1 << 33), B.AGG_E_UNSUPPORTED),
    (dict(ld_token=1 << 26), B.AGG_E_UNSUPPORTED), (dict(table=None), B.AGG_E_ARG), (dict(table=FAKE + 2), B.AGG_E_ARG),
    (dict(lt=7), B.AGG_E_ARG), (dict(lt=1 << 33), B.AGG_E_UNSUPPORTED), (dict(seqs=-1), B.AGG_E_ARG),
    (dict(seq_pages=-1), B.AGG_E_ARG), (dict(seqs=1 << 31), B.AGG_E_UNSUPPORTED),
    (dict(seq_pages=1 << 27, lt=1 << 27), B.AGG_E_UNSUPPORTED), (dict(seq_pages=1 << 62, lt=1 << 62), B.AGG_E_UNSUPPORTED)])
def test_caches_and_tables_rejected(lib, call, kw, code):
    assert call(lib, **kw) == code
    assert B.last_error()


@pytest.mark.parametrize("kw", [
    dict(tokens=0, k_in=None, positions=None), dict(q_heads=0, q=None, qo=None), dict(rope=None, rope_rows=0, rope_dim=0),
    dict(rope_dim=16), dict(pairs=1), dict(rope_rows=0), dict(lq=264, qo=2 * FAKE, lqo=512, lk=136, lv=1024), dict(q_heads=1024, lq=65536, lqo=65536),
    dict(tokens=1, lqo=512)])
def test_write_args_ok(lib, kw):
    assert _write(lib, **kw) == B.AGG_OK, B.last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), B.AGG_E_ARG), (dict(tokens=(1 << 30) + 1), B.AGG_E_UNSUPPORTED), (dict(q_heads=-1), B.AGG_E_ARG),
    (dict(q_heads=1025), B.AGG_E_ARG), (dict(q=None), B.AGG_E_ARG), (dict(qo=None), B.AGG_E_ARG), (dict(q=FAKE + 8), B.AGG_E_ARG),
    (dict(lq=248), B.AGG_E_ARG), (dict(lq=260), B.AGG_E_ARG), (dict(lqo=255), B.AGG_E_ARG), (dict(lq=1 << 32), B.AGG_E_UNSUPPORTED),
    (dict(lqo=512), B.AGG_E_ARG), (dict(k_in=None), B.AGG_E_ARG), (dict(v_in=None), B.AGG_E_ARG), (dict(lk=120), B.AGG_E_ARG),
    (dict(lv=129), B.AGG_E_ARG), (dict(v_in=FAKE + 4), B.AGG_E_ARG), (dict(rope=None), B.AGG_E_ARG), (dict(rope_dim=0), B.AGG_E_ARG),
    (dict(rope_dim=8), B.AGG_E_ARG), (dict(rope_dim=80), B.AGG_E_ARG), (dict(rope_dim=-16), B.AGG_E_ARG),
    (dict(rope_rows=-1), B.AGG_E_ARG), (dict(rope_rows=1 << 31), B.AGG_E_UNSUPPORTED), (dict(rope=FAKE + 4), B.AGG_E_ARG),
    (dict(pairs=2), B.AGG_E_ARG), (dict(positions=None), B.AGG_E_ARG), (dict(positions=FAKE + 1), B.AGG_E_ARG)])
def test_write_args_rejected(lib, kw, code):
    assert _write(lib, **kw) == code
    assert B.last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(), B.AGG_OK), (dict(tokens=0, ko=None, vo=None, positions=None), B.AGG_OK), (dict(od=B.AGG_FP32), B.AGG_OK),
    (dict(od=B.AGG_FP32, lk=132, lv=140), B.AGG_OK), (dict(tokens=-1), B.AGG_E_ARG), (dict(od=B.AGG_FP8_E4M3), B.AGG_E_ARG),
    (dict(ko=None), B.AGG_E_ARG), (dict(vo=None), B.AGG_E_ARG), (dict(ko=FAKE + 8), B.AGG_E_ARG), (dict(lk=127), B.AGG_E_ARG),
    (dict(lv=132), B.AGG_E_ARG), (dict(lv=1 << 40), B.AGG_E_UNSUPPORTED), (dict(positions=None), B.AGG_E_ARG),
    (dict(tokens=(1 << 30) + 1), B.AGG_E_UNSUPPORTED)])
def test_read_args(lib, kw, code):
    assert _read(lib, **kw) == code
    assert bool(B.last_error()) == (code != B.AGG_OK)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0, q=None, out=None, lens=None), B.AGG_OK), (dict(window=5), B.AGG_OK), (dict(window=1 << 62), B.AGG_OK),
    (dict(od=B.AGG_FP32, lo=260), B.AGG_OK), (dict(scale=0.0), B.AGG_OK), (dict(scale=-1.0), B.AGG_OK),
    (dict(q_heads=2, lq=128, lo=128), B.AGG_OK), (dict(q_heads=1024, lq=65536, lo=65536), B.AGG_OK),
    (dict(rows=-1), B.AGG_E_ARG), (dict(rows=(1 << 20) + 1), B.AGG_E_UNSUPPORTED), (dict(window=-1), B.AGG_E_ARG),
    (dict(q_heads=0), B.AGG_E_ARG), (dict(q_heads=3), B.AGG_E_ARG), (dict(q_heads=1026), B.AGG_E_ARG),
    (dict(scale=float("nan")), B.AGG_E_ARG), (dict(scale=float("inf")), B.AGG_E_ARG), (dict(scale=3e38), B.AGG_E_ARG),
    (dict(od=B.AGG_FP8_E4M3), B.AGG_E_ARG), (dict(q=None), B.AGG_E_ARG), (dict(q=FAKE + 8), B.AGG_E_ARG), (dict(lq=252), B.AGG_E_ARG),
    (dict(lq=260), B.AGG_E_ARG), (dict(out=None), B.AGG_E_ARG), (dict(lo=255), B.AGG_E_ARG), (dict(lo=260), B.AGG_E_ARG),
    (dict(lens=None), B.AGG_E_ARG), (dict(lens=FAKE + 2), B.AGG_E_ARG)])
def test_attn_args(lib, kw, code):
    assert _attn(lib, **kw) == code
    assert bool(B.last_error()) == (code != B.AGG_OK)


def test_a_call_without_a_ctx_is_refused(lib):
    c = _cache()
    rows = (FAKE, 128)
    assert lib.kv_write(None, _ref(c), 4, 0, None, 0, None, 0, *rows, *rows, None, 0, 0, 0, FAKE, None, FAKE, 4, 8, 8,
                        None) == B.AGG_E_ARG
    assert lib.kv_read(None, _ref(c), 4, FAKE, None, FAKE, 4, 8, 8, B.AGG_BF16, *rows, *rows, None) == B.AGG_E_ARG
    assert lib.paged_attn(None, _ref(c), 4, 2, *rows, 0.1, FAKE, None, FAKE, 4, 8, 8, 0, B.AGG_BF16, *rows, None,
                          None) == B.AGG_E_ARG


def _refused(call):
    with pytest.raises(B.AggError) as e:
        call()
    assert e.value.code == B.AGG_E_ARG


def test_binding_refuses_what_the_call_would_read_wrongly():
    bf16, i32 = torch.bfloat16, torch.int32
    k = torch.zeros(0, 16, 2, 64, dtype=bf16)
    cache = B.KvCache(k, k)                                                      # (no pages: nothing to lie on a device)
    for bad in (lambda: B.KvCache(k, k.half()), lambda: B.KvCache(k.float(), k.float()),
                lambda: B.KvCache(k, torch.zeros(1, 16, 2, 64, dtype=bf16)), lambda: B.KvCache(k[..., 0], k[..., 0]),
                lambda: B.KvCache(torch.zeros(3, 16, 2, 64, dtype=bf16), torch.zeros(3, 16, 2, 64, dtype=bf16)),
                lambda: B.KvCache(torch.zeros(3, 16, 2, 64, dtype=bf16), torch.zeros(3, 2, 16, 64, dtype=bf16).transpose(1, 2)),
                lambda: B.KvCache(torch.zeros(3, 16, 64, 2, dtype=bf16).transpose(2, 3), torch.zeros(3, 16, 64, 2, dtype=bf16).transpose(2, 3)),
                lambda: B.KvCache(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn))):
        _refused(bad)
    rows, pos, table = torch.zeros(4, 128, dtype=bf16), torch.zeros(4, dtype=i32), torch.zeros(4, 8, dtype=i32)
    q = torch.zeros(4, 256, dtype=bf16)
    _refused(lambda: B.kv_write(None, cache, 4, rows, rows, pos, table))         # host tensors
    _refused(lambda: B.kv_write(None, cache, 5, rows, rows, pos, table))         # fewer rows than tokens
    _refused(lambda: B.kv_write(None, cache, 0, rows.float(), rows, pos, table))
    _refused(lambda: B.kv_write(None, cache, 0, rows, rows, pos, table, q=q))    # no q_out
    _refused(lambda: B.kv_write(None, cache, 0, rows, rows, pos, table, rope=torch.zeros(5)))
    _refused(lambda: B.kv_write(None, cache, 4, rows[:0], rows, pos, table))
    _refused(lambda: B.kv_read(None, cache, 0, pos, table, rows, rows.float()))
    _refused(lambda: B.kv_read(None, cache, 0, pos, table.long(), rows, rows))
    _refused(lambda: B.kv_read(None, cache, 0, pos, table[0], rows, rows))
    _refused(lambda: B.kv_read(None, cache, 0, pos.long(), table[:, :0], rows, rows))
    _refused(lambda: B.paged_attn(None, cache, 0, q[:, :100], pos, table[:, :0], q, scale=1.0))    # no whole heads
    _refused(lambda: B.paged_attn(None, cache, 0, q.float(), pos, table[:, :0], q, scale=1.0))
    _refused(lambda: B.paged_attn(None, cache, 3, q[:0], pos, table[:2, :0], q, scale=1.0, row_seq=None))


# ------------------------------------------------------------------------------ paged_attn's workspace

def _workspace(lib, rows, q_heads, seq_pages, window=0, **kw):
    n = ctypes.c_int64(-1)
    c = _cache(**kw)
    assert lib.agg_paged_attn_workspace(_ref(c), rows, q_heads, seq_pages, window, ctypes.byref(n)) == B.AGG_OK, B.last_error()
    return n.value


@pytest.mark.parametrize("rows,q_heads,kv_heads,dim,seq_pages,window,most", [
    # (rows * heads * (positions / 32 + 2) / 2 results of a head's queries, dim + 4 floats a query)
    (0, 8, 1, 128, 100, 0, 0), (1, 8, 1, 128, 1, 0, 1 * 4224), (1, 8, 1, 128, 32, 0, 9 * 4224),
    (16, 64, 8, 128, 4, 0, 256 * 4224), (16, 64, 8, 128, 1 << 20, 64, 256 * 4224), (64, 1, 1, 64, 2, 0, 96 * 272),
    (1 << 20, 1024, 16, 128, 1 << 15, 0, 4 * 256 * 64 * 528)])                                     # four a workgroup
def test_the_workspace_is_no_more_than_the_rows_can_need(lib, rows, q_heads, kv_heads, dim, seq_pages, window, most):
    """Every capture keeps one as long as its ctx lives."""
    kw = dict(kv_heads=kv_heads, head_dim=dim, ld_head=dim, ld_token=dim * kv_heads, ld_page=16 * dim * kv_heads)
    assert _workspace(lib, rows, q_heads, seq_pages, window, **kw) <= most


@pytest.mark.parametrize("q_heads,kv_heads,dim", [(8, 1, 128), (64, 8, 128), (20, 20, 80), (33, 1, 64), (130, 2, 256)])
def test_the_workspace_holds_every_plan(lib, q_heads, kv_heads, dim):
    """The kernel cuts a row of t tiles into ceil(t / s) parts, s one of some multiples of an even share of all tiles and four
    at least, or, where there is a workgroup for every tile, a 32nd of the longest row and four at least; a row of one
    part takes no place. Whatever the lengths, the places of all parts are inside the workspace."""
    import random
    rng = random.Random(q_heads + dim)
    group = q_heads // kv_heads
    tiles16 = 1 if group <= 16 else 2 if group <= 32 or dim > 128 else 4
    grid = 256 * (2 if tiles16 == 1 and dim <= 128 else 1)
    items = -(-group // (16 * tiles16)) * kv_heads
    slot = min(group, 16 * tiles16) * (dim + 4) * 4
    kw = dict(kv_heads=kv_heads, head_dim=dim, ld_head=dim, ld_token=dim * kv_heads, ld_page=16 * dim * kv_heads)
    for _ in range(400):
        rows, room = int(2 ** rng.uniform(0, 9)), 16 * int(2 ** rng.uniform(0, 13))
        window = rng.choice([0, 0, int(2 ** rng.uniform(0, 14))])
        lens = [rng.choice([room, rng.randint(0, room), int(2 ** rng.uniform(0, 17)) % (room + 1)]) for _ in range(rows)]
        tiles = []
        for n in lens:
            lo = max(0, n - window) if window else 0
            tiles.append(-(-n // 32) - lo // 32 if n > lo else 1)
        total = sum(tiles) * items
        some = max(4, -(-total // grid))
        sizes = {max(4, -(-some * q // 4)) for q in (2, 4, 5, 6, 8, 16)}
        if rows <= 64 and total <= grid:
            sizes = {max(tiles)} if max(tiles) <= 8 else {max(4, -(-max(tiles) // 32))}
        held = _workspace(lib, rows, q_heads, room // 16, window, **kw) // slot
        for s in sizes:
            parts = [-(-t // s) for t in tiles]
            assert sum(p for p in parts if p > 1) * items <= held, (rows, room, window, s)
            assert max(parts) <= 32 * 32, (rows, room, window, s)      # (what two steps join)


def test_the_workspace_of_refused_sizes(lib):
    n = ctypes.c_int64()
    c = _cache()
    for args in ((_ref(c), -1, 2, 4, 0), (_ref(c), 1, 3, 4, 0), (_ref(c), 1, 2, -4, 0), (_ref(c), 1, 2, 4, -1), (None, 1, 2, 4, 0),
                 (_ref(c), (1 << 20) + 1, 2, 4, 0), (_ref(c), 1, 2, 1 << 62, 0)):
        assert lib.agg_paged_attn_workspace(*args, ctypes.byref(n)) != B.AGG_OK and B.last_error()
    assert lib.agg_paged_attn_workspace(_ref(c), 1, 2, 4, 0, None) == B.AGG_E_ARG


@pytest.mark.parametrize("off", [1, 2, 3])
def test_optional_arrays_that_are_not_aligned_are_refused(lib, off):
    """The sequences of the tokens or rows, and the logarithms of the sums: words of four bytes, as every array here."""
    c, rows = _cache(), (FAKE, 128)
    for what, call in (
            ("token_seq", lambda p, n: lib.kv_write(None, _ref(c), n, 0, None, 0, None, 0, *rows, *rows, None, 0, 0, 0, FAKE, p,
                                                    FAKE, 4, 8, 8, None)),
            ("token_seq", lambda p, n: lib.kv_read(None, _ref(c), n, FAKE, p, FAKE, 4, 8, 8, B.AGG_BF16, *rows, *rows, None)),
            ("row_seq", lambda p, n: lib.paged_attn(None, _ref(c), n, 2, *rows, 0.1, FAKE, p, FAKE, 4, 8, 8, 0, B.AGG_BF16, *rows,
                                                    None, None)),
            ("lse", lambda p, n: lib.paged_attn(None, _ref(c), n, 2, *rows, 0.1, FAKE, None, FAKE, 4, 8, 8, 0, B.AGG_BF16, *rows,
                                                p, None))):
        assert call(FAKE + off, 4) == B.AGG_E_ARG and what in B.last_error(), what
        assert call(FAKE + 4, 4) == B.AGG_E_ARG and "ctx" in B.last_error(), what          # (only the ctx is missing)
        assert call(FAKE + off, 0) == B.AGG_E_ARG and "ctx" in B.last_error(), what        # (no tokens: not looked at)
