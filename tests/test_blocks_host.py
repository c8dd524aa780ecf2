"""Page tables, rotary positions of several axes and selected blocks on the CPU: the
tables of axes, plans, and refusals before any launch (fake, never dereferenced pointers)."""
import ctypes

import numpy as np
import pytest

import blocks_ref as ref
import kv_cache_decode_gb300 as kvd

FAKE = 0x10000000
INV, UNS, SMALL = kvd.ERR_INVALID_ARG, kvd.ERR_UNSUPPORTED, kvd.ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module")
def lib():
    from kv_cache_decode_gb300 import _build
    _build.build()
    return kvd.load()


@pytest.mark.parametrize("sections", [(16, 24, 24), (8,), (1, 7), (2, 3, 3), (1, 1, 1, 5), (40, 40, 48)])
def test_axes_tables(lib, sections):
    n = sum(sections)
    plain, _ = kvd.rope_table(2 * n, 5e5)
    for order in ("blocks", "dealt"):
        turns, axes, f = kvd.rope_axes_table(sections, 5e5, order)
        assert f == 1.0 and np.array_equal(turns, plain)
        assert np.array_equal(axes, ref.axes_of(sections, order == "dealt"))
        assert [int((axes == a).sum()) for a in range(len(sections))] == list(sections)


def test_axes_tables_of_their_own(lib):
    for order in ("blocks", "dealt"):
        turns, axes, _ = kvd.rope_axes_table((8, 16, 40), 1e4, order, per_axis=True, scaling="linear", factor=2.0)
        for a, n in enumerate((8, 16, 40)):
            assert np.array_equal(turns[axes == a], kvd.rope_table(2 * n, 1e4, "linear", 2.0)[0])


@pytest.mark.parametrize("kw", [dict(sections=()), dict(sections=(8, 0)), dict(sections=(-8, 16)), dict(sections=(4,)), dict(sections=(8, 4)),
                                dict(sections=(2, 2, 2, 1, 1)), dict(sections=(129, 7)), dict(sections=(64, 72)), dict(per_axis=True, sections=(4, 4)),
                                dict(base=1.0), dict(scaling="linear", factor=0.5)])
def test_axes_table_refuses(lib, kw):
    with pytest.raises(kvd.KvdError) as e:
        kvd.rope_axes_table(**{"sections": (8, 8), **kw})
    assert e.value.status == INV


def test_axes_table_refuses_words(lib):
    with pytest.raises(ValueError):
        kvd.rope_axes_table((8,), order="other")
    with pytest.raises(ValueError):
        kvd.rope_axes_table((8,), scaling="other")


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def _call(fn, names, defaults, **kw):
    a = dict(defaults)
    for k, v in kw.items():
        assert k in a, k
        a[k] = v
    return fn(*[a[n] for n in names])


PAGES = dict(table=FAKE, free=FAKE + 0x10000, count=FAKE + 0x20000, lens=FAKE + 0x30000, new=FAKE + 0x40000, batch=4, max_blocks=8, page=16,
             pages=100, pos=FAKE + 0x50000, off=FAKE + 0x60000, slots=FAKE + 0x70000, positions=FAKE + 0x80000, rows=64, status=None, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(table=None), INV), (dict(free=None), INV), (dict(count=None), INV), (dict(lens=None), INV), (dict(new=None), INV),
    (dict(table=FAKE + 2), INV), (dict(slots=FAKE + 0x70001), INV), (dict(status=FAKE + 0x90002), INV), (dict(batch=-1), INV), (dict(max_blocks=0), INV),
    (dict(page=8), INV), (dict(page=48), INV), (dict(page=8192), INV), (dict(pages=0), INV), (dict(pages=1 << 27), INV), (dict(rows=-1), INV),
    (dict(rows=1 << 31), INV), (dict(batch=8193), UNS), (dict(batch=8000, max_blocks=1 << 19), INV), (dict(lens=FAKE + 0x40000), INV),
    (dict(slots=FAKE + 0x80010), INV), (dict(pos=FAKE), INV), (dict(count=FAKE + 0x10004), INV),
])
def test_pages_refuses(lib, kw, want):
    assert _call(lib.kvd_pages_update, list(PAGES), PAGES, **kw) == want


def _axes(**kw):
    a = dict(turns=FAKE, axes=FAKE + 0x1000, factor=1.0, rotary_dim=64, interleaved=0, n_axes=3)
    a.update(kw)
    return kvd._CRopeAxes(*a.values())


TURN = dict(rope=None, x=FAKE + 0x10000, xs=1024, xd=0, y=FAKE + 0x900000, ys=1024, yd=0, pos=FAKE + 0x2000, axis=10, rows=10, H=8, D=128,
            stream=None)


@pytest.mark.parametrize("rope,kw,want", [
    (None, {}, INV), (dict(turns=None), {}, INV), (dict(turns=FAKE + 4), {}, INV), (dict(axes=None), {}, INV), (dict(axes=FAKE + 4), {}, INV), (dict(rotary_dim=24), {}, INV),
    (dict(rotary_dim=144), {}, INV), (dict(n_axes=0), {}, INV), (dict(n_axes=5), {}, INV), (dict(factor=float("nan")), {}, INV),
    ({}, dict(pos=None), INV), ({}, dict(pos=FAKE + 2), INV), ({}, dict(axis=9), INV), ({}, dict(axis=-1), INV), ({}, dict(rows=-1), INV),
    ({}, dict(rows=1 << 31), INV), ({}, dict(H=0), INV), ({}, dict(D=100), INV), ({}, dict(D=2048), UNS), ({}, dict(xs=1000), INV),
    ({}, dict(xs=1028), INV), ({}, dict(x=FAKE + 8), INV), ({}, dict(xd=2), INV), ({}, dict(y=FAKE + 0x10010), INV),
    ({}, dict(y=FAKE + 0x10000, yd=1), INV), ({}, dict(pos=FAKE + 0x900004), INV),
])
def test_turn_refuses(lib, rope, kw, want):
    st = None if rope is None else _axes(**rope)
    a = {**TURN, "rope": None if st is None else ctypes.addressof(st)}
    assert _call(lib.kvd_rope_apply_axes, list(TURN), a, **kw) == want


APPEND = dict(cache=None, rope=None, q=FAKE + 0x100000, qs=1024, qo=FAKE + 0x200000, qos=1024, k=FAKE + 0x300000, ks=256, v=FAKE + 0x400000, vs=256,
              slots=FAKE + 0x1000, pos=FAKE + 0x2000, axis=10, batch=0, rows=10, Hq=8, Hkv=2, D=128, status=None, stream=None)


def _cache(**kw):
    a = dict(k=FAKE + 0x1000000, v=FAKE + 0x2000000, k_scales=None, v_scales=None, block_table=None, s_max=0, max_blocks=0, page_size=16, num_pages=10,
             fp8=0)
    a.update(kw)
    return kvd._CCache(*a.values())


@pytest.mark.parametrize("cache,kw,want", [
    (None, {}, INV), (dict(k=None), {}, INV), (dict(v=FAKE + 8), {}, INV), (dict(k_scales=FAKE), {}, INV), (dict(fp8=1), {}, INV), (dict(page_size=24), {}, INV),
    (dict(num_pages=0), {}, INV), (dict(page_size=0, num_pages=0), {}, INV), (dict(num_pages=1 << 28), {}, INV), (dict(v=FAKE + 0x1000000), {}, INV),
    ({}, dict(q=None), INV), ({}, dict(slots=None), INV), ({}, dict(slots=FAKE + 1), INV), ({}, dict(pos=None), INV), ({}, dict(axis=3), INV),
    ({}, dict(rows=-1), INV), ({}, dict(Hkv=0), INV), ({}, dict(Hq=0), INV), ({}, dict(D=132), INV), ({}, dict(D=1032, qs=8256, qos=8256, ks=2064, vs=2064), UNS),
    ({}, dict(ks=255), INV), ({}, dict(k=FAKE + 0x300008), INV), ({}, dict(qo=FAKE + 0x100010), INV), ({}, dict(qo=FAKE + 0x300000), INV),
    ({}, dict(k=FAKE + 0x1000000), INV), ({}, dict(slots=FAKE + 0x1000010), INV), ({}, dict(pos=FAKE + 0x200000), INV), ({}, dict(status=FAKE + 1), INV),
    (dict(k_scales=FAKE + 0x3000000, v_scales=FAKE + 0x4000000), dict(D=80, qs=640, qos=640, ks=160, vs=160), UNS),
    (dict(k_scales=FAKE + 0x3000000, v_scales=FAKE + 0x3000000), {}, INV),
])
def test_append_refuses(lib, cache, kw, want):
    c, r = None if cache is None else _cache(**cache), _axes()
    a = {**APPEND, "cache": None if c is None else ctypes.addressof(c), "rope": ctypes.addressof(r)}
    assert _call(lib.kvd_kv_append_axes, list(APPEND), a, **kw) == want


def _bounds(**kw):
    a = dict(codes=FAKE + 0x1000000, scales=FAKE + 0x2000000, block_table=FAKE + 0x100, s_max=0, max_blocks=8, page_size=64, num_pages=10, block_tokens=32)
    a.update(kw)
    return kvd._CBlockBounds(*a.values())


BOUNDS = dict(k=FAKE + 0x4000000, bounds=None, frm=None, lens=FAKE + 0x10000, batch=2, most=64, Hkv=2, D=128, status=None, stream=None)
BAD_BOUNDS = [(None, {}, INV), (dict(codes=None), {}, INV), (dict(codes=FAKE + 8), {}, INV), (dict(scales=FAKE + 2), {}, INV), (dict(block_tokens=8), {}, INV),
              (dict(block_tokens=48), {}, INV), (dict(block_tokens=128), {}, INV), (dict(page_size=40), {}, INV), (dict(block_table=None), {}, INV),
              (dict(block_table=FAKE + 1), {}, INV), ({}, dict(batch=-1), INV), ({}, dict(Hkv=0), INV), ({}, dict(D=96), UNS), ({}, dict(lens=None), INV),
              ({}, dict(lens=FAKE + 2), INV), ({}, dict(status=FAKE + 2), INV)]


@pytest.mark.parametrize("bounds,kw,want", BAD_BOUNDS + [
    ({}, dict(k=None), INV), ({}, dict(k=FAKE + 2), INV), ({}, dict(most=-1), INV), ({}, dict(frm=FAKE + 1), INV), ({}, dict(k=FAKE + 0x1000000), INV),
    ({}, dict(lens=FAKE + 0x2000000), INV)])
def test_bounds_refuses(lib, bounds, kw, want):
    b = None if bounds is None else _bounds(**bounds)
    a = {**BOUNDS, "bounds": None if b is None else ctypes.addressof(b)}
    assert _call(lib.kvd_kv_block_bounds, list(BOUNDS), a, **kw) == want


SELECT = dict(bounds=None, q=FAKE + 0x4000000, lens=FAKE + 0x10000, batch=2, T=1, max_len=512, keep=8, first=1, last=2, Hq=8, Hkv=2, D=128,
              ws=FAKE + 0x5000000, wb=1 << 20, out=FAKE + 0x6000000, status=None, stream=None)


@pytest.mark.parametrize("bounds,kw,want", BAD_BOUNDS + [
    ({}, dict(q=None), INV), ({}, dict(q=FAKE + 8), INV), ({}, dict(out=None), INV), ({}, dict(out=FAKE + 1), INV), ({}, dict(T=0), INV), ({}, dict(T=65), UNS),
    ({}, dict(max_len=-1), INV), ({}, dict(max_len=544), INV), ({}, dict(keep=0, first=0), INV), ({}, dict(keep=2), INV), ({}, dict(first=-1), INV),
    ({}, dict(last=0), INV), ({}, dict(first=2 ** 31 - 1, last=2 ** 31 - 1), INV), ({}, dict(keep=(1 << 20) + 1), UNS), ({}, dict(Hq=7), INV), ({}, dict(Hq=130), UNS),
    ({}, dict(ws=None), SMALL), ({}, dict(wb=255), SMALL), ({}, dict(ws=FAKE + 0x5000010), INV), ({}, dict(out=FAKE + 0x4000000), INV),
    ({}, dict(ws=FAKE + 0x1000000), INV)])
def test_select_refuses(lib, bounds, kw, want):
    b = None if bounds is None else _bounds(**bounds)
    a = {**SELECT, "bounds": None if b is None else ctypes.addressof(b)}
    assert _call(lib.kvd_block_select, list(SELECT), a, **kw) == want


def test_plans(lib):
    assert kvd.block_select_plan(2, 3, 4, 1000, 64) == -(-2 * 3 * 4 * 15 * 4 // 256) * 256
    assert kvd.block_select_plan(2, 1, 4, 10, 64) == 0
    # enough pairs for the machine: nothing to join; one pair of a long list: several clusters' float32 rows
    assert kvd.decode_blocks_plan(64, 1, 32, 8, 128, 64, 64, num_sms=152) == 0
    assert kvd.decode_blocks_plan(1, 1, 32, 8, 128, 32, 64, num_sms=152) == 0
    n = kvd.decode_blocks_plan(1, 1, 8, 1, 128, 256, 128, num_sms=152)
    assert n > 0 and n % 256 == 0
    for kw in (dict(block_tokens=8), dict(block_tokens=100), dict(n_blocks=0), dict(n_tokens=0), dict(n_heads_q=7)):
        with pytest.raises(kvd.KvdError) as e:
            kvd.decode_blocks_plan(**{**dict(batch=1, n_tokens=1, n_heads_q=8, n_heads_kv=2, head_dim=128, n_blocks=4, block_tokens=64, num_sms=152), **kw})
        assert e.value.status == INV
    for kw in (dict(n_tokens=65), dict(n_blocks=(1 << 20) + 1), dict(head_dim=96), dict(n_heads_q=130), dict(n_blocks=1 << 19, block_tokens=4096)):
        with pytest.raises(kvd.KvdError) as e:
            kvd.decode_blocks_plan(**{**dict(batch=1, n_tokens=1, n_heads_q=8, n_heads_kv=2, head_dim=128, n_blocks=4, block_tokens=64, num_sms=152), **kw})
        assert e.value.status == UNS


DECODE = dict(cache=None, q=FAKE, blocks=FAKE + 0x10000, lens=FAKE + 0x20000, batch=2, T=1, K=4, block=64, Hq=8, Hkv=2, D=128, scale=0.1, ws=None, wb=0,
              out=FAKE + 0x30000, dt=0, lse=None, status=None, stream=None)


@pytest.mark.parametrize("cache,kw,want", [
    (None, {}, INV), (dict(k=None), {}, INV), (dict(v=FAKE + 8), {}, INV), (dict(k_scales=FAKE, v_scales=FAKE), {}, UNS), (dict(fp8=1), {}, UNS),
    (dict(page_size=24), {}, INV), (dict(block_table=None), {}, INV), (dict(block_table=FAKE + 1), {}, INV),
    (dict(block_table=None, s_max=1 << 30), {}, UNS), ({}, dict(q=None), INV), ({}, dict(blocks=None), INV), ({}, dict(blocks=FAKE + 2), INV), ({}, dict(lens=None), INV),
    ({}, dict(out=None), INV), ({}, dict(out=FAKE + 8), INV), ({}, dict(lse=FAKE + 2), INV), ({}, dict(batch=-1), INV), ({}, dict(T=0), INV), ({}, dict(T=65), UNS),
    ({}, dict(K=0), INV), ({}, dict(block=24), INV), ({}, dict(block=8192), INV), ({}, dict(Hq=9), INV), ({}, dict(Hq=256), UNS), ({}, dict(D=96), UNS),
    ({}, dict(scale=float("inf")), INV), ({}, dict(dt=3), INV)])
def test_decode_refuses(lib, cache, kw, want):
    c = None if cache is None else _cache(**{**dict(block_table=FAKE + 0x100, max_blocks=8), **cache})
    a = {**DECODE, "cache": None if c is None else ctypes.addressof(c)}
    assert _call(lib.kvd_decode_blocks, list(DECODE), a, **kw) == want
