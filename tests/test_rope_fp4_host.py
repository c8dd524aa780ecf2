"""Rotary tables, the fp4 format and the new entry points' argument checks, on
the CPU: the frequency tables against 50-digit arithmetic, the fp4 oracle
against its definition's bounds, and refusals before any launch (fake,
never dereferenced pointers)."""
import ctypes
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest

import kv_cache_decode_gb300 as kvd
import oracle
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

FAKE = 0x10000000


@pytest.fixture(scope="module")
def lib():
    from kv_cache_decode_gb300 import _build
    _build.build()
    return kvd.load()


# ---------------------------------------------------------------------------
# rotary tables
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("R,base", [(16, 10000.0), (64, 10000.0), (128, 500000.0), (256, 1e6), (96, 10000.0)])
def test_table_against_50_digits(lib, R, base):
    getcontext().prec = 50
    pi = Decimal("3.14159265358979323846264338327950288419716939937510")
    turns, f = kvd.rope_table(R, base)
    assert f == 1.0 and turns.dtype == np.uint64 and turns.shape == (R // 2,)
    ln_base = Decimal(base).ln()
    for i in range(R // 2):
        want = (-2 * i * ln_base / R).exp() / (2 * pi) * (1 << 64)
        # The frequency is a double, within a few units of 2^-53.
        assert abs(Decimal(int(turns[i])) - want) <= want * Decimal(2) ** -49 + 1


def _radians(turns):
    return turns.astype(np.float64) / 2.0 ** 64 * 2 * np.pi


def test_scalings(lib):
    R, base, f, orig = 128, 10000.0, 8.0, 4096.0
    plain = _radians(kvd.rope_table(R, base)[0])
    assert np.allclose(_radians(kvd.rope_table(R, base, "linear", f)[0]), plain / f, rtol=1e-12)
    assert np.allclose(_radians(kvd.rope_table(R, base, "base", f)[0]),
                       (base * f ** (R / (R - 2.0))) ** (-np.arange(0, R, 2) / R), rtol=1e-12)
    w, g = kvd.rope_table(R, base, "wavelength", f, orig)
    w = _radians(w)
    turns = orig * plain / (2 * np.pi)
    assert g == 1.0
    assert np.allclose(w[turns >= 4], plain[turns >= 4], rtol=1e-12)
    assert np.allclose(w[turns <= 1], plain[turns <= 1] / f, rtol=1e-12)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and ((w[mid] > plain[mid] / f) & (w[mid] < plain[mid])).all()
    w, g = kvd.rope_table(R, base, "parts", f, orig)
    w = _radians(w)
    assert g == pytest.approx(0.1 * math.log(f) + 1, abs=1e-6)
    at = lambda n: R * math.log(orig / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = math.floor(at(32)), math.ceil(at(1))
    ramp = np.clip((np.arange(R // 2) - lo) / (hi - lo), 0, 1)
    assert np.allclose(w, plain * (1 - ramp) + plain / f * ramp, rtol=1e-12)
    assert kvd.rope_table(R, base, "parts", f, orig, attn_factor=1.25)[1] == 1.25
    # a factor of one changes nothing, whatever the scaling
    for s in ("linear", "base", "parts", "wavelength"):
        assert np.allclose(_radians(kvd.rope_table(R, base, s, 1.0, orig)[0]), plain, rtol=1e-12)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=8), dict(rotary_dim=24), dict(rotary_dim=272), dict(rotary_dim=0), dict(rotary_dim=-16),
    dict(base=1.0), dict(base=float("inf")), dict(base=float("nan")), dict(scaling="linear", factor=0.5),
    dict(scaling="linear", factor=float("nan")), dict(scaling="parts", factor=2.0, original_len=0.0),
    dict(scaling="wavelength", factor=2.0, original_len=4096.0, slow=4.0, fast=4.0),
    dict(scaling="wavelength", factor=2.0, original_len=4096.0, slow=0.0),
    dict(attn_factor=-1.0), dict(attn_factor=float("inf")),
])
def test_table_refuses(lib, kw):
    with pytest.raises(kvd.KvdError) as e:
        kvd.rope_table(**{"rotary_dim": 64, **kw})
    assert e.value.status == kvd.ERR_INVALID_ARG


def test_table_refuses_unknown_scaling(lib):
    with pytest.raises(ValueError):
        kvd.rope_table(64, scaling="other")
    f = ctypes.c_float()
    buf = (ctypes.c_uint64 * 32)()
    assert lib.kvd_rope_table(64, 1e4, 9, 1, 0, 0, 0, 0, buf, ctypes.byref(f)) == kvd.ERR_INVALID_ARG
    assert lib.kvd_rope_table(64, 1e4, 0, 1, 0, 0, 0, 0, None, ctypes.byref(f)) == kvd.ERR_INVALID_ARG
    assert lib.kvd_rope_table(64, 1e4, 0, 1, 0, 0, 0, 0, buf, None) == kvd.ERR_INVALID_ARG


# ---------------------------------------------------------------------------
# the fp4 format (oracle)
# ---------------------------------------------------------------------------

def _bits(x):
    return f32_to_bf16_bits(np.ascontiguousarray(x, np.float32))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_fp4_error_bound_and_pack(D):
    r = np.random.default_rng(D)
    x = r.standard_normal((3, 32, D)).astype(np.float32) * np.exp2(r.integers(-20, 20, (3, 32, 1))).astype(np.float32)
    x[0, 3] = 0.0
    x[1, 5, 1:] = 0.0
    x[2, 7, :16] *= 2.0 ** -24
    bits = _bits(x)
    codes, sb, exps = oracle.quantize_fp4(bits)
    back = oracle.dequantize_fp4(codes, sb, exps)
    ref = bf16_bits_to_f32(bits).astype(np.float64)
    # Largest code spacing is 2 (4..6) for values up to 6 s: at most half of it
    # off, plus what the scale's own rounding (2^-4 relative, which may push the largest
    # value past 6 s) and the smallest scale 2^-9 * 2^e leave.
    amax = np.abs(ref.reshape(3, 32, D // 16, 16)).max(-1)
    unit = np.exp2(exps.astype(np.float64) - 127)[..., None]
    bound = amax * (1.0 / 6.0) * (1 + 2.0 ** -4) + amax * 2.0 ** -4 + 6 * 2.0 ** -10 * unit
    err = np.abs(back - ref).reshape(3, 32, D // 16, 16).max(-1)
    assert (err <= bound + 1e-300).all()
    assert (back[0, 3] == 0).all() and exps[0, 3] == 0 and (codes[0, 3] == 0).all()
    # the row exponent is the smallest that reaches the row's largest value
    a = np.abs(ref).max(-1)
    nz = a > 0
    assert (a[nz] <= 2688 * unit[..., 0][nz]).all() and (a[nz] > 1344 * unit[..., 0][nz]).all()
    blk = oracle.pack_fp4(codes, sb, exps)
    assert blk.shape == (3, 2, kvd.fp4_block_bytes(D)) and blk.shape[-1] == 9 * D + 16
    for p, q in zip(oracle.unpack_fp4(blk, D), (codes, sb, exps)):
        assert np.array_equal(p, q)
    # bf16 holds every value read back
    assert np.array_equal(bf16_bits_to_f32(_bits(back.astype(np.float32))).astype(np.float64), back)


def test_fp4_exact_values():
    # Rows that the format holds exactly come back as they are, ties go to the even code.
    row = np.zeros((1, 64), np.float32)
    row[0, :16] = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -.5, -1, -1.5, -2, -3, -4, -6, 0]) * 448
    row[0, 16:32] = row[0, :16] / 2
    codes, sb, exps = oracle.quantize_fp4(_bits(row))
    assert exps[0] == 127 and sb[0, 0] == 0x7e
    assert np.array_equal(oracle.dequantize_fp4(codes, sb, exps), row.astype(np.float64))
    row = np.zeros((1, 64), np.float32)
    row[0, :16] = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0]) * 448
    codes, _, _ = oracle.quantize_fp4(_bits(row))
    assert codes[0, :16].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 0, 10, 10, 12, 12, 14, 14, 0]


def test_block_bytes(lib):
    assert [lib.kvd_fp4_block_bytes(d) for d in (64, 128, 256, 96, 0, -64)] == [592, 1168, 2320, 0, 0, 0]
    with pytest.raises(ValueError):
        kvd.fp4_block_bytes(96)
    with pytest.raises(ValueError):
        kvd.alloc_cache_fp4(1, 1, 64, 24, device="cpu")
    assert kvd.alloc_cache_fp4(2, 3, 64, 32, device="cpu").shape == (2, 3, 2, 592)


def test_rope_oracle_is_a_rotation():
    r = np.random.default_rng(3)
    turns, _ = kvd.rope_table(64)
    x = r.standard_normal((5, 2, 80))
    pos = np.array([0, 1, -7, 2 ** 31 - 1, -2 ** 31])
    ph = oracle.rope_phases(pos, turns)
    for inter in (False, True):
        y = oracle.rope(x, ph, 1.0, inter)
        assert np.allclose(y[0], x[0]) and np.array_equal(y[..., 64:], x[..., 64:])
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        back = oracle.rope(y, -ph, 1.0, inter)
        assert np.allclose(back, x)
        # scores depend on the distance alone
        q, k = r.standard_normal((2, 1, 1, 64))
        dot = [float((oracle.rope(q, oracle.rope_phases([a], turns), 1.0, inter)
                      * oracle.rope(k, oracle.rope_phases([b], turns), 1.0, inter)).sum())
               for a, b in ((5, 2), (100005, 100002))]
        assert dot[0] == pytest.approx(dot[1], abs=1e-9)


# ---------------------------------------------------------------------------
# refusals, before any launch
# ---------------------------------------------------------------------------

def _rope(**over):
    a = dict(turns=FAKE, factor=1.0, rotary_dim=64, interleaved=0)
    a.update(over)
    return kvd._CRope(a["turns"], a["factor"], a["rotary_dim"], a["interleaved"])


def _apply(lib, rope=None, **over):
    a = dict(x=FAKE, xs=1024, idt=0, y=FAKE * 2, ys=1024, odt=0, pos=FAKE * 3, rows=4, H=8, D=128)
    a.update(over)
    return lib.kvd_rope_apply(ctypes.byref(rope or _rope()), a["x"], a["xs"], a["idt"], a["y"], a["ys"], a["odt"], a["pos"],
                              a["rows"], a["H"], a["D"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(x=None), 1), (dict(y=None), 1), (dict(pos=None), 1), (dict(x=FAKE + 8), 1), (dict(y=FAKE * 2 + 4), 1),
    (dict(pos=FAKE * 3 + 2), 1), (dict(xs=1023), 1), (dict(ys=1020), 1), (dict(ys=1028), 1), (dict(rows=-1), 1),
    (dict(rows=1 << 31), 1), (dict(H=0), 1), (dict(D=12), 1), (dict(D=0), 1), (dict(D=1032, xs=8256, ys=8256), 2),
    (dict(idt=5), 1), (dict(odt=-1), 1), (dict(D=48, xs=384, ys=384), 1),   # rotary_dim 64 past the head
    (dict(y=FAKE + 2048), 1), (dict(y=FAKE + 1024, xs=2048, ys=2048), 1),     # overlaps x
    (dict(y=FAKE, ys=2048), 1), (dict(y=FAKE, odt=1), 1),                     # in place with another stride or type
    (dict(pos=FAKE * 2 + 16), 1),                                             # positions inside y
    (dict(rows=0), 0), (dict(rows=0, y=FAKE), 0),
])
def test_rope_apply_refuses(lib, over, expect):
    assert _apply(lib, **over) == expect


@pytest.mark.parametrize("rope", [dict(turns=None), dict(turns=FAKE + 4), dict(rotary_dim=8), dict(rotary_dim=20),
                                  dict(rotary_dim=144), dict(factor=float("nan"))])
def test_rope_refuses(lib, rope):
    assert _apply(lib, rope=_rope(**rope)) == kvd.ERR_INVALID_ARG
    assert lib.kvd_rope_apply(None, FAKE, 1024, 0, FAKE * 2, 1024, 0, FAKE * 3, 4, 8, 128, None) == kvd.ERR_INVALID_ARG


def _append(lib, fp4=False, rope="rope", cache=None, **over):
    a = dict(q=FAKE, qs=1024, qo=FAKE * 2, qos=1024, k=FAKE * 3, ks=256, v=FAKE * 4, vs=256, pos=FAKE * 5, off=None, B=2,
             N=6, Hq=8, Hkv=2, D=128, status=None)
    a.update(over)
    if fp4:
        c = kvd._CCacheFp4(FAKE * 6, FAKE * 7, None, 64, 0, 0, 0)
        fn = lib.kvd_kv_append_fp4
    else:
        c = kvd._CCache(FAKE * 6, FAKE * 7, None, None, None, 64, 0, 0, 0, 0)
        fn = lib.kvd_kv_append_rope
    for k, v in (cache or {}).items():
        setattr(c, k, v)
    r = _rope() if rope == "rope" else rope
    return fn(ctypes.byref(c), None if r is None else ctypes.byref(r), a["q"], a["qs"], a["qo"], a["qos"], a["k"], a["ks"],
              a["v"], a["vs"], a["pos"], a["off"], a["B"], a["N"], a["Hq"], a["Hkv"], a["D"], a["status"], None)


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "fp4"])
@pytest.mark.parametrize("over,expect", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(pos=None), 1), (dict(k=FAKE * 3 + 8), 1), (dict(ks=248), 1), (dict(vs=260), 1),
    (dict(qs=1000), 1), (dict(qos=1023), 1), (dict(q=None), 1), (dict(qo=None), 1), (dict(B=-1), 1), (dict(N=5), 1),
    (dict(N=-2), 1), (dict(N=1 << 31), 1), (dict(Hkv=0), 1), (dict(Hq=0), 1), (dict(D=100), None), (dict(off=FAKE + 2), 1),
    (dict(status=FAKE + 1), 1), (dict(qo=FAKE + 512), 1), (dict(qo=FAKE, qos=2048), 1),
    (dict(qo=FAKE * 3), 1), (dict(qo=FAKE * 4 + 512), 1), (dict(qo=FAKE * 6), 1), (dict(k=FAKE * 7), 1),
    (dict(pos=FAKE * 6 + 64), 1), (dict(qo=FAKE * 9, pos=FAKE * 9 + 16), 1), (dict(off=FAKE * 7 + 64), 1),  # indices inside what is written
    (dict(qo=FAKE * 9, off=FAKE * 9 + 16), 1),
    (dict(cache=dict(k=None)), 1), (dict(cache=dict(v=FAKE * 6)), 1), (dict(cache=dict(v=FAKE * 6 + 1024)), 1),
    (dict(cache=dict(block_table=FAKE * 8, max_blocks=2, page_size=24, num_pages=4)), 1),
    (dict(cache=dict(block_table=FAKE * 8, max_blocks=0, page_size=16, num_pages=4)), 1),
    (dict(cache=dict(block_table=FAKE * 8 + 2, max_blocks=2, page_size=16, num_pages=4)), 1),
    (dict(N=0), 0), (dict(B=0, N=0), 0), (dict(B=0, N=2), 1),
])
def test_append_refuses(lib, fp4, over, expect):
    if expect is None:
        expect = kvd.ERR_UNSUPPORTED if fp4 else kvd.ERR_INVALID_ARG
    assert _append(lib, fp4, **over) == expect


def test_append_refuses_forms(lib):
    assert _append(lib, rope=None) == kvd.ERR_INVALID_ARG                       # the plain append has its own calls
    assert _append(lib, True, rope=None) == kvd.ERR_INVALID_ARG                 # q without a rotation
    assert _append(lib, True, rope=None, q=None, qo=None, N=0) == kvd.OK
    assert _append(lib, True, cache=dict(s_max=40)) == kvd.ERR_INVALID_ARG      # not whole blocks
    assert _append(lib, cache=dict(k_scales=FAKE * 8)) == kvd.ERR_INVALID_ARG   # one scale array
    assert _append(lib, cache=dict(fp8=1)) == kvd.ERR_INVALID_ARG               # fp8 without scales
    two = dict(k_scales=FAKE * 8, v_scales=FAKE * 9)
    assert _append(lib, D=96, qs=768, qos=768, cache=two) == kvd.ERR_UNSUPPORTED
    assert _append(lib, cache=dict(k_scales=FAKE * 8, v_scales=FAKE * 8)) == kvd.ERR_INVALID_ARG
    assert _append(lib, cache=dict(k_scales=FAKE * 8, v_scales=FAKE * 9 + 2)) == kvd.ERR_INVALID_ARG
    assert _append(lib, N=0, cache=two) == kvd.OK


def _decode4(lib, cache=None, **over):
    a = dict(q=FAKE, lens=FAKE * 2, B=2, T=1, mx=64, Hq=8, Hkv=2, D=128, scale=0.1, n=4, ws=FAKE * 3, wsb=0, out=FAKE * 4, dt=0,
             lse=None, kn=None, vn=None, pos=None, status=None)
    a.update(over)
    c = kvd._CCacheFp4(FAKE * 6, FAKE * 7, None, 64, 0, 0, 0)
    for k, v in (cache or {}).items():
        setattr(c, k, v)
    return lib.kvd_decode_fp4(ctypes.byref(c), a["q"], a["lens"], a["B"], a["T"], a["mx"], a["Hq"], a["Hkv"], a["D"], a["scale"],
                              a["n"], a["ws"], a["wsb"], a["out"], a["dt"], a["lse"], a["kn"], a["vn"], a["pos"], a["status"],
                              None)


@pytest.mark.parametrize("over,expect", [
    (dict(), 3), (dict(ws=None, wsb=1 << 30), 3), (dict(ws=FAKE * 3 + 16, wsb=1 << 30), 1), (dict(q=None), 1), (dict(out=None), 1),
    (dict(lens=None), 1), (dict(q=FAKE + 2), 1), (dict(out=FAKE * 4 + 8), 1), (dict(lens=FAKE + 1), 1), (dict(lse=FAKE + 2), 1),
    (dict(status=FAKE + 2), 1), (dict(B=-1), 1), (dict(T=0), 1), (dict(T=65), 2), (dict(mx=65), 1), (dict(mx=-1), 1),
    (dict(Hq=7), 1), (dict(Hq=130), 2), (dict(D=96), 2), (dict(scale=float("nan")), 1), (dict(n=-1), 1), (dict(dt=2), 1),
    (dict(kn=FAKE), 1), (dict(kn=FAKE, vn=FAKE), 1), (dict(pos=FAKE), 1), (dict(cache=dict(k=None)), 1),
    (dict(cache=dict(v=FAKE + 8)), 1), (dict(cache=dict(s_max=0)), 1), (dict(cache=dict(s_max=72)), 1),
    (dict(cache=dict(block_table=FAKE, max_blocks=2, page_size=8, num_pages=4)), 1), (dict(B=0, wsb=1 << 30), 0),
])
def test_decode_fp4_refuses(lib, over, expect):
    assert _decode4(lib, **over) == expect


def test_plan_fp4(lib):
    assert kvd.decode_plan_fp4(1, 1, 8, 1, 128, 256, num_sms=152) == (1, 0)
    n, ws = kvd.decode_plan_fp4(128, 1, 32, 8, 128, 8192, num_sms=152)
    assert n >= 152 and ws > 0
    # a pair's rows in blocks share the resident CTAs
    n2, _ = kvd.decode_plan_fp4(64, 1, 48, 1, 256, 2048, num_sms=152)
    assert 1 <= n2 <= 152
    assert kvd.decode_plan_fp4(3, 5, 8, 2, 64, 100, num_sms=152, n_split=7)[0] == 7
    for bad, st in ((dict(batch=-1), 1), (dict(n_tokens=0), 1), (dict(n_tokens=65), 2), (dict(head_dim=96), 2),
                    (dict(n_heads_q=130, n_heads_kv=2), 2), (dict(n_split=-1), 1), (dict(max_seq_len=-1), 1)):
        a = dict(batch=1, n_tokens=1, n_heads_q=8, n_heads_kv=2, head_dim=128, max_seq_len=64, num_sms=152, n_split=0)
        a.update(bad)
        with pytest.raises(kvd.KvdError) as e:
            kvd.decode_plan_fp4(**a)
        assert e.value.status == st


@pytest.mark.parametrize("args,expect", [
    # cache, blocks, lens, B, S, S_blocks, max, Hkv, D
    ((None, FAKE * 2, FAKE, 2, 64, 64, 64, 2, 128), 1), ((FAKE * 3, None, FAKE, 2, 64, 64, 64, 2, 128), 1),
    ((FAKE * 3, FAKE * 2, None, 2, 64, 64, 64, 2, 128), 1), ((FAKE * 3, FAKE * 2 + 8, FAKE, 2, 64, 64, 64, 2, 128), 1),
    ((FAKE * 3, FAKE * 2, FAKE, 2, 64, 72, 64, 2, 128), 1), ((FAKE * 3, FAKE * 2, FAKE, 2, 64, 48, 64, 2, 128), 1),
    ((FAKE * 3, FAKE * 2, FAKE, 2, 48, 64, 64, 2, 128), 1), ((FAKE * 3, FAKE * 2, FAKE, 2, 64, 64, 64, 2, 96), 2),
    ((FAKE * 3, FAKE * 3 + 1024, FAKE, 2, 64, 64, 64, 2, 128), 1), ((FAKE * 3, FAKE * 2, FAKE, -1, 64, 64, 64, 2, 128), 1),
    ((FAKE * 3, FAKE * 2, FAKE, 0, 64, 64, 64, 2, 128), 0), ((FAKE * 3, FAKE * 2, FAKE, 2, 64, 64, 0, 2, 128), 0),
])
def test_quantize_fp4_refuses(lib, args, expect):
    cache, blocks, lens, B, S, Sb, mx, H, D = args
    assert lib.kvd_kv_quantize_fp4(cache, blocks, lens, B, S, Sb, mx, H, D, None) == expect
    # the way back: out in the cache's place
    assert lib.kvd_kv_read_fp4(blocks, None, Sb, 0, 0, 0, cache, S, lens, B, mx, H, D, None, None) == expect


def test_fp4_token_limit(lib):
    top = 0x7ffffc00
    c = dict(s_max=0x7ffffff0)
    assert _decode4(lib, cache=c, mx=top) == kvd.ERR_WORKSPACE_TOO_SMALL
    assert _decode4(lib, cache=c, mx=top + 1) == kvd.ERR_UNSUPPORTED
    assert lib.kvd_kv_quantize_fp4(FAKE, FAKE * 2, FAKE * 3, 0, 0x7ffffff0, 0x7ffffff0, top + 1, 1, 64, None) == kvd.ERR_UNSUPPORTED
    assert lib.kvd_kv_read_fp4(FAKE, None, 0x7ffffff0, 0, 0, 0, FAKE * 2, 0x7ffffff0, FAKE * 3, 0, top + 1, 1, 64, None,
                               None) == kvd.ERR_UNSUPPORTED
    assert lib.kvd_kv_quantize_fp4(FAKE, FAKE * 2, FAKE * 3, 0, 0x7ffffff0, 0x7ffffff0, top, 1, 64, None) == kvd.OK


def test_read_fp4_refuses_pages(lib):
    ok = dict(max_blocks=4, page=16, pages=9, mx=64, status=None)

    def call(**over):
        a = {**ok, **over}
        return lib.kvd_kv_read_fp4(FAKE, FAKE * 2, 0, a["max_blocks"], a["page"], a["pages"], FAKE * 3, 64, FAKE * 4, 0, a["mx"], 2,
                                   128, a["status"], None)
    assert call() == kvd.OK
    for over in (dict(max_blocks=0), dict(page=24), dict(page=8), dict(pages=0), dict(max_blocks=3), dict(status=FAKE + 2)):
        assert call(**over) == kvd.ERR_INVALID_ARG, over


def test_python_refusals():
    import torch
    r = kvd.RopeTable(64, device="cpu")
    assert r.turns.shape == (32,) and r.factor == 1.0
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    for fn in (lambda: kvd.rope_apply(r, x, torch.zeros(4, dtype=torch.int32), x),
               lambda: kvd.decode_fp4(x, x, x, x, 4, 1.0, x),
               lambda: kvd.kv_append_rope(r, x[None], x[None], x, x, torch.zeros(4, dtype=torch.int32)),
               lambda: kvd.kv_append_fp4(None, x, x, x, x), lambda: kvd.kv_append_fp4(x, None, x, x, x),
               lambda: kvd.decode_fp4(x, None, x, x, 4, 1.0, x), lambda: kvd.decode_fp4(None, x, x, x, 4, 1.0, x),
               lambda: kvd.rope_apply(None, x, x, x), lambda: kvd.rope_apply(r, None, x, x),
               lambda: kvd.kv_append_rope(r, None, x, x, x, x), lambda: kvd.kv_append_rope(r, x, x, None, x, x),
               lambda: kvd.kv_quantize_fp4(None, x, x, 3), lambda: kvd.kv_read_fp4(x, None, x, 3),
               lambda: kvd.kv_quantize_fp4(x, x, x, 3), lambda: kvd.kv_read_fp4(x, x, x, 3)):
        with pytest.raises((ValueError, TypeError)):
            fn()


def test_plan_fp4_short_sequences(lib):
    """A CTA for every pair, however short, as far as the SMs hold them."""
    for B, T, Hq, Hkv, D, L in ((41, 1, 64, 8, 256, 1), (108, 1, 2, 2, 128, 31), (7, 4, 8, 8, 64, 16)):
        n, _ = kvd.decode_plan_fp4(B, T, Hq, Hkv, D, L, num_sms=152)
        assert min(B * Hkv, 152) <= n <= B * Hkv
    assert kvd.decode_plan_fp4(5, 1, 8, 1, 128, 0, num_sms=152)[0] == 1


# ---------------------------------------------------------------------------
# shapes, before any launch: CPU tensors that say they lie on a device
# ---------------------------------------------------------------------------

@pytest.fixture
def on_device(monkeypatch):
    """(a maker of tensors, the list of launches): nothing is launched, the call's name is noted."""
    import torch

    class There(torch.Tensor):
        def get_device(self):
            return 0

    made, launched = [], []

    def make(*shape, dtype=torch.bfloat16):
        made.append(torch.zeros(*shape, dtype=dtype).as_subclass(There))
        return made[-1]
    monkeypatch.setattr(kvd, "_launch", lambda fn, what, dev, stream, *args: launched.append(what))
    monkeypatch.setattr(kvd, "_rope_on", lambda rope, dev, what: rope._ref)
    return make, launched


def _append_call(make, form, **shapes):
    import torch
    B, Hq, Hkv, D, S = 3, 4, 2, 64, 32
    a = dict(k_new=(B, 4, Hkv, D), v_new=(B, 4, Hkv, D), q=(B, 4, Hq, D), q_out=(B, 4, Hq, D), offsets=None)
    a.update(shapes)
    kw = dict(q=make(*a["q"]) if a["q"] else None, q_out=make(*a["q_out"]) if a["q"] else None,
              row_offsets=None if a["offsets"] is None else make(B + 1, dtype=torch.int32))
    args = make(*a["k_new"]), make(*a["v_new"]), make(B, dtype=torch.int32)
    rope = kvd.RopeTable(64, device="cpu")
    if form == "fp4":
        kvd.kv_append_fp4(*(make(B, Hkv, S // 16, 9 * D + 16, dtype=torch.uint8) for _ in range(2)), *args, rope=rope, **kw)
    else:
        kvd.kv_append_rope(rope, *(make(B, S, Hkv, D) for _ in range(2)), *args, **kw)


@pytest.mark.parametrize("form", ["bf16", "fp4"])
def test_new_rows_of_another_batch_are_refused(lib, on_device, form):
    """[T, B, H, D] where [B, T, H, D] is asked has as many rows, but they are other sequences'."""
    make, launched = on_device
    flat = dict(k_new=(12, 2, 64), v_new=(12, 2, 64), q=(12, 4, 64), q_out=(12, 4, 64))
    _append_call(make, form)
    _append_call(make, form, q=None)
    _append_call(make, form, **flat)                                  # packed rows, 4 to a sequence
    _append_call(make, form, offsets=True, **flat)
    _append_call(make, form, offsets=True, **{n: (1,) + s for n, s in flat.items()})
    _append_call(make, form, k_new=(3, 2, 64), v_new=(3, 1, 2, 64), q=(3, 1, 4, 64), q_out=(3, 4, 64))
    assert len(launched) == 6
    for name in ("k_new", "v_new", "q", "q_out"):
        heads = 4 if name in ("q", "q_out") else 2
        for lead in ((4, 3), (2, 6), (1, 12), (12, 1)):
            with pytest.raises(ValueError):
                _append_call(make, form, **{name: lead + (heads, 64)})
        with pytest.raises(ValueError):
            _append_call(make, form, offsets=True, **{**flat, name: (3, 4, heads, 64)})
    assert len(launched) == 6


def test_positions_and_results_of_another_shape_are_refused(lib, on_device):
    import torch
    make, launched = on_device
    r = kvd.RopeTable(64, device="cpu")

    def call(x, pos, out):
        kvd.rope_apply(r, make(*x), make(*pos, dtype=torch.int32), make(*out))
    right = [((3, 4, 2, 64), (3, 4), (3, 4, 2, 64)), ((3, 4, 2, 64), (12,), (3, 4, 2, 64)), ((12, 2, 64), (12,), (12, 2, 64)),
             ((12, 2, 64), (3, 4), (3, 4, 2, 64)), ((3, 4, 2, 64), (3, 4), (12, 2, 64)),
             ((3, 4, 2, 64), (12, 1), (1, 12, 2, 64))]  # (a one is no batch: the rows in order)
    for x, pos, out in right:
        call(x, pos, out)
    assert len(launched) == len(right)
    for x, pos, out in (((3, 4, 2, 64), (4, 3), (3, 4, 2, 64)), ((3, 4, 2, 64), (3, 4), (4, 3, 2, 64)),
                        ((12, 2, 64), (4, 3), (3, 4, 2, 64)), ((3, 4, 2, 64), (12,), (2, 6, 2, 64)), ((12, 2, 64), (11,), (12, 2, 64))):
        with pytest.raises(ValueError):
            call(x, pos, out)
    assert len(launched) == len(right)


def test_packed_structs_are_the_declared_ones():
    """The bytes that the calls send are the C structs', field by field and to their full size."""
    for pack, struct_type in ((kvd._pack_cache, kvd._CCache), (kvd._pack_fp4, kvd._CCacheFp4)):
        n = len(struct_type._fields_)
        for values in ([0x1111111111111111 * (i + 1) if t is ctypes.c_void_p else 0x01020304 * (i + 1)
                        for i, (_, t) in enumerate(struct_type._fields_)], [0] * n):
            s = struct_type(*values)
            assert len(pack(*values)) == ctypes.sizeof(s)
            assert pack(*values) == bytes(s)
