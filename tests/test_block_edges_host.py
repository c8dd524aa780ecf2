"""Rotary sections of each axis' own table on the CPU, of any size from 8 pairs: frequencies against their formulas."""
import math

import numpy as np
import pytest

import blocks_ref as ref
import kv_cache_decode_gb300 as kvd


@pytest.fixture(scope="module")
def lib():
    from kv_cache_decode_gb300 import _build
    _build.build()
    return kvd.load()


def _turns(n, base, scaling, scale, original, slow, fast):
    """Turns per position of an axis' n pairs, as the header has them, in float64: units of 2^-64 turn."""
    R, out = 2.0 * n, []
    if scaling == "base":
        base *= scale ** (R / (R - 2))
    place = lambda t: R * math.log(original / (2 * math.pi * t)) / (2 * math.log(base))  # noqa: E731
    lo, hi = (max(math.floor(place(fast)), 0), min(math.ceil(place(slow)), R - 1)) if scaling == "parts" else (0, 1)
    for i in range(n):
        w = base ** (-2 * i / R)
        keep = 0.0 if scaling == "linear" else 1.0
        if scaling == "parts":
            keep = 1 - (i - lo) / (hi - lo)
        if scaling == "wavelength":
            keep = (original * w / (2 * math.pi) - slow) / (fast - slow)
        keep = min(1.0, max(0.0, keep))
        out.append((w * keep + w / scale * (1 - keep)) / (2 * math.pi) * 2.0 ** 64)
    return np.array(out)


@pytest.mark.parametrize("order", ["blocks", "dealt"])
@pytest.mark.parametrize("sections", [(20, 20), (22, 21, 21), (8, 28, 28), (9, 15), (13, 43, 13, 11), (16, 24, 24), (31, 33)])
@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=4.0)),
                                        ("parts", dict(factor=8.0, original_len=4096.0, slow=1.0, fast=32.0)),
                                        ("wavelength", dict(factor=8.0, original_len=8192.0, slow=1.0, fast=4.0))])
def test_tables_of_each_axis(lib, sections, order, scaling, kw):
    """Ordinary splits of a head over rows and columns, or frames, rows and columns: not multiples of 8 pairs."""
    turns, axes, factor = kvd.rope_axes_table(sections, 1e4, order, per_axis=True, scaling=scaling, **kw)
    assert np.array_equal(axes, ref.axes_of(sections, order == "dealt"))
    assert factor == np.float32(0.1 * math.log(8.0) + 1 if scaling == "parts" else 1)
    for a, n in enumerate(sections):
        want = _turns(n, 1e4, scaling, kw.get("factor", 1.0), kw.get("original_len", 0.0), kw.get("slow"), kw.get("fast"))
        got = turns[axes == a].astype(np.float64)
        # powers, quotients and logarithms of float64, a few roundings each of a power of up to 2^17: 1e-13 of the value
        assert got.shape == want.shape and (np.abs(got - want) <= 1e-13 * want + 1).all()
        if n % 8 == 0:
            slow_fast = {k: kw[k] for k in ("slow", "fast") if k in kw}
            assert np.array_equal(turns[axes == a], kvd.rope_table(2 * n, 1e4, scaling, kw.get("factor", 1.0), kw.get("original_len", 0.0),
                                                                   **slow_fast)[0])


@pytest.mark.parametrize("sections", [(20, 21), (7, 17), (18, 18), (8, 0), (120, 16), (20, 20, 20, 20, 20)])
def test_tables_of_each_axis_refused(lib, sections):
    """All pairs together still are a multiple of 8, up to 128, of at most four axes; each axis has 8 at least."""
    with pytest.raises(kvd.KvdError) as e:
        kvd.rope_axes_table(sections, 1e4, per_axis=True)
    assert e.value.status == kvd.ERR_INVALID_ARG
