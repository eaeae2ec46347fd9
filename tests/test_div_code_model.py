"""The E4M3 code of a corrected FP32 quotient equals the code of the IEEE
quotient fl32(x / s) (CPU replay of the checkpoint kernels' quantization).

The kernels form q1 = q0 + (x - q0 s) y from q0 = x y and y = RN(1 / s).  Why
its code is that of fl32(x / s):
* away from an E4M3 midpoint m both quotients, within an ulp or two of x / s, lie
  on the same side of it;
* the codes could differ only where x / s is next to one of the FP32 rounding
  midpoints beside m, m + h and m - h with h half an ulp.  There x y is off by
  less than one ulp (y by half an ulp), so q0 is one of the two floats around,
  half an ulp from x / s; x - q0 s is exact, and the error left is that of y in
  (x - q0 s) y: below 2^-25 ulp.  But x / s cannot be that close: x - s m is a
  multiple of 2^-27 and s h of 2^-47 (in units of the exponents of s and m), so
  their difference is 0 or at least 2^-24 ulp of the quotient, and 0 it cannot
  be, as s (m + h) has more than 24 significant bits.
The replay goes through every bf16 amax mantissa against every bf16 value below
it, and through FP32 values placed next to those points.
"""
import ctypes
import shutil
import subprocess
from pathlib import Path

import numpy as np
import pytest

import oracle

HERE = Path(__file__).resolve().parent


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    out = tmp_path_factory.mktemp("div") / "libdiv.so"
    subprocess.run([cc, "-O2", "-ffp-contract=off", "-shared", "-fPIC", str(HERE / "div_code_model.c"), "-o", str(out),
                    "-lm"], check=True)
    lib = ctypes.CDLL(str(out))
    lib.quotients.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                              ctypes.c_void_p]

    def run(x, s, nudge=0):
        x, s = (np.ascontiguousarray(v, dtype=np.float32) for v in (x, s))
        q, ok = np.empty_like(x), np.empty(x.size, np.uint8)
        lib.quotients(x.ctypes.data, s.ctypes.data, x.size, nudge, q.ctypes.data, ok.ctypes.data)
        return q, ok.astype(bool)

    return run


def _codes_equal(x, s, q):
    with np.errstate(over="ignore"):
        exact = (x / s).astype(np.float32)
    a, b = oracle.e4m3_encode_array(q), oracle.e4m3_encode_array(exact)
    bad = np.flatnonzero(a != b)
    assert bad.size == 0, (x[bad[:3]], s[bad[:3]], a[bad[:3]], b[bad[:3]])


@pytest.mark.parametrize("shift", [0, -70, 110])
def test_every_bf16_value_under_every_bf16_amax(model, shift):
    """All 128 amax mantissas; every bf16 value of the 21 binades below (a scale
    of 2^shift moves both alike)."""
    man = (1.0 + np.arange(128) / 128.0).astype(np.float64)
    vals = np.concatenate([man * 2.0 ** e for e in range(-20, 1)])
    for amax in man:
        a = np.float32(amax * 2.0 ** shift)
        x = (vals[vals <= amax] * 2.0 ** shift).astype(np.float32)
        s = np.full(x.size, a / np.float32(448.0), np.float32)
        for sign in (1, -1):
            q, ok = model(sign * x, s)
            assert ok.all()
            _codes_equal(sign * x, s, q)


def test_fp32_values_next_to_the_critical_points(model):
    """x = the FP32 values around s m and s (m +- h) for every E4M3 midpoint m and
    random scales: quotients as close to the critical points as they can come."""
    rng = np.random.default_rng(1)
    dec = np.sort(oracle.e4m3_decode_table()[:0x7F])
    mid = (dec[1:] + dec[:-1]) / 2                      # 126 midpoints, the subnormal ones among them
    s = (1.0 + rng.random(3000)).astype(np.float32) * np.float32(2.0) ** rng.integers(-60, 60, 3000).astype(np.float32)
    x = []
    for off in (0.0, 2.0 ** -24, -2.0 ** -24, 2.0 ** -25, -2.0 ** -25):
        x.append((s[:, None].astype(np.float64) * (mid * (1 + off))[None, :]).astype(np.float32))
    x = np.stack(x)
    for step in (0, 1, -1):
        y = x.copy()
        if step:
            y = np.nextafter(y, np.float32(np.inf if step > 0 else 0)).astype(np.float32)
        ss = np.broadcast_to(s[None, :, None], y.shape)
        q, ok = model(y.reshape(-1), ss.reshape(-1))
        assert ok.all()
        _codes_equal(y.reshape(-1), np.ascontiguousarray(ss).reshape(-1), q)


def test_zeros_keep_their_sign_and_tiny_values_give_zero(model):
    x = np.array([0.0, -0.0, 1e-38, -1e-38, 1e-45, -1e-45], np.float32)
    for s in (np.float32(1.0), np.float32(2.0 ** -80), np.float32(7.5e35)):
        q, _ = model(x, np.full(x.size, s, np.float32))
        tiny = np.abs(q) < 2.0 ** -10
        assert np.array_equal(np.signbit(q), np.signbit(x))
        assert tiny[:2].all() and (s != 1.0 or tiny.all())


def test_the_check_rejects_a_reciprocal_that_is_an_ulp_off(model):
    rng = np.random.default_rng(2)
    s = (1.0 + rng.random(20000)).astype(np.float32)
    assert model(s, s)[1].all()
    for nudge in (-1, 1, 2):
        assert not model(s, s, nudge)[1].any()
