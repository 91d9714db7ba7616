"""The polynomial of capped scores, as the host computes it for a call."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from paged_kv_attention_25_gb300 import pkv

CSRC = os.path.join(os.path.dirname(pkv.__file__), "csrc")
LOG2E = np.float32(1.4426950408889634)


@pytest.fixture(scope="module")
def cap_poly(tmp_path_factory):
    """(base, cap_out) -> small, [q0 .. q3], as numpy floats of 32 bits."""
    d = tmp_path_factory.mktemp("cap")
    src, lib = d / "cap.cpp", d / "cap.so"
    src.write_text('#include "score_cap.h"\nextern "C" void cap(float b, float c, float* out) {\n'
                   "  const pkv::CapPoly p = pkv::cap_poly(b, c);\n  out[0] = p.small;\n"
                   "  for (int i = 0; i < 4; ++i) out[1 + i] = p.q[i];\n}\n")
    subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)],
                   check=True)
    fn = ctypes.CDLL(str(lib)).cap
    fn.argtypes = [ctypes.c_float, ctypes.c_float, ctypes.POINTER(ctypes.c_float)]
    fn.restype = None

    def call(base, cap_out):
        out = (ctypes.c_float * 5)()
        fn(base, cap_out, out)
        return np.float32(out[0]), np.array(out[1:], np.float32)
    return call


def base_of(scale, k_scale, softcap):
    return np.float32(np.float32(np.float32(scale) * np.float32(k_scale)) / np.float32(softcap))


def check(small, q, base, cap_out):
    """Off by 6e-7 of the score as a polynomial, and by half a step of fp32 for each coefficient, whose terms' magnitudes add up
    to at most (1 + 1/12 + 1/120 + 1/1400) of the score's bound y: 2^-23 of it in all."""
    x = np.linspace(0, float(small), 4001)[1:]
    want = float(cap_out) * np.tanh(float(base) * x)
    z = x * x
    c = q.astype(np.float64)
    got = x * (c[0] + z * (c[1] + z * (c[2] + z * c[3])))
    assert (np.abs(got - want) <= (6e-7 + 2.0 ** -23) * float(cap_out) * float(base) * x).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("k_scale", [1.0, 0.03, 2.0 ** -6, 4 / 448, 2 / 448])
@pytest.mark.parametrize("softcap", [5.0, 30.0, 50.0])
def test_common_scales_and_caps_have_the_short_way(cap_poly, d, k_scale, softcap):
    """Scales of FP8 pools whose largest value is 2 or 4, and no scale, with the caps that models use."""
    base, cap_out = base_of(d ** -0.5, k_scale, softcap), np.float32(softcap) * LOG2E
    small, q = cap_poly(base, cap_out)
    assert small == np.float32(0.5) / base
    check(small, q, base, cap_out)


def test_no_coefficient_leaves_the_range(cap_poly):
    """Over all scales and caps that are accepted: a coefficient is a normal number, or no score counts as small."""
    lo, hi = float(np.finfo(np.float32).tiny), float(np.finfo(np.float32).max)
    some = none = 0
    for scale in 2.0 ** np.arange(-90, 91, 3):
        for softcap in 2.0 ** np.arange(-30, 31, 3):
            base, cap_out = base_of(scale, 1.0, softcap), np.float32(softcap) * LOG2E
            small, q = cap_poly(base, cap_out)
            if small == 0:
                none += 1
                assert (q == 0).all()
            else:
                some += 1
                assert ((np.abs(q) >= lo) & (np.abs(q) <= hi)).all()
                check(small, q, base, cap_out)
    assert some > 100 and none > 100
