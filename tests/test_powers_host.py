"""The powers of two behind the draw's weights (csrc/exq_powers.h), compiled for the host as they stand, against 40 digits."""
import ctypes
import os
import subprocess
from decimal import Decimal, localcontext

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixed_bitrate_quantized_amd", "csrc")

SOURCE = """
#include <cmath>
#define __host__
#define __device__
#define __forceinline__ inline
#include "exq_powers.h"
extern "C" void powers(double* table, const double* t, double* out, int n) {
    for (int i = 0; i < exq::kPowers; ++i) table[i] = exq::exp2_series((double)i / exq::kPowers);
    for (int i = 0; i < n; ++i) out[i] = exq::power_of(table, t[i]);
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("powers")
    src, so = str(d / "powers.cpp"), str(d / "powers.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-w", "-shared", "-fPIC", "-I" + CSRC, src, "-o", so], check=True)
    return ctypes.CDLL(so)


def computed(lib, t):
    t = np.ascontiguousarray(t, dtype=np.float64)
    table, out = np.zeros(256), np.zeros(t.size)
    at = lambda x: x.ctypes.data_as(ctypes.POINTER(ctypes.c_double))
    lib.powers(at(table), at(t), at(out), t.size)
    return table, out


def errors(values, t):
    """Relative, of values that should be 2^(t / 256)."""
    with localcontext() as context:
        context.prec = 40
        ln2 = Decimal(2).ln()
        return np.array([float(abs(Decimal(float(v)) / (Decimal(float(x)) / 256 * ln2).exp() - 1)) for v, x in zip(values, t)])


def test_table_entries(lib):
    """A step of the series rounds its two factors and its sum, 2^-53 each, and passes ln(2) / i of what came before it on:
    (1 + 0.7 * 3 + 0.24 * 3 + ..) * 2^-53 is below 2^-51."""
    table, _ = computed(lib, [0.0])
    assert errors(table, np.arange(256)).max() <= 2.0 ** -51


def test_powers_between_entries(lib):
    """All entries, at the ends and the middle of what lies between them and where the cut series is worst, and far powers."""
    f = np.concatenate([np.linspace(-0.5, 0.5, 9), [-0.49999, 0.49999, 0.354, -0.354]])
    t = np.concatenate([(np.arange(-256, 0)[:, None] + f[None, :]).ravel(), [0.0, -1e-9, -2560.5, -12345.25, -16383.5, -200000.49]])
    t = t[t <= 0]
    _, out = computed(lib, t)
    assert errors(out, t).max() <= 2.0 ** -45
    assert computed(lib, [0.0])[1][0] == 1.0
