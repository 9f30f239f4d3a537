"""The polynomials compiled into the masked-attention kernels, checked on the
host: the coefficients are read out of the source and their error measured
against numpy's 2^x and tanh in f64, so that a mistyped coefficient fails here,
without a GPU."""
import pathlib
import re

import numpy as np
import pytest

SRC = (pathlib.Path(__file__).resolve().parents[1] / "jepa_video_encoder_b200" / "csrc" / "masked_attention.cu").read_text()


def _exp2_coefficients():
    body = SRC[SRC.index("void ex2_poly2("):]
    body = body[:body.index("float ya, yb")]
    first, second = body.split("} else {")
    take = lambda s: [float(a) for a, b in re.findall(r"f2_pack\((\d\.\d+)f, (\d\.\d+)f\)", s) if a == b]  # noqa: E731
    return take(first[first.index("if constexpr (BF)"):]), take(second)


@pytest.mark.parametrize("which,terms,bound", [(0, 4, 7.6e-5), (1, 5, 2.7e-6)])
def test_exp2_polynomial(which, terms, bound):
    c = _exp2_coefficients()[which]
    assert len(c) == terms
    f = np.linspace(-0.5, 0.5, 100001)
    y = np.zeros_like(f)
    for v in c:   # in Horner's order: the highest first
        y = y * f + np.float64(np.float32(v))
    assert np.abs(y / np.exp2(f) - 1).max() <= bound


@pytest.mark.parametrize("bf16,terms,bound", [("true", 5, 7.0e-6), ("false", 6, 6.2e-7)])
def test_tanh_polynomial(bf16, terms, bound):
    body = SRC[SRC.index(f"struct TanhPoly<{bf16}>"):]
    vals = re.search(r"constexpr float v\[\d\] = \{([^}]*)\}", body).group(1)
    c = [float(x.strip().rstrip("f")) for x in vals.split(",")]
    assert len(c) == terms
    z = np.linspace(1e-4, 1, 100001)
    y = np.zeros_like(z)
    for v in reversed(c):
        y = y * z * z + np.float64(np.float32(v))
    assert np.abs(y * z / np.tanh(z) - 1).max() <= bound
