"""The quotient of the capped scores, on the host: the kernels' coefficients have
the error that their comment states."""
import importlib.util
import os
import re

import numpy as np

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_compression_fkv_b200", "csrc")


def load():
    spec = importlib.util.spec_from_file_location("fit_tanh", os.path.join(CSRC, "fit_tanh.py"))
    fit = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fit)
    with open(os.path.join(CSRC, "paged_common.cuh")) as f:
        text = f.read()

    def numbers(name):
        found = re.search(name + r" = (?:\{([^}]*)\}|([^,;{]*))", text)
        body = found.group(1) or found.group(2)
        return np.array([float(x.strip().rstrip("f")) for x in body.split(",")])

    return fit, numbers


def test_error_of_the_kernels_quotient():
    fit, numbers = load()
    P, Q = numbers(r"constexpr float P\[5\]"), numbers(r"constexpr float Q\[4\]")
    most = numbers("kTanhMost")[0]
    assert most == fit.LIMIT and len(P) == 5 and len(Q) == 4
    assert np.polyval(Q[::-1], most ** 2) < 176  # four of them share a reciprocal
    y = np.concatenate([np.logspace(-30, -2, 4000), np.linspace(0.01, 20, 400001)])
    z = np.minimum(y, most)
    exact = np.tanh(y)
    quotient = z * np.polyval(P[::-1], z * z) / np.polyval(Q[::-1], z * z)
    # the fit's 2.63e-7; its coefficients rounded to fp32, half a step (2^-24
    # of P, of whose terms all but one small one are positive, and of Q); at and
    # behind the cut 1 - tanh(8) = 2.3e-7 more
    bound = 2.64e-7 + 2 * 2.0 ** -24
    assert np.max(np.abs(quotient / exact - 1)[y <= most]) <= bound
    assert np.max(np.abs(quotient / exact - 1)) <= bound + 2.3e-7
    y32 = np.concatenate([y, -y]).astype(np.float32)
    got = fit.tanh32(P, Q, y32).astype(np.float64)
    assert np.max(np.abs(got / np.tanh(y32.astype(np.float64)) - 1)) <= 9 * 2.0 ** -24


def test_error_of_the_form_for_small_scores():
    fit, numbers = load()
    S, small = numbers(r"constexpr float S\[4\]"), numbers("kTanhSmall")[0]
    assert small == fit.SMALL and len(S) == 4
    y = np.concatenate([np.logspace(-30, -2, 4000), np.linspace(0.01, small, 400001)])
    u = y * y
    # the fit's 1.5e-8; coefficients off by half a step, in a sum that is below 1/12
    assert np.max(np.abs((1 + u * np.polyval(S[::-1], u)) * y / np.tanh(y) - 1)) <= 1.51e-8 + 2.0 ** -24 / 12
    got = fit.small32(S, np.concatenate([y, -y])).astype(np.float64)
    y32 = np.concatenate([y, -y]).astype(np.float32).astype(np.float64)
    assert np.max(np.abs(got / np.tanh(y32) - 1)) <= 2 * 2.0 ** -24


def test_the_fits_have_not_moved():
    fit, _ = load()
    assert fit.fit(points=600)[2] <= 2.65e-7
    assert fit.fit_small()[1] <= 1.51e-8
