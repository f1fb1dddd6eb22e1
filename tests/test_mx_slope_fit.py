"""CPU check of the fit behind GELU's derivative: besides its absolute error, its relative one where
the derivative is small, with the kernel's own coefficients and order of roundings."""

import importlib.util
import os
import re

import numpy as np

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiled_dense_gemm_tlg_b200", "csrc")


def test_gelu_slope_is_relative_where_it_is_small():
    spec = importlib.util.spec_from_file_location("fit_gelu_slope", os.path.join(CSRC, "fit_gelu_slope.py"))
    fit = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fit)
    src = open(os.path.join(CSRC, "tlg_mx_device.cuh")).read()
    vals = re.search(r"gelu_slope_coef\(int k\).*?c\[\d+\] = \{([^}]*)\}", src, flags=re.S).group(1)
    kernel = np.array([float(v.strip().rstrip("f")) for v in vals.split(",")], dtype=np.float32)
    x = np.linspace(-12, -2, 400001).astype(np.float32)
    assert np.abs(fit.gelu_slope_f32(x, kernel) / fit.gelu_slope_exact(x) - 1).max() < 1e-5
    x = np.array([-13, -14, -100, -1e30, -np.inf, 14, 1e30, np.inf], dtype=np.float32)
    assert np.abs(fit.gelu_slope_f32(x, kernel) - (x > 0)).max() < 1e-35
