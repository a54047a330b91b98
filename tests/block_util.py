"""Shared helpers of the tests of layer normalisation and attention.

Tolerances.  A bf16 rounding has a relative error of at most 2^-9; the
attention kernels round three times on the way to an output (the softmax
weight or its gradient, the stored o behind the backward's row sums, the
output), so the norm-wise bound is 3 * 2^-9 = 5.9e-3, and layer
normalisation, which rounds its output alone, stays under 2^-9 plus its fp32
sums' errors.  fp32 results carry sums of at most a few thousand terms:
sqrt(4096) * 2^-24 = 4e-6 for random signs, bounded here by 1e-5.  The
largest single error is held to ten of the norm-wise bounds of the larger of
the element and the tensor's root mean square."""

import numpy as np

TOL = {"f32": 1e-5, "bf16": 6e-3}
NORM_TOL = {"f32": 1e-5, "bf16": 2.1e-3}


def assert_near(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, what
    if not ref.size:
        return
    special = ~np.isfinite(ref)
    assert np.array_equal(got[special], ref[special], equal_nan=True), f"{what}: special values"
    got, ref = got[~special], ref[~special]
    assert np.isfinite(got).all(), f"{what}: not finite"
    d, norm = got - ref, np.linalg.norm(ref)
    rms = norm / np.sqrt(max(1, ref.size))
    if norm == 0:
        assert np.abs(d).max(initial=0.0) <= tol, what
        return
    rel = np.linalg.norm(d) / norm
    worst = (np.abs(d) / np.maximum(rms, np.abs(ref))).max()
    assert rel <= tol, f"{what}: rel {rel:.3e} > {tol:.1e}"
    assert worst <= 10 * tol, f"{what}: worst {worst:.3e} > {10 * tol:.1e}"
