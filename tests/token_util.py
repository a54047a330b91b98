"""Shared helpers of the tests of rotary positions, log probabilities and dropout."""

import numpy as np
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# half a step of the output's type, relative to the value
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
U = 2.0 ** -24  # of fp32 arithmetic


def rand(r, shape, act, scale=1.0, mean=0.0):
    x = torch.from_numpy((mean + scale * r.standard_normal(shape)).astype(np.float32))
    return x.to(DT[act]).cuda()


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def nan(shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def within(got, ref, bound, what):
    """|got - ref| <= bound, element by element; infinities and NaN equal."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, what
    special = ~np.isfinite(ref)
    assert np.array_equal(got[special], ref[special], equal_nan=True), f"{what}: special values"
    bound = np.broadcast_to(bound, ref.shape)
    got, ref, bound = got[~special], ref[~special], bound[~special]
    ok = np.abs(got - ref) <= bound
    if not ok.all():
        over = np.abs(got - ref) / np.maximum(bound, 1e-300)
        raise AssertionError(f"{what}: {np.count_nonzero(~ok)} of {ok.size} beyond the bound, "
                             f"worst {np.nanmax(over):.2f} times")
