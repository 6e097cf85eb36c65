"""The check of rotated and moved rows that an unwritten component fails.

A comparison with NaN is false, so ``err > bound`` passes a component that is NaN,
which is what outputs are filled with before the call.  Here a component is right
only if it lies within its bound.
"""
import numpy as np

# relative: half a step of bf16; of |a| + |b| of a pair: the angle's error (tests/test_gpu_operators.py
# derives both)
HALF_STEP = 2.0 ** -8
ANGLE = 2.0 ** -19


def check_written(got, want, size, what):
    """got: float64 array; want and size as oracle.operators gives them."""
    bound = np.where(size > 0, HALF_STEP * np.abs(want) + ANGLE * (1 + HALF_STEP) * size, 0.0)
    with np.errstate(invalid="ignore"):
        err = np.abs(got - want)
        right = err <= bound
    assert right.all(), (f"{what}: {int((~right).sum())} components off, {int(np.isnan(got).sum())} of them NaN, "
                         f"first at {np.argwhere(~right)[0].tolist()}")
