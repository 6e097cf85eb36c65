"""Host-side edges of the rotary, compaction and beam-selection calls and of the
block manager calls that go with them (no GPU)."""
import math

import numpy as np
import pytest

from oracle import operators as ref
from tests.written import check_written


def test_an_unwritten_component_fails_the_check():
    """NaN, infinity and a stale value fail; what the formula gives, rounded, passes."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 16))
    want, size = ref.rotate(x, 77, ref.angular_frequencies(8), False)      # components 8 .. 15 pass unchanged
    check_written(want, want, size, "as it should be")
    for at in ((0, 0), (1, 7), (2, 8), (2, 15)):
        for bad in (math.nan, math.inf, -math.inf, want[at] + 1.0):
            got = want.copy()
            got[at] = bad
            with pytest.raises(AssertionError):
                check_written(got, want, size, "planted")
    with pytest.raises(AssertionError):
        check_written(np.full_like(want, math.nan), want, size, "nothing written")
