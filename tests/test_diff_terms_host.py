"""PA_DIFF_ONE_TERM is prefill's flag alone (no GPU: every call is refused, or has nothing to
do, before anything is launched)."""
import ctypes

import pytest

from tests.test_step_operators_host import INVALID, B, _decode_diff, _prefill_diff  # noqa: F401


@pytest.mark.parametrize("keys", [0, 1])
def test_one_term_is_of_prefill_alone(B, keys):  # noqa: F811
    assert _prefill_diff(B, seqs=0, dflags=B.PA_DIFF_ONE_TERM | keys) == 0
    assert _prefill_diff(B, seqs=0, dflags=4 | keys) == INVALID
    assert _decode_diff(B, seqs=0, dflags=B.PA_DIFF_ONE_TERM | keys) == INVALID


def test_the_flags_value_is_the_headers(B):  # noqa: F811
    import os
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pa.h")
    with open(header) as f:
        line = next(x for x in f if x.startswith("#define PA_DIFF_ONE_TERM"))
    assert int(line.split()[2].rstrip("u"), 0) == B.PA_DIFF_ONE_TERM
    assert ctypes.sizeof(B.PaDiff) == 32
