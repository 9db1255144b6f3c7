"""The verification pass's entry points at the ends of their ranges, on the host."""
import ctypes as C

import pytest

import speculative_decoding_drafter_head_b200 as ds

F = C.c_void_p(0x10000)          # never dereferenced: every call below fails its host checks
INVALID, SMALL = 1, 3


@pytest.mark.parametrize("scale, status", [(3e38, INVALID), (-3e38, INVALID), (2e38, SMALL)])
def test_scale_in_base_two_is_finite(scale, status):
    """The kernel's scores are in base two: a scale that is finite, but not times log2(e), would
    make every score NaN or infinite."""
    st = ds.load().dspark_verify_attention(F, F, F, F, F, F, 4, 8, 32, 8, 128, 16, 64, 64, scale, F,
                                           F, 16, None)
    assert st == status
