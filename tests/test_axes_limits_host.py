"""The most tokens that the rotation with several axes and the append by a slot map take, without a GPU: one
more is refused before any launch, whatever a workgroup's work is."""
import ctypes

import pytest

from packed_varlen_rotary_rope_amd import attention as A

EINVAL = -1
FAKE, OTHER = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000)  # never dereferenced: every call is refused


@pytest.mark.parametrize("D,tokens", [(2, 16), (64, 16), (256, 16), (258, 15), (384, 10), (512, 8)])
@pytest.mark.parametrize("heads", [1, 300])
def test_one_token_too_many(D, tokens, heads):
    T = 33554431 * tokens + 1
    sections = (ctypes.c_int32 * 1)(D // 2)
    assert A._lib.rope_qk_apply_axes(FAKE, OTHER, FAKE, OTHER, T, heads, 1, D, 0, 0, 0, 0, FAKE, T, sections, 1, 0,
                                     1e4, 1.0, 1, 1, None) == EINVAL
    assert A._lib.kv_append_slots(FAKE, OTHER, FAKE, FAKE, OTHER, OTHER, T, heads, 1, D, 0, 0, 0, 0, 9, 16, 16 * D, D, D,
                                  FAKE, FAKE, T, sections, 1, 0, 1e4, 1.0, 1, None) == EINVAL
