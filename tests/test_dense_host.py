"""Host-side refusals of the dense attention that need no GPU: nothing is launched."""
import ctypes
import math

import pytest

from test_rope_host import INVALID, A, BatchC, CacheC, Geo, lib  # noqa: F401  (lib: the fixture)


@pytest.mark.parametrize("scale", [4.4e12, 1e31, 2.4e38, 3e38, math.inf, math.nan, 0.0, -1.0])
def test_scales_without_a_score_in_range_are_refused(lib, scale):  # noqa: F811
    r = ctypes.byref
    geo = Geo(64, 4, 128, 128, 128, 16, 1, 0)
    need = lib.msa_dense_attn_workspace_size(r(geo), 1, 1, 1)
    for T in (1, 0):
        assert lib.msa_dense_attn(r(geo), r(BatchC(1, T, A, A, A, 16, 1)), r(CacheC(A, None, 0, 8)), A, scale, A, need, A,
                                  None, None, None) == INVALID
    assert lib.msa_dense_attn(r(geo), r(BatchC(1, 0, A, A, A, 16, 1)), r(CacheC(A, None, 0, 8)), A, 2.0 ** 42, A, need, A,
                              None, None, None) == 0
