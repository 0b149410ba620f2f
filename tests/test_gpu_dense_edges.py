"""GPU tests of the dense attention at the ends of what its description allows, against 64-bit arithmetic on the
cache's own rows; the element tolerance of one call is derived in test_gpu_dense.py."""
import numpy as np
import pytest

from test_gpu_dense import Case, msa  # noqa: F401  (msa: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("qbyte,kbyte,scale", [(0x7E, 0x7E, 0.65), (0x01, 0x01, 2.0 ** 30)])
@pytest.mark.parametrize("n", [200, 1500, 9000])
@pytest.mark.parametrize("q", [1, 8, 20])
def test_scores_as_far_out_as_is_allowed(msa, q, n, qbyte, kbyte, scale):  # noqa: F811
    """|z| up to 1.67e7, from the lowest on the first key to the highest on the last one that all tokens see: the
    largest queries and keys at an ordinary scale, the smallest at a large one. Queries are one value and keys
    multiples of one, so that the scores are exact in any order: equal ones weigh the same, others 4,096 or more apart."""
    c = Case(msa, [n], [q], seed=31)
    c.q8.fill_(qbyte)
    c.q8[:, 1::2, 3] = qbyte | 0x80
    c.kv[:, 0::2, 8192:] = kbyte
    c.kv[int(c.table[0, 0]), 0::2, :64] = 0xFF  # every element the lowest
    last = n - q
    c.kv[int(c.table[0, last // 128]), 0::2, 64 * (last % 128):64 * (last % 128) + 64] = 0x77  # the highest
    out, lse = c.run(msa, scale=scale)
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    c.check(out, lse, scale=float(np.float32(scale)), tokens=[0, q - 1])
