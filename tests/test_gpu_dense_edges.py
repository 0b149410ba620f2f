"""GPU tests of the dense attention at the ends of what its description allows: scores as far out as they may be, and
a context attended in shards whose rows are joined by their log-sum-exp. Against 64-bit arithmetic on the
cache's own rows; the element tolerance of one call is derived in test_gpu_dense.py."""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_dense import SCALE, Case, msa  # noqa: F401  (msa: the fixture)

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


@pytest.mark.parametrize("lens,qs,cuts", [
    ([1000, 700, 129], [1, 1, 1], [3]), ([3000, 1500, 260, 140], [1, 5, 8, 8], [1, 2, 9]),
    ([20000, 300], [1, 3], [2, 100])])
def test_shards_of_a_context_join_by_log_sum_exp(msa, lens, qs, cuts):  # noqa: F811
    """As the description has it: one query token a sequence, lengths what the token sees of the shard, tokens that
    see nothing of it left out. Rows err by at most what one call's may, each shard's weighted by its share (the
    shares sum to 1, and so do the bounds); the shares come from two log-sum-exps off by 2^-16 (1 + Z)
    each, and every shard's output is rounded to bf16: (2^-7 + 2^-10 + 2^-15 (1 + Z)) A + 2^-27 E."""
    c = Case(msa, lens, qs, seed=32)
    owner = np.repeat(np.arange(len(qs)), qs)
    pos = np.concatenate([np.arange(n - q, n) for n, q in zip(lens, qs)])
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    parts = []
    for b0, b1 in zip([0] + cuts, cuts + [c.table.shape[1]]):
        seen = np.minimum(pos + 1, 128 * b1) - 128 * b0
        here = np.flatnonzero(seen > 0)
        batch = msa.Batch(dev(np.arange(len(here) + 1)), dev(seen[here]), dev(c.table[owner[here], b0:b1]), 1, T=len(here))
        out = torch.empty(len(here), 64, 128, dtype=torch.uint16, device="cuda")
        lse = torch.empty(len(here), 64, device="cuda")
        ws = torch.empty(msa.msa_dense_attn_workspace_size(len(here), len(here), 1), dtype=torch.uint8, device="cuda")
        msa.msa_dense_attn(batch, c.cache, c.q8[torch.from_numpy(here).cuda()], SCALE, out, ws, lse, status)
        o, s = np.zeros((c.T, 64, 128)), np.full((c.T, 64), -np.inf)
        o[here], s[here] = out.view(torch.bfloat16).double().cpu().numpy(), lse.double().cpu().numpy()
        parts.append((o, s))
    assert msa.status_bits(status) == 0
    total = np.logaddexp.reduce([s for _, s in parts])
    got = sum(np.exp(s - total)[..., None] * o for o, s in parts)
    q64 = oracle.e4m3_decode(c.q8.cpu().numpy())
    for b in range(len(lens)):
        K, V = c.rows(b)
        for t in np.flatnonzero(owner == b):
            for g in range(4):
                hs = slice(16 * g, 16 * g + 16)
                k, v = K[:pos[t] + 1, g], V[:pos[t] + 1, g]
                z = q64[t, hs] @ k.T * SCALE
                m = z.max(-1, keepdims=True)
                e = np.exp(z - m)
                l = e.sum(-1, keepdims=True)
                Z = (np.abs(q64[t, hs]) @ np.abs(k).T).max() * SCALE
                tol = (2.0 ** -7 + 2.0 ** -10 + 2.0 ** -15 * (1 + Z)) * (e / l @ np.abs(v)) + 2.0 ** -27 * np.abs(v).sum(0) / l
                assert (np.abs(got[t, hs] - e / l @ v) <= tol).all(), (b, t, g)
                assert np.abs(total[t, hs] - (m + np.log(l))[:, 0]).max() <= 2.0 ** -16 * (1 + Z)
