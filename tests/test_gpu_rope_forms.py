"""GPU parity of the forms that the rotation and the append take from some size on: many rows a half warp, a
half warp a token. Sizes come from the rules' own thresholds; the tolerances are test_gpu_rope.py's."""
import numpy as np
import pytest
import torch

from test_gpu_rope import check_e4m3, fp32_slack, make_rows, msa, rotated64  # noqa: F401  (msa: the fixture)

pytestmark = pytest.mark.gpu
SMS = 152  # the rules' own count; test_rope_rules.py holds these sizes to the rules
MANY_ROWS = 6 * 16 * SMS + 1
FEW_HEADS_ROWS = 8 * 6 * 16 * SMS + 1
MANY_HEADS = 8  # of 16 bits, from which MANY_ROWS holds
MANY_TOKENS = 3 * 16 * SMS // 2
FORMS = [(0, 64, True, True), (1, 128, True, True), (1, 32, True, False), (0, 128, False, True), (0, 16, True, False),
         (1, 96, False, False), (0, 0, True, True), (0, 112, False, False), (1, 16, True, True)]


@pytest.mark.parametrize("heads,layout,rot,norm,packed", [(64, *f) for f in FORMS] + [
    (h, *f) for h in (8, 9, 24, 100) for f in (FORMS[1], FORMS[3], FORMS[5])])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_rope_fp8_of_many_rows(msa, dt, heads, layout, rot, norm, packed, rows=MANY_ROWS):  # noqa: F811
    """From the threshold on: the last CTA not full, tokens of 8 to 100 rows, so that a CTA's 64 (fp32: 32) rows touch up
    to nine tokens and as little as a part of one."""
    T = -(-rows // heads) + 3
    rng = np.random.default_rng(T + rot)
    x = make_rows(T, heads, dt, packed, T)
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    pos[[0, T // 2, T - 1]] = [2 ** 31 - 1, -5, 131071]
    w = rng.uniform(0.5, 1.5, 128).astype(np.float32) if norm else None
    freq = 5e6 ** (-np.arange(rot // 2) / max(rot // 2, 1))
    rope = msa.Rope(torch.from_numpy(freq).cuda() if rot else None, layout, 1.2)
    out = torch.full((T * heads * 128 + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    msa.msa_rope_fp8(x, torch.from_numpy(pos).cuda(), rope, out, None if w is None else torch.from_numpy(w).cuda(), 1e-5)
    torch.cuda.synchronize()
    got = out.cpu().numpy()
    assert (got[T * heads * 128:] == 0xAB).all()
    y = rotated64(x.float().cpu().numpy(), pos, freq, layout, 1.2, w, 1e-5)
    check_e4m3(got[:T * heads * 128].reshape(T, heads, 128), y, fp32_slack(y))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("heads,layout,rot", [(1, 0, 128), (1, 1, 16), (4, 0, 64), (7, 1, 96)])
def test_rope_fp8_of_many_tokens_with_few_heads(msa, dt, heads, layout, rot):  # noqa: F811
    """As many rows of few heads: mostly a row a half warp, up to 16 tokens a CTA."""
    test_rope_fp8_of_many_rows(msa, dt, heads, layout, rot, True, True)


@pytest.mark.parametrize("dt,heads,layout,rot,norm", [("bf16", 4, 0, 64, True), ("f16", 5, 1, 128, False), ("f32", 2, 0, 128, True)])
def test_rope_fp8_of_very_many_tokens_with_few_heads(msa, dt, heads, layout, rot, norm):  # noqa: F811
    """Many rows a half warp with up to 17 tokens a CTA, the most that one takes."""
    test_rope_fp8_of_many_rows(msa, dt, heads, layout, rot, norm, True, FEW_HEADS_ROWS)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("heads", [64, 9])
def test_both_forms_give_the_same_bytes(msa, dt, heads):  # noqa: F811
    """A call from the threshold on and one below it: a row's bytes do not depend on its batch."""
    T = -(-MANY_ROWS // heads)
    x = make_rows(T, heads, dt, True, T)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 977
    rope, w = msa.Rope.frequencies(64, 5e6), torch.rand(128, device="cuda") + 0.5
    a, b = (torch.zeros(T, heads, 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    assert T * heads >= MANY_ROWS > (T - 1) * heads
    msa.msa_rope_fp8(x, pos, rope, a, w)
    msa.msa_rope_fp8(x[:T - 1], pos, rope, b, w)
    assert torch.equal(a[:T - 1], b[:T - 1])
