"""GPU tests of the append's two forms (a half warp a row, and from MANY_TOKENS on a half warp a token): bytes of
msa_kv_insert, slots out of range, values that are not finite. Every byte against the definition."""
import math

import pytest
import torch

from test_gpu_rope import msa  # noqa: F401  (the fixture)
from test_gpu_rope_forms import MANY_TOKENS

pytestmark = pytest.mark.gpu
SIZES = [6, 700, MANY_TOKENS - 1, MANY_TOKENS, MANY_TOKENS + 9]


def rows(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(n, *s, generator=g, device="cuda") * 3 for s in ((4, 128), (4, 128), (128,))]


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("n", SIZES)
def test_unrotated_fp32_rows_are_kv_insert(msa, n, index):  # noqa: F811
    k, v, ik = rows(n, n)
    k[5], v[4], ik[3], k[n - 1], v[n - 2] = 0.0, 1e9, 1e-7, 1e9, 0.0
    pages = n // 128 + 2
    slots = torch.randperm(pages * 128, device="cuda")[:n]
    slots[2::7] = -1
    a, b = msa.Cache.empty(pages, index), msa.Cache.empty(pages, index)
    msa.msa_kv_insert(k, v, ik, slots, a)
    msa.msa_rope_kv_insert(k, v, ik, None, slots, msa.Rope(None), b)
    assert torch.equal(a.kv_pages, b.kv_pages) and torch.equal(a.index_pages, b.index_pages)
    assert (b.kv_pages != 0).any() and (b.index_pages != 0).any()


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", SIZES)
def test_bad_slots_write_nothing(msa, n, dt, index):  # noqa: F811
    """Slots out of range in either half of a warp, alone and next to each other, and one token past the last warp's
    whole ones: the status, the good tokens' bytes, and nothing else, page 0 least of all."""
    k, v, ik = (x.to(dt) for x in rows(n, n))
    pages = n // 128 + 3
    slots = 128 + torch.randperm((pages - 1) * 128, device="cuda")[:n]  # page 0 holds no token's row
    limit = pages * 128
    bad = {0: -2, 3: limit, 4: limit + 1, 5: 1 << 62, n - 1: -(1 << 62)}
    if n > 100:
        bad.update({34: -2, 35: -128, 66: limit, n // 2: limit + 127, n - 20: (1 << 32) + 130, n - 3: -(1 << 32) + 130})
    good = slots.clone()
    for at, s in bad.items():
        slots[at], good[at] = s, -1
    pos = torch.arange(n, dtype=torch.int32, device="cuda") + 1000
    rope, w = msa.Rope.frequencies(64, 1e4), torch.rand(128, device="cuda") + 0.5
    caches = []
    for s in (slots, good):
        c = msa.Cache.empty(pages, index)
        c.kv_pages.fill_(0x5A)
        c.index_pages.fill_(0x5A)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        msa.msa_rope_kv_insert(k, v, ik, pos, s, rope, c, w, w, status=status)
        assert msa.status_bits(status) == (1 << msa.MSA_ERR_DEVICE_FAULT if s is slots else 0)
        caches.append(c)
    a, b = caches
    assert torch.equal(a.kv_pages, b.kv_pages) and torch.equal(a.index_pages, b.index_pages)
    assert (a.kv_pages[:msa.KV_PAGE_BYTES] == 0x5A).all()
    assert (a.index_pages[:msa.INDEX_PAGE_BYTES[index]] == 0x5A).all()
    msa.msa_rope_kv_insert(k, v, ik, pos, slots, rope, a, w, w)  # no status word: skipped all the same
    assert torch.equal(a.kv_pages, b.kv_pages) and torch.equal(a.index_pages, b.index_pages)


def nvfp4(x):
    """The E4M3 bytes that the cache's form of x [.., 128] stands for (CPU tensor, fp32)."""
    grp = x.unflatten(-1, (8, 16))
    amax = torch.nan_to_num(grp.abs(), nan=0.0, posinf=math.inf).amax(-1, keepdim=True)
    scale = (amax / 6).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    r = torch.nan_to_num(grp / scale, nan=0.0, posinf=math.inf, neginf=-math.inf)
    r = torch.where(scale == 0, torch.zeros(()), r)
    mag = torch.zeros_like(r)
    for lo, hi, to_even in ((0, .5, 0), (.5, 1, 1), (1, 1.5, 1), (1.5, 2, 2), (2, 3, 2), (3, 4, 4), (4, 6, 4)):
        a, mid = r.abs(), (lo + hi) / 2
        mag = torch.where((a > mid) | ((a == mid) & (to_even == hi)), torch.tensor(float(hi)), mag)
    want = (torch.copysign(mag, r) * scale).clamp(-448.0, 448.0)
    return torch.where(mag == 0, torch.zeros(()), want).to(torch.float8_e4m3fn).view(torch.uint8).view(x.shape)


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("n", SIZES)
def test_values_that_are_not_finite(msa, n, index):  # noqa: F811
    """NVFP4: an infinity saturates its group's scale and itself, a NaN becomes 0 and counts for no maximum. An FP8 index
    key: an infinity becomes 448, a NaN stays one. The rest of a row is as ever, whichever row of a warp it is."""
    inf, nan = math.inf, math.nan
    g = torch.Generator().manual_seed(4)
    x = torch.randn(n, 4, 128, generator=g)
    x[0::6, :, 0], x[0::6, :, 17], x[0::6, :, 33], x[0::6, :, 47] = inf, -inf, nan, 3e38
    x[1::6, :, 5], x[1::6, :, 6], x[1::6, :, 14] = nan, inf, 1e30
    x[2::6, :, :16], x[2::6, :, 16:32], x[2::6, :, 32:48] = nan, inf, -inf
    x[3::6, :, :16], x[3::6, :, 16:32], x[3::6, :, 32:48] = 0.0, 1e-40, -1e-3
    x[4::6, :, 96:] = nan
    pages = n // 128 + 2
    slots = torch.randperm(pages * 128, generator=g)[:n].cuda()
    cache = msa.Cache.empty(pages, index)
    xg = x.cuda()
    msa.msa_rope_kv_insert(xg, xg, xg[:, 1], None, slots, msa.Rope(None), cache)
    k, v = (torch.empty(n, 4, 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    ik = torch.empty(n, 128, dtype=torch.uint8, device="cuda")
    msa.msa_kv_read(slots, cache, k, v, ik)
    want = nvfp4(x)
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)
    if index == 1:
        want = x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        want[x.isnan()] = 0x7F
    assert torch.equal(ik.cpu(), want[:, 1])
