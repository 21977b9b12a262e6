"""The 8-bit grouped-query cache where its numbers are furthest apart, against
the 64-bit definition (tests/gqa8_ref.py) and the bounds derived there."""

import pytest
import torch

import bit_kv_cache_nvfp4_gb300 as kv
import gqa8_ref as ref
from test_gpu_gqa8 import BF16, F16, dev, ints

pytestmark = pytest.mark.gpu

# query heads a kv head: items of 8, 16 and 24 rows, and the prompt kernel's
HEADS = [(4, 128, BF16), (4, 64, F16), (16, 128, BF16), (12, 64, F16), (20, 128, F16), (40, 64, BF16), (40, 128, F16)]
OCTAVES = [12, 16, 20, 24, 40, 90]


def check(c, news, hq, dtype, window=0, sm_scale=None, q=None, seed=0):
    """Attention against its definition; a value beyond f16's range is an
    infinity there, as in any rounding to the type.  The bounds' 2^-25 is half of
    f16's least step: bf16, whose least is 2^-133, does without."""
    device, d = c.pool.device, c.pool.shape[4]
    cu = ref.cu_of(news)
    if q is None:
        g = torch.Generator(device=device).manual_seed(seed)
        q = torch.randn(cu[-1], hq, d, device=device, generator=g).to(dtype)
    scale = d ** -0.5 if sm_scale is None else sm_scale
    err = torch.zeros(1, dtype=torch.int32, device=device)
    out, lse = kv.attention_gqa8(q, c.pool, c.scales, c.page_table, c.seq_lens, ints(cu, device), max(news), scale,
                                 window=window, dev_err=err)
    want = ref.attention(q, c.pool, c.scales, c.table, c.lens, cu, scale, window)
    tol, lse_tol = ref.bounds(*want, dtype, d)
    if dtype == BF16:
        tol = tol - 2.0 ** -25 + 2.0 ** -134
    top = torch.finfo(dtype).max
    assert int(err.item()) == 0 and not out.isnan().any()
    off = (out.double().clamp(-top, top) - want[0].clamp(-top, top)).abs()
    worst = float((off / tol).max())
    assert worst <= 1, f"out error {float(off.max()):.3g}, {worst:.3g} of its bound"
    worst = float(((lse.double() - want[1]).abs() / lse_tol).max())
    assert worst <= 1, f"lse error {worst:.3g} of its bound"


def apart(c, b, big, octaves):
    """V of request b: page `big` of each pair `octaves` above the other one."""
    for i, page in enumerate(c.table[b]):
        if page >= 0:
            c.scales[page, :, 1] = 127 + (octaves // 2 if i % 2 == big else -(octaves - octaves // 2))


# ---------------------------------------------------------------------------
# neighbouring pages of a tile, their values far apart: a row is held to the
# mean of |v| under its own softmax, in which a page that it does not see, or
# that has next to no weight, does not count.
# (A weight enters its product with 2^-8 or 2^-11 of itself, or, where weight *
# 2^e is below 2^-14 of the tile's largest, 2^-22 of that: which is what the
# bounds say, for the largest weight * 2^e stands for the largest weight * |v|.)
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("octaves", OCTAVES)
@pytest.mark.parametrize("g,d,dtype", HEADS[:2] + HEADS[5:])
def test_drafts_across_a_page_border(octaves, g, d, dtype):
    """The first rows see the small page alone, the last ones both."""
    c = ref.Cache([66, 194, 300], 2, d, dev(), seed=octaves)
    for b in range(3):
        apart(c, b, 1, octaves)
    check(c, [5, 4, 1], 2 * g, dtype, seed=g)


@pytest.mark.parametrize("octaves", OCTAVES)
@pytest.mark.parametrize("g,d,dtype", HEADS[:2] + HEADS[5:])
def test_windows_that_leave_the_large_page(octaves, g, d, dtype):
    """A window that the first rows' keys of the large page fall into and the
    last rows' do not."""
    c = ref.Cache([128, 258, 640], 2, d, dev(), seed=octaves)
    for b in range(3):
        apart(c, b, 0, octaves)
    check(c, [5, 4, 6], 2 * g, dtype, window=62, seed=g)


@pytest.mark.parametrize("octaves", OCTAVES)
@pytest.mark.parametrize("nats", [5.0, 60.0])
@pytest.mark.parametrize("g,d,dtype", HEADS)
def test_large_values_of_little_weight(octaves, nats, g, d, dtype):
    """Every second page has large values whose scores are `nats` below the
    others': k = -1 against rows of q that sum to nats / sm_scale."""
    device, hkv = dev(), 2
    c = ref.Cache([128, 100, 1000, 5000], hkv, d, device, seed=octaves)
    for b in range(4):
        apart(c, b, b % 2, octaves)
        for i, page in enumerate(c.table[b]):
            if page < 0:
                continue
            c.scales[page, :, 0] = 127
            c.pool[page, :, 0] = 0xB8 if i % 2 == b % 2 else 0            # -1 and 0
    gen = torch.Generator(device=device).manual_seed(g)
    q = torch.full((4, hkv * g, d), nats * d ** -0.5, device=device)
    q = (q * (1 + 0.01 * torch.randn(q.shape, device=device, generator=gen))).to(dtype)
    check(c, [1, 1, 1, 1], hkv * g, dtype, q=q)


@pytest.mark.parametrize("octaves", OCTAVES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_one_page_of_large_values_in_a_long_context(octaves, dtype):
    """Tiles on either side of it, and pieces that other blocks continue, are
    joined across the same distance."""
    c = ref.Cache([20000, 300], 2, 128, dev(), seed=octaves)
    for i in (0, 70, 155, 311):
        c.scales[c.table[0][i], :, 1] = 127 - 6 + octaves // 2
    c.scales[c.table[1][1], :, 1] = 127 + 40 - octaves
    check(c, [1, 1], 16, dtype)
    check(c, [30, 30], 8, dtype)


# ---------------------------------------------------------------------------
# q at the ends of its type
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("news", [[1, 1], [3, 40]])
@pytest.mark.parametrize("top", [2.0 ** 126, 2.0 ** 127, 3.3e38])
def test_queries_near_the_largest_bf16(news, top):
    """With an sm_scale that brings the scores back: the row's exponent has to
    reach 120 (2^128 / 448)."""
    device = dev()
    c = ref.Cache([100, 300], 1, 128, device, seed=3)
    g = torch.Generator(device=device).manual_seed(5)
    q = (torch.rand(sum(news), 4, 128, device=device, generator=g) * 2 - 1)
    q[:, :, 7] = 1.0                                             # every row's largest is `top`
    q = (q * top).to(BF16)
    assert q.isfinite().all()
    check(c, news, 4, BF16, q=q, sm_scale=2.0 ** -126)


# ---------------------------------------------------------------------------
# every code at every kind of exponent byte, read back
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
def test_read_of_every_code_and_exponent_byte(d, dtype):
    """code * 2^(byte - 127) rounded once for all 256 bytes; a NaN code is a NaN
    in both types, and f16 saturates at 65504."""
    device = dev()
    pages = 256
    pool = torch.arange(256, dtype=torch.int32).repeat(64 * d // 256).view(64, d).to(torch.uint8).to(device)
    pool = pool[None, None, None].expand(pages, 1, 2, 64, d).contiguous()
    scales = torch.arange(256, device=device).to(torch.uint8)[:, None, None].expand(pages, 1, 2).contiguous()
    table = torch.arange(pages, dtype=torch.int32, device=device)[None].contiguous()
    n = pages * 64
    got = kv.read_gqa8(pool, scales, table, ints([0], device), ints([0, n], device), n, dtype=dtype)
    want = ref.values(pool, scales, table[0].tolist(), 0, n)[0]           # [2, n, D]
    if dtype == F16:
        want = want.clamp(-65504, 65504)
    for s in range(2):
        x, y = got[s][:, 0], want[s].to(dtype)
        assert torch.equal(x.isnan(), y.isnan())
        assert torch.equal(x.nan_to_num(nan=0.0), y.nan_to_num(nan=0.0))
