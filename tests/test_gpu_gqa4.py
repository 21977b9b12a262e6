"""The 4-bit grouped-query cache on the GPU against its 64-bit definition
(tests/gqa4_ref.py): the append bit for bit, the read-back exactly, the attention
within bounds derived there."""
import math

import pytest
import torch

import bit_kv_cache_nvfp4_gb300 as kv
import gqa4_ref as ref

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    return torch.device("cuda", torch.cuda.current_device())


def ints(x, device):
    return torch.tensor(x, dtype=torch.int32, device=device)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def run_append(k, v, cu, c):
    pool, scales = c.pool.clone(), c.scales.clone()
    err = torch.zeros(1, dtype=torch.int32, device=k.device)
    kv.append_gqa4(k, v, ints(cu, k.device), c.page_table, c.seq_lens, pool, scales, dev_err=err)
    want_pool, want_scales = c.pool.cpu().clone(), c.scales.cpu().clone()
    ref.append(k.double().cpu(), v.double().cpu(), cu, c.table, c.lens, want_pool, want_scales)
    assert torch.equal(scales.cpu(), want_scales)
    assert torch.equal(pool.cpu(), want_pool)
    return int(err.item())


@pytest.mark.parametrize("d,dtype,hkv", [(128, BF16, 2), (64, F16, 3), (128, F16, 1), (64, BF16, 8)])
@pytest.mark.parametrize("lens,news", [
    ([1], [1]), ([64, 65, 63], [64, 65, 63]), ([65, 64, 128, 200], [1, 1, 1, 1]),
    ([300, 7, 129, 0, 70], [200, 7, 2, 0, 69]), ([5, 0, 90], [9, 2, 90]),
])
def test_append_matches_the_definition(d, dtype, hkv, lens, news):
    device = dev()
    g = torch.Generator(device=device).manual_seed(len(lens) + d)
    c = ref.Cache(lens, hkv, d, device, seed=d + hkv)
    cu = ref.cu_of(news)
    x = torch.randn(cu[-1] + 3, 2, hkv, d, device=device, generator=g)
    x = (x * torch.exp2(torch.randint(-9, 9, (cu[-1] + 3, 1, hkv, 1), device=device, generator=g).float())).to(dtype)
    assert run_append(x[:, 0], x[:, 1], cu, c) == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n", [7, 40])
def test_append_borders_between_codes_and_scales(dtype, n):
    """Elements at every border between two codes of every scale, one step of
    their type below and above it, and amax at borders between scales: each of
    them decided as the quotient in 64 bits is."""
    device = dev()
    scales = ref.e4m3_values()[1:127]
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    rows = torch.zeros(126, 8, 16, dtype=torch.float64)
    x = scales[:, None] * border                                         # [126, 7]
    for i, sign in enumerate((1, -1)):
        at = (x * sign).to(dtype)
        bits = at.view(torch.int16)
        for j, step in enumerate((0, 1, -1)):
            rows[:, 3 * i + j, 1:8] = (bits + step).view(dtype).double()
            rows[:, 3 * i + j, 8:15] = -rows[:, 3 * i + j, 1:8]
    mid = (ref.e4m3_values()[0:126] + ref.e4m3_values()[1:127]) / 2 * 6
    rows[:, 6, 0], rows[:, 7, 0] = mid, -mid
    rows[:, :6, 0] = (scales * 6)[:, None]                               # amax that gives the scale
    rows[:, 7, 1] = torch.nextafter(mid.to(torch.float32), torch.tensor(1e30)).double()
    x = rows.reshape(-1, 16).to(dtype).to(device)
    x = x[:x.shape[0] // 8 * 8].view(-1, 1, 128)
    for a in range(0, x.shape[0], n):
        part = x[a:a + n]
        c = ref.Cache([part.shape[0]], 1, 128, device, seed=a)
        assert run_append(part, part.flip(-1), [0, part.shape[0]], c) == 0


def test_append_limits_and_zero_blocks():
    """The smallest scale and below it, the largest and beyond it, zeros of both
    signs."""
    device = dev()
    x = torch.zeros(64, 1, 64, device=device, dtype=BF16)
    for i, big in enumerate([0.0, 6 * 2.0 ** -10, 6.05 * 2.0 ** -10, 2.0 ** -7, 2688.0, 2700.0, 3e38, 1e-38, -0.0, 6 * 448.0]):
        x[i, 0, 5], x[i, 0, 6] = -big, big / 3
        x[i + 20, 0, :] = big
        x[i + 40, 0, 17] = big
        x[i + 40, 0, 18:30] = -big / 12
    c = ref.Cache([64], 1, 64, device, seed=5)
    assert run_append(x, x.flip(0), [0, 64], c) == 0


def test_append_token_by_token_leaves_the_others():
    device = dev()
    c = ref.Cache([1], 2, 64, device, seed=3)
    pool, scales, want_pool, want_scales = c.pool, c.scales, c.pool.cpu().clone(), c.scales.cpu().clone()
    g = torch.Generator(device=device).manual_seed(1)
    for n in range(1, 65):
        x = (torch.randn(1, 2, 2, 64, device=device, generator=g) * 2.0 ** ((n * 7) % 23 - 8)).to(BF16)
        kv.append_gqa4(x[:, 0], x[:, 1], ints([0, 1], device), c.page_table, ints([n], device), pool, scales)
        ref.append(x[:, 0].double().cpu(), x[:, 1].double().cpu(), [0, 1], c.table, [n], want_pool, want_scales)
    assert torch.equal(scales.cpu(), want_scales) and torch.equal(pool.cpu(), want_pool)


@pytest.mark.parametrize("n", [7, 70])
def test_append_flags_and_sanitizes_nonfinite_values(n):
    device = dev()
    lens = [n] * (1 if n > 7 else 3)
    c = ref.Cache(lens, 1, 64, device, seed=5)
    x = torch.randn(sum(lens), 1, 64, device=device).to(BF16)
    x[3, 0, 7], x[4, 0, 8], x[-1, 0, 1] = math.nan, math.inf, -math.inf
    x[5, 0, 16:32] = math.inf                                    # nothing else in the block
    y = torch.randn(sum(lens), 1, 64, device=device).to(BF16)
    assert run_append(x, y, ref.cu_of(lens), c) == kv.DEV_NONFINITE


@pytest.mark.parametrize("news", [[300, 100], [3, 2]])
def test_append_skips_bad_pages(news):
    device = dev()
    c = ref.Cache([200, 100], 1, 64, device, seed=6, extra_columns=0)
    c.table[0][1], c.table[1][0], c.table[0][3] = c.pool.shape[0], -5, -1
    c.page_table = ints(c.table, device)
    c.lens = [300 if news[0] > 3 else 130, 100 if news[0] > 3 else 2]    # beyond the table as well
    c.seq_lens = ints(c.lens, device)
    x = torch.randn(sum(news), 1, 64, device=device).to(BF16)
    assert run_append(x, x, ref.cu_of(news), c) == kv.DEV_BAD_PAGE


@pytest.mark.parametrize("B,news", [(33, (1,)), (40, (0, 3, 70)), (1030, (1, 0, 2)), (1100, (9, 0, 1)), (70, (1,))])
def test_append_and_read_many_requests(B, news):
    """More requests than a warp looks at in one round, in two rounds; some without
    a token, a token each, and one that is not request t's."""
    device = dev()
    news = [news[i % len(news)] for i in range(B)]
    if B == 70:
        news[0] = 0
    lens = [n + (i * 13) % 90 for i, n in enumerate(news)]
    c = ref.Cache(lens, 1, 64, device, seed=B)
    cu = ref.cu_of(news)
    g = torch.Generator(device=device).manual_seed(B)
    x = (torch.randn(cu[-1], 2, 1, 64, device=device, generator=g) * 4).to(BF16)
    assert run_append(x[:, 0], x[:, 1], cu, c) == 0
    k, v = kv.read_gqa4(c.pool, c.scales, c.page_table, ints([n - m for n, m in zip(lens, news)], device),
                        ints(cu, device), cu[-1])
    for b in range(0, B, 7):
        want = ref.values(c.pool, c.scales, c.table[b], lens[b] - news[b], lens[b])
        assert torch.equal(k[cu[b]:cu[b + 1]].double(), want[:, 0].transpose(0, 1))
        assert torch.equal(v[cu[b]:cu[b + 1]].double(), want[:, 1].transpose(0, 1))


# ---------------------------------------------------------------------------
# read-back
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d,dtype,hkv", [(128, BF16, 2), (64, F16, 3), (128, F16, 8), (64, BF16, 1)])
def test_read_is_exact(d, dtype, hkv):
    device = dev()
    c = ref.Cache([200, 64, 1, 300, 10], hkv, d, device, seed=d, spread=8)
    starts, news = [63, 0, 0, 129, 4], [130, 64, 1, 171, 0]
    cu = ref.cu_of(news)
    total = cu[-1] + 2
    k = torch.full((total, hkv, d), 7.0, dtype=dtype, device=device)
    v = torch.full((total, hkv, d), 8.0, dtype=dtype, device=device)
    err = torch.zeros(1, dtype=torch.int32, device=device)
    got = kv.read_gqa4(c.pool, c.scales, c.page_table, ints(starts, device), ints(cu, device), total,
                       dtype=dtype, k_out=k, v_out=v, dev_err=err)
    assert got[0] is k and got[1] is v and int(err.item()) == 0
    for b in range(5):
        x = ref.values(c.pool, c.scales, c.table[b], starts[b], starts[b] + news[b])
        rows = slice(cu[b], cu[b + 1])
        assert torch.equal(k[rows].double(), x[:, 0].transpose(0, 1))
        assert torch.equal(v[rows].double(), x[:, 1].transpose(0, 1))
    assert (k[cu[-1]:] == 7).all() and (v[cu[-1]:] == 8).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_read_takes_any_byte_and_zeroes_bad_pages(dtype):
    """All 256 bytes of codes with all 256 of scales: a NaN scale gives NaNs, a
    negative one the negative."""
    device = dev()
    c = ref.Cache([256, 64], 1, 64, device, seed=1)
    scale = torch.arange(256, dtype=torch.uint8, device=device)
    for i, page in enumerate(c.table[0][:4]):
        c.scales[page] = scale[64 * i:64 * i + 64].view(1, 1, 64, 1)
        c.pool[page, 0] = torch.randint(0, 256, (2, 64, 32), device=device).to(torch.uint8)
    c.pool[c.table[0][0], 0, 0] = (torch.arange(64, device=device)[:, None] * 4 + torch.arange(32, device=device) % 4).to(torch.uint8)
    table = [c.table[0], [c.pool.shape[0]] + c.table[1][1:]]
    err = torch.zeros(1, dtype=torch.int32, device=device)
    k, v = kv.read_gqa4(c.pool, c.scales, ints(table, device), ints([0, 0], device), ints([0, 256, 320], device),
                        320, dtype=dtype, dev_err=err)
    x = ref.values(c.pool, c.scales, c.table[0], 0, 256)
    assert torch.equal(k[:256].double().nan_to_num(9e9), x[:, 0].transpose(0, 1).nan_to_num(9e9))
    assert torch.equal(v[:256].double().nan_to_num(9e9), x[:, 1].transpose(0, 1).nan_to_num(9e9))
    assert (k[256:] == 0).all() and (v[256:] == 0).all() and int(err.item()) == kv.DEV_BAD_PAGE


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def check_attention(c, news, hq, dtype, window=0, sm_scale=None, q=None, max_new=None, seed=0, gain=1.0):
    device, d = c.pool.device, 2 * c.pool.shape[4]
    cu = ref.cu_of(news)
    if q is None:
        g = torch.Generator(device=device).manual_seed(seed)
        q = (torch.randn(cu[-1], hq, d, device=device, generator=g) * gain).to(dtype)
    scale = d ** -0.5 if sm_scale is None else sm_scale
    out = torch.full((q.shape[0], hq, d), 3.0, dtype=dtype, device=device)
    lse = torch.full((q.shape[0], hq), 3.0, device=device)
    err = torch.zeros(1, dtype=torch.int32, device=device)
    kv.attention_gqa4(q, c.pool, c.scales, c.page_table, c.seq_lens, ints(cu, device),
                      max(news) if max_new is None else max_new, scale, window=window, out=out, lse=lse,
                      dev_err=err)
    want = ref.attention(q[:cu[-1]], c.pool, c.scales, c.table, c.lens, cu, scale, window)
    tol, lse_tol = ref.bounds(*want, dtype, d)
    n = cu[-1]
    assert (out[n:] == 3).all() and (lse[n:] == 3).all()         # rows behind the last request
    assert out[:n].isfinite().all()
    off = (out[:n].double() - want[0]).abs()
    worst = float((off / tol).max()) if n else 0.0
    assert worst <= 1, f"out error {float(off.max()):.3g}, {worst:.3g} of its bound"
    empty = want[1] == -math.inf
    assert torch.equal(lse[:n] == -math.inf, empty)
    off = (lse[:n].double() - want[1]).masked_fill(empty, 0).abs()
    worst = float((off / lse_tol).max()) if n else 0.0
    assert worst <= 1, f"lse error {float(off.max()):.3g}, {worst:.3g} of its bound"
    assert (out[:n][empty] == 0).all()
    return int(err.item()), out, lse


EDGES = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 513]


@pytest.mark.parametrize("g,hkv,d,dtype", [(1, 2, 128, BF16), (4, 2, 128, BF16), (8, 1, 64, BF16), (7, 3, 64, F16),
                                           (3, 1, 128, F16), (16, 2, 128, BF16), (12, 1, 64, F16), (20, 1, 128, F16),
                                           (24, 1, 64, BF16), (32, 1, 128, BF16), (40, 1, 64, F16), (48, 1, 64, BF16),
                                           (33, 1, 128, BF16), (64, 1, 64, F16), (128, 1, 128, F16)])
def test_attention_single_tokens(g, hkv, d, dtype):
    """Every height of item, and groups that only the prompt kernel takes."""
    c = ref.Cache(EDGES, hkv, d, dev(), seed=g, spread=1)
    assert check_attention(c, [1] * len(EDGES), g * hkv, dtype, seed=g)[0] == 0


@pytest.mark.parametrize("g,hkv,d,dtype", [(8, 1, 128, BF16), (5, 2, 64, F16), (1, 3, 128, F16), (4, 2, 64, BF16)])
@pytest.mark.parametrize("news", [[2, 3, 4, 1, 0, 4], [5, 3, 5, 1, 0, 4], [9, 1, 30, 64, 65, 2], [130, 257, 1, 200, 33, 64]])
@pytest.mark.parametrize("window", [0, 1, 50, 100])
def test_attention_several_tokens(g, hkv, d, dtype, news, window):
    lens = [max(n, m) for n, m in zip(news, [2, 300, 64, 129, 40, 1000])]
    c = ref.Cache(lens, hkv, d, dev(), seed=g + window)
    assert check_attention(c, news, g * hkv, dtype, window=window, seed=g)[0] == 0


@pytest.mark.parametrize("news", [[3, 2, 4, 1, 1], [90, 1, 40, 0, 100]])
@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, F16)])
def test_attention_rows_without_a_key(news, d, dtype):
    """Sequences of length zero, and fewer tokens than rows: 0 and -inf."""
    c = ref.Cache([2, 0, 1, 1, 0], 2, d, dev(), seed=2)
    check_attention(c, news, 8, dtype)


@pytest.mark.parametrize("news", [[1, 1, 1], [7, 5, 3], [70, 40, 1]])
def test_attention_masks_bad_pages(news):
    c = ref.Cache([300, 400, 130], 2, 128, dev(), seed=4, extra_columns=0)
    c.table[0][1], c.table[0][4], c.table[1][6] = -1, c.pool.shape[0], 1 << 30
    c.table[2][:3] = [-7, -7, -7]                                # nothing left of this one
    c.page_table = ints(c.table, c.pool.device)
    c.lens[1] = 700                                              # beyond the table
    c.seq_lens = ints(c.lens, c.pool.device)
    assert check_attention(c, news, 8, BF16)[0] == kv.DEV_BAD_PAGE


@pytest.mark.parametrize("news", [[1, 1], [6, 5], [5, 40]])
@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, F16)])
def test_attention_scales_of_very_different_size(news, d, dtype):
    """Scales from the smallest subnormal to 240 side by side."""
    c = ref.Cache([700, 1000], 1, d, dev(), seed=8, spread=8)
    check_attention(c, news, 4, dtype, sm_scale=2.0 ** -14)


@pytest.mark.parametrize("n", [1, 7, 40])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("nats", [8.0, 14.0])
def test_attention_first_token_draws_most(n, dtype, nats):
    """One key far above many small ones, whose weights together still count."""
    device = dev()
    c = ref.Cache([20000], 1, 64, device, seed=9)
    page = c.table[0][0]
    c.pool[page, 0, 0, 0] = 0x02                                 # 1.0 in the even elements
    c.scales[page, 0, 0, 0] = 0x38
    g = torch.Generator(device=device).manual_seed(3)
    q = torch.zeros(n, 4, 64, device=device)
    q[..., 0::2] = nats / 4
    q += 0.02 * torch.randn(n, 4, 64, device=device, generator=g)
    check_attention(c, [n], 4, dtype, q=q.to(dtype))


@pytest.mark.parametrize("news", [[1, 1, 1], [6, 7, 1], [2, 33, 1]])
def test_attention_scales_of_q(news):
    """Rows of q from 2^-100 to 2^60 and zero rows; negative and zero sm_scale."""
    device = dev()
    c = ref.Cache([100, 90, 70], 1, 128, device, seed=10)
    g = torch.Generator(device=device).manual_seed(3)
    q = torch.randn(sum(news), 4, 128, device=device, generator=g)
    e = torch.tensor([-100.0, 0.0, -20.0, 3.0], device=device)
    q = (q * torch.exp2(e)[None, :, None]).to(BF16)
    q[0, 1] = 0
    for s in (0.125, -0.07, 0.0):
        check_attention(c, news, 4, BF16, q=q, sm_scale=s)
    check_attention(c, news, 4, BF16, q=(q.float() * 2.0 ** 60).to(BF16), sm_scale=2.0 ** -63)
    wide = torch.randn(sum(news), 4, 128, device=device, generator=g)
    wide[..., ::3] *= 2.0 ** -20                                 # small beside the row's largest
    wide[..., 1::3] *= 2.0 ** -30
    check_attention(c, news, 4, BF16, q=wide.to(BF16))


@pytest.mark.parametrize("news", [[1, 1], [6, 2], [3, 40]])
def test_attention_nonfinite_queries_stay_in_their_rows(news):
    device = dev()
    c = ref.Cache([100, 200], 1, 128, device, seed=11)
    q = torch.randn(sum(news), 4, 128, device=device).to(BF16)
    clean = check_attention(c, news, 4, BF16, q=q)[1:]
    bad = q.clone()
    bad[0, 1, 5], bad[-1, 2, 0] = math.nan, math.inf
    out, lse = kv.attention_gqa4(bad, c.pool, c.scales, c.page_table, c.seq_lens, ints(ref.cu_of(news), device),
                                 max(news), 128 ** -0.5)
    for t, h in ((0, 1), (q.shape[0] - 1, 2)):
        assert out[t, h].isnan().all() and lse[t, h].isnan()
        out[t, h], lse[t, h] = clean[0][t, h], clean[1][t, h]
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


def test_attention_strided_queries_and_behind_the_last_request():
    device = dev()
    c = ref.Cache([100, 40], 2, 128, device, seed=12)
    x = torch.randn(9, 3, 4, 128, device=device).to(BF16)
    check_attention(c, [2, 5], 4, BF16, q=x[:, 1])               # two rows behind the last
    y = torch.randn(4, 50, 128, device=device).to(BF16).transpose(0, 1)
    check_attention(c, [40, 10], 4, BF16, q=y)                   # head-major


@pytest.mark.parametrize("dtype,n,window", [(BF16, 1, 0), (F16, 3, 0), (F16, 7, 0), (BF16, 100, 0), (BF16, 2, 5000)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_long_contexts(dtype, n, window, d):
    c = ref.Cache([30011, 9, 16384], 2, d, dev(), seed=13)
    assert check_attention(c, [n, min(n, 9), n], 8, dtype, window=window)[0] == 0


@pytest.mark.parametrize("n", [9, 17, 24, 25, 33, 41, 49, 100, 128, 129, 140, 256, 257])
@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, F16)])
def test_attention_items_of_every_height(n, d, dtype):
    """One kv head, so n rows: below and above what an item and each of its row
    tiles hold, with one tile of keys, an odd and an even number of them, and cut
    along the keys."""
    c = ref.Cache([n, 300, 500, 5000], 1, d, dev(), seed=n, spread=1)
    check_attention(c, [n, min(n, 300), n, n], 1, dtype, seed=n)
    check_attention(c, [n, min(n, 300), n, n], 1, dtype, window=200, seed=n)


@pytest.mark.parametrize("seed", range(4))
def test_attention_short_items_between_long_ones(seed):
    """Items of a tile or two, whose warps are at the next item's rows while others
    still store the one before, on either kernel."""
    lens = [(4971, 176, 70, 4, 613, 297, 164, 838, 5, 531)[(i * 3 + seed) % 10] for i in range(38)]
    c = ref.Cache(lens, 3, 64, dev(), seed=seed)
    for _ in range(3):
        check_attention(c, [5] * 38, 36, F16, seed=seed)
        check_attention(c, [2] * 38, 12, F16, seed=seed)


def test_attention_many_requests():
    lens = [(i * 37) % 400 for i in range(300)]
    c = ref.Cache(lens, 1, 64, dev(), seed=14)
    check_attention(c, [min(1, n) for n in lens], 4, BF16)


def test_attention_mixed_batch():
    """Prompt chunks and single tokens in one call."""
    news = [200, 1, 1, 0, 77, 1, 1, 129]
    lens = [200, 1000, 64, 50, 600, 1, 333, 500]
    c = ref.Cache(lens, 2, 128, dev(), seed=15)
    check_attention(c, news, 8, BF16)


@pytest.mark.parametrize("B", [1, 7, 150, 160, 400])
@pytest.mark.parametrize("news", [(1,), (1, 0, 2, 1), (1, 40, 0, 1, 9, 200)])
@pytest.mark.parametrize("d,dtype,g", [(128, BF16, 4), (64, F16, 12)])
def test_attention_short_tables(B, news, d, dtype, g):
    """Tables of 8 pages at most, whose items are never cut: a block for each
    item, or several."""
    lens = [(i * 89) % 449 for i in range(B)]
    news = [min(news[i % len(news)], n) for i, n in enumerate(lens)]
    if sum(news) == 0:
        lens[0] = news[0] = 1
    c = ref.Cache(lens, 2, d, dev(), seed=B)
    assert c.page_table.shape[1] <= 8
    assert check_attention(c, news, 2 * g, dtype, seed=B)[0] == 0


@pytest.mark.parametrize("wide", [1, 20])
def test_attention_flags_a_request_beyond_max_new(wide):
    """With tables whose items are never cut, and with others."""
    device = dev()
    c = ref.Cache([100, 50, 80], 1, 64, device, seed=16, extra_columns=wide)
    news, cu = [1, 3, 1], ref.cu_of([1, 3, 1])
    q = torch.randn(5, 2, 64, device=device).to(BF16)
    err = torch.zeros(1, dtype=torch.int32, device=device)
    out, lse = (torch.full((5, 2, 64), 3.0, dtype=BF16, device=device), torch.full((5, 2), 3.0, device=device))
    kv.attention_gqa4(q, c.pool, c.scales, c.page_table, c.seq_lens, ints(cu, device), 1, 0.125, out=out, lse=lse,
                      dev_err=err)
    assert int(err.item()) == kv.DEV_BAD_LENGTH
    whole = check_attention(c, news, 2, BF16, q=q, sm_scale=0.125)
    for t in (0, 4):
        assert torch.equal(out[t], whole[1][t]) and torch.equal(lse[t], whole[2][t])
    assert (out[1:4] == 3).all() and (lse[1:4] == 3).all()


@pytest.mark.parametrize("B,columns,d", [(64, 1 << 19, 128), (32, 1 << 20, 64)])
def test_attention_by_tables_with_room_for_more_than_an_int_of_work(B, columns, d):
    """The tables could name 2^30 units of work and more, though the requests are
    short: single tokens, drafts and a prompt's chunk."""
    news = [300, 1, 0, 9, 2, 64] + [1] * (B - 6)
    lens = [333, 70, 40, 9, 129, 64] + [1 + 37 * i % 500 for i in range(B - 6)]
    c = ref.Cache(lens, 8, d, dev(), seed=B)
    wide = torch.full((B, columns), -1, dtype=torch.int32, device=c.pool.device)
    wide[:, :c.page_table.shape[1]] = c.page_table
    c.page_table = wide
    assert check_attention(c, news, 32, BF16, seed=B)[0] == 0


# ---------------------------------------------------------------------------
# every tile counts
# ---------------------------------------------------------------------------
def needles(n, d, device, seed=0):
    """A request of n tokens over one kv head, and a row of q for each 64 keys: keys
    have elements of +-1/4 or less, but one of each 64 is 6 in dimension t % d, of a
    sign by t // d, where row t of q makes that a score of 18 (sm_scale d^-0.5); the
    others' are at most 0.75, so that with 30000 keys the one has over 99 % of the
    weight."""
    c = ref.Cache([n], 1, d, "cpu", seed=seed)
    tiles = -(-n // 64)
    pages = torch.tensor(c.table[0][:tiles])
    c.pool[pages, 0, 0] &= 0x99                                  # codes of 0 and 0.5
    c.scales[pages, 0, 0] = 0x30                                 # 0.5
    q = torch.zeros(tiles, d)
    for t in range(tiles):
        at = (t * 37) % min(64, n - t * 64)
        sign, dim = (t // d) % 2, t % d
        page, byte = c.table[0][t], dim // 2
        c.scales[page, 0, 0, at, dim // 16] = 0x38               # 1
        c.pool[page, 0, 0, at, dim // 16 * 8:dim // 16 * 8 + 8] = 0
        c.pool[page, 0, 0, at, byte] = (7 + 8 * sign) << (4 * (dim % 2))
        q[t, dim] = (1 - 2 * sign) * 3 * d ** 0.5
    c.pool, c.scales = c.pool.to(device), c.scales.to(device)
    c.page_table, c.seq_lens = c.page_table.to(device), c.seq_lens.to(device)
    return c, q.to(device)


@pytest.mark.parametrize("n,d,dtype", [(8011, 128, BF16), (4099, 64, F16), (900, 128, F16)])
@pytest.mark.parametrize("m", [1, 8, 16, 24, 32, 60, 130])
def test_rows_see_every_page(n, d, dtype, m):
    """Rows that each ask for a page of their own, as heads of single tokens and as
    rows of chunks (m of them): items of every height, cut over the blocks."""
    c, q = needles(n, d, dev())
    for t in range(0, q.shape[0], max(m, 8)):
        rows = q[t:t + max(m, 8)]
        rows = torch.cat([rows[:1].expand(max(m, 8) - rows.shape[0], -1), rows]).to(dtype)
        if m <= 32:
            check_attention(c, [1], rows.shape[0], dtype, q=rows[None])
        if m >= 8:
            check_attention(c, [rows.shape[0]], 1, dtype, q=rows[:, None])


# ---------------------------------------------------------------------------
# together, streams, graphs
# ---------------------------------------------------------------------------
def serve(device, steps, d=128, hkv=2, hq=8, dtype=BF16, graph=False):
    """A prompt chunk of three sessions, then `steps` single tokens each, turned by
    their positions first: the attention's outputs, and q, K, V as they were
    given."""
    g = torch.Generator(device=device).manual_seed(77)
    prompts, B, width = [100, 63, 1], 3, 4
    pool = torch.randint(0, 256, (B * width, hkv, 2, 64, d // 2), dtype=torch.uint8, device=device, generator=g)
    scales = torch.randint(0, 256, (B * width, hkv, 2, 64, d // 16), dtype=torch.uint8, device=device, generator=g)
    table = torch.randperm(B * width, device=device, generator=g).to(torch.int32).view(B, width)
    cu, lens = ints(ref.cu_of(prompts), device), ints(prompts, device)
    freq = kv.rotary_frequencies(d // 2, scaling="ramp", stretch=4.0, device=device)
    x = torch.randn(sum(prompts), hq + 2 * hkv, d, device=device, generator=g).to(dtype)
    pos = torch.cat([torch.arange(n, device=device) for n in prompts]).to(torch.int32)
    q, k = kv.rotary(x[:, :hq], x[:, hq:hq + hkv], pos, freq)
    kv.append_gqa4(k, x[:, hq + hkv:], cu, table, lens, pool, scales)
    outs = [kv.attention_gqa4(q, pool, scales, table, lens, cu, max(prompts), d ** -0.5)[0]]
    cu1 = ints([0, 1, 2, 3], device)
    tokens = torch.randn(steps, B, hq + 2 * hkv, d, device=device, generator=g).to(dtype)
    buf = torch.empty_like(tokens[0])

    def step():
        qt, kt = kv.rotary(buf[:, :hq], buf[:, hq:hq + hkv], lens, freq)
        lens.add_(1)
        kv.append_gqa4(kt, buf[:, hq + hkv:], cu1, table, lens, pool, scales)
        return kv.attention_gqa4(qt, pool, scales, table, lens, cu1, 1, d ** -0.5)[0]

    if graph:
        warm = (lens.clone(), pool.clone(), scales.clone())
        buf.copy_(tokens[0])
        step()
        torch.cuda.synchronize()
        for t, w in zip((lens, pool, scales), warm):
            t.copy_(w)
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            kept = step()
    for i in range(steps):
        buf.copy_(tokens[i])
        if graph:
            captured.replay()
            outs.append(kept.clone())
        else:
            outs.append(step())
    return outs, x, tokens, pool, scales, table, freq


def turned(x, pos, freq):
    """Halves of the first 2 n elements by 64-bit angles, rounded to x's type."""
    n = freq.numel()
    a = pos.double()[:, None, None] * freq.double()
    u, v = x[..., :n].double(), x[..., n:2 * n].double()
    y = torch.cat([u * a.cos() - v * a.sin(), u * a.sin() + v * a.cos(), x[..., 2 * n:].double()], -1)
    return y


def test_serving_run():
    """Prompt, then 70 steps (pages fill and new ones begin), position by position:
    what the cache holds is the quantized k and v (k turned; an element that rounds
    to its type the other way than in 64 bits, about one in 2^16, changes its block's
    codes by a step at most: allowed in one block of 200), and the outputs
    are the attention over what it holds."""
    device = dev()
    outs, x, tokens, pool, scales, table, freq = serve(device, 70)
    hq, hkv, d, prompts = 8, 2, 128, [100, 63, 1]
    cu = ref.cu_of(prompts)
    for b in range(3):
        rows = torch.cat([x[cu[b]:cu[b + 1]], tokens[:, b]])
        n = rows.shape[0]
        pos = torch.arange(n, device=device)
        held = ref.values(pool, scales, table[b].tolist(), 0, n)
        k = turned(rows[:, hq:hq + hkv], pos, freq).to(BF16)
        for side, want in ((0, k), (1, rows[:, hq + hkv:])):
            y = ref.dequantize(*ref.quantize(want.double().cpu())).to(device).transpose(0, 1)
            other = (held[:, side] != y).unflatten(-1, (-1, 16)).any(-1)
            assert float(other.double().mean()) <= (0.005 if side == 0 else 0.0)
        q = turned(rows[:, :hq], pos, freq).to(BF16)
        got = torch.cat([outs[0][cu[b]:cu[b + 1]]] + [o[b:b + 1] for o in outs[1:]])
        want = ref.attention(q, pool, scales, [table[b].tolist()], [n], [0, n], d ** -0.5)
        # (the same one in 2^16 of q's elements: 2^-8 of an element of a score's 128)
        tol = ref.bounds(*want, BF16, d)[0] + 2 * 2.0 ** -8 * want[2][0] * q.double().abs().amax(-1, keepdim=True) * d ** -0.5 * 6
        assert ((got.double() - want[0]).abs() <= tol).all()


def test_serving_run_captured_in_a_graph_gives_the_same_bits():
    device = dev()
    a, b = serve(device, 70), serve(device, 70, graph=True)
    for x, y in zip(a[0], b[0]):
        assert torch.equal(x, y)
    assert torch.equal(a[3], b[3]) and torch.equal(a[4], b[4])


def test_equal_calls_give_equal_bits():
    device = dev()
    c = ref.Cache([20000, 700, 3000, 90], 2, 128, device, seed=19)
    for news, hq in (([1, 1, 1, 1], 16), ([5, 1, 5, 3], 8), ([100, 3, 200, 1], 8)):
        q = torch.randn(sum(news), hq, 128, device=device).to(BF16)
        args = (q, c.pool, c.scales, c.page_table, c.seq_lens, ints(ref.cu_of(news), device), max(news), 0.09)
        first = kv.attention_gqa4(*args)
        for _ in range(5):
            again = kv.attention_gqa4(*args)
            assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_calls_on_two_streams_do_not_share_anything():
    """Two calls in flight on two streams, each split over the SMs."""
    device = dev()
    cs = [ref.Cache([20000], 2, 128, device, seed=s) for s in (20, 21)]
    q = torch.randn(1, 8, 128, device=device).to(BF16)
    args = [(q, c.pool, c.scales, c.page_table, c.seq_lens, ints([0, 1], device), 1, 0.09) for c in cs]
    want = [kv.attention_gqa4(*a) for a in args]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(kv.attention_gqa4(*args[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_two_graphs_replayed_at_once():
    device = dev()
    c = ref.Cache([20000, 300], 2, 128, device, seed=22)
    qs = [torch.randn(2, 8, 128, device=device).to(BF16) for _ in range(2)]
    args = (c.pool, c.scales, c.page_table, c.seq_lens, ints([0, 1, 2], device), 1, 0.09)
    want = [kv.attention_gqa4(q, *args) for q in qs]
    graphs, got = [], []
    for q in qs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            got.append(kv.attention_gqa4(q, *args))
        graphs.append(gr)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])


@pytest.mark.parametrize("n", [1, 6, 70])
def test_own_workspace_and_its_refusal(n):
    device = dev()
    c = ref.Cache([20000], 2, 128, device, seed=23)
    q = torch.randn(n, 8, 128, device=device).to(BF16)
    args = (q, c.pool, c.scales, c.page_table, c.seq_lens, ints([0, n], device), n, 0.09)
    want = kv.attention_gqa4(*args)
    size = kv.attention_gqa4_workspace(1, n, n, 8, 2, 128)
    ws = torch.full((max(size, 1),), 255, dtype=torch.uint8, device=device)
    got = kv.attention_gqa4(*args, workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(kv.Kv4Error) as e:
        kv.attention_gqa4(*args, workspace=ws[:size - 16])
    assert e.value.status == 5


@pytest.mark.parametrize("d,dtype,hq,n", [(128, BF16, 4, 1), (128, F16, 24, 1), (64, BF16, 4, 3), (128, BF16, 8, 7),
                                          (128, BF16, 4, 40), (64, F16, 8, 70)])
def test_a_wait_that_runs_out(d, dtype, hq, n):
    """A wait on a barrier that nothing arrives on gives up after its limit, in the
    middle of several items: KV4_DEV_TIMEOUT, the call ends, no row behind the last
    request is written, and the next call is whole."""
    device = dev()
    B = 700 if n < 8 else 250
    lens = [n + (i * 53) % 700 for i in range(B)]
    c = ref.Cache(lens, 2, d, device, seed=25)
    q = torch.randn(n * B + 5, hq, d, device=device).to(dtype)
    args = (q, c.pool, c.scales, c.page_table, c.seq_lens, ints(ref.cu_of([n] * B), device), n, 0.09)
    want = kv.attention_gqa4(*args)
    err = torch.zeros(1, dtype=torch.int32, device=device)
    out, lse = (torch.full((n * B + 5, hq, d), 3.0, dtype=dtype, device=device),
                torch.full((n * B + 5, hq), 3.0, device=device))
    kv.set_wait_limit(1_000_000, 1)
    try:
        kv.attention_gqa4(*args, out=out, lse=lse, dev_err=err)
        torch.cuda.synchronize()
    finally:
        kv.set_wait_limit()
    assert int(err.item()) == kv.DEV_TIMEOUT
    assert (out[n * B:] == 3).all() and (lse[n * B:] == 3).all()
    got = kv.attention_gqa4(*args)
    assert torch.equal(got[0][:n * B], want[0][:n * B]) and torch.equal(got[1][:n * B], want[1][:n * B])


@pytest.mark.parametrize("limit", [1, 1500, 4000, 12000])
@pytest.mark.parametrize("d,dtype,hq,n,B,length", [
    (128, BF16, 16, 1, 150, 3000), (128, F16, 4, 1, 3, 60000), (64, BF16, 16, 1, 150, 5000), (64, F16, 10, 5, 60, 3000),
    (64, BF16, 48, 2, 60, 3000), (128, BF16, 8, 70, 40, 3000), (64, F16, 4, 300, 30, 3000)])
def test_waits_that_give_up_with_copies_on_their_way(d, dtype, hq, n, B, length, limit):
    """A limit as short as a copy's own time: any wait of a block may be the one that
    gives up, on whatever is on its way (or none, where the hardware's own suspension of a
    waiting thread outlasts them all: a short call may still be whole, but not without
    saying so otherwise).  The call ends, what it does not own stays as it is, and the next
    call is whole."""
    device = dev()
    lens = [max(n, length - 37 * (i % 40)) for i in range(B)]
    c = ref.Cache(lens, 2, d, device, seed=26)
    q = torch.randn(n * B + 3, hq, d, device=device).to(dtype)
    args = (q, c.pool, c.scales, c.page_table, c.seq_lens, ints(ref.cu_of([n] * B), device), n, 0.09)
    size = kv.attention_gqa4_workspace(B, n, n * B + 3, hq, 2, d)
    ws = torch.full((size + 4096,), 7, dtype=torch.uint8, device=device)
    want = kv.attention_gqa4(*args, workspace=ws[:size])
    held = c.pool.clone(), c.scales.clone(), q.clone()
    out, lse = (torch.full((n * B + 3, hq, d), 3.0, dtype=dtype, device=device),
                torch.full((n * B + 3, hq), 3.0, device=device))
    kv.set_wait_limit(limit)
    try:
        for _ in range(5):
            err = torch.zeros(1, dtype=torch.int32, device=device)
            kv.attention_gqa4(*args, out=out, lse=lse, workspace=ws[:size], dev_err=err)
            torch.cuda.synchronize()
            assert int(err.item()) in (0, kv.DEV_TIMEOUT)
            if int(err.item()) == 0:
                assert torch.equal(out[:n * B], want[0][:n * B]) and torch.equal(lse[:n * B], want[1][:n * B])
    finally:
        kv.set_wait_limit()
    assert (out[n * B:] == 3).all() and (lse[n * B:] == 3).all() and (ws[size:] == 7).all()
    assert all(torch.equal(x, y) for x, y in zip(held, (c.pool, c.scales, q)))
    got = kv.attention_gqa4(*args, workspace=ws[:size])
    assert torch.equal(got[0][:n * B], want[0][:n * B]) and torch.equal(got[1][:n * B], want[1][:n * B])


# ---------------------------------------------------------------------------
# what the binding takes and refuses
# ---------------------------------------------------------------------------
def call_args(device):
    """A small valid call of each kind, by argument name."""
    c = ref.Cache([100, 30], 2, 64, device, seed=27)
    x = torch.randn(5, 2, 64, device=device).to(BF16)
    cu = ints([0, 3, 5], device)
    cache = dict(pool=c.pool, scales=c.scales, page_table=c.page_table)
    return {"append": (kv.append_gqa4, dict(k=x, v=x.clone(), cu_seqlens=cu, seq_lens=c.seq_lens, **cache)),
            "read": (kv.read_gqa4, dict(starts=ints([3, 0], device), cu_seqlens=cu, total=5, **cache)),
            "attention": (kv.attention_gqa4, dict(q=x.repeat(1, 2, 1), seq_lens=c.seq_lens, cu_seqlens=cu, max_new=3,
                                                  sm_scale=0.125, **cache))}


def unaligned(t):
    return torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view_as(t).copy_(t)


CACHE_REFUSALS = [
    ("pool", lambda t: t.cpu(), TypeError), ("pool", lambda t: t.view(torch.int8), TypeError),
    ("pool", lambda t: t[:, :, :1], ValueError), ("pool", lambda t: t[..., :16], ValueError),
    ("pool", lambda t: t.flatten(3), ValueError), ("pool", lambda t: t.transpose(0, 1), ValueError),
    ("pool", unaligned, kv.Kv4Error), ("pool", lambda t: t[:0], ValueError),
    ("scales", lambda t: t[:-1], ValueError), ("scales", lambda t: t.float(), TypeError),
    ("scales", lambda t: t[..., :2], ValueError), ("scales", lambda t: t[..., 0], ValueError),
    ("scales", unaligned, kv.Kv4Error), ("scales", lambda t: None, TypeError),
    ("page_table", lambda t: t.long(), TypeError), ("page_table", lambda t: t[:1], ValueError),
    ("page_table", lambda t: t[0], ValueError), ("page_table", lambda t: t[:, :0], kv.Kv4Error),
    ("cu_seqlens", lambda t: t[:2], ValueError), ("cu_seqlens", lambda t: t.cpu(), TypeError),
    ("dev_err", lambda t: torch.zeros(1), TypeError),
]
INPUT_REFUSALS = [
    (lambda t: t.float(), TypeError), (lambda t: t[:, :, :32], ValueError), (lambda t: t[..., ::2], ValueError),
    (lambda t: t[:, :1], ValueError), (lambda t: unaligned(t), ValueError), (lambda t: t.cpu(), TypeError),
    (lambda t: torch.empty(5, 1, 64, dtype=BF16, device=t.device).expand(t.shape), kv.Kv4Error),
]
REFUSALS = (
    [(f, name, change, e) for f in ("append", "read", "attention") for name, change, e in CACHE_REFUSALS]
    + [("append", name, change, e) for name in ("k", "v") for change, e in INPUT_REFUSALS]
    + [("attention", "q", change, e) for change, e in INPUT_REFUSALS]
    + [("append", "v", lambda t: t.half(), TypeError), ("read", "starts", lambda t: t.long(), TypeError),
       ("read", "total", lambda n: -1, ValueError), ("read", "dtype", lambda t: torch.float32, TypeError),
       ("read", "k_out", lambda t: torch.empty(4, 2, 64, dtype=BF16, device="cuda"), ValueError),
       ("attention", "max_new", lambda n: 0, kv.Kv4Error), ("attention", "window", lambda n: -1, ValueError),
       ("attention", "sm_scale", lambda x: math.nan, kv.Kv4Error),
       ("attention", "out", lambda t: torch.empty(5, 4, 64, dtype=F16, device="cuda"), TypeError),
       ("attention", "workspace", lambda t: torch.empty(1 << 26, dtype=torch.int32, device="cuda"), TypeError)])


@pytest.mark.parametrize("i", range(len(REFUSALS)))
def test_binding_refuses(i):
    """Nothing is launched, and the next call is as if there had been none."""
    f, name, change, error = REFUSALS[i]
    fn, args = call_args(dev())[f]
    pool = args["pool"].clone()
    with pytest.raises(error):
        fn(**{**args, name: change(args.get(name))})
    assert torch.equal(args["pool"], pool)
    fn(**args)
    torch.cuda.synchronize()


def test_written_tensors_count_it_and_results_carry_no_gradient():
    device = dev()
    calls = call_args(device)
    fn, args = calls["append"]
    before = args["pool"]._version, args["scales"]._version, args["k"]._version
    fn(**args)
    assert (args["pool"]._version, args["scales"]._version, args["k"]._version) == (before[0] + 1, before[1] + 1, before[2])
    fn, args = calls["attention"]
    out, lse = fn(**{**args, "q": args["q"].clone().requires_grad_()})
    assert not out.requires_grad and not lse.requires_grad


def test_empty_calls():
    device = dev()
    c = ref.Cache([100, 30], 2, 64, device, seed=28)
    x = torch.empty(0, 2, 64, dtype=BF16, device=device)
    cu, none = ints([0, 0, 0], device), ints([0], device)
    pool = c.pool.clone()
    kv.append_gqa4(x, x, cu, c.page_table, c.seq_lens, c.pool, c.scales)
    k, v = kv.read_gqa4(c.pool, c.scales, c.page_table, ints([0, 0], device), cu, 0)
    out, lse = kv.attention_gqa4(x, c.pool, c.scales, c.page_table, c.seq_lens, cu, 0, 0.1)
    assert k.shape == v.shape == out.shape == (0, 2, 64) and lse.shape == (0, 2)
    x = torch.ones(3, 2, 64, dtype=BF16, device=device)          # no request at all
    kv.append_gqa4(x, x, none, c.page_table[:0], c.seq_lens[:0], c.pool, c.scales)
    out, lse = torch.full((3, 2, 64), 3.0, dtype=BF16, device=device), torch.full((3, 2), 3.0, device=device)
    kv.attention_gqa4(x, c.pool, c.scales, c.page_table[:0], c.seq_lens[:0], none, 1, 0.1, out=out, lse=lse)
    assert torch.equal(c.pool, pool) and (out == 3).all() and (lse == 3).all()


@pytest.mark.parametrize("cu", [[0, 40, 20, 70], [-9, 5, 2 ** 31 - 1, 3], [70, 0, -2 ** 31, 90], [0, 70, 70, 70], [0, 1, 2, 3]])
@pytest.mark.parametrize("lens", [[2 ** 31 - 1, -2 ** 31, 5], [3, 2 ** 31 - 1, 2 ** 31 - 40], [90, 20, 60]])
def test_lengths_and_pages_out_of_range_stay_in_bounds(cu, lens):
    """Rows, lengths and page numbers that nobody should pass: what lies around
    the call's tensors is left as it was.  (Every one of them is held to the call's
    sizes before it makes an address.)"""
    device = dev()
    hq, hkv, d, pages = 8, 2, 64, 8
    g = torch.Generator(device=device).manual_seed(3)
    pool = torch.randint(0, 256, (pages + 2, hkv, 2, 64, d // 2), dtype=torch.uint8, device=device, generator=g)
    scales = torch.randint(0, 120, (pages + 2, hkv, 2, 64, d // 16), dtype=torch.uint8, device=device, generator=g)
    table = ints([[0, 7, 2 ** 31 - 1, 3], [-2 ** 31, 1, 8, 2], [4, 4, 5, -1]], device)
    guard_pool, guard_scales = pool.clone(), scales.clone()
    cu_t, lens_t = ints(cu, device), ints(lens, device)
    cache = (pool[1:-1], scales[1:-1])
    for T in (70, 23):                                           # blocks of pages, of tokens
        x = torch.randn(T, hq + 2 * hkv, d, device=device, generator=g).to(BF16)
        for max_new in (1, 5, 70):
            out = torch.full((T + 2, hq, d), 3.0, dtype=BF16, device=device)
            lse = torch.full((T + 2, hq), 3.0, device=device)
            kv.attention_gqa4(x[:, :hq], *cache, table, lens_t, cu_t, max_new, 0.125, out=out[1:-1], lse=lse[1:-1])
            for t in (out, lse):
                assert (t[0] == 3).all() and (t[-1] == 3).all()
        ko = torch.full((T + 2, hkv, d), 3.0, dtype=BF16, device=device)
        vo = ko.clone()
        kv.read_gqa4(*cache, table, lens_t, cu_t, T, k_out=ko[1:-1], v_out=vo[1:-1])
        for t in (ko, vo):
            assert (t[0] == 3).all() and (t[-1] == 3).all()
        kv.append_gqa4(x[:, hq:hq + hkv], x[:, hq + hkv:], cu_t, table, lens_t, *cache)
        for t, was in ((pool, guard_pool), (scales, guard_scales)):
            assert torch.equal(t[0], was[0]) and torch.equal(t[-1], was[-1])


# ---------------------------------------------------------------------------
# offsets beyond 32 bits
# ---------------------------------------------------------------------------
def test_pool_beyond_32_bits():
    """A pool of 6.5 GB, its last pages used: as in a small one."""
    device, pages = dev(), 400_000
    lens, news = [300, 65, 1], [40, 1, 1]
    c = ref.Cache(lens, 2, 128, device, seed=30)
    n, cu = c.pool.shape[0], ints(ref.cu_of(news), device)
    pool = torch.empty(pages, 2, 2, 64, 64, dtype=torch.uint8, device=device)
    scales = torch.empty(pages, 2, 2, 64, 8, dtype=torch.uint8, device=device)
    pool[pages - n:], scales[pages - n:] = c.pool, c.scales
    table = torch.where(c.page_table < 0, c.page_table, c.page_table + (pages - n))
    x = torch.randn(42, 12, 128, device=device).to(BF16)
    starts = ints([9, 0, 0], device)
    got = []
    for p, s, t in ((c.pool, c.scales, c.page_table), (pool, scales, table)):
        kv.append_gqa4(x[:, 8:10], x[:, 10:], cu, t, c.seq_lens, p, s)
        kv.append_gqa4(x[-2:, 8:10], x[-2:, 10:], ints([0, 0, 1, 2], device), t, c.seq_lens, p, s)
        got.append((p[-n:], s[-n:], *kv.read_gqa4(p, s, t, starts, cu, 42),
                    *kv.attention_gqa4(x[:, :8], p, s, t, c.seq_lens, cu, 40, 0.09),
                    *kv.attention_gqa4(x[:3, :8], p, s, t, c.seq_lens, ints([0, 1, 2, 3], device), 1, 0.09)))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_outputs_beyond_32_bits():
    """2.7e9 elements of out and of the read-back."""
    device = dev()
    B, hkv, g, d = 65535, 16, 20, 128
    c = ref.Cache([500], hkv, d, device, seed=32)
    table = c.page_table[:, :8].expand(B, -1).contiguous()       # every request the same pages
    lens = torch.randint(1, 500, (B,), dtype=torch.int32, device=device)
    cu = torch.arange(B + 1, dtype=torch.int32, device=device)
    q = torch.empty(B, hkv * g, d, dtype=BF16, device=device)
    q[-9:] = torch.randn(9, hkv * g, d, device=device).to(BF16)
    q[:-9] = q[-9:-8]
    out, lse = kv.attention_gqa4(q, c.pool, c.scales, table, lens, cu, 1, 0.09)
    want = ref.attention(q[-9:], c.pool, c.scales, c.table * 9, lens[-9:].tolist(), list(range(10)), 0.09)
    tol, lse_tol = ref.bounds(*want, BF16, d)
    assert ((out[-9:].double() - want[0]).abs() <= tol).all()
    assert ((lse[-9:].double() - want[1]).abs() <= lse_tol).all()
    del q, out, lse
    n = 1_300_000                                                # tokens of a request that repeats its pages
    row = c.page_table[0, :7].repeat(n // 448 + 1)[None].contiguous()
    k, v = kv.read_gqa4(c.pool, c.scales, row, ints([0], device), ints([0, n], device), n)
    last = kv.read_gqa4(c.pool, c.scales, row, ints([n - 100], device), ints([0, 100], device), 100)
    assert torch.equal(k[-100:], last[0]) and torch.equal(v[-100:], last[1])
