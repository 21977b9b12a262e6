"""The 8-bit grouped-query cache on the GPU against its 64-bit definition
(tests/gqa8_ref.py): the append bit for bit, the read-back exactly, the
attention within bounds derived there."""
import math

import pytest
import torch

import bit_kv_cache_nvfp4_gb300 as kv
import gqa8_ref as ref

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
def run_append(k, v, cu, c, pool=None, scales=None):
    pool, scales = c.pool.clone(), c.scales.clone()
    err = torch.zeros(1, dtype=torch.int32, device=k.device)
    kv.append_gqa8(k, v, ints(cu, k.device), c.page_table, c.seq_lens, pool, scales, dev_err=err)
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


def test_append_exponent_limits_and_zero_blocks():
    """Blocks at and beyond both ends of the exponent's range, all-zero blocks,
    amax exactly 448 * 2^e and one step above it."""
    device = dev()
    rows = [0.0, 448.0, 450.0, 1.75, 1.7578125, 2.0 ** -60, 3e38, 2.0 ** -40 * 448, 1e-38]
    for i, big in enumerate(rows):
        c = ref.Cache([40], 1, 64, device, seed=i)
        x = torch.zeros(40, 1, 64, device=device, dtype=BF16)
        x[3, 0, 5] = -big
        x[9, 0, :] = big / 3
        assert run_append(x, x.flip(0), [0, 40], c) == 0


def test_append_keeps_earlier_tokens_of_the_page():
    """Token by token: the exponent of a page rises with a large token and the
    earlier codes are re-rounded, also when the write starts at row 1 or 63."""
    device = dev()
    c = ref.Cache([1], 2, 64, device, seed=3)
    pool, scales = c.pool, c.scales
    table, page = c.page_table, c.table[0][0]
    want_pool, want_scales = pool.cpu().clone(), scales.cpu().clone()
    g = torch.Generator(device=device).manual_seed(1)
    for n in range(1, 65):
        x = (torch.randn(1, 2, 2, 64, device=device, generator=g) * 2.0 ** ((n * 7) % 23 - 8)).to(BF16)
        kv.append_gqa8(x[:, 0], x[:, 1], ints([0, 1], device), table, ints([n], device), pool, scales)
        ref.append(x[:, 0].double().cpu(), x[:, 1].double().cpu(), [0, 1], c.table, [n], want_pool, want_scales)
        assert torch.equal(scales.cpu()[page], want_scales[page]), n
        assert torch.equal(pool.cpu()[page], want_pool[page]), n


def test_append_flags_and_sanitizes_nonfinite_values():
    device = dev()
    c = ref.Cache([70], 1, 64, device, seed=5)
    x = torch.randn(70, 1, 64, device=device).to(BF16)
    x[3, 0, 7], x[4, 0, 8], x[69, 0, 1] = math.nan, math.inf, -math.inf
    y = torch.randn(70, 1, 64, device=device).to(BF16)
    assert run_append(x, y, [0, 70], c) == kv.DEV_NONFINITE


def test_append_skips_bad_pages():
    device = dev()
    c = ref.Cache([200, 100], 1, 64, device, seed=6, extra_columns=0)
    c.table[0][1], c.table[1][0] = c.pool.shape[0], -5
    c.page_table = ints(c.table, device)
    c.lens = [300, 100]                     # beyond the table as well
    c.seq_lens = ints(c.lens, device)
    x = torch.randn(400, 1, 64, device=device).to(BF16)
    assert run_append(x, x, [0, 300, 400], c) == kv.DEV_BAD_PAGE


# ---------------------------------------------------------------------------
# read-back
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d,dtype,hkv", [(128, BF16, 2), (64, F16, 3), (128, F16, 8), (64, BF16, 1)])
def test_read_is_exact(d, dtype, hkv):
    device = dev()
    c = ref.Cache([200, 64, 1, 300, 10], hkv, d, device, seed=d, spread=3)
    starts, news = [63, 0, 0, 129, 4], [130, 64, 1, 171, 0]
    cu = ref.cu_of(news)
    total = cu[-1] + 2
    k = torch.full((total, hkv, d), 7.0, dtype=dtype, device=device)
    v = torch.full((total, hkv, d), 8.0, dtype=dtype, device=device)
    err = torch.zeros(1, dtype=torch.int32, device=device)
    got = kv.read_gqa8(c.pool, c.scales, c.page_table, ints(starts, device), ints(cu, device), total,
                       dtype=dtype, k_out=k, v_out=v, dev_err=err)
    assert got[0] is k and got[1] is v and int(err.item()) == 0
    for b in range(5):
        x = ref.values(c.pool, c.scales, c.table[b], starts[b], starts[b] + news[b])
        rows = slice(cu[b], cu[b + 1])
        assert torch.equal(k[rows].double(), x[:, 0].transpose(0, 1).to(dtype).double())
        assert torch.equal(v[rows].double(), x[:, 1].transpose(0, 1).to(dtype).double())
    assert (k[cu[-1]:] == 7).all() and (v[cu[-1]:] == 8).all()


def test_read_saturates_f16_and_zeroes_bad_pages():
    device = dev()
    c = ref.Cache([64, 64], 1, 64, device, seed=1)
    c.pool[c.table[0][0]] = 0x7E                                 # 448
    c.scales[c.table[0][0]] = 127 + 8                            # 114688
    table = [c.table[0], [c.pool.shape[0]] + c.table[1][1:]]
    err = torch.zeros(1, dtype=torch.int32, device=device)
    k, v = kv.read_gqa8(c.pool, c.scales, ints(table, device), ints([0, 0], device), ints([0, 64, 128], device),
                        128, dtype=F16, dev_err=err)
    assert (k[:64] == 65504).all() and (v[:64] == 65504).all()
    assert (k[64:] == 0).all() and (v[64:] == 0).all() and int(err.item()) == kv.DEV_BAD_PAGE


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def check_attention(c, news, hq, dtype, window=0, sm_scale=None, q=None, max_new=None, seed=0, gain=1.0):
    device, d = c.pool.device, c.pool.shape[4]
    cu = ref.cu_of(news)
    if q is None:
        g = torch.Generator(device=device).manual_seed(seed)
        q = (torch.randn(cu[-1], hq, d, device=device, generator=g) * gain).to(dtype)
    scale = d ** -0.5 if sm_scale is None else sm_scale
    out = torch.full((q.shape[0], hq, d), 3.0, dtype=dtype, device=device)
    lse = torch.full((q.shape[0], hq), 3.0, device=device)
    err = torch.zeros(1, dtype=torch.int32, device=device)
    kv.attention_gqa8(q, c.pool, c.scales, c.page_table, c.seq_lens, ints(cu, device),
                      max(news) if max_new is None else max_new, scale, window=window, out=out, lse=lse,
                      dev_err=err)
    want = ref.attention(q[:cu[-1]], c.pool, c.scales, c.table, c.lens, cu, scale, window)
    tol, lse_tol = ref.bounds(*want, dtype, d)
    n = cu[-1]
    assert (out[n:] == 3).all() and (lse[n:] == 3).all()         # rows behind the last request
    off = (out[:n].double() - want[0]).abs()
    assert out[:n].isfinite().all()
    worst = float((off / tol).max()) if n else 0.0
    assert worst <= 1, f"out error {float(off.max()):.3g}, {worst:.3g} of its bound"
    empty = want[1] == -math.inf
    assert torch.equal(lse[:n] == -math.inf, empty)
    off = (lse[:n].double() - want[1]).masked_fill(empty, 0).abs()
    worst = float((off / lse_tol).max()) if n else 0.0
    assert worst <= 1, f"lse error {float(off.max()):.3g}, {worst:.3g} of its bound"
    assert (out[:n][empty] == 0).all()
    return int(err.item()), out, lse


EDGES = [1, 2, 63, 64, 65, 127, 128, 129, 200, 513]


@pytest.mark.parametrize("g,hkv,d,dtype", [(1, 2, 128, BF16), (4, 2, 128, BF16), (8, 1, 64, BF16), (7, 3, 64, F16),
                                           (3, 1, 128, F16), (16, 2, 128, BF16), (12, 1, 64, F16), (33, 1, 128, BF16)])
def test_attention_single_tokens(g, hkv, d, dtype):
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
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attention_rows_without_a_key(news, dtype):
    """Sequences of length zero, and fewer tokens than rows: 0 and -inf."""
    c = ref.Cache([2, 0, 1, 1, 0], 2, 128, dev(), seed=2)
    check_attention(c, news, 8, dtype)


@pytest.mark.parametrize("news", [[1, 1, 1], [70, 40, 1]])
def test_attention_masks_bad_pages(news):
    c = ref.Cache([300, 400, 130], 2, 128, dev(), seed=4, extra_columns=0)
    c.table[0][1], c.table[0][4], c.table[1][6] = -1, c.pool.shape[0], 1 << 30
    c.table[2][:3] = [-7, -7, -7]                                # nothing left of this one
    c.page_table = ints(c.table, c.pool.device)
    c.lens[1] = 700                                              # beyond the table
    c.seq_lens = ints(c.lens, c.pool.device)
    assert check_attention(c, news, 8, BF16)[0] == kv.DEV_BAD_PAGE


@pytest.mark.parametrize("news", [[1, 1], [5, 40]])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attention_blocks_of_very_different_size(news, dtype):
    """Page exponents up to 24 octaves apart; the last pages tiny."""
    c = ref.Cache([700, 1000], 1, 128, dev(), seed=8, spread=12)
    check_attention(c, news, 4, dtype, sm_scale=2.0 ** -16)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("nats", [8.0, 14.0])
def test_attention_first_token_draws_most(n, dtype, nats):
    """One key far above many small ones, whose weights together still count."""
    device = dev()
    c = ref.Cache([20000], 1, 64, device, seed=9)
    page = c.table[0][0]
    c.pool[page, 0, 0, 0] = 0x38                                 # 1.0
    c.pool[page, 0, 0, 1:] = 0
    c.scales[page, 0, 0] = 127
    g = torch.Generator(device=device).manual_seed(3)
    q = torch.full((n, 4, 64), nats / 8, device=device) + 0.02 * torch.randn(n, 4, 64, device=device, generator=g)
    check_attention(c, [n], 4, dtype, q=q.to(dtype))


@pytest.mark.parametrize("news", [[1, 1, 1], [2, 33, 1]])
def test_attention_scales_of_q(news):
    """Rows of q from 2^-100 to 2^60 and zero rows; negative and zero sm_scale."""
    device = dev()
    c = ref.Cache([100, 90, 70], 1, 128, device, seed=10)
    t = sum(news)
    g = torch.Generator(device=device).manual_seed(3)
    q = torch.randn(t, 4, 128, device=device, generator=g)
    e = torch.tensor([-100.0, 0.0, -20.0, 3.0], device=device)
    q = (q * torch.exp2(e)[None, :, None]).to(BF16)
    q[0, 1] = 0
    for s in (0.125, -0.07, 0.0):
        check_attention(c, news, 4, BF16, q=q, sm_scale=s)
    check_attention(c, news, 4, BF16, q=(q.float() * 2.0 ** 60).to(BF16), sm_scale=2.0 ** -63)


@pytest.mark.parametrize("news", [[1, 1], [3, 40]])
def test_attention_nonfinite_queries_stay_in_their_rows(news):
    device = dev()
    c = ref.Cache([100, 200], 1, 128, device, seed=11)
    q = torch.randn(sum(news), 4, 128, device=device).to(BF16)
    clean = check_attention(c, news, 4, BF16, q=q)[1:]
    bad = q.clone()
    bad[0, 1, 5], bad[-1, 2, 0] = math.nan, math.inf
    out, lse = kv.attention_gqa8(bad, c.pool, c.scales, c.page_table, c.seq_lens, ints(ref.cu_of(news), device),
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


@pytest.mark.parametrize("dtype,n,window", [(BF16, 1, 0), (F16, 3, 0), (BF16, 100, 0), (BF16, 2, 5000)])
def test_attention_long_contexts(dtype, n, window):
    c = ref.Cache([30011, 9, 16384], 2, 128, dev(), seed=13)
    assert check_attention(c, [n, min(n, 9), n], 8, dtype, window=window)[0] == 0


@pytest.mark.parametrize("n", [9, 33, 100, 128, 129, 140, 256, 257])
@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, F16)])
def test_attention_items_of_every_height(n, d, dtype):
    """One kv head, so n rows: below and above what an item and each of its two
    row tiles hold, with one tile of keys, an odd and an even number of them,
    and cut along the keys."""
    c = ref.Cache([n, 300, 500, 5000], 1, d, dev(), seed=n, spread=1)
    check_attention(c, [n, min(n, 300), n, n], 1, dtype, seed=n)
    check_attention(c, [n, min(n, 300), n, n], 1, dtype, window=200, seed=n)


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


def test_attention_flags_a_request_beyond_max_new():
    device = dev()
    c = ref.Cache([100, 50, 80], 1, 64, device, seed=16)
    news, cu = [1, 3, 1], ref.cu_of([1, 3, 1])
    q = torch.randn(5, 2, 64, device=device).to(BF16)
    err = torch.zeros(1, dtype=torch.int32, device=device)
    out, lse = (torch.full((5, 2, 64), 3.0, dtype=BF16, device=device), torch.full((5, 2), 3.0, device=device))
    kv.attention_gqa8(q, c.pool, c.scales, c.page_table, c.seq_lens, ints(cu, device), 1, 0.125, out=out, lse=lse,
                      dev_err=err)
    assert int(err.item()) == kv.DEV_BAD_LENGTH
    whole = check_attention(c, news, 2, BF16, q=q, sm_scale=0.125)
    for t in (0, 4):
        assert torch.equal(out[t], whole[1][t]) and torch.equal(lse[t], whole[2][t])
    assert (out[1:4] == 3).all() and (lse[1:4] == 3).all()


# ---------------------------------------------------------------------------
# together, streams, graphs
# ---------------------------------------------------------------------------
def serve(device, steps, d=128, hkv=2, hq=8, dtype=BF16, graph=False):
    """A prompt chunk of three sessions, then `steps` single tokens each: the
    attention's outputs and the K, V written."""
    g = torch.Generator(device=device).manual_seed(77)
    prompts, B = [100, 63, 1], 3
    width = 4
    pool = torch.randint(0, 256, (B * width, hkv, 2, 64, d), dtype=torch.uint8, device=device, generator=g)
    scales = torch.full((B * width, hkv, 2), 127, dtype=torch.uint8, device=device)
    table = torch.randperm(B * width, device=device, generator=g).to(torch.int32).view(B, width)
    cu, lens = ints(ref.cu_of(prompts), device), ints(prompts, device)
    x = torch.randn(sum(prompts), hq + 2 * hkv, d, device=device, generator=g).to(dtype)
    kv.append_gqa8(x[:, hq:hq + hkv], x[:, hq + hkv:], cu, table, lens, pool, scales)
    outs = [kv.attention_gqa8(x[:, :hq], pool, scales, table, lens, cu, max(prompts), d ** -0.5)[0]]
    cu1 = ints([0, 1, 2, 3], device)
    tokens = torch.randn(steps, B, hq + 2 * hkv, d, device=device, generator=g).to(dtype)
    buf = torch.empty_like(tokens[0])

    def step():
        lens.add_(1)
        kv.append_gqa8(buf[:, hq:hq + hkv], buf[:, hq + hkv:], cu1, table, lens, pool, scales)
        return kv.attention_gqa8(buf[:, :hq], pool, scales, table, lens, cu1, 1, d ** -0.5)[0]

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
    return outs, x, tokens, pool, scales


def test_serving_run_against_the_unquantized_attention():
    """Prompt, then 70 steps (pages fill and new ones begin).  Against
    attention over the values as they were given: each k, v element is off by
    at most 2^-4 of itself, or 2^-10 of its page's largest (subnormal codes),
    twice where its page's exponent rose; |q.k| sums of 128 random signs keep
    the scores within 0.15 of theirs (6 standard deviations of 128 products
    each off by 2^-4 / sqrt(3) at most), so out within exp(0.3) - 1 + 2^-3 of
    the softmax mean of |v| -- and far closer on average."""
    device = dev()
    outs, x, tokens, pool, scales = serve(device, 70)
    hq, hkv, d, prompts = 8, 2, 128, [100, 63, 1]
    cu = ref.cu_of(prompts)
    for b in range(3):
        ks = torch.cat([x[cu[b]:cu[b + 1], hq:hq + hkv], tokens[:, b, hq:hq + hkv]]).double()
        vs = torch.cat([x[cu[b]:cu[b + 1], hq + hkv:], tokens[:, b, hq + hkv:]]).double()
        qs = torch.cat([x[cu[b]:cu[b + 1], :hq], tokens[:, b, :hq]]).double()
        got = torch.cat([outs[0][cu[b]:cu[b + 1]]] + [o[b:b + 1] for o in outs[1:]]).double()
        n = ks.shape[0]
        ok = torch.ones(n, n, dtype=torch.bool, device=device).tril()
        for h in range(hq):
            s = (qs[:, h] @ ks[:, h // 4].T * d ** -0.5).masked_fill(~ok, -math.inf)
            p = torch.softmax(s, -1)
            want, mean = p @ vs[:, h // 4], p @ vs[:, h // 4].abs()
            assert ((got[:, h] - want).abs() <= 0.48 * mean + 0.01).all()
            assert float((got[:, h] - want).norm() / want.norm()) < 0.1


def test_serving_run_captured_in_a_graph_gives_the_same_bits():
    device = dev()
    a, b = serve(device, 70), serve(device, 70, graph=True)
    for x, y in zip(a[0], b[0]):
        assert torch.equal(x, y)
    assert torch.equal(a[3], b[3]) and torch.equal(a[4], b[4])


def test_calls_on_two_streams_do_not_share_anything():
    """Two calls in flight on two streams, each split over the SMs."""
    device = dev()
    cs = [ref.Cache([20000], 2, 128, device, seed=s) for s in (20, 21)]
    q = torch.randn(1, 8, 128, device=device).to(BF16)
    args = [(q, c.pool, c.scales, c.page_table, c.seq_lens, ints([0, 1], device), 1, 0.09) for c in cs]
    want = [kv.attention_gqa8(*a) for a in args]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(kv.attention_gqa8(*args[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_two_graphs_replayed_at_once():
    device = dev()
    c = ref.Cache([20000, 300], 2, 128, device, seed=22)
    qs = [torch.randn(2, 8, 128, device=device).to(BF16) for _ in range(2)]
    args = (c.pool, c.scales, c.page_table, c.seq_lens, ints([0, 1, 2], device), 1, 0.09)
    want = [kv.attention_gqa8(q, *args) for q in qs]
    graphs, got = [], []
    for q in qs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            got.append(kv.attention_gqa8(q, *args))
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


def test_own_workspace_and_its_refusal():
    device = dev()
    c = ref.Cache([20000], 2, 128, device, seed=23)
    q = torch.randn(1, 8, 128, device=device).to(BF16)
    args = (q, c.pool, c.scales, c.page_table, c.seq_lens, ints([0, 1], device), 1, 0.09)
    want = kv.attention_gqa8(*args)
    n = kv.attention_gqa8_workspace(1, 1, 1, 8, 2, 128)
    ws = torch.full((max(n, 1),), 255, dtype=torch.uint8, device=device)
    got = kv.attention_gqa8(*args, workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    if n:
        with pytest.raises(kv.Kv4Error) as e:
            kv.attention_gqa8(*args, workspace=ws[:n - 16])
        assert e.value.status == 5


def test_attention_reports_a_wait_that_runs_out():
    """A wait on a barrier that nothing arrives on gives up after its limit:
    KV4_DEV_TIMEOUT, and the call ends."""
    device = dev()
    c = ref.Cache([1000, 30], 1, 128, device, seed=24)
    for n in (1, 30):
        q = torch.randn(2 * n, 4, 128, device=device).to(BF16)
        args = (q, c.pool, c.scales, c.page_table, c.seq_lens, ints([0, n, 2 * n], device), n, 0.09)
        want = kv.attention_gqa8(*args)
        err = torch.zeros(1, dtype=torch.int32, device=device)
        kv.set_wait_limit(2_000_000, 1)
        try:
            kv.attention_gqa8(*args, dev_err=err)
            torch.cuda.synchronize()
        finally:
            kv.set_wait_limit()
        assert int(err.item()) == kv.DEV_TIMEOUT
        got = kv.attention_gqa8(*args)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("d,dtype,hq,n", [(128, BF16, 4, 1), (128, F16, 12, 1), (64, BF16, 4, 3), (128, BF16, 4, 40),
                                          (64, F16, 8, 70)])
def test_a_wait_that_runs_out_with_work_left(d, dtype, hq, n):
    """Blocks that give up in the middle of several items: the call ends, no row
    behind the last request is written, and the next call is whole."""
    device = dev()
    B = 700 if n < 8 else 250
    lens = [n + (i * 53) % 700 for i in range(B)]
    c = ref.Cache(lens, 2, d, device, seed=25)
    q = torch.randn(n * B + 5, hq, d, device=device).to(dtype)
    args = (q, c.pool, c.scales, c.page_table, c.seq_lens, ints(ref.cu_of([n] * B), device), n, 0.09)
    want = kv.attention_gqa8(*args)
    err = torch.zeros(1, dtype=torch.int32, device=device)
    out, lse = (torch.full((n * B + 5, hq, d), 3.0, dtype=dtype, device=device),
                torch.full((n * B + 5, hq), 3.0, device=device))
    kv.set_wait_limit(1_000_000, 1)
    try:
        kv.attention_gqa8(*args, out=out, lse=lse, dev_err=err)
        torch.cuda.synchronize()
    finally:
        kv.set_wait_limit()
    assert int(err.item()) == kv.DEV_TIMEOUT
    assert (out[n * B:] == 3).all() and (lse[n * B:] == 3).all()
    got = kv.attention_gqa8(*args)
    assert torch.equal(got[0][:n * B], want[0][:n * B]) and torch.equal(got[1][:n * B], want[1][:n * B])


@pytest.mark.parametrize("B,news", [(33, (1,)), (40, (0, 3, 70)), (1030, (1, 0, 2)), (1100, (9, 0, 1))])
def test_append_and_read_many_requests(B, news):
    """More requests than a warp looks at in one round, in two rounds; some
    without a token."""
    device = dev()
    news = [news[i % len(news)] for i in range(B)]
    lens = [n + (i * 13) % 90 for i, n in enumerate(news)]
    c = ref.Cache(lens, 1, 64, device, seed=B)
    cu = ref.cu_of(news)
    g = torch.Generator(device=device).manual_seed(B)
    x = (torch.randn(cu[-1], 2, 1, 64, device=device, generator=g) * 4).to(BF16)
    assert run_append(x[:, 0], x[:, 1], cu, c) == 0
    k, v = kv.read_gqa8(c.pool, c.scales, c.page_table, ints([n - m for n, m in zip(lens, news)], device),
                        ints(cu, device), cu[-1])
    for b in range(0, B, 7):
        want = ref.values(c.pool, c.scales, c.table[b], lens[b] - news[b], lens[b])
        assert torch.equal(k[cu[b]:cu[b + 1]].double(), want[:, 0].transpose(0, 1))
        assert torch.equal(v[cu[b]:cu[b + 1]].double(), want[:, 1].transpose(0, 1))


# ---------------------------------------------------------------------------
# what the binding takes and refuses
# ---------------------------------------------------------------------------
def test_strides_of_single_elements_do_not_matter():
    """One token, or one head: a contiguous tensor may have any stride there."""
    device = dev()
    c = ref.Cache([100], 1, 64, device, seed=26)
    x = torch.randn(1, 1, 64, device=device).to(BF16)
    odd = torch.as_strided(x.clone(), (1, 1, 64), (3, 5, 1))
    assert odd.is_contiguous()
    pools = []
    for t in (x, odd):
        pool, scales = c.pool.clone(), c.scales.clone()
        kv.append_gqa8(t, t, ints([0, 1], device), c.page_table, c.seq_lens, pool, scales)
        pools.append((pool, scales))
    assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])
    a = [kv.attention_gqa8(t, c.pool, c.scales, c.page_table, c.seq_lens, ints([0, 1], device), 1, 0.125)
         for t in (x, odd)]
    assert torch.equal(a[0][0], a[1][0]) and torch.equal(a[0][1], a[1][1])


def call_args(device):
    """A small valid call of each kind, by argument name."""
    c = ref.Cache([100, 30], 2, 64, device, seed=27)
    x = torch.randn(5, 2, 64, device=device).to(BF16)
    cu = ints([0, 3, 5], device)
    cache = dict(pool=c.pool, scales=c.scales, page_table=c.page_table)
    return {"append": (kv.append_gqa8, dict(k=x, v=x.clone(), cu_seqlens=cu, seq_lens=c.seq_lens, **cache)),
            "read": (kv.read_gqa8, dict(starts=ints([3, 0], device), cu_seqlens=cu, total=5, **cache)),
            "attention": (kv.attention_gqa8, dict(q=x.repeat(1, 2, 1), seq_lens=c.seq_lens, cu_seqlens=cu, max_new=3,
                                                  sm_scale=0.125, **cache))}


def unaligned(t):
    return torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view_as(t).copy_(t)


CACHE_REFUSALS = [
    ("pool", lambda t: t.cpu(), TypeError), ("pool", lambda t: t.view(torch.int8), TypeError),
    ("pool", lambda t: t[:, :, :1], ValueError), ("pool", lambda t: t[..., :32], ValueError),
    ("pool", lambda t: t.flatten(3), ValueError), ("pool", lambda t: t.transpose(0, 1), ValueError),
    ("pool", unaligned, kv.Kv4Error), ("pool", lambda t: t[:0], ValueError),
    ("scales", lambda t: t[:-1], ValueError), ("scales", lambda t: t.float(), TypeError),
    ("scales", lambda t: None, TypeError), ("page_table", lambda t: t.long(), TypeError),
    ("page_table", lambda t: t[:1], ValueError), ("page_table", lambda t: t[0], ValueError),
    ("page_table", lambda t: t[:, ::2], ValueError), ("page_table", lambda t: t[:, :0], kv.Kv4Error),
    ("cu_seqlens", lambda t: t[:2], ValueError), ("cu_seqlens", lambda t: t.cpu(), TypeError),
    ("dev_err", lambda t: torch.zeros(1), TypeError),
]
INPUT_REFUSALS = [
    (lambda t: t.float(), TypeError), (lambda t: t[:, :, :32], ValueError), (lambda t: t[..., ::2], ValueError),
    (lambda t: t[:, :1], ValueError), (lambda t: unaligned(t), ValueError), (lambda t: t.cpu(), TypeError),
    (lambda t: torch.empty(5, 1, 64, dtype=BF16, device=t.device).expand(t.shape), kv.Kv4Error),
    (lambda t: torch.empty(5, t.shape[1], 68, dtype=BF16, device=t.device)[..., :64], ValueError),
]
REFUSALS = (
    [(f, name, change, e) for f in ("append", "read", "attention") for name, change, e in CACHE_REFUSALS]
    + [("append", name, change, e) for name in ("k", "v") for change, e in INPUT_REFUSALS]
    + [("attention", "q", change, e) for change, e in INPUT_REFUSALS]
    + [("append", "v", lambda t: t.half(), TypeError), ("append", "v", lambda t: t[:4], ValueError),
       ("append", "seq_lens", lambda t: t[:1], ValueError), ("read", "starts", lambda t: t.long(), TypeError),
       ("read", "total", lambda n: -1, ValueError), ("read", "total", lambda n: 2 ** 31, ValueError),
       ("read", "total", lambda n: 5.0, TypeError), ("read", "dtype", lambda t: torch.float32, TypeError),
       ("read", "k_out", lambda t: torch.empty(4, 2, 64, dtype=BF16, device="cuda"), ValueError),
       ("read", "v_out", lambda t: torch.empty(5, 2, 64, dtype=F16, device="cuda"), TypeError),
       ("read", "v_out", lambda t: torch.empty(5, 64, 2, dtype=BF16, device="cuda").mT, ValueError),
       ("attention", "max_new", lambda n: 0, kv.Kv4Error), ("attention", "max_new", lambda n: -1, ValueError),
       ("attention", "window", lambda n: -1, ValueError), ("attention", "sm_scale", lambda x: "a", TypeError),
       ("attention", "sm_scale", lambda x: 1e300, kv.Kv4Error), ("attention", "sm_scale", lambda x: math.nan, kv.Kv4Error),
       ("attention", "out", lambda t: torch.empty(5, 4, 64, dtype=F16, device="cuda"), TypeError),
       ("attention", "lse", lambda t: torch.empty(4, 5, device="cuda").T, ValueError),
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


def test_empty_calls():
    device = dev()
    c = ref.Cache([100, 30], 2, 64, device, seed=28)
    x = torch.empty(0, 2, 64, dtype=BF16, device=device)
    cu, none = ints([0, 0, 0], device), ints([0], device)
    pool = c.pool.clone()
    kv.append_gqa8(x, x, cu, c.page_table, c.seq_lens, c.pool, c.scales)
    k, v = kv.read_gqa8(c.pool, c.scales, c.page_table, ints([0, 0], device), cu, 0)
    out, lse = kv.attention_gqa8(x, c.pool, c.scales, c.page_table, c.seq_lens, cu, 0, 0.1)
    assert k.shape == v.shape == out.shape == (0, 2, 64) and lse.shape == (0, 2)
    x = torch.ones(3, 2, 64, dtype=BF16, device=device)          # no request at all
    kv.append_gqa8(x, x, none, c.page_table[:0], c.seq_lens[:0], c.pool, c.scales)
    out, lse = torch.full((3, 2, 64), 3.0, dtype=BF16, device=device), torch.full((3, 2), 3.0, device=device)
    kv.attention_gqa8(x, c.pool, c.scales, c.page_table[:0], c.seq_lens[:0], none, 1, 0.1, out=out, lse=lse)
    assert torch.equal(c.pool, pool) and (out == 3).all() and (lse == 3).all()


@pytest.mark.parametrize("cu", [[0, 40, 20, 70], [-9, 5, 2 ** 31 - 1, 3], [70, 0, -2 ** 31, 90], [0, 70, 70, 70]])
@pytest.mark.parametrize("lens", [[2 ** 31 - 1, -2 ** 31, 5], [3, 2 ** 31 - 1, 2 ** 31 - 40], [90, 20, 60]])
def test_lengths_and_pages_out_of_range_stay_in_bounds(cu, lens):
    """Rows, lengths and page numbers that nobody should pass: what lies around
    the call's tensors is left as it was.  (Every one of them is held to the
    call's sizes before it makes an address.)"""
    device = dev()
    T, hq, hkv, d, pages = 70, 8, 2, 64, 8
    g = torch.Generator(device=device).manual_seed(3)
    pool = torch.randint(0, 126, (pages + 2, hkv, 2, 64, d), dtype=torch.uint8, device=device, generator=g)
    scales = torch.full((pages + 2, hkv, 2), 127, dtype=torch.uint8, device=device)
    table = ints([[0, 7, 2 ** 31 - 1, 3], [-2 ** 31, 1, 8, 2], [4, 4, 5, -1]], device)
    guard_pool, guard_scales = pool.clone(), scales.clone()
    cu_t, lens_t = ints(cu, device), ints(lens, device)
    x = torch.randn(T, hq + 2 * hkv, d, device=device, generator=g).to(BF16)
    cache = (pool[1:-1], scales[1:-1])
    for max_new in (1, 70):
        out = torch.full((T + 2, hq, d), 3.0, dtype=BF16, device=device)
        lse = torch.full((T + 2, hq), 3.0, device=device)
        kv.attention_gqa8(x[:, :hq], *cache, table, lens_t, cu_t, max_new, 0.125, out=out[1:-1], lse=lse[1:-1])
        for t in (out, lse):
            assert (t[0] == 3).all() and (t[-1] == 3).all()
    ko = torch.full((T + 2, hkv, d), 3.0, dtype=BF16, device=device)
    vo = ko.clone()
    kv.read_gqa8(*cache, table, lens_t, cu_t, T, k_out=ko[1:-1], v_out=vo[1:-1])
    for t in (ko, vo):
        assert (t[0] == 3).all() and (t[-1] == 3).all()
    kv.append_gqa8(x[:, hq:hq + hkv], x[:, hq + hkv:], cu_t, table, lens_t, *cache)
    for t, was in ((pool, guard_pool), (scales, guard_scales)):
        assert torch.equal(t[0], was[0]) and torch.equal(t[-1], was[-1])


FIRST_CALLS = """
import sys
import torch
sys.path.insert(0, sys.argv[1])
import bit_kv_cache_nvfp4_gb300 as kv
i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
pool = torch.zeros(8, 2, 2, 64, 64, dtype=torch.uint8, device="cuda")
scales = torch.full((8, 2, 2), 127, dtype=torch.uint8, device="cuda")
table, lens, cu = i([[0, 1, 2, 3], [4, 5, 6, 7]]), i([200, 1]), i([0, 200, 201])
x = torch.randn(201, 12, 64, device="cuda").to(torch.bfloat16)
starts = i([0, 0])
def calls():
    kv.append_gqa8(x[:, 8:10], x[:, 10:], cu, table, lens, pool, scales)
    return (*kv.read_gqa8(pool, scales, table, starts, cu, 201),
            *kv.attention_gqa8(x[:, :8], pool, scales, table, lens, cu, 200, 0.125))
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    kept = calls()
g.replay()
torch.cuda.synchronize()
kept = [t.clone() for t in kept]
assert all(torch.equal(a, b) for a, b in zip(kept, calls()))
"""


def test_first_calls_of_a_process_can_be_captured():
    import pathlib
    import subprocess
    import sys
    dev()
    root = str(pathlib.Path(__file__).resolve().parents[1])
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_calls_from_two_threads():
    import threading
    device = dev()
    c = ref.Cache([3000, 70], 2, 128, device, seed=29)
    q = torch.randn(41, 8, 128, device=device).to(BF16)
    args = (q, c.pool, c.scales, c.page_table, c.seq_lens, ints([0, 1, 41], device), 40, 0.09)
    want = kv.attention_gqa8(*args)
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i].append(kv.attention_gqa8(*args))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for out, lse in got[0] + got[1]:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ---------------------------------------------------------------------------
# offsets beyond 32 bits
# ---------------------------------------------------------------------------
def test_pool_beyond_32_bits():
    """A pool of 6.5 GB, its last pages used: as in a small one."""
    device, pages = dev(), 200_000
    lens, news = [300, 65, 1], [40, 1, 1]
    c = ref.Cache(lens, 2, 128, device, seed=30)
    n, cu = c.pool.shape[0], ints(ref.cu_of(news), device)
    pool = torch.empty(pages, 2, 2, 64, 128, dtype=torch.uint8, device=device)
    scales = torch.empty(pages, 2, 2, dtype=torch.uint8, device=device)
    pool[pages - n:], scales[pages - n:] = c.pool, c.scales
    table = torch.where(c.page_table < 0, c.page_table, c.page_table + (pages - n))
    x = torch.randn(42, 12, 128, device=device).to(BF16)
    starts = ints([9, 0, 0], device)
    got = []
    for p, s, t in ((c.pool, c.scales, c.page_table), (pool, scales, table)):
        kv.append_gqa8(x[:, 8:10], x[:, 10:], cu, t, c.seq_lens, p, s)
        got.append((p[-n:], s[-n:], *kv.read_gqa8(p, s, t, starts, cu, 42),
                    *kv.attention_gqa8(x[:, :8], p, s, t, c.seq_lens, cu, 40, 0.09)))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_input_strides_beyond_32_bits():
    """Tokens 1.5e9 elements apart."""
    device = dev()
    far = torch.empty(2 * 1_500_000_000 + 12 * 128, dtype=BF16, device=device)
    x = torch.as_strided(far, (3, 12, 128), (1_500_000_000, 128, 1))
    near = torch.randn(3, 12, 128, device=device).to(BF16)
    x.copy_(near)
    c = ref.Cache([80, 3], 2, 128, device, seed=31)
    cu = ints([0, 2, 3], device)
    got = []
    for y in (near, x):
        pool, scales = c.pool.clone(), c.scales.clone()
        kv.append_gqa8(y[:, 8:10], y[:, 10:], cu, c.page_table, c.seq_lens, pool, scales)
        got.append((pool, scales, *kv.attention_gqa8(y[:, :8], pool, scales, c.page_table, c.seq_lens, cu, 2, 0.09)))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_outputs_beyond_32_bits():
    """2.7e9 elements of out and of the read-back.  The last rows of out within
    their bounds, not bit for bit as in a call of their own: which of the two
    warpgroups gets an item's even tiles depends on the tiles before it, and
    with that the order in which a row's partial sums are added (a + b in fp32
    is off by up to 2^-24 of itself either way, which the bounds count)."""
    device = dev()
    B, hkv, g, d = 65535, 16, 20, 128
    c = ref.Cache([500], hkv, d, device, seed=32)
    table = c.page_table[:, :8].expand(B, -1).contiguous()       # every request the same pages
    lens = torch.randint(1, 500, (B,), dtype=torch.int32, device=device)
    cu = torch.arange(B + 1, dtype=torch.int32, device=device)
    q = torch.empty(B, hkv * g, d, dtype=BF16, device=device)
    q[-9:] = torch.randn(9, hkv * g, d, device=device).to(BF16)
    q[:-9] = q[-9:-8]
    out, lse = kv.attention_gqa8(q, c.pool, c.scales, table, lens, cu, 1, 0.09)
    want = ref.attention(q[-9:], c.pool, c.scales, c.table * 9, lens[-9:].tolist(), list(range(10)), 0.09)
    tol, lse_tol = ref.bounds(*want, BF16, d)
    assert ((out[-9:].double() - want[0]).abs() <= tol).all()
    assert ((lse[-9:].double() - want[1]).abs() <= lse_tol).all()
    del q, out, lse
    n = 1_300_000                                                # tokens of a request that repeats its pages
    row = c.page_table[0, :7].repeat(n // 448 + 1)[None].contiguous()
    k, v = kv.read_gqa8(c.pool, c.scales, row, ints([0], device), ints([0, n], device), n)
    last = kv.read_gqa8(c.pool, c.scales, row, ints([n - 100], device), ints([0, 100], device), 100)
    assert torch.equal(k[-100:], last[0]) and torch.equal(v[-100:], last[1])


def test_prompt_of_many_row_groups_and_its_last_rows():
    """A prompt whose rows fill hundreds of items: its last rows as when they
    are the only new ones, within the bounds of both."""
    device = dev()
    n, hq, d = 20011, 8, 64
    c = ref.Cache([n], 1, d, device, seed=33)
    q = torch.randn(n, hq, d, device=device).to(BF16)
    out, lse = kv.attention_gqa8(q, c.pool, c.scales, c.page_table, c.seq_lens, ints([0, n], device), n, 0.125)
    for first, count in ((0, 65), (10000, 30), (n - 33, 33)):
        lens = [first + count]
        want = ref.attention(q[first:first + count], c.pool, c.scales, c.table, lens, [0, count], 0.125, 0)
        tol, lse_tol = ref.bounds(*want, BF16, d)
        assert ((out[first:first + count].double() - want[0]).abs() <= tol).all()
        assert ((lse[first:first + count].double() - want[1]).abs() <= lse_tol).all()
