"""How the grouped-query attention joins the pieces of items that were cut: the kernels
of few rows and of many, items of up to 8 pieces and of more, 8 rows a block (many
requests and heads) and one."""
import pytest
import torch

import bit_kv_cache_nvfp4_gb300 as kv
import gqa4_ref
import gqa8_ref
import test_gpu_gqa4
import test_gpu_gqa8
from test_gpu_gqa4 import BF16, F16, dev, ints

pytestmark = pytest.mark.gpu
BITS = {4: (gqa4_ref, test_gpu_gqa4.check_attention, kv.attention_gqa4),
        8: (gqa8_ref, test_gpu_gqa8.check_attention, kv.attention_gqa8)}


def one_long(length, others):
    """Contexts of 46 requests, the 20th of them long."""
    lens = [i * 31 % (others + 1) for i in range(46)]
    lens[20] = length
    return lens


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d,dtype,g,n", [(128, BF16, 8, 1), (128, F16, 3, 1), (64, BF16, 4, 3), (64, F16, 6, 4), (128, BF16, 8, 4),
                                         (64, F16, 16, 3)])
@pytest.mark.parametrize("others", [0, 150])
def test_a_long_context_among_many_requests(bits, d, dtype, g, n, others):
    """An item of some 200 pieces beside many of one: 3, 8, 12, 24, 32 and 48 rows, by 8 a
    block."""
    ref, check, _ = BITS[bits]
    lens = one_long(100000, others)
    c = ref.Cache(lens, 1, d, dev(), seed=31)
    assert check(c, [min(n, x) for x in lens], g, dtype)[0] == 0


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("hkv,lens", [(1, [100000]), (2, [40000, 90, 700]), (1, [1000]), (2, [3000] * 46), (1, [6000] * 50)])
@pytest.mark.parametrize("d,dtype,n", [(128, F16, 1), (64, BF16, 3)])
def test_items_of_few_rows(bits, hkv, lens, d, dtype, n):
    """By rows and by blocks of rows, of many pieces and of few."""
    ref, check, _ = BITS[bits]
    c = ref.Cache(lens, hkv, d, dev(), seed=32)
    assert check(c, [n] * len(lens), 5 * hkv, dtype)[0] == 0


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("lens,news", [([100000], [40]), ([60000, 80, 300], [70, 5, 0]), ([9000], [300]), ([2000] * 30, [50] * 30)])
@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, F16)])
def test_items_of_many_rows(bits, lens, news, d, dtype):
    ref, check, _ = BITS[bits]
    c = ref.Cache(lens, 1, d, dev(), seed=33)
    assert check(c, news, 2, dtype)[0] == 0


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d,n", [(128, 1), (64, 3)])
def test_nonfinite_rows_of_a_long_context(bits, d, n):
    """A NaN or an infinity of q stays in its row, through any number of pieces."""
    ref, _, attention = BITS[bits]
    device, lens = dev(), one_long(100000, 64)
    news = [min(n, x) for x in lens]
    c = ref.Cache(lens, 1, d, device, seed=34)
    cu = ref.cu_of(news)
    q = torch.randn(cu[-1], 8, d, device=device).to(BF16)
    row = cu[20]
    odd = torch.zeros(cu[-1], 8, dtype=torch.bool, device=device)
    odd[row, 1] = odd[row, 7] = odd[row + n - 1, 4] = True
    # (a row's reference moves with those beside it, and its last bits with that: the
    # others are compared with the definition)
    want = ref.attention(q, c.pool, c.scales, c.table, c.lens, cu, d ** -0.5)
    tol, lse_tol = ref.bounds(*want, BF16, d)
    q[row, 1, 5], q[row, 7, 0], q[row + n - 1, 4, 63] = float("nan"), float("inf"), float("-inf")
    out, lse = attention(q, c.pool, c.scales, c.page_table, c.seq_lens, ints(cu, device), n, d ** -0.5)
    assert out[odd].isnan().all() and lse[odd].isnan().all()
    assert ((out.double() - want[0]).abs() <= tol)[~odd].all()
    assert ((lse.double() - want[1]).abs() <= lse_tol)[~odd].all()


@pytest.mark.parametrize("bits", [4, 8])
def test_joins_give_equal_bits(bits):
    ref, _, attention = BITS[bits]
    device, lens = dev(), one_long(100000, 150)
    c = ref.Cache(lens, 2, 128, device, seed=35)
    news = [min(1, x) for x in lens]
    q = torch.randn(sum(news), 16, 128, device=device).to(F16)
    args = (q, c.pool, c.scales, c.page_table, c.seq_lens, ints(ref.cu_of(news), device), 1, 0.09)
    first = attention(*args)
    for _ in range(20):
        again = attention(*args)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
