"""Every tile of keys counts: queries that one key in each tile answers to, so
that a tile that was lost, or taken twice, is far outside a row's bounds."""
import pytest
import torch

import gqa8_ref as ref
from test_gpu_gqa8 import BF16, F16, dev
from test_gpu_gqa8_values import check

TILE = 128


def needles(n, d, device, dtype, seed=0):
    """A request of n tokens over one kv head, and a row of q for each tile of
    128 keys.  Keys are random with a standard deviation of 1/8; one key of tile
    t is 7/8 in dimension t % d, of a sign by t // d, where row t of q has a
    component that makes that a score of 17.5 (sm_scale d^-0.5) and of the others
    2.5 times a random number: with 30000 keys the one has 98 % of the weight."""
    c = ref.Cache([n], 1, d, "cpu", seed=seed)
    tiles = -(-n // TILE)
    assert tiles <= 2 * d
    pages = torch.tensor(c.table[0][:-(-n // 64)])
    c.scales[pages, 0, 0] = 127 - 9
    q = torch.zeros(tiles, d)
    for t in range(tiles):
        at = t * TILE + (t * 37) % min(TILE, n - t * TILE)
        sign = t // d
        c.pool[c.table[0][at // 64], 0, 0, at % 64, t % d] = 0x7E | sign << 7           # +-448 * 2^-9
        q[t, t % d] = (1 - 2 * sign) * 20 * d ** 0.5
    c.pool, c.scales = c.pool.to(device), c.scales.to(device)
    c.page_table, c.seq_lens = c.page_table.to(device), c.seq_lens.to(device)
    return c, q.to(device=device, dtype=dtype)


@pytest.mark.parametrize("n,d,dtype", [(30011, 128, BF16), (16384, 64, F16)])
def test_a_lost_tile_is_outside_the_bounds(n, d, dtype):
    """Of the reference itself, on the host: without the values of its tile, or
    with them twice, a row is several times its bound off."""
    c, q = needles(n, d, "cpu", dtype)
    for t in sorted({0, 1, q.shape[0] - 1, *range(5, q.shape[0], 47)}):
        row = q[t].view(1, 1, d)
        want = ref.attention(row, c.pool, c.scales, c.table, c.lens, [0, 1], d ** -0.5)
        tol, _ = ref.bounds(*want, dtype, d)
        pool = c.pool.clone()
        pool[c.table[0][2 * t:2 * t + 2], :, 1] = 0
        lost = ref.attention(row, pool, c.scales, c.table, c.lens, [0, 1], d ** -0.5)[0]
        off = float(((lost - want[0]).abs() / tol).max())
        assert off > 20, (t, off)


@pytest.mark.gpu
@pytest.mark.parametrize("g", [8, 16, 24])
@pytest.mark.parametrize("n,d,dtype", [(30011, 128, BF16), (16384, 64, F16), (900, 128, F16)])
def test_single_tokens_see_every_tile(n, d, dtype, g):
    """A long request cut over the SMs' blocks, for items of each height."""
    c, q = needles(n, d, dev(), dtype)
    for t in range(0, q.shape[0], g):
        rows = q[t:t + g]
        rows = torch.cat([rows, rows[:1].expand(g - rows.shape[0], -1)])
        check(c, [1], g, dtype, q=rows[None])


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, 9000])
@pytest.mark.parametrize("n,d,dtype", [(30011, 128, BF16), (16384, 64, F16), (900, 128, F16)])
def test_prompt_rows_see_every_tile(n, d, dtype, window):
    """Row t of a chunk asks for tile t; items of up to 128 rows and of more."""
    c, q = needles(n, d, dev(), dtype)
    for m in (q.shape[0], 60, 128, 130):
        for t in range(0, q.shape[0], m):
            rows = q[t:t + m]
            rows = torch.cat([rows[:1].expand(m - rows.shape[0], -1), rows])
            check(c, [m], 1, dtype, q=rows[:, None], window=window)


@pytest.mark.gpu
def test_requests_of_many_lengths_see_every_tile():
    """33 requests of one length after the other share their blocks."""
    device, d = dev(), 128
    cs = [needles(n, d, "cpu", BF16, seed=n) for n in range(1, 4300, 131)]
    big = ref.Cache([n for c, _ in cs for n in c.lens], 1, d, "cpu")
    for b, (c, _) in enumerate(cs):
        for i, page in enumerate(big.table[b]):
            if page >= 0:
                big.pool[page], big.scales[page] = c.pool[c.table[0][i]], c.scales[c.table[0][i]]
    for name in ("pool", "scales", "page_table", "seq_lens"):
        setattr(big, name, getattr(big, name).to(device))
    for t in range(0, 34, 8):
        q = torch.stack([c_q[torch.arange(t, t + 8) % c_q.shape[0]] for _, c_q in cs]).to(device)
        check(big, [1] * len(cs), 8, BF16, q=q)


@pytest.mark.gpu
@pytest.mark.parametrize("g", [25, 31, 48, 64, 100, 128])
@pytest.mark.parametrize("d,dtype", [(128, F16), (64, BF16), (64, F16), (128, BF16)])
def test_many_heads_a_group(g, d, dtype):
    """Multi-query groups, which the prompt kernel takes also for single tokens."""
    c = ref.Cache([1, 64, 130, 513, 3000], 2, d, dev(), seed=g, spread=1)
    check(c, [1, 1, 1, 1, 1], 2 * g, dtype, seed=g)
    check(c, [1, 3, 2, 5, 4], 2 * g, dtype, window=100, seed=g)
