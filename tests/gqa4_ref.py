"""The 4-bit grouped-query cache in 64 bits: plain implementations that the GPU
tests compare against, and inputs for them.

Nothing here uses the library.  A row holds E2M1 codes (sign, 2 exponent bits with
bias 1, 1 fraction bit), two a byte with the even element low, and an E4M3 scale
for each 16 elements; value = code * scale."""
from __future__ import annotations

import math

import torch

from gqa8_ref import cu_of, e4m3_values  # noqa: F401  (E4M3's 256 values)

PAGE = 64
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def nearest(grid: torch.Tensor, x: torch.Tensor) -> torch.Tensor:
    """Index of the value of a rising grid that is nearest to x >= 0 (saturating),
    ties to the even index."""
    a = x.clamp(max=float(grid[-1]))
    hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - grid[lo], grid[hi] - a
    return torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def quantize(x: torch.Tensor):
    """float64 [.., D] (host) -> code bytes [.., D / 2], scale bytes [.., D / 16]."""
    b = x.unflatten(-1, (-1, 16))
    fin = b.isfinite()
    amax = torch.where(fin, b, 0.0).abs().amax(-1)
    scale = nearest(e4m3_values()[:127], amax / 6)
    s = e4m3_values()[scale][..., None]
    y = torch.where(b.isnan(), 0.0, b) / torch.where(s > 0, s, 1.0)
    code = nearest(E2M1[:8], y.abs()) + 8 * (torch.signbit(b) & ~b.isnan()).long()
    code = torch.where(s > 0, code, 0).flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.to(torch.uint8)


def dequantize(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    s = e4m3_values().to(codes.device)[scales.long()]
    return (E2M1.to(codes.device)[c].unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def append(k, v, cu, table, lens, pool, scales):
    """The append on host copies: k, v float64 [T, Hkv, D]; pool, scales uint8
    (changed in place)."""
    for b in range(len(lens)):
        start = lens[b] - (cu[b + 1] - cu[b])
        for pos in range(max(start, 0), lens[b]):
            page = pos // PAGE
            if page < len(table[b]) and 0 <= table[b][page] < pool.shape[0]:
                row = cu[b] + pos - start
                code, scale = quantize(torch.stack([k[row], v[row]], 1))
                pool[table[b][page], :, :, pos % PAGE] = code
                scales[table[b][page], :, :, pos % PAGE] = scale


def values(pool, scales, table_b, first: int, last: int):
    """K and V of positions [first, last): float64 [Hkv, 2, n, D]; a page the
    table does not have gives NaN."""
    shape = (*pool.shape[1:4], 2 * pool.shape[4])
    out = []
    for page in range(first // PAGE, -(-last // PAGE)):
        if page < len(table_b) and 0 <= table_b[page] < pool.shape[0]:
            out.append(dequantize(pool[table_b[page]], scales[table_b[page]]))
        else:
            out.append(torch.full(shape, math.nan, dtype=torch.float64, device=pool.device))
    if not out:
        return torch.zeros(shape[0], 2, 0, shape[3], dtype=torch.float64, device=pool.device)
    return torch.cat(out, dim=2)[:, :, first % PAGE:first % PAGE + last - first]


def attention(q, pool, scales, table, lens, cu, sm_scale, window=0):
    """(out, lse, sizes) in 64 bits.  sizes: what rounding errors are multiplied
    by, per row: the softmax mean of |v| [T, Hq, D], sm_scale * max_j sum_d |q_d
    k_jd|, the largest |q| times the largest sum_d |k_jd| sm_scale, the largest
    |v|, and the number of keys."""
    T, hq, d = q.shape
    g, dev = hq // pool.shape[1], q.device
    out = torch.zeros(T, hq, d, dtype=torch.float64, device=dev)
    weight = torch.zeros_like(out)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device=dev)
    spread, wide, top, keys = (torch.zeros(T, hq, dtype=torch.float64, device=dev) for _ in range(4))
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        if n <= 0 or lens[b] <= 0:
            continue
        pos = torch.arange(lens[b] - n, lens[b], device=dev)
        lo = max(0, lens[b] - n - window + 1) // PAGE * PAGE if window else 0
        x = values(pool, scales, table[b], lo, lens[b])
        key = torch.arange(lo, lens[b], device=dev)
        ok = key[None] <= pos[:, None]
        if window:
            ok = ok & (key[None] > pos[:, None] - window)
        ok = ok & x[0, 0, :, 0].isfinite()[None]
        rows = slice(cu[b], cu[b + 1])
        for h in range(hq):
            k, v = x[h // g, 0].nan_to_num(), x[h // g, 1].nan_to_num()
            qq = q[rows, h].double()
            s = (qq @ k.T * sm_scale).masked_fill(~ok, -math.inf)
            m = s.amax(-1, keepdim=True)
            m = m.masked_fill(m == -math.inf, 0)
            p = torch.exp(s - m).masked_fill(~ok, 0)
            l = p.sum(-1, keepdim=True)
            p = p / l.masked_fill(l == 0, 1)
            out[rows, h], weight[rows, h] = p @ v, p @ v.abs()
            lse[rows, h] = (m + l.log())[:, 0]
            spread[rows, h] = (qq.abs() @ k.abs().T * abs(sm_scale)).masked_fill(~ok, 0).amax(-1)
            wide[rows, h] = (qq.abs().amax(-1, keepdim=True) * k.abs().sum(-1)[None] * abs(sm_scale)).masked_fill(~ok, 0).amax(-1)
            top[rows, h] = (v.abs().amax(-1)[None] * ok).amax(-1)
            keys[rows, h] = ok.sum(-1).double()
    return out, lse, (weight, spread, wide, top, keys)


def bounds(out, lse, sizes, dtype, D):
    """Elementwise bounds on |out error| and |lse error|.

    Scores: exact products summed in fp32, D additions and the scale, each off by
    2^-23 of the running sum at most (the tensor core need not round to nearest):
    (D + 16) 2^-23 spread; q's elements below 2^-22 of their row's largest are off
    by 2^-32 of that: 2^-32 wide.  exp2 and its fp32 argument (up to 2^7 in magnitude
    where a weight matters): 2^-17.  A weight enters its product rounded by half an
    f16 step, 2^-11, or below f16's normal range by 2^-32 of the row's largest.  A
    row's sums, of weights and of weights times v: n keys, 2^-23 each, in either
    product and for the join, twice.  The output is rounded once: eps / 2 of itself
    (fp16's subnormals: 2^-25)."""
    weight, spread, wide, top, n = sizes
    ds = (D + 16) * 2.0 ** -23 * spread + 2.0 ** -32 * wide + 2.0 ** -17
    half = torch.finfo(dtype).eps / 2
    sums = 2 * (n + 16) * 2.0 ** -23
    tol = half * out.abs() + (1 + half) * weight * (2.0 ** -11 + 2 * ds + sums)[..., None]
    tol = tol + (n * 2.0 ** -32 * top)[..., None] + 2.0 ** -25
    lse_tol = ds + sums + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0, neginf=0.0)
    return tol, lse_tol


class Cache:
    """A random cache of B requests on `device`: pool, scales, table with shuffled
    pages; bytes nobody wrote are random, NaN and negative scales among them.
    `spread`: octaves up and down that a token's scales lie apart."""

    def __init__(self, lens, hkv, d, device, seed=0, spare=2, spread=0, extra_columns=1):
        g = torch.Generator().manual_seed(seed)
        self.lens = list(lens)
        need = [-(-max(n, 0) // PAGE) for n in lens]
        pages = sum(need) + spare
        perm = torch.randperm(pages, generator=g).tolist()
        width = max(1, max(need)) + extra_columns
        self.table = []
        pool = torch.randint(0, 256, (pages, hkv, 2, PAGE, d // 2), generator=g, dtype=torch.uint8)
        scales = torch.randint(0, 256, (pages, hkv, 2, PAGE, d // 16), generator=g, dtype=torch.uint8)
        at = 0
        for b, n in enumerate(lens):
            row = perm[at:at + need[b]]
            at += need[b]
            self.table.append(row + [-1] * (width - need[b]))
            if need[b]:
                # codes at random with small ones in front, E4M3 scales near 1/2
                mag = torch.randint(0, 8, (2, need[b], hkv, 2, PAGE, d // 2), generator=g)
                mag = torch.minimum(mag, torch.randint(0, 9, mag.shape, generator=g).clamp(max=7))
                code = mag + 8 * torch.randint(0, 2, mag.shape, generator=g)
                e = torch.randint(6 - spread, 7 + spread, (need[b], hkv, 2, PAGE, 1), generator=g).clamp(0, 14)
                s = e * 8 + torch.randint(0, 8, (need[b], hkv, 2, PAGE, d // 16), generator=g)
                live = torch.arange(need[b] * PAGE).view(need[b], 1, 1, PAGE, 1) < n
                pool[row] = torch.where(live, (code[0] | code[1] << 4).to(torch.uint8), pool[row])
                scales[row] = torch.where(live, s.to(torch.uint8), scales[row])
        self.pool, self.scales = pool.to(device), scales.to(device)
        self.page_table = torch.tensor(self.table, dtype=torch.int32, device=device)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=device)
