"""The 8-bit grouped-query cache in 64 bits: plain implementations that the
GPU tests compare against, and inputs for them.

Nothing here uses the library.  A code is E4M3 (sign, 4 exponent bits with
bias 7, 3 fraction bits, 0x7F / 0xFF NaN), a block's value is code * 2^e with
the least e such that amax <= 448 * 2^e, -48 <= e <= 48."""
from __future__ import annotations

import math

import torch

PAGE = 64


def e4m3_values() -> torch.Tensor:
    out = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = math.nan if c & 127 == 127 else (f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10))
        out.append(-v if c & 128 else v)
    return torch.tensor(out, dtype=torch.float64)


def encode(x: torch.Tensor) -> torch.Tensor:
    """Nearest E4M3 code of float64 x (|x| <= 448 after saturation), ties to
    the even code."""
    pos = e4m3_values()[:127]                           # 0 .. 448, rising
    a = x.abs().clamp(max=448.0).cpu()
    hi = torch.searchsorted(pos, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return torch.where(torch.signbit(x.cpu()), code + 128, code).to(torch.uint8)


def least_exponent(amax: float) -> int:
    e = -48
    while e < 48 and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def append(k, v, cu, table, lens, pool, scales):
    """The append on host copies: k, v float64 [T, Hkv, D]; pool, scales
    uint8 (changed in place)."""
    vals = e4m3_values()
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        start = lens[b] - n
        for page in range(max(start, 0) // PAGE, -(-lens[b] // PAGE)):
            first, last = max(start, page * PAGE, 0), min(lens[b], page * PAGE + PAGE)
            if first >= last:
                continue
            if not (page < len(table[b]) and 0 <= table[b][page] < pool.shape[0]):
                continue
            pg, off = table[b][page], first - page * PAGE
            rows = slice(cu[b] + first - start, cu[b] + last - start)
            for h in range(pool.shape[1]):
                for s, src in enumerate((k, v)):
                    x = src[rows, h]
                    fin = x[x.isfinite()]
                    e = least_exponent(float(fin.abs().max()) if fin.numel() else 0.0)
                    if off > 0:
                        old = int(scales[pg, h, s]) - 127
                        e = max(e, old)
                        if e > old:
                            kept = vals[pool[pg, h, s, :off].long()] * 2.0 ** (old - e)
                            pool[pg, h, s, :off] = encode(kept)
                    y = torch.nan_to_num(x, nan=0.0, posinf=math.inf, neginf=-math.inf) * 2.0 ** -e
                    pool[pg, h, s, off:off + last - first] = encode(y)
                    scales[pg, h, s] = e + 127


def values(pool, scales, table_b, first: int, last: int):
    """K and V of positions [first, last): float64 [Hkv, 2, n, D]; a page the
    table does not have gives NaN."""
    vals = e4m3_values().to(pool.device)
    out = []
    for page in range(first // PAGE, -(-last // PAGE)):
        if page < len(table_b) and 0 <= table_b[page] < pool.shape[0]:
            x = vals[pool[table_b[page]].long()]
            out.append(x * torch.exp2(scales[table_b[page]].double() - 127)[..., None, None])
        else:
            out.append(torch.full(pool.shape[1:], math.nan, dtype=torch.float64, device=pool.device))
    if not out:
        return torch.zeros(pool.shape[1], 2, 0, pool.shape[4], dtype=torch.float64, device=pool.device)
    x = torch.cat(out, dim=2)
    return x[:, :, first % PAGE:first % PAGE + last - first]


def attention(q, pool, scales, table, lens, cu, sm_scale, window=0):
    """(out, lse, weight, spread) in 64 bits.  weight [T, Hq, D] is the mean of
    |v| under the softmax, spread [T, Hq] = sm_scale * max_j sum_d |q_d k_jd|
    and the largest |q| times the largest sum_d |k_jd|: what rounding errors of
    p and of the scores are multiplied by."""
    T, hq, d = q.shape
    hkv = pool.shape[1]
    g = hq // hkv
    dev = q.device
    out = torch.zeros(T, hq, d, dtype=torch.float64, device=dev)
    weight, top = torch.zeros_like(out), torch.zeros_like(out)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device=dev)
    spread, wide = torch.zeros_like(lse).fill_(0), torch.zeros_like(lse).fill_(0)
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
        held = torch.tensor([j // PAGE < len(table[b]) and 0 <= table[b][j // PAGE] < pool.shape[0]
                             for j in range(lo, lens[b])], device=dev)
        ok = ok & held[None]
        for h in range(hq):
            k, v = x[h // g, 0].nan_to_num(), x[h // g, 1].nan_to_num()
            qq = q[cu[b]:cu[b + 1], h].double()
            s = (qq @ k.T * sm_scale).masked_fill(~ok, -math.inf)
            m = s.amax(-1, keepdim=True)
            m = m.masked_fill(m == -math.inf, 0)
            p = torch.exp(s - m).masked_fill(~ok, 0)
            l = p.sum(-1, keepdim=True)
            p = p / l.masked_fill(l == 0, 1)
            rows = slice(cu[b], cu[b + 1])
            out[rows, h] = p @ v
            weight[rows, h] = p @ v.abs()
            lse[rows, h] = (m + l.log())[:, 0]
            spread[rows, h] = (qq.abs() @ k.abs().T * abs(sm_scale)).masked_fill(~ok, 0).amax(-1)
            wide[rows, h] = (qq.abs().amax(-1, keepdim=True) * k.abs().sum(-1)[None] *
                             abs(sm_scale)).masked_fill(~ok, 0).amax(-1)
    return out, lse, weight, (spread, wide)


def bounds(out, lse, weight, spread, dtype, D):
    """Elementwise bounds on |out error| and |lse error|.

    Scores: products of exact operands summed in fp32, D + 8 additions and the
    scale, each off by 2^-24 of the running sum: (D + 10) 2^-24 spread; q may
    enter with elements below 2^-10 of its row's largest rounded to 2^-18 of
    that: 2^-18 wide.  exp2 and its fp32 argument (up to 2^7 in magnitude where
    p matters): 2^-17 more at most.  p enters its product rounded by at most
    half a bf16 step, 2^-8 (bf16 calls), or half an f16 step, 2^-11 (f16
    calls), or, where p is below 2^-14 of its tile's largest, by 2^-22 of that:
    the 128 keys of a tile together 2^-15 of the weight's largest.  The output
    is rounded once: eps / 2 of itself (fp16's subnormals: 2^-25)."""
    ds = (D + 10) * 2.0 ** -24 * spread[0] + 2.0 ** -18 * spread[1] + 2.0 ** -17
    ep = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    half = torch.finfo(dtype).eps / 2
    tol = half * out.abs() + (1 + half) * weight * (ep + 2 * ds[..., None])
    tol = tol + 2.0 ** -15 * weight.amax(-1, keepdim=True) + 2.0 ** -25
    lse_tol = ds + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0, neginf=0.0)
    return tol, lse_tol


class Cache:
    """A random cache of B requests on `device`: pool, scales, table with
    shuffled pages; bytes nobody wrote are random, NaN codes among them."""

    def __init__(self, lens, hkv, d, device, seed=0, dtype=torch.bfloat16, spare=2, spread=0,
                 extra_columns=1):
        g = torch.Generator().manual_seed(seed)
        self.lens = list(lens)
        need = [-(-max(n, 0) // PAGE) for n in lens]
        pages = sum(need) + spare
        perm = torch.randperm(pages, generator=g).tolist()
        width = max(1, max(need)) + extra_columns
        self.table = []
        pool = torch.randint(0, 256, (pages, hkv, 2, PAGE, d), generator=g, dtype=torch.uint8)
        scales = torch.randint(100, 140, (pages, hkv, 2), generator=g, dtype=torch.uint8)
        at = 0
        for b, n in enumerate(lens):
            row = perm[at:at + need[b]] + [-1] * (width - need[b])
            at += need[b]
            self.table.append(row)
            if need[b]:
                x = torch.randn(need[b], hkv, 2, PAGE, d, generator=g, dtype=torch.float64)
                e = torch.randint(-6 - spread, -5 + spread, (need[b], hkv, 2), generator=g)
                live = torch.arange(need[b] * PAGE).view(need[b], 1, 1, PAGE, 1) < n
                code = encode(x * 64.0).view(x.shape)
                pool[row[:need[b]]] = torch.where(live, code, pool[row[:need[b]]])
                scales[row[:need[b]]] = (e + 127).to(torch.uint8)
        self.pool, self.scales = pool.to(device), scales.to(device)
        self.page_table = torch.tensor(self.table, dtype=torch.int32, device=device)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=device)


def cu_of(news):
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    return cu
