"""Rotary positions and the 4-bit grouped-query cache, measured: the rotation of
new queries and keys, the cache's write, its read-back and the attention that
reads it, over the range of calls a serving loop makes.

The cache.  Each request's keys and values live in 64-token pages:

    pool    uint8 [num_pages, Hkv, 2, 64, D / 2]   E2M1 codes; index 2: K, V;
                                                   element 2j in a byte's low half
    scales  uint8 [num_pages, Hkv, 2, 64, D / 16]  E4M3, one per 16 elements of a
                                                   token's head: value = code * scale

A block's scale is E4M3(amax / 6) and its codes are E2M1(x / scale), both
rounded half to even and saturating (448 and 6); a block whose scale is 0 has
codes of 0.  ``page_table`` int32 [B, stride] gives the physical page of each
logical one; ``seq_lens`` int32 [B] counts the tokens of each request, its new
ones included; ``cu_seqlens`` int32 [B + 1] are the bounds of each request's
new tokens in the flat [T, ...] inputs.

The operators.
  rotary     pairs of elements of q's and k's heads, turned by position *
             frequency and multiplied by a factor: neighbours, or elements half
             the turned part apart; the rest of a head stays as it is.
  append     the new tokens' K and V into their pages.
  read       the values of a range of each request's tokens, flat.
  attention  softmax(q k^T * sm_scale) v of the new tokens over the cache,
             causal, optionally with a sliding window; also the log-sum-exp.
             A row without a key gives 0 and -inf.

An append is followed by the read-back of the pages it touched: what the 4-bit
cache holds is returned as the values it stands for.
"""
import math
import random

import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a decode step of a full server: one token of each session, somewhere in a long context
        dict(name="rotary_step", op="rotary", t=64, hq=64, hk=8, d=128, rot=128, at=0, pairs="half", dtype="bf16",
             far=204800, stretch=8),
        # draft tokens of latent attention: the last part of q's heads, neighbours paired, one shared key row
        dict(name="rotary_drafts", op="rotary", t=256, hq=64, hk=1, d=576, rot=64, at=512, pairs="near", dtype="bf16",
             far=131072, stretch=1),
        # a ragged batch of prompts, a quarter of each head left as it is
        dict(name="rotary_prompts", op="rotary", t=16381, hq=32, hk=8, d=128, rot=96, at=0, pairs="half", dtype="f16",
             far=32768, stretch=4),
        # a decode step of a full server, pages filled to anywhere
        dict(name="append_step", op="append", B=128, hkv=8, d=128, dtype="bf16", new=1, lo=1, hi=4000),
        # prompts of odd lengths behind a cached prefix
        dict(name="append_prompts", op="append", B=9, hkv=8, d=128, dtype="bf16", new=4099, lo=4099, hi=9001),
        # a short prefix read back for a small model's prompt chunk
        dict(name="read_short", op="read", B=3, hkv=2, d=64, dtype="f16", new=500, lo=500, hi=777),
        # long prefixes read back
        dict(name="read_long", op="read", B=12, hkv=8, d=128, dtype="bf16", new=8191, lo=8191, hi=30000),
        # a session's first replies: the smallest attention
        dict(name="attend_one", op="attention", B=1, hkv=8, g=4, d=128, dtype="bf16", new=1, lo=333, hi=333, window=0),
        # a decode step of a full server, contexts far apart
        dict(name="attend_step", op="attention", B=64, hkv=8, g=8, d=128, dtype="bf16", new=1, lo=500, hi=32768, window=0),
        # few sessions with very long contexts: the work is split along them
        dict(name="attend_far", op="attention", B=2, hkv=8, g=8, d=128, dtype="bf16", new=1, lo=204800, hi=204800, window=0),
        # five drafted tokens checked at once, a sliding window, a padded slot without tokens
        dict(name="attend_drafts", op="attention", B=24, hkv=4, g=7, d=64, dtype="f16", new=5, lo=0, hi=20001, window=4096),
        # a chunk of a long prompt over its cached part
        dict(name="attend_chunk", op="attention", B=2, hkv=8, g=4, d=128, dtype="bf16", new=2048, lo=9000, hi=16384, window=0),
    ]


def draw(rng):
    logint = lambda a, b: max(a, min(b, round(math.exp(rng.uniform(math.log(a), math.log(b))))))  # noqa: E731
    op = rng.choice(["rotary", "append", "read", "attention", "attention", "attention"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "rotary":
        d = rng.choice([64, 80, 96, 128, 192, 256, 576])
        rot = rng.choice([d, d // 2, 2 * rng.randint(1, d // 2)])
        hk = rng.choice([1, 2, 3, 4, 8])
        hq = hk * rng.choice([1, 2, 4, 7, 8])
        return dict(op=op, t=logint(1, max(1, min(16384, 83000000 // ((hq + hk) * d)))), hq=hq, hk=hk, d=d, rot=rot,
                    at=rng.choice([0, 0, d - rot]), pairs=rng.choice(["half", "near"]), dtype=dtype,
                    far=logint(64, 1000000), stretch=rng.choice([1, 1, 4, 32]))
    c = dict(op=op, hkv=rng.choice([1, 2, 3, 4, 8]), d=rng.choice([64, 128]), dtype=dtype)
    if op == "append":
        c["new"] = rng.choice([1, 1, logint(2, 8), logint(9, 8192)])
        c["B"] = logint(1, max(1, min(256, 36000 // c["new"])))
    elif op == "read":
        c["new"] = logint(1, 16384)
        c["B"] = logint(1, max(1, min(64, 90000 // c["new"])))
    else:
        c["g"] = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        c["new"] = rng.choice([1, 1, logint(2, 8), logint(9, 4096)])
        c["window"] = rng.choice([0, 0, 0, logint(16, 8192)])
        hq = c["hkv"] * c["g"]
        c["B"] = logint(1, max(1, min(128, (1 << 17) // (hq * c["new"]))))
        # scores of the plain form, codes of the cache
        far = min(131072, (1 << 30) // (c["B"] * hq * c["new"]), 1000000000 // (c["B"] * c["hkv"] * c["d"]))
        c["hi"] = logint(c["new"], max(c["new"], far))
        c["lo"] = rng.choice([c["hi"], max(1, c["hi"] // 3), max(0, c["new"] - 1)])
        if c["B"] > 1 and 8 < c["new"] and rng.random() < 0.3:
            c["one"] = c["B"] // 2                                # some sessions decode beside the chunks
        return c
    c["hi"] = c["new"] + rng.choice([0, logint(1, 3000)])
    c["lo"] = c["new"] + (c["hi"] - c["new"]) // rng.choice([1, 2, 5])
    return c


def shape_of(case):
    """(tokens, new tokens) of each request; of the case alone, so that its work is known."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    lens = [r.randint(min(case["lo"], case["hi"]), case["hi"]) for _ in range(case["B"])]
    lens[0] = case["hi"]
    news = [case["new"]] * case["B"]
    for b in range(case["B"] - case.get("one", 0), case["B"]):
        news[b] = 1
    if case["op"] != "attention" and case["new"] > 8:          # ragged prompts and ranges
        news = [case["new"]] + [r.randint(case["new"] // 2, case["new"]) for _ in range(case["B"] - 1)]
    if case["op"] == "attention" and case["lo"] == 0 and case["B"] > 1:
        lens[-1] = 0                                            # a padded slot
    return lens, news


def work(case):
    if case["op"] == "rotary":
        n = case["t"] * (case["hq"] * case["d"] + case["hk"] * key_width(case))
        return {"bytes": 4 * n + 8 * case["t"], "flops": 0}
    lens, news = shape_of(case)
    hkv, d = case["hkv"], case["d"]
    held = d * 9 // 16                                          # bytes of a token's head in the cache
    if case["op"] == "append":
        # inputs in 16 bits; rows written; the touched pages' rows read back and their values written
        read = sum(n + (l - n) % PAGE for l, n in zip(lens, news))
        return {"bytes": (sum(news) + read) * hkv * 2 * (2 * d + held), "flops": 0}
    if case["op"] == "read":
        return {"bytes": sum(news) * hkv * 2 * (2 * d + held), "flops": 0}
    hq, w = hkv * case["g"], case["window"]
    pairs, keys = 0, 0
    for l, n in zip(lens, news):
        first = max(0, l - n)
        m = l - first                                          # rows with a key
        if w:
            full = max(0, min(m, l - max(first, w - 1)))       # rows that see a whole window
            short = m - full                                   # rows at first .. first + short - 1
            pairs += full * w + short * (first + 1) + short * (short - 1) // 2
            keys += l - max(0, first - w + 1)
        else:
            pairs += m * (first + 1) + m * (m - 1) // 2
            keys += l
    t = sum(news)
    return {"bytes": keys * hkv * held * 2 + t * hq * (d * 4 + 4), "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def key_width(case):
    """Of k's rows: one that all heads share holds the turned part alone."""
    return case["rot"] if case["at"] > 0 else case["d"]


def frequencies(case):
    """Frequencies of the pairs, fp32; slow ones divided by `stretch`, fast ones kept, a ramp between."""
    n = case["rot"] // 2
    f = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / max(n, 1))
    turns = 8192 * f / (2 * math.pi)                            # over the length that a model was trained on
    keep = ((turns - 1) / 31).clamp(0, 1)
    return (f * (keep + (1 - keep) / case["stretch"])).float()


def magnitude(x):
    """Scales and codes of blocks of 16 of the last dimension: (E4M3 as fp32 [..., n], codes int [..., 16 n])."""
    b = x.float().unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1) / 6).clamp_max(448).to(torch.float8_e4m3fn).float()
    y = torch.where(s[..., None] > 0, b.abs() / s[..., None], 0)
    c = ((y > 0.25).int() + (y >= 0.75).int() + (y > 1.25).int() + (y >= 1.75).int() + (y > 2.5).int()
         + (y >= 3.5).int() + (y > 5).int())
    c = torch.where((b < 0) & (s[..., None] > 0), c + 8, c)
    return s, c.flatten(-2)


def pack(c):
    c = c.to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def scale_bytes(s):
    return s.to(torch.float8_e4m3fn).view(torch.uint8)


def decode(codes, scales):
    """The 32-bit values of packed codes [..., D / 2] and scale bytes [..., D / 16]."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    s = scales.view(torch.float8_e4m3fn).float()
    return (grid[c].unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def prepare_rotary(case, dev, randn, gen):
    t, d, dt = case["t"], case["d"], DTYPES[case["dtype"]]
    kw = key_width(case)
    # a fused projection's output: q and k are slices of its rows
    wide = randn(t, case["hq"] * d + case["hk"] * kw + 64)
    wide[::13] *= 4
    wide = wide.to(dt)
    q = wide[:, :case["hq"] * d].unflatten(1, (case["hq"], d))
    k = wide[:, case["hq"] * d:case["hq"] * d + case["hk"] * kw].unflatten(1, (case["hk"], kw))
    # runs of neighbouring positions, as ragged prompts have them, up to the last one
    pos = torch.arange(t, device=dev) % max(1, case["far"])
    at = torch.randint(0, max(1, case["far"]), (t // 64 + 1,), device=dev, generator=gen)
    pos = (pos + at[torch.arange(t, device=dev) // 64]) % max(1, case["far"])
    pos[-1] = case["far"] - 1
    return dict(op="rotary", q=q, k=k, positions=pos, inv_freq=frequencies(case).to(dev), near=case["pairs"] == "near",
                q_at=case["at"], k_at=0 if case["at"] > 0 else case["at"], factor=1.0 + 0.1 * math.log(case["stretch"]))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, device=dev, generator=gen)  # noqa: E731
    if case["op"] == "rotary":
        return prepare_rotary(case, dev, randn, gen)
    lens, news = shape_of(case)
    B, hkv, d, dt = case["B"], case["hkv"], case["d"], DTYPES[case["dtype"]]
    need = [-(-n // PAGE) for n in lens]
    stride = max(1, max(need))
    total = sum(need)
    num_pages = total + 3
    perm = torch.randperm(num_pages, device=dev, generator=gen).to(torch.int32)
    table = torch.full((B, stride), -1, dtype=torch.int32, device=dev)
    # pages that nothing was written to, and rows past a request's end, hold any bytes
    pool = torch.empty((num_pages, hkv, 2, PAGE, d // 2), dtype=torch.uint8, device=dev)
    pool.random_(0, 256, generator=gen)
    scales = torch.empty((num_pages, hkv, 2, PAGE, d // 16), dtype=torch.uint8, device=dev)
    scales.random_(0, 256, generator=gen)
    # keys with a few strong channels, heads of different size, a first token that draws attention
    channel = torch.ones(2, d, device=dev)
    channel[0, torch.randperm(d, device=dev, generator=gen)[: d // 32]] = 3.0
    head = torch.exp2(torch.rand(hkv, 2, 1, 1, device=dev, generator=gen) * 2 - 1)
    sink = randn(hkv, d)
    sink = sink / sink.norm(dim=-1, keepdim=True) * d ** 0.5
    at = 0
    for b in range(B):
        held = lens[b] if case["op"] != "append" else max(0, lens[b] - news[b])
        pages = perm[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = pages
        for p0 in range(0, -(-held // PAGE), 512):
            pg = pages[p0:min(p0 + 512, -(-held // PAGE))].long()
            x = randn(len(pg), hkv, 2, PAGE, d) * channel[None, None, :, None, :] * head
            if p0 == 0:
                x[0, :, 0, 0, :] = 1.5 * sink
            s, c = magnitude(x.to(dt))
            live = (p0 * PAGE + torch.arange(len(pg) * PAGE, device=dev)).view(-1, 1, 1, PAGE, 1) < held
            pool[pg] = torch.where(live, pack(c), pool[pg])
            scales[pg] = torch.where(live, scale_bytes(s), scales[pg])
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(news), 0)
    s = dict(op=case["op"], pool=pool, scales=scales, page_table=table, d=d, hkv=hkv, dtype=dt, B=B,
             seq_lens=torch.tensor(lens, dtype=torch.int32, device=dev), cu_seqlens=cu.to(dev),
             total=sum(news), max_len=max(lens), max_new=max(news))
    if case["op"] == "attention":
        hq, t = hkv * case["g"], sum(news)
        q = randn(t, hq, d) + 0.3 * sink.repeat_interleave(case["g"], 0)
        n = case.get("one", 0)
        s.update(q=q.to(dt), g=case["g"], window=case["window"], sm_scale=d ** -0.5, ones=n,
                 max_first=max(lens[:B - n]), max_ones=max(lens[B - n:], default=0), rows_first=sum(news[:B - n]))
    elif case["op"] == "append":
        # a fused projection's output: K and V are slices of its rows
        kv = (randn(s["total"], 2, hkv, d) * channel[None, :, None, :] * 1.5).to(dt)
        kv[::17] *= 2
        kv[3::29, :, :, :16] = 0                                 # blocks of zeros
        kv[5::31] *= 1e-3                                        # and of values near the smallest scale
        starts = [(l - n) // PAGE * PAGE for l, n in zip(lens, news)]
        cu_read = torch.zeros(B + 1, dtype=torch.int32)
        cu_read[1:] = torch.cumsum(torch.tensor([l - f for l, f in zip(lens, starts)]), 0)
        s.update(k=kv[:, 0], v=kv[:, 1], starts=torch.tensor(starts, dtype=torch.int32, device=dev),
                 cu_read=cu_read.to(dev), total_read=int(cu_read[-1]))
    else:
        s.update(starts=torch.tensor([l - n for l, n in zip(lens, news)], dtype=torch.int32, device=dev),
                 cu_read=s["cu_seqlens"], total_read=s["total"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        import bit_kv_cache_nvfp4_gb300 as kv
        if s["op"] == "rotary":
            q, k = kv.rotary(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=s["near"], q_offset=s["q_at"],
                             k_offset=s["k_at"], factor=s["factor"])
            return {"q": q, "k": k}
        if s["op"] == "attention":
            out, lse = kv.attention_gqa4(s["q"], s["pool"], s["scales"], s["page_table"], s["seq_lens"],
                                         s["cu_seqlens"], s["max_new"], s["sm_scale"], window=s["window"])
            return {"out": out, "lse": lse}
        if s["op"] == "append":
            kv.append_gqa4(s["k"], s["v"], s["cu_seqlens"], s["page_table"], s["seq_lens"], s["pool"], s["scales"])
        k, v = kv.read_gqa4(s["pool"], s["scales"], s["page_table"], s["starts"], s["cu_read"], s["total_read"],
                            dtype=s["dtype"])
        return {"k": k, "v": v}
    if s["op"] == "rotary":
        return {"q": plain_rotary(s, s["q"], s["q_at"]), "k": plain_rotary(s, s["k"], s["k_at"])}
    if s["op"] == "attention":
        first, n = s["B"] - s["ones"], s["rows_first"]
        if not s["ones"]:
            out, lse = plain_attention(s, s["q"], slice(0, first), s["cu_seqlens"], s["max_new"], s["max_len"])
            return {"out": out, "lse": lse}
        # sessions that decode apart from the prompt's chunk, so that neither is padded to the other
        a = plain_attention(s, s["q"][:n], slice(0, first), s["cu_seqlens"][:first + 1], s["max_new"], s["max_first"])
        o = plain_attention(s, s["q"][n:], slice(first, None), s["cu_seqlens"][first:] - n, 1, s["max_ones"])
        return {"out": torch.cat([a[0], o[0]]), "lse": torch.cat([a[1], o[1]])}
    if s["op"] == "append":
        plain_append(s)
    k, v = plain_read(s)
    return {"k": k, "v": v}


def plain_rotary(s, x, at):
    n = s["inv_freq"].numel()
    # (a far position times a frequency needs more than 32 bits to keep its angle)
    a = s["positions"].double()[:, None] * s["inv_freq"].double()
    c, z = (a.cos() * s["factor"]).float()[:, None], (a.sin() * s["factor"]).float()[:, None]
    out = x.clone()
    part = x[..., at:at + 2 * n].float()
    if s["near"]:
        u, v = part[..., 0::2], part[..., 1::2]
        y = torch.stack([u * c - v * z, u * z + v * c], -1).flatten(-2)
    else:
        u, v = part[..., :n], part[..., n:]
        y = torch.cat([u * c - v * z, u * z + v * c], -1)
    out[..., at:at + 2 * n] = y.to(x.dtype)
    return out


def request_of(cu, t):
    """Request of each of t flat tokens, and the token's place in it."""
    tok = torch.arange(t, device=cu.device)
    b = torch.searchsorted(cu[1:].long(), tok, right=True)
    return b, tok - cu[b]


def plain_append(s):
    b, i = request_of(s["cu_seqlens"], s["total"])
    start = (s["seq_lens"] - s["cu_seqlens"].diff()).long()
    pos = start[b] + i
    page, off = s["page_table"][b, pos // PAGE].long(), pos % PAGE
    sc, c = magnitude(torch.stack([s["k"], s["v"]], dim=2))               # [T, Hkv, 2, D]
    s["pool"][page, :, :, off] = pack(c)
    s["scales"][page, :, :, off] = scale_bytes(sc)


def plain_read(s):
    b, i = request_of(s["cu_read"], s["total_read"])
    pos = s["starts"].long()[b] + i
    page, off = s["page_table"][b, pos // PAGE].long(), pos % PAGE
    x = decode(s["pool"][page, :, :, off], s["scales"][page, :, :, off]).to(s["dtype"])
    return x[:, :, 0].contiguous(), x[:, :, 1].contiguous()


def plain_attention(s, q, which, cu, max_new, max_len):
    d, hkv, g = s["d"], s["hkv"], s["g"]
    lens, n = s["seq_lens"][which].long(), cu.diff().long()
    B, npg = lens.shape[0], max(1, -(-max_len // PAGE))
    pages = s["page_table"][which, :npg].clamp_min(0).long()
    key = torch.arange(npg * PAGE, device=q.device)
    held = (key[None] < lens[:, None])[:, None, :, None]
    side = lambda j: decode(s["pool"][pages, :, j], s["scales"][pages, :, j]).transpose(1, 2).reshape(  # noqa: E731
        B, hkv, npg * PAGE, d).masked_fill(~held, 0)
    i = torch.arange(max_new, device=q.device)
    tok = (cu[:-1].long()[:, None] + i[None]).clamp_max(q.shape[0] - 1)
    qb = q[tok].float().view(B, max_new, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, max_new * g, d)
    pos = (lens - n)[:, None] + i[None]                                                # [B, max_new]
    ok = (key[None, None] <= pos[..., None]) & (key[None, None] < lens[:, None, None])
    if s["window"]:
        ok = ok & (key[None, None] > pos[..., None] - s["window"])
    sc = (qb @ side(0).transpose(2, 3)).mul_(s["sm_scale"]).view(B, hkv, max_new, g, npg * PAGE)
    sc.masked_fill_(~ok[:, None, :, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, hkv, max_new * g, -1) @ side(1)).view(B, hkv, max_new, g, d) / l.masked_fill(l == 0, 1)
    lse = (m + l.log())[..., 0]
    b, j = request_of(cu, q.shape[0])
    return (o[b, :, j].reshape(q.shape).to(s["dtype"]), lse[b, :, j].reshape(q.shape[:2]))


# ---------------------------------------------------------------------------
# the same in 64 bits, from the definition
# ---------------------------------------------------------------------------
def minifloat(exponent_bits, fraction_bits, bias, dev):
    """All values of a small format, by their codes, sign first (E4M3's code of all ones is NaN)."""
    vals = []
    for c in range(2 << (exponent_bits + fraction_bits)):
        e, f = (c >> fraction_bits) & ((1 << exponent_bits) - 1), c & ((1 << fraction_bits) - 1)
        x = (f * 2.0 ** (1 - bias) if e == 0 else ((1 << fraction_bits) + f) * 2.0 ** (e - bias)) / (1 << fraction_bits)
        if exponent_bits == 4 and (c & 127) == 127:
            x = math.nan
        vals.append(-x if c >> (exponent_bits + fraction_bits) else x)
    return torch.tensor(vals, dtype=torch.float64, device=dev)


def nearest(x, fraction_bits, least_exponent, top):
    """x rounded to a small format's values, half to even, saturating, in 64 bits."""
    grid = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** least_exponent))) - fraction_bits)
    return (torch.round(x / grid) * grid).clamp(-top, top)


def exact(case, seed):
    s = prepare(case, seed)
    dev = torch.device("cuda")
    if case["op"] == "rotary":
        n, out = case["rot"] // 2, {}
        for name, at in (("q", s["q_at"]), ("k", s["k_at"])):
            y = s[name].double()
            first = at + torch.arange(n, device=dev) * (2 if s["near"] else 1)
            second = first + (1 if s["near"] else n)
            turn = torch.polar(torch.full((case["t"], n), s["factor"], dtype=torch.float64, device=dev),
                               s["positions"].double()[:, None] * s["inv_freq"].double())
            z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
            y[..., first], y[..., second] = z.real, z.imag
            out[name] = y
        return out
    e2m1, e4m3 = minifloat(2, 1, 1, dev), minifloat(4, 3, 7, dev)
    lens, news = shape_of(case)
    hkv, d = case["hkv"], case["d"]
    table = s["page_table"].tolist()

    def values(b, first, last):
        """K and V of request b's tokens [first, last): [Hkv, 2, n, D]."""
        pg = torch.tensor(table[b][first // PAGE:-(-last // PAGE)], dtype=torch.long, device=dev)
        c = s["pool"][pg].long()
        x = torch.stack([e2m1[c % 16], e2m1[c // 16]], -1).flatten(-2)
        x = x * e4m3[s["scales"][pg].long()].repeat_interleave(16, -1)
        x = x.permute(1, 2, 0, 3, 4).reshape(hkv, 2, -1, d)
        return x[:, :, first % PAGE:first % PAGE + last - first]

    if case["op"] == "attention":
        g, w, at = case["g"], case["window"], 0
        out = torch.zeros(s["total"], hkv * g, d, dtype=torch.float64, device=dev)
        lse = torch.full((s["total"], hkv * g), -math.inf, dtype=torch.float64, device=dev)
        for b, (l, n) in enumerate(zip(lens, news)):
            pos = torch.arange(l - n, l, device=dev)
            lo = max(0, l - n - w + 1) // PAGE * PAGE if w else 0
            if l > 0:
                x = values(b, lo, l)
                key = torch.arange(lo, l, device=dev)
                ok = key[None] <= pos[:, None]
                if w:
                    ok &= key[None] > pos[:, None] - w
                some = ok.any(-1)
                for h in range(hkv * g):
                    q = s["q"][at:at + n, h].double()
                    sc = (q @ x[h // g, 0].T * s["sm_scale"]).masked_fill_(~ok, -math.inf)
                    z = torch.logsumexp(sc, -1)
                    p = torch.exp(sc.sub_(z.masked_fill(~some, 0)[:, None]))
                    out[at:at + n, h] = p @ x[h // g, 1]
                    lse[at:at + n, h] = z
            at += n
        return {"out": out, "lse": lse}
    if case["op"] == "read":
        x = torch.cat([values(b, l - n, l) for b, (l, n) in enumerate(zip(lens, news))], 2)
        return {"k": x[:, 0].transpose(0, 1), "v": x[:, 1].transpose(0, 1)}
    got, at = [], 0
    for b, (l, n) in enumerate(zip(lens, news)):
        first = (l - n) // PAGE * PAGE
        x = torch.stack([s["k"][at:at + n], s["v"][at:at + n]], 0).double().permute(2, 0, 1, 3)   # [Hkv, 2, n, D]
        at += n
        x = x.unflatten(-1, (-1, 16))
        sc = nearest(x.abs().amax(-1, keepdim=True) / 6, 3, -6, 448.0)
        y = torch.where(sc > 0, nearest(x / torch.where(sc > 0, sc, 1), 1, 0, 6.0) * sc, 0).flatten(-2)
        got.append(torch.cat([values(b, first, l - n), y], 2) if l - n > first else y)
    y = torch.cat(got, 2)
    return {"k": y[:, 0].transpose(0, 1), "v": y[:, 1].transpose(0, 1)}
