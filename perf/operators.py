"""The 8-bit grouped-query cache, measured: its write, its read-back and the
attention that reads it, over the range of calls a serving loop makes.

The cache.  Each request's keys and values live in 64-token pages:

    pool    uint8 [num_pages, Hkv, 2, 64, D]   E4M3 codes; index 2: K, V
    scales  uint8 [num_pages, Hkv, 2]          one E8M0 byte per page, head
                                               and side: value = code * 2^(byte - 127)

with the exponent of a page's block the smallest e with
amax <= 448 * 2^e (-48 <= e <= 48).  ``page_table`` int32 [B, stride] gives
the physical page of each logical one; ``seq_lens`` int32 [B] counts the
tokens of each request, its new ones included; ``cu_seqlens`` int32 [B + 1]
are the bounds of each request's new tokens in the flat [T, ...] inputs.

The operators.
  append     the new tokens' K and V into their pages.  A page that already
             holds earlier tokens of the request keeps them: its exponent
             only rises, and their codes are re-rounded when it does.
  read       the values of a range of each request's tokens, flat.
  attention  softmax(q k^T * sm_scale) v of the new tokens over the cache,
             causal, optionally with a sliding window; also the log-sum-exp.
             A row without a key gives 0 and -inf.

An append is followed by the read-back of the pages it touched, as a prompt
chunk's attention in the model's type does: what the 8-bit cache holds is
returned as the values it stands for.
"""
import math
import random

import torch

own = False

PAGE = 64
E_MIN, E_MAX, BIAS = -48, 48, 127
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one session's next token: latency alone counts
        dict(name="append_one", op="append", B=1, hkv=8, d=128, dtype="bf16", new=1, lo=90, hi=90),
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
        # a whole prompt at once
        dict(name="attend_prompt", op="attention", B=1, hkv=8, g=4, d=128, dtype="bf16", new=8192, lo=8192, hi=8192, window=0),
        # a prompt chunk in the same batch as sessions that decode
        dict(name="attend_mixed", op="attention", B=33, hkv=8, g=4, d=128, dtype="bf16", new=1000, one=32, lo=300, hi=8192, window=0),
    ]


def draw(rng):
    logint = lambda a, b: max(a, min(b, round(math.exp(rng.uniform(math.log(a), math.log(b))))))  # noqa: E731
    c = dict(op=rng.choice(["append", "read", "attention", "attention", "attention"]),
             hkv=rng.choice([1, 2, 3, 4, 8]), d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "bf16", "f16"]))
    if c["op"] == "append":
        c["new"] = rng.choice([1, 1, logint(2, 8), logint(9, 8192)])
        c["B"] = logint(1, max(1, min(256, 40000 // c["new"])))
    elif c["op"] == "read":
        c["new"] = logint(1, 16384)
        c["B"] = logint(1, max(1, min(64, 98000 // c["new"])))
    else:
        c["g"] = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        c["new"] = rng.choice([1, 1, logint(2, 8), logint(9, 4096)])
        c["window"] = rng.choice([0, 0, 0, logint(16, 8192)])
        hq = c["hkv"] * c["g"]
        c["B"] = logint(1, max(1, min(128, (1 << 17) // (hq * c["new"]))))
        # scores of the plain form, codes of the cache
        far = min(131072, (1 << 30) // (c["B"] * hq * c["new"]), 1500000000 // (c["B"] * c["hkv"] * c["d"] * 2))
        c["hi"] = logint(c["new"], max(c["new"], far))
        c["lo"] = rng.choice([c["hi"], max(1, c["hi"] // 3), max(0, c["new"] - 1)])
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
    lens, news = shape_of(case)
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "append":
        # inputs in 16 bits; codes written; the touched pages' codes read back and their values written
        read = sum(n + (l - n) % PAGE for l, n in zip(lens, news))
        return {"bytes": sum(news) * hkv * d * 2 * 3 + read * hkv * d * 2 * 3, "flops": 0}
    if case["op"] == "read":
        return {"bytes": sum(news) * hkv * d * 2 * 3, "flops": 0}
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
    return {"bytes": keys * hkv * d * 2 + t * hq * (d * 4 + 4), "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def exponent_of(amax):
    """Smallest e with amax <= 448 * 2^e, in [E_MIN, E_MAX] (int32)."""
    m, e = torch.frexp(amax.float())
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(amax > 0, e.clamp(E_MIN, E_MAX), torch.full_like(e, E_MIN))


def encode(x, e):
    """E4M3 codes of x * 2^-e (e broadcast), round half to even, saturating."""
    return (x.float() * torch.exp2(-e.float())).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def decode(codes, e):
    """The 32-bit values of E4M3 codes at exponent e (broadcast)."""
    return codes.view(torch.float8_e4m3fn).float() * torch.exp2(e.float())


def prepare(case, seed):
    dev = torch.device("cuda")
    lens, news = shape_of(case)
    B, hkv, d, dt = case["B"], case["hkv"], case["d"], DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, device=dev, generator=gen)  # noqa: E731
    need = [-(-n // PAGE) for n in lens]
    stride = max(1, max(need))
    total = sum(need)
    num_pages = total + 3
    perm = torch.randperm(num_pages, device=dev, generator=gen).to(torch.int32)
    table = torch.full((B, stride), -1, dtype=torch.int32, device=dev)
    # pages that nothing was written to, and rows past a request's end, hold any bytes
    pool = torch.empty((num_pages, hkv, 2, PAGE, d), dtype=torch.uint8, device=dev)
    pool.random_(0, 256, generator=gen)
    scales = torch.full((num_pages, hkv, 2), BIAS, dtype=torch.uint8, device=dev)
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
        np_ = -(-held // PAGE)
        if np_ == 0:
            continue
        x = randn(np_, hkv, 2, PAGE, d) * channel[None, None, :, None, :] * head
        x[0, :, 0, 0, :] = 1.5 * sink
        live = torch.arange(np_ * PAGE, device=dev).view(np_, 1, 1, PAGE, 1) < held
        x = x.to(dt).float() * live
        e = exponent_of(x.abs().amax(dim=(3, 4)))
        codes = encode(x, e[..., None, None])
        pg = pages[:np_].long()
        pool[pg] = torch.where(live, codes, pool[pg])
        scales[pg] = (e + BIAS).to(torch.uint8)
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(news), 0)
    s = dict(op=case["op"], pool=pool, scales=scales, page_table=table, d=d, hkv=hkv, dtype=dt, B=B,
             seq_lens=torch.tensor(lens, dtype=torch.int32, device=dev), cu_seqlens=cu.to(dev),
             total=sum(news), max_len=max(lens), max_new=max(news), spare=perm[-1].long())
    if case["op"] == "attention":
        hq, t = hkv * case["g"], sum(news)
        q = randn(t, hq, d) + 0.3 * sink.repeat_interleave(case["g"], 0)
        n = case.get("one", 0)
        s.update(q=q.to(dt), g=case["g"], window=case["window"], sm_scale=d ** -0.5, ones=n,
                 max_first=max(lens[:B - n]), max_ones=max(lens[B - n:], default=0), rows_first=sum(news[:B - n]))
    elif case["op"] == "append":
        # a fused projection's output: K and V are slices of its rows
        kv = (randn(s["total"], 2, hkv, d) * channel[None, :, None, :] * 1.5).to(dt)
        kv[::17] *= 2                                            # some tokens raise their page's exponent
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
        if s["op"] == "attention":
            out, lse = kv.attention_gqa8(s["q"], s["pool"], s["scales"], s["page_table"], s["seq_lens"],
                                         s["cu_seqlens"], s["max_new"], s["sm_scale"], window=s["window"])
            return {"out": out, "lse": lse}
        if s["op"] == "append":
            kv.append_gqa8(s["k"], s["v"], s["cu_seqlens"], s["page_table"], s["seq_lens"], s["pool"], s["scales"])
        k, v = kv.read_gqa8(s["pool"], s["scales"], s["page_table"], s["starts"], s["cu_read"], s["total_read"],
                            dtype=s["dtype"])
        return {"k": k, "v": v}
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


def request_of(cu, t):
    """Request of each of t flat tokens, and the token's place in it."""
    tok = torch.arange(t, device=cu.device)
    b = torch.searchsorted(cu[1:].long(), tok, right=True)
    return b, tok - cu[b]


def plain_append(s):
    b, i = request_of(s["cu_seqlens"], s["total"])
    n = s["cu_seqlens"].diff()
    start = (s["seq_lens"] - n).long()
    pos = start[b] + i
    page, off = s["page_table"][b, pos // PAGE].long(), pos % PAGE
    kv = torch.stack([s["k"], s["v"]], dim=2).float()                      # [T, Hkv, 2, D]
    need = exponent_of(kv.abs().amax(-1))                                 # [T, Hkv, 2]
    old = s["scales"].int() - BIAS
    e = torch.full_like(old, -1000).index_reduce_(0, page, need, "amax")
    # the first page of a request that starts inside it keeps its tokens
    kept = ((start % PAGE) > 0) & (n > 0)
    p0 = s["page_table"].gather(1, (start // PAGE).clamp_max(s["page_table"].shape[1] - 1)[:, None])[:, 0].long()
    p0 = torch.where(kept, p0, s["spare"])                                # a page of nobody's, put back as it is
    raised = torch.where(kept[:, None, None], torch.maximum(e[p0], old[p0]), torch.full_like(old[p0], -1000))
    e = e.index_reduce(0, p0, raised, "amax")
    e = torch.where(e > -1000, e, old)
    first = s["pool"][p0]
    live = kept.view(-1, 1, 1, 1, 1) & (torch.arange(PAGE, device=pos.device).view(1, 1, 1, PAGE, 1)
                                        < (start % PAGE).view(-1, 1, 1, 1, 1))
    again = encode(decode(first, old[p0][..., None, None]), e[p0][..., None, None])
    s["pool"][p0] = torch.where(live, again, first)
    s["pool"][page, :, :, off] = encode(kv, e[page][..., None])
    s["scales"].copy_((e + BIAS).to(torch.uint8))


def plain_read(s):
    b, i = request_of(s["cu_read"], s["total_read"])
    pos = s["starts"].long()[b] + i
    page, off = s["page_table"][b, pos // PAGE].long(), pos % PAGE
    x = decode(s["pool"][page, :, :, off], (s["scales"][page].int() - BIAS)[..., None])
    if s["dtype"] == torch.float16:
        x = x.clamp(-65504, 65504)
    x = x.to(s["dtype"])
    return x[:, :, 0].contiguous(), x[:, :, 1].contiguous()


def plain_attention(s, q, which, cu, max_new, max_len):
    d, hkv, g = s["d"], s["hkv"], s["g"]
    lens, n = s["seq_lens"][which].long(), cu.diff().long()
    B, npg = lens.shape[0], max(1, -(-max_len // PAGE))
    pages = s["page_table"][which, :npg].clamp_min(0).long()
    x = decode(s["pool"][pages], (s["scales"][pages].int() - BIAS)[..., None, None])   # [B, npg, Hkv, 2, 64, D]
    key = torch.arange(npg * PAGE, device=q.device)
    held = (key[None] < lens[:, None])[:, None, :, None]
    k = x[:, :, :, 0].transpose(1, 2).reshape(B, hkv, npg * PAGE, d).masked_fill(~held, 0)
    v = x[:, :, :, 1].transpose(1, 2).reshape(B, hkv, npg * PAGE, d).masked_fill(~held, 0)
    i = torch.arange(max_new, device=q.device)
    tok = (cu[:-1].long()[:, None] + i[None]).clamp_max(q.shape[0] - 1)
    qb = q[tok].float().view(B, max_new, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, max_new * g, d)
    pos = (lens - n)[:, None] + i[None]                                                # [B, max_new]
    ok = (key[None, None] <= pos[..., None]) & (key[None, None] < lens[:, None, None])
    if s["window"]:
        ok = ok & (key[None, None] > pos[..., None] - s["window"])
    sc = (qb @ k.transpose(2, 3)).mul_(s["sm_scale"]).view(B, hkv, max_new, g, npg * PAGE)
    sc.masked_fill_(~ok[:, None, :, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, hkv, max_new * g, -1) @ v).view(B, hkv, max_new, g, d) / l.masked_fill(l == 0, 1)
    lse = (m + l.log())[..., 0]
    b, j = request_of(cu, q.shape[0])
    return (o[b, :, j].reshape(q.shape).to(s["dtype"]), lse[b, :, j].reshape(q.shape[:2]))


# ---------------------------------------------------------------------------
# the same in 64 bits, from the definition
# ---------------------------------------------------------------------------
def e4m3_table(dev):
    """The 256 values of E4M3: sign, 4 exponent bits (bias 7), 3 fraction bits; 0x7F is NaN."""
    vals = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = math.nan if (c & 127) == 127 else (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
        vals.append(-x if c & 128 else x)
    return torch.tensor(vals, dtype=torch.float64, device=dev)


def nearest(x, e):
    """x rounded to the grid of E4M3 values times 2^e, in 64 bits."""
    y = x * 2.0 ** -e
    grid = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(y / grid) * grid).clamp(-448, 448) * 2.0 ** e


def least_exponent(amax):
    e = E_MIN
    while e < E_MAX and amax > 448 * 2.0 ** e:
        e += 1
    return e


def exact(case, seed):
    s = prepare(case, seed)
    dev, tab = s["pool"].device, e4m3_table(s["pool"].device)
    lens, news = shape_of(case)
    hkv, d = case["hkv"], case["d"]
    table, scales = s["page_table"].tolist(), s["scales"].cpu()
    two = torch.exp2(s["scales"].double() - BIAS)

    def values(b, first, last):
        """K and V of request b's tokens [first, last): [Hkv, 2, n, D]."""
        pg = torch.tensor(table[b][first // PAGE:-(-last // PAGE)], dtype=torch.long, device=dev)
        x = tab[s["pool"][pg].long()] * two[pg][..., None, None]
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
        ks = [values(b, l - n, l) for b, (l, n) in enumerate(zip(lens, news))]
        x = torch.cat(ks, 2)
        top = 65504.0 if case["dtype"] == "f16" else math.inf
        return {"k": x[:, 0].transpose(0, 1).clamp(-top, top), "v": x[:, 1].transpose(0, 1).clamp(-top, top)}
    got, at = [], 0
    for b, (l, n) in enumerate(zip(lens, news)):
        first = (l - n) // PAGE * PAGE
        old = l - n - first
        x = torch.stack([s["k"][at:at + n], s["v"][at:at + n]], 0).double()          # [2, n, Hkv, D]
        at += n
        span = torch.zeros(2, -(-(l - first) // PAGE) * PAGE, hkv, d, dtype=torch.float64, device=dev)
        if old:
            span[:, :old] = values(b, first, l - n).permute(1, 2, 0, 3)
        amax = span.clone()
        amax[:, :old] = 0
        amax[:, old:l - first] = x
        amax = amax.abs().view(2, -1, PAGE, hkv, d).amax((2, 4)).cpu()               # [2, pages, Hkv]
        e = torch.tensor([[[max(least_exponent(float(amax[j, p, h])),
                                int(scales[table[b][first // PAGE], h, j]) - BIAS if p == 0 and old else E_MIN)
                            for h in range(hkv)] for p in range(amax.shape[1])] for j in range(2)], dtype=torch.float64, device=dev)
        span[:, old:l - first] = x
        y = nearest(span, e.repeat_interleave(PAGE, 1)[..., None])
        got.append(y[:, :l - first])
    y = torch.cat(got, 1)
    top = 65504.0 if case["dtype"] == "f16" else math.inf
    return {"k": y[0].clamp(-top, top), "v": y[1].clamp(-top, top)}
