"""Rotary positions on the GPU against the formula in 64 bits."""
import math

import pytest
import torch

import bit_kv_cache_nvfp4_gb300 as kv

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    return torch.device("cuda", torch.cuda.current_device())


def turned(x, pos, freq, near, at, factor):
    """(value, size of the terms it is the sum of), float64."""
    n = freq.numel()
    a = (pos.double()[:, None] * freq.double())[:, None]
    first = at + torch.arange(n, device=x.device) * (2 if near else 1)
    second = first + (1 if near else n)
    y, size = x.double(), x.double().abs()
    u, v = y[..., first].clone(), y[..., second].clone()
    c, s = a.cos() * factor, a.sin() * factor
    y[..., first], y[..., second] = u * c - v * s, u * s + v * c
    both = ((u.abs() + v.abs()) * abs(factor))
    size[..., first], size[..., second] = both, both
    return y, size


def close(got, want, freq):
    """An angle is held to 2^-29 of a turn and given to sincospi in fp32 (2^-25 of
    pi), which is good to 2 ulp or so, then the factor: 2^-22 of the terms in all; two
    products and a sum in fp32, 2^-23; the result is rounded once to its type."""
    y, size = want
    eps = torch.finfo(got.dtype).eps / 2
    tol = eps * y.abs() + (1 + eps) * 2.0 ** -21 * size + (2.0 ** -25 if got.dtype == F16 else 2.0 ** -134)
    assert ((got.double() - y).abs() <= tol).all()


def check(t, hq, hk, dq, dk, n, near, dtype, q_at=0, k_at=0, far=100000, factor=1.0, wide=True, pad=0, seed=0, scale=1.0):
    device = dev()
    g = torch.Generator(device=device).manual_seed(seed)
    x = torch.randn(t, hq * dq + hk * dk + pad, device=device, generator=g).mul_(scale).to(dtype)
    q = x[:, :hq * dq].unflatten(1, (hq, dq))
    k = x[:, hq * dq:hq * dq + hk * dk].unflatten(1, (hk, dk)) if hk else None
    pos = torch.randint(-far // 4, far, (t,), device=device, generator=g)
    pos = pos if wide else pos.to(torch.int32)
    freq = kv.rotary_frequencies(2 * n, device=device)
    gq, gk = kv.rotary(q, k, pos, freq, interleaved=near, q_offset=q_at, k_offset=k_at, factor=factor)
    close(gq, turned(q, pos, freq, near, q_at, factor), freq)
    rest = torch.ones(dq, dtype=torch.bool, device=device)
    rest[q_at:q_at + 2 * n] = False
    assert torch.equal(gq[..., rest], q[..., rest])
    if hk:
        close(gk, turned(k, pos, freq, near, k_at, factor), freq)
        rest = torch.ones(dk, dtype=torch.bool, device=device)
        rest[k_at:k_at + 2 * n] = False
        assert torch.equal(gk[..., rest], k[..., rest])
    else:
        assert gk is None
    return q, k, pos, freq, gq, gk


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("t,hq,hk,d", [(1, 32, 8, 128), (3, 4, 1, 64), (64, 8, 2, 96), (257, 7, 1, 80), (700, 1, 1, 64),
                                       (3000, 5, 2, 128), (9000, 2, 1, 64)])
def test_whole_heads(t, hq, hk, d, near, dtype):
    """A single token, several heads a thread, several tokens a block."""
    check(t, hq, hk, d, d, d // 2, near, dtype, wide=bool(t % 2), seed=t)


@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("n,at,d", [(32, 512, 576), (1, 0, 64), (1, 61, 64), (31, 1, 64), (20, 24, 64), (24, 16, 72),
                                    (6, 4, 16), (2, 0, 6), (61, 6, 128), (48, 0, 128), (300, 0, 601), (512, 0, 1024)])
def test_part_of_a_head(n, at, d, near):
    """Parts that begin and end at any element, heads of any length: vectors of every
    width, down to single elements."""
    check(5, 3, 2, d, d, n, near, BF16, q_at=at, k_at=at, seed=n)
    check(1300, 3, 1, d, 2 * n, n, near, F16, q_at=at, pad=3, seed=n)


def test_latent_queries_and_their_one_key():
    """The rope part of latent attention: q's heads from element 512 on, one key row."""
    check(64, 64, 1, 576, 64, 32, True, BF16, q_at=512)
    check(3, 16, 0, 576, 0, 32, True, BF16, q_at=512)


@pytest.mark.parametrize("pad", [0, 1, 2, 4, 8])
def test_strides_of_any_alignment(pad):
    check(50, 4, 2, 64, 64, 32, False, BF16, pad=pad)
    check(50, 4, 2, 64, 64, 32, True, F16, pad=pad)


@pytest.mark.parametrize("wide", [False, True])
def test_far_positions(wide):
    """Up to 2^31 - 1: fp32 angles would be wrong by many turns."""
    check(500, 2, 1, 64, 64, 32, False, BF16, far=2 ** 31 - 1, wide=wide)
    check(500, 2, 1, 64, 64, 32, True, F16, far=2 ** 31 - 1, wide=wide, factor=1.3)


def test_frequencies_of_every_size():
    """0, subnormal, tiny and above one; negative ones turn the other way."""
    device = dev()
    freq = torch.tensor([0.0, 1e-42, 2.0 ** -60, 1e-10, 0.3, 1.0, 1.999, 2.0, 3.999, -0.7, -1.5, 2.0 ** -20], device=device)
    x = torch.randn(200, 2, 24, device=device).to(BF16)
    pos = torch.randint(0, 300000, (200,), device=device)
    got, none = kv.rotary(x, None, pos, freq)
    assert none is None
    close(got, turned(x, pos, freq, False, 0, 1.0), freq)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_values_of_every_size(dtype):
    """Subnormals and the largest, infinities and NaN in their own pairs only."""
    check(40, 2, 1, 64, 64, 32, False, dtype, scale=2.0 ** -20 if dtype == F16 else 1e-30)
    check(40, 2, 1, 64, 64, 32, True, dtype, scale=1e4 if dtype == F16 else 1e30)
    device = dev()
    x = torch.randn(9, 2, 64, device=device).to(dtype)
    pos, freq = torch.arange(9, device=device), kv.rotary_frequencies(64, device=device)
    clean, _ = kv.rotary(x, None, pos, freq)
    bad = x.clone()
    bad[3, 1, 5], bad[4, 0, 40] = math.nan, math.inf
    got, _ = kv.rotary(bad, None, pos, freq)
    for t, h, i in ((3, 1, 5), (4, 0, 8)):
        assert not got[t, h, [i, i + 32]].isfinite().any()
        got[t, h, [i, i + 32]] = clean[t, h, [i, i + 32]]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("t", [1, 100, 2000])
def test_in_place_and_into_given_outputs(near, t):
    q, k, pos, freq, gq, gk = check(t, 6, 2, 128, 128, 48, near, BF16, q_at=8, k_at=8)
    big = torch.full((t + 2, 8, 128), 3.0, dtype=BF16, device=q.device)
    oq, ok = big[1:-1, :6], big[1:-1, 6:]
    r = kv.rotary(q, k, pos, freq, interleaved=near, q_offset=8, k_offset=8, q_out=oq, k_out=ok)
    assert r[0] is oq and r[1] is ok and torch.equal(oq, gq) and torch.equal(ok, gk)
    assert (big[0] == 3).all() and (big[-1] == 3).all()
    mine = torch.cat([q, k], 1)
    was = mine._version
    kv.rotary(mine[:, :6], mine[:, 6:], pos, freq, interleaved=near, q_offset=8, k_offset=8, q_out=mine[:, :6],
              k_out=mine[:, 6:])
    assert mine._version > was and torch.equal(mine[:, :6], gq) and torch.equal(mine[:, 6:], gk)
    part = torch.cat([q, k], 1)[..., 8:104]                      # a slice that turns whole
    kv.rotary(part, None, pos, freq, interleaved=near, q_out=part)
    assert torch.equal(part, torch.cat([gq, gk], 1)[..., 8:104])


def test_turning_back_gives_the_inputs():
    """The gradient of a rotation is the rotation back: dot products with it agree."""
    device = dev()
    x = torch.randn(300, 4, 64, device=device).to(BF16)
    w = torch.randn(300, 4, 64, device=device).to(BF16)
    pos, freq = torch.randint(0, 10000, (300,), device=device), kv.rotary_frequencies(64, device=device)
    y, _ = kv.rotary(x, None, pos, freq)
    back, _ = kv.rotary(w, None, -pos, freq)
    a, b = (y.double() * w.double()).sum(-1), (x.double() * back.double()).sum(-1)
    # (64 terms, each side off by half a bf16 step of its result)
    size = (y.double().abs() * w.double().abs()).sum(-1) + (x.double().abs() * back.double().abs()).sum(-1)
    assert ((a - b).abs() <= (2.0 ** -8 + 2.0 ** -19) * size + 2.0 ** -19 * 64).all()


def refusals(device):
    q = torch.randn(5, 4, 64, device=device).to(BF16)
    good = dict(q=q, k=q[:, :1].clone(), positions=torch.arange(5, device=device), inv_freq=torch.ones(16, device=device))
    return good, [
        ("q", q.float(), TypeError), ("q", q.cpu(), TypeError), ("q", q[0], ValueError), ("q", q[..., ::2], ValueError),
        ("q", q.half(), TypeError), ("k", q[:4], ValueError), ("k", q.half(), TypeError), ("k", q[..., :30], ValueError),
        ("positions", torch.arange(5.0, device=device), TypeError), ("positions", torch.arange(4, device=device), ValueError),
        ("positions", torch.arange(5), TypeError), ("positions", torch.arange(10, device=device)[::2], ValueError),
        ("inv_freq", torch.ones(16, device=device).double(), TypeError), ("inv_freq", torch.ones(33, device=device), ValueError),
        ("inv_freq", torch.ones(0, device=device), kv.Kv4Error), ("inv_freq", torch.ones(4, 4, device=device), ValueError),
        ("q_offset", 33, ValueError), ("q_offset", -1, ValueError), ("k_offset", 40, ValueError), ("k_offset", 1.5, TypeError),
        ("factor", "a", TypeError), ("factor", math.inf, kv.Kv4Error),
        ("q_out", torch.empty(5, 4, 32, dtype=BF16, device=device), ValueError),
        ("q_out", torch.empty(5, 4, 64, dtype=F16, device=device), TypeError),
        ("q_out", torch.empty(5, 1, 64, dtype=BF16, device=device).expand(5, 4, 64), kv.Kv4Error),
        ("q_out", torch.empty(5, 64, 4, dtype=BF16, device=device).mT, ValueError),
    ]


def test_refusals():
    device = dev()
    good, bad = refusals(device)
    for name, value, error in bad:
        with pytest.raises(error):
            kv.rotary(**{**good, name: value})
    buf = torch.randn(6, 4, 64, device=device).to(BF16)
    with pytest.raises(ValueError):                              # a shifted view of the input
        kv.rotary(buf[:5], None, good["positions"], good["inv_freq"], q_out=buf[1:])
    with pytest.raises(ValueError):
        kv.rotary(good["q"], None, good["positions"], good["inv_freq"], k_out=good["k"])
    with pytest.raises(TypeError):
        kv.rotary(None, None, good["positions"], good["inv_freq"])
    kv.rotary(**good)
    torch.cuda.synchronize()


def test_outputs_that_share_elements_with_the_other_side_are_refused():
    device = dev()
    freq = kv.rotary_frequencies(64, device=device)
    for t in (1, 7):
        pos = torch.arange(t, device=device) + 9
        x = torch.randn(t, 4, 64, device=device).to(BF16)
        y, z = x.clone(), torch.empty(t, 9, 64, dtype=BF16, device=device)
        for q, k, out in ((x, x, dict(q_out=x)), (x, x, dict(k_out=x)), (x, y, dict(q_out=y)), (x, y, dict(k_out=x)),
                          (x, y, dict(q_out=z[:, :4], k_out=z[:, 3:7])), (x, y, dict(q_out=z[:, 5:], k_out=z[:, 3:7])),
                          (x, y, dict(q_out=z[:, ::2][:, :4], k_out=z[:, 2:6])),
                          (x, y[:, :1], dict(q_out=z[:, :4], k_out=z[:, 3:4])),
                          (x[..., :32], y[..., :32], dict(q_out=z[:, :4, :32], k_out=z[:, :4, 31:63]))):
            freq_of = freq[:q.shape[2] // 2]
            with pytest.raises(ValueError, match="apart"):
                kv.rotary(q, k, pos, freq_of, **out)
    torch.cuda.synchronize()


@pytest.mark.parametrize("t", [1, 7, 300])
@pytest.mark.parametrize("near", [False, True])
def test_slices_of_one_tensor_turn_in_place(t, near):
    """By tokens [T, q heads | k heads | v heads, D], by heads [T, heads, q | k | v, D], and
    tokens behind one another."""
    device = dev()
    freq, pos = kv.rotary_frequencies(64, device=device), torch.arange(t, device=device) * 3 + 1
    rows = torch.randn(t, 9, 64, device=device).to(BF16)
    heads = torch.randn(t, 4, 3, 64, device=device).to(BF16)
    whole = torch.randn(2 * t, 4, 64, device=device).to(BF16)
    for q, k in ((rows[:, :6], rows[:, 6:8]), (rows[:, 8:], rows[:, 2:5]), (heads[:, :, 0], heads[:, :, 1]),
                 (heads[:, :, 2], heads[:, :1, 1]), (whole[:t], whole[t:])):
        want = kv.rotary(q, k, pos, freq, interleaved=near)
        assert all(not torch.equal(a, b) for a, b in zip(want, (q, k)))
        kv.rotary(q, k, pos, freq, interleaved=near, q_out=q, k_out=k)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_outputs_whose_own_rows_meet_are_refused():
    """Sliding windows, out of place and in place; nothing is written.  Rows that lie
    between one another's, tokens inside heads among them, are fine."""
    device = dev()
    freq, pos = kv.rotary_frequencies(64, device=device), torch.arange(6, device=device) + 3
    x = torch.randn(6, 3, 64, device=device).to(BF16)
    want = kv.rotary(x, None, pos, freq)[0]
    flat = torch.randn(6000, device=device).to(BF16)
    kept = flat.clone()
    for strides in ((64, 64, 1), (128, 64, 1), (64, 128, 1), (128, 192, 1), (129, 65, 1), (330, 192, 1)):
        slide = flat.as_strided((6, 3, 64), strides)
        for q in (x, slide):
            with pytest.raises(kv.Kv4Error):
                kv.rotary(q, None, pos, freq, q_out=slide)
    torch.cuda.synchronize()
    assert torch.equal(flat, kept)
    for strides in ((192, 64, 1), (64, 384, 1), (64, 400, 1), (250, 70, 1), (512, 192, 1), (320, 192, 1), (384, 704, 1)):
        out = flat.as_strided((6, 3, 64), strides)
        kv.rotary(x, None, pos, freq, q_out=out)
        assert torch.equal(out, want)
        out.copy_(x)
        kv.rotary(out, None, pos, freq, q_out=out)
        assert torch.equal(out, want)


def test_interleaved_without_a_truth_value_is_refused():
    """Before anything is written, in place."""
    device = dev()
    good, _ = refusals(device)
    q, k = good["q"].clone(), good["k"].clone()
    for value in (torch.ones(2), torch.ones(2, device=device)):
        with pytest.raises(TypeError, match="interleaved"):
            kv.rotary(**{**good, "q": q, "k": k, "interleaved": value, "q_out": q, "k_out": k})
    torch.cuda.synchronize()
    assert torch.equal(q, good["q"]) and torch.equal(k, good["k"])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("n", [16, 5])
def test_frequencies_that_are_not_finite_give_nan_in_their_pairs(n, near, dtype):
    """At position 0 too (0 * inf is NaN); the other pairs and what does not turn are as
    without them."""
    device = dev()
    x = torch.randn(40, 3, 40, device=device).to(dtype)
    pos = torch.arange(40, device=device) * 7
    freq = kv.rotary_frequencies(2 * n, device=device)
    want = kv.rotary(x, None, pos, freq, interleaved=near, q_offset=3)[0]
    bad = {0: math.nan, 2: math.inf, n - 1: -math.inf}
    odd = freq.clone()
    for i, value in bad.items():
        odd[i] = value
        first = 3 + (2 * i if near else i)
        want[..., first] = want[..., first + (1 if near else n)] = math.nan
    got = kv.rotary(x, None, pos, odd, interleaved=near, q_offset=3)[0]
    assert torch.equal(got.isnan(), want.isnan()) and int(got.isnan().sum()) == 40 * 3 * 6
    assert torch.equal(got.nan_to_num(), want.nan_to_num())


def test_empty_calls():
    device = dev()
    freq, pos = torch.ones(4, device=device), torch.zeros(0, dtype=torch.int64, device=device)
    x = torch.empty(0, 3, 16, dtype=BF16, device=device)
    q, k = kv.rotary(x, x[:, :1], pos, freq)
    assert q.shape == (0, 3, 16) and k.shape == (0, 1, 16)
    none, k = kv.rotary(None, torch.ones(2, 1, 8, dtype=BF16, device=device), torch.zeros(2, dtype=torch.int32, device=device), freq)
    assert none is None and (k == 1).all()


def test_streams_and_graphs():
    device = dev()
    q = torch.randn(300, 8, 128, device=device).to(BF16)
    pos, freq = torch.arange(300, device=device), kv.rotary_frequencies(128, device=device)
    want = kv.rotary(q, q[:, :2], pos, freq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = kv.rotary(q, q[:, :2], pos, freq)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(streams[0]):
            graph.replay()
        with torch.cuda.stream(streams[1]):
            got = kv.rotary(q, q[:, :2], pos, freq)
    torch.cuda.synchronize()
    for a, b, c in zip(want, kept, got):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_rows_beyond_32_bits():
    """Tokens 1.5e9 elements apart, and more than 2^32 elements of output."""
    device = dev()
    far = torch.empty(2 * 1_500_000_000 + 3 * 64, dtype=BF16, device=device)
    x = torch.as_strided(far, (3, 3, 64), (1_500_000_000, 64, 1))
    near = torch.randn(3, 3, 64, device=device).to(BF16)
    x.copy_(near)
    pos, freq = torch.tensor([5, 70, 900], device=device), kv.rotary_frequencies(64, device=device)
    assert torch.equal(kv.rotary(x, None, pos, freq)[0], kv.rotary(near, None, pos, freq)[0])
    del far, x
    T = 600_000
    x = torch.randn(1000, 64, 128, device=device).to(BF16).repeat(T // 1000, 1, 1)
    pos = torch.arange(1000, device=device).repeat(T // 1000)
    freq = kv.rotary_frequencies(128, device=device)
    y = kv.rotary(x, None, pos, freq)[0]
    assert torch.equal(y[-1000:], y[:1000])
