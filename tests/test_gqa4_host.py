"""The 4-bit grouped-query and rotary entry points without a GPU: what they refuse,
frequencies, and the reference's own pieces."""
import ctypes
import math

import pytest
import torch

import bit_kv_cache_nvfp4_gb300 as kv
import gqa4_ref as ref
from test_gqa8_host import (BAD, SHARED, UNSUPPORTED, append_args, attention_args, lib, mem,  # noqa: F401
                            read_args)

ALIGNED = [("pool", 8), ("scales", 8)]


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(lens=None), BAD), (dict(ks0=132), BAD), (dict(vs1=4), BAD),
    (dict(ks1=32), BAD), (dict(ks0=-128), BAD), (dict(pages=0), BAD)])
def test_append_refuses(lib, mem, change, status):  # noqa: F811
    assert lib.kv4_append_gqa4(*append_args(mem[1], **change)) == status


@pytest.mark.parametrize("change,status", SHARED + [(dict(starts=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD)])
def test_read_refuses(lib, mem, change, status):  # noqa: F811
    assert lib.kv4_read_gqa4(*read_args(mem[1], **change)) == status


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(q=None), BAD), (dict(lens=None), BAD), (dict(out=None), BAD), (dict(lse=None), BAD), (dict(hq=7), BAD),
    (dict(hq=1), BAD), (dict(hq=2 * 129), UNSUPPORTED), (dict(window=-1), BAD), (dict(max_new=0), BAD),
    (dict(max_new=-1), BAD), (dict(scale=math.inf), BAD), (dict(scale=math.nan), BAD), (dict(qs0=513), BAD)])
def test_attention_refuses(lib, mem, change, status):  # noqa: F811
    assert lib.kv4_attention_gqa4(*attention_args(mem[1], **change)) == status


@pytest.mark.parametrize("name,off", ALIGNED)
def test_alignment(lib, mem, name, off):  # noqa: F811
    """Codes and scales move in 16-byte pieces."""
    change = {name: mem[1] + off}
    assert lib.kv4_append_gqa4(*append_args(mem[1], **change)) == BAD
    assert lib.kv4_read_gqa4(*read_args(mem[1], **change)) == BAD
    assert lib.kv4_attention_gqa4(*attention_args(mem[1], **change)) == BAD


def test_empty_calls_need_no_device(lib, mem):  # noqa: F811
    for args in (dict(T=0), dict(B=0)):
        assert lib.kv4_append_gqa4(*append_args(mem[1], **args)) == 0
        assert lib.kv4_read_gqa4(*read_args(mem[1], **args)) == 0
        assert lib.kv4_attention_gqa4(*attention_args(mem[1], **args)) == 0


# ---------------------------------------------------------------------------
# rotary
# ---------------------------------------------------------------------------
def rotary_args(p, **kw):
    a = dict(q=p, qs0=256, qs1=64, hq=4, dq=64, qo=0, qout=p, qos0=256, qos1=64, k=p, ks0=64, ks1=64, hk=1, dk=64, ko=0,
             kout=p, kos0=64, kos1=64, dtype=0, T=3, pos=p, bits=32, freq=p, n=32, near=0, factor=1.0, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("change,status", [
    (dict(q=None), BAD), (dict(qout=None), BAD), (dict(k=None), BAD), (dict(kout=None), BAD), (dict(pos=None), BAD),
    (dict(freq=None), BAD), (dict(T=-1), BAD), (dict(T=2 ** 31), BAD), (dict(hq=-1), BAD), (dict(hq=65536), BAD),
    (dict(hq=65535, qos1=64, qs1=64), UNSUPPORTED), (dict(n=0), BAD), (dict(n=33), BAD), (dict(n=513, dq=2000), UNSUPPORTED),
    (dict(qo=1), BAD), (dict(qo=-1), BAD), (dict(ko=2 ** 31 - 1), BAD), (dict(dq=0), BAD), (dict(dk=65537), BAD),
    (dict(dtype=2), UNSUPPORTED), (dict(bits=16), UNSUPPORTED), (dict(factor=math.inf), BAD), (dict(factor=math.nan), BAD),
    (dict(qs0=-1), BAD), (dict(qos1=63), BAD), (dict(kos0=63), BAD), (dict(qos0=512), BAD), (dict(qs1=128), BAD)])
def test_rotary_refuses(lib, mem, change, status):  # noqa: F811
    assert lib.kv4_rotary(*rotary_args(mem[1], **change)) == status


def rows_meet(t, token, h, head, d):
    """Whether two of the rows [i * token + j * head, + d) share an element, by looking."""
    at = sorted(i * token + j * head for i in range(t) for j in range(h))
    return any(y - x < d for x, y in zip(at, at[1:]))


def test_rotary_refuses_outputs_whose_rows_meet(lib, mem):  # noqa: F811
    """All strides of small outputs, out of place and in place: a step that is at least a
    row long is not enough, and rows of one dimension may lie between the other's."""
    refused = accepted = 0
    for t in range(1, 6):
        for h in range(1, 5):
            for token in range(1, 27):
                for head in range(1, 19):
                    meet = rows_meet(t, token, h, head, 4)
                    refused, accepted = refused + meet, accepted + (not meet)
                    if not meet and torch.cuda.is_available():
                        continue                                  # (it would be launched)
                    one = dict(T=t, n=2, k=None, kout=None, hk=0, hq=h, dq=4, qos0=token, qos1=head)
                    for args in (dict(one, qs0=64, qs1=8, qout=mem[1] + 64), dict(one, qs0=token, qs1=head)):
                        assert (lib.kv4_rotary(*rotary_args(mem[1], **args)) == BAD) == meet, (t, token, h, head)
    assert refused > 1000 and accepted > 1000
    # sizes at which a product of steps and strides would leave 64 bits
    for t, token, h, head, meet in ((2 ** 31 - 1, 2 ** 62, 65535, 2 ** 62, True), (2 ** 31 - 1, 64, 65535, 64, True),
                                    (2 ** 31 - 1, 64, 65535, 2 ** 31 * 64 - 128, True), (2 ** 20, 2 ** 61 + 1, 3, 2 ** 62, True)):
        args = dict(T=t, n=2, k=None, kout=None, hk=0, hq=h, dq=4, qos0=token, qos1=head, qs0=0, qs1=0, qout=mem[1] + 64)
        assert (lib.kv4_rotary(*rotary_args(mem[1], **args)) == BAD) == meet


def test_rotary_alignment(lib, mem):  # noqa: F811
    for change in (dict(q=mem[1] + 1), dict(kout=mem[1] + 3), dict(pos=mem[1] + 2), dict(pos=mem[1] + 4, bits=64),
                   dict(freq=mem[1] + 2)):
        assert lib.kv4_rotary(*rotary_args(mem[1], **change)) == BAD


def test_rotary_of_nothing(lib, mem):  # noqa: F811
    none = dict(q=None, qout=None, hq=0, k=None, kout=None, hk=0)
    assert lib.kv4_rotary(*rotary_args(mem[1], **none)) == 0
    assert lib.kv4_rotary(*rotary_args(mem[1], T=0)) == 0


def test_frequencies():
    f = kv.rotary_frequencies(64)
    i = torch.arange(32, dtype=torch.float64)
    want = 10000.0 ** (-i / 32)
    assert f.dtype == torch.float32 and torch.equal(f, want.float())
    assert torch.equal(kv.rotary_frequencies(64, scaling="linear", stretch=8.0), (want / 8).float())
    base = kv.rotary_frequencies(64, scaling="base", stretch=8.0)
    assert base[0] == 1 and abs(float(base[-1]) / float(want[-1] / 8) - 1) < 1e-6
    ramp = kv.rotary_frequencies(64, scaling="ramp", stretch=8.0, original_length=4096, slow=1.0, fast=32.0).double()
    turns = 4096 * want / (2 * math.pi)
    r = ramp / want
    assert ((r - 1).abs()[turns > 32] < 1e-6).all() and ((r * 8 - 1).abs()[turns < 1] < 1e-6).all()
    between = (turns > 1) & (turns < 32)
    assert between.any() and (r[between] > 1 / 8).all() and (r[between] < 1).all()
    assert (r[1:] <= r[:-1] * (1 + 2.0 ** -22)).all()            # (rounded to fp32: 2^-24 of each)
    assert torch.equal(kv.rotary_frequencies(2), torch.ones(1))


def test_frequencies_of_a_ramp_by_index():
    """64 turned elements over 4096 tokens: 32 turns are at pair 10.47, 1 turn at 22.52,
    so pairs up to 10 are kept, those from 23 on divided, pair 16 six thirteenths between."""
    want = [10000.0 ** (-i / 32) for i in range(32)]
    assert math.floor(64 * math.log(4096 / (64 * math.pi)) / (2 * math.log(1e4))) == 10
    assert math.ceil(64 * math.log(4096 / (2 * math.pi)) / (2 * math.log(1e4))) == 23
    for i in range(32):
        keep = min(max((23 - i) / 13, 0.0), 1.0)
        want[i] *= keep + (1 - keep) / 40
    args = dict(stretch=40.0, original_length=4096, slow=1.0, fast=32.0)
    got = kv.rotary_frequencies(64, scaling="index_ramp", **args)
    assert got.dtype == torch.float32
    # (each rounded once: half a step of fp32)
    assert (got.double() / torch.tensor(want, dtype=torch.float64) - 1).abs().max() <= 2.0 ** -24 * (1 + 2.0 ** -20)
    by_turns = kv.rotary_frequencies(64, scaling="ramp", **args)
    ratio = (by_turns / got).tolist()
    assert all(abs(r - 1) < 1e-6 for r in ratio[:10] + ratio[24:]) and abs(ratio[11] - 0.93) < 0.01 and min(ratio) < 0.24
    # a step, where both ends are one index, and ends beyond the pairs
    step = kv.rotary_frequencies(64, scaling="index_ramp", stretch=4.0, original_length=2 * math.pi * 1.5, slow=1.0, fast=1.2)
    assert step[0] == 1 and abs(float(step[2]) / 10000.0 ** (-2 / 32) - 0.25) < 1e-6
    short = kv.rotary_frequencies(8, scaling="index_ramp", stretch=4.0, original_length=3)
    assert torch.allclose(short.double(), 10000.0 ** (-torch.arange(4, dtype=torch.float64) / 4) / 4 * torch.tensor([4.0, 1, 1, 1]), rtol=1e-6)


@pytest.mark.parametrize("args", [dict(dim=0), dict(dim=7), dict(dim=8, base=0.0), dict(dim=8, stretch=-1.0),
                                  dict(dim=2, scaling="base", stretch=2.0), dict(dim=8, scaling="ramp", slow=4.0, fast=4.0),
                                  dict(dim=8, scaling="other"), dict(dim=8, base=math.inf), dict(dim=8, stretch=math.nan)])
def test_frequencies_refuse(args):
    with pytest.raises(ValueError):
        kv.rotary_frequencies(**args)


@pytest.mark.parametrize("args", [dict(slow=2.0, fast=2.0), dict(slow=0.0), dict(slow=-1.0), dict(base=1.0), dict(base=0.5),
                                  dict(original_length=0), dict(original_length=math.nan), dict(original_length=math.inf),
                                  dict(fast=math.nan), dict(fast=math.inf)])
def test_frequencies_of_a_ramp_by_index_refuse(args):
    with pytest.raises(ValueError):
        kv.rotary_frequencies(64, scaling="index_ramp", stretch=8.0, **args)


# ---------------------------------------------------------------------------
# the reference
# ---------------------------------------------------------------------------
def test_reference_codes_by_hand():
    """A block of amax 6: scale 1 and codes of the values themselves, ties to even;
    one of amax 12: scale 2; a block of zeros."""
    x = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.26, 0.5, 1, 1.5, 2, 3, -4], dtype=torch.float64)
    codes, scale = ref.quantize(torch.cat([x, 2 * x, 0 * x]))
    assert scale.tolist() == [0x38, 0x40, 0]
    half = torch.stack([codes[:8] & 15, codes[:8] >> 4], -1).flatten().tolist()
    assert half == [7, 0, 2, 2, 4, 4, 6, 6, 8, 9, 1, 2, 3, 4, 5, 14]
    assert torch.equal(codes[:8], codes[8:16]) and (codes[16:] == 0).all()


def test_reference_round_trip():
    """Every code of every positive scale comes back."""
    s = torch.arange(1, 127, dtype=torch.uint8)
    code = torch.arange(16, dtype=torch.uint8)
    x = ref.dequantize((code[0::2] | code[1::2] << 4).expand(126, 8), s[:, None])
    codes, scales = ref.quantize(x)
    assert torch.equal(scales[:, 0], s)
    assert torch.equal(ref.dequantize(codes, scales), x)


def test_bounds_see_a_lost_page():
    """Of the reference itself: without the values of one page of a request whose
    query asks for it, a row is many times its bound off."""
    c = ref.Cache([300], 1, 64, "cpu", seed=1)
    q = torch.randn(1, 1, 64) * 0.1
    want = ref.attention(q, c.pool, c.scales, c.table, c.lens, [0, 1], 0.125)
    tol, _ = ref.bounds(*want, torch.bfloat16, 64)
    c.scales[c.table[0][2], :, 1] = 0
    lost = ref.attention(q, c.pool, c.scales, c.table, c.lens, [0, 1], 0.125)[0]
    assert float(((lost - want[0]).abs() / tol).max()) > 20
