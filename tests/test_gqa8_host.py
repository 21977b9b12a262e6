"""The 8-bit grouped-query entry points without a GPU: what they refuse, and
the reference's own pieces."""
import ctypes
import math

import pytest
import torch

import bit_kv_cache_nvfp4_gb300 as kv
import gqa8_ref as ref

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    return kv.load_library()


@pytest.fixture(scope="module")
def mem():
    buf = ctypes.create_string_buffer(1 << 12)
    return buf, (ctypes.addressof(buf) + 255) & ~255


def append_args(p, **kw):
    a = dict(k=p, ks0=128, ks1=64, v=p, vs0=128, vs1=64, dtype=0, T=4, cu=p, pt=p, stride=2, page=64, lens=p, B=1,
             hkv=2, d=64, pool=p, scales=p, pages=3, err=None, stream=None)
    a.update(kw)
    return list(a.values())


def read_args(p, **kw):
    a = dict(pool=p, scales=p, pages=3, pt=p, stride=2, page=64, starts=p, cu=p, T=4, B=1, hkv=2, d=64, dtype=0, k=p,
             v=p, err=None, stream=None)
    a.update(kw)
    return list(a.values())


def attention_args(p, **kw):
    a = dict(q=p, qs0=512, qs1=64, dtype=0, T=4, cu=p, max_new=2, pool=p, scales=p, pages=3, pt=p, stride=2, page=64,
             lens=p, B=2, hq=8, hkv=2, d=64, window=0, scale=0.1, out=p, lse=p, ws=p, wsn=0, err=None, stream=None)
    a.update(kw)
    return list(a.values())


BAD = 1
UNSUPPORTED = 2
SHARED = [(dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(page=32), UNSUPPORTED),
          (dict(dtype=2), UNSUPPORTED), (dict(T=-1), BAD), (dict(B=-1), BAD), (dict(B=65536), BAD), (dict(hkv=0), BAD),
          (dict(pages=-1), BAD), (dict(pages=2 ** 31 - 1), BAD), (dict(stride=0), BAD), (dict(T=2 ** 31), BAD),
          (dict(pool=None), BAD), (dict(scales=None), BAD), (dict(cu=None), BAD), (dict(pt=None), BAD)]


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(lens=None), BAD), (dict(ks0=132), BAD), (dict(vs1=4), BAD),
    (dict(ks1=32), BAD), (dict(ks0=-128), BAD)])
def test_append_refuses(lib, mem, change, status):
    assert lib.kv4_append_gqa8(*append_args(mem[1], **change)) == status


@pytest.mark.parametrize("change,status", SHARED + [(dict(starts=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD)])
def test_read_refuses(lib, mem, change, status):
    assert lib.kv4_read_gqa8(*read_args(mem[1], **change)) == status


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(q=None), BAD), (dict(lens=None), BAD), (dict(out=None), BAD), (dict(lse=None), BAD), (dict(hq=7), BAD),
    (dict(hq=1), BAD), (dict(hq=2 * 129), UNSUPPORTED), (dict(window=-1), BAD), (dict(max_new=0), BAD),
    (dict(max_new=-1), BAD), (dict(scale=math.inf), BAD), (dict(scale=math.nan), BAD), (dict(qs0=513), BAD)])
def test_attention_refuses(lib, mem, change, status):
    assert lib.kv4_attention_gqa8(*attention_args(mem[1], **change)) == status


@pytest.mark.parametrize("change,status", [(dict(pages=0), BAD), (dict(hkv=32768, ks1=64, vs1=64), UNSUPPORTED)])
def test_no_pages_and_too_many_heads_are_refused(lib, mem, change, status):
    rest = {k: v for k, v in change.items() if k not in ("ks1", "vs1")}
    assert lib.kv4_append_gqa8(*append_args(mem[1], **change)) == status
    assert lib.kv4_read_gqa8(*read_args(mem[1], **rest)) == status
    hq = {"hq": rest["hkv"]} if "hkv" in rest else {}
    assert lib.kv4_attention_gqa8(*attention_args(mem[1], **rest, **hq)) == status


def test_misaligned_pointers_are_refused(lib, mem):
    p = mem[1]
    assert lib.kv4_append_gqa8(*append_args(p, pool=p + 64)) == BAD
    assert lib.kv4_append_gqa8(*append_args(p, k=p + 8)) == BAD
    assert lib.kv4_append_gqa8(*append_args(p, cu=p + 2)) == BAD
    assert lib.kv4_read_gqa8(*read_args(p, v=p + 8)) == BAD
    assert lib.kv4_attention_gqa8(*attention_args(p, out=p + 8)) == BAD
    assert lib.kv4_attention_gqa8(*attention_args(p, lse=p + 2)) == BAD


def test_empty_calls_do_nothing(lib):
    none = dict(pool=None, scales=None, cu=None, pt=None)
    assert lib.kv4_append_gqa8(*append_args(None, T=0)) == 0
    assert lib.kv4_append_gqa8(*append_args(None, B=0, **none)) == 0
    assert lib.kv4_read_gqa8(*read_args(None, T=0)) == 0
    assert lib.kv4_attention_gqa8(*attention_args(None, T=0, max_new=0)) == 0
    assert lib.kv4_attention_gqa8(*attention_args(None, B=0)) == 0


def test_plan_refuses(lib):
    n = ctypes.c_size_t()
    plan = lambda **kw: lib.kv4_attention_gqa8_plan(*{**dict(B=1, m=1, T=1, hq=8, hkv=2, d=64), **kw}.values(),  # noqa: E731
                                                    ctypes.byref(n))
    assert plan(hq=7) == BAD and plan(hkv=0) == BAD and plan(m=-1) == BAD and plan(T=-1) == BAD
    assert plan(d=32) == UNSUPPORTED and plan(hq=258) == UNSUPPORTED


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    pool, scales = torch.zeros(1, 2, 2, 64, 64, dtype=torch.uint8), torch.zeros(1, 2, 2, dtype=torch.uint8)
    i = torch.zeros(1, dtype=torch.int32)
    table, cu = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        kv.append_gqa8(x, x, cu, table, i, pool, scales)
    with pytest.raises(TypeError):
        kv.read_gqa8(pool, scales, table, i, cu, 1)
    with pytest.raises(TypeError):
        kv.attention_gqa8(x, pool, scales, table, i, cu, 1, 0.1)


def test_reference_encoding_round_trips_and_rounds_to_even():
    vals = ref.e4m3_values()
    codes = torch.tensor([c for c in range(256) if c & 127 != 127])
    assert torch.equal(ref.encode(vals[codes]).long(), codes)
    mid = (vals[16:120] + vals[17:121]) / 2                     # ties between neighbours
    assert (ref.encode(mid) % 2 == 0).all()
    x = torch.linspace(-448, 448, 20001, dtype=torch.float64)
    assert torch.equal(ref.encode(x), x.float().to(torch.float8_e4m3fn).view(torch.uint8))
    assert [ref.least_exponent(a) for a in (448.0, 448.1, 1.75, 0.0, 1e30)] == [0, 1, -8, -48, 48]
