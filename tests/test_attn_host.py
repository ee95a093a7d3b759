"""The cache and attention entry points without a GPU: sizes, refusals on the host, the binding's
checks, and the tests' own layout reader against its writer."""
import ctypes

import numpy as np
import pytest
import torch

import hadamard_bit_quant_hbl_b200 as hbl
from hadamard_bit_quant_hbl_b200 import _build
from attn_ref import join_records, k_bit, record_bytes, split_records, v_bit

FAKE = 1 << 20  # a 256-byte aligned non-null address; never dereferenced on these paths
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    _build.build()
    return hbl.lib()


def test_cache_bytes(L):
    assert hbl.hbl_kv_cache_bytes(7, 64, 8, 128, 3) == 7 * 8 * 4 * (4 * 128 * 3 + 128)
    assert hbl.hbl_kv_cache_bytes(1, 16, 1, 64, 2) == 640
    assert hbl.hbl_kv_cache_bytes(0, 16, 1, 64, 2) == 0
    # a cache of more than 4 GiB: sizes are formed in 64 bits
    assert hbl.hbl_kv_cache_bytes(1 << 20, 64, 8, 128, 8) == (1 << 20) * 8 * 4 * (4 * 128 * 8 + 128)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bits", [2, 3, 4, 8])
def test_layout_is_a_bijection(D, bits):
    k = [k_bit(d, i, bits) for d in range(D) for i in range(bits)]
    assert sorted(k) == list(range(D * bits))
    v = [16 * u + b for u, b in (v_bit(d, i, bits) for d in range(D) for i in range(bits))]
    assert sorted(v) == list(range(D * bits))
    rng = np.random.default_rng(D + bits)
    T, H = 64, 3
    uk, uv = rng.integers(0, 1 << bits, (2, T, H, D))
    gk, gv = rng.uniform(0.1, 2, (2, T, H)).astype(np.float32)
    cache = join_records(uk, uv, gk, gv, bits, 32)
    assert cache.size == T // 16 * H * record_bytes(D, bits)
    for a, b in zip(split_records(cache, H, D, bits, 32), (uk, uv, gk, gv)):
        np.testing.assert_array_equal(a, b)


def test_kv_append_refuses(L):
    ok = dict(Q=FAKE, qs=512, K=FAKE, ks=256, V=FAKE, vs=256, pos=FAKE, slots=FAKE, theta=1e4, T=5, Hq=4, Hkv=2, D=128,
              bits=3, cache=FAKE, cb=BIG, np=4, ps=64, qo=FAKE + 4096, qos=512)

    def call(**kw):
        a = {**ok, **kw}
        return L.hbl_kv_append(a["Q"], a["qs"], a["K"], a["ks"], a["V"], a["vs"], a["pos"], a["slots"], a["theta"],
                               a["T"], a["Hq"], a["Hkv"], a["D"], a["bits"], a["cache"], a["cb"], a["np"], a["ps"],
                               a["qo"], a["qos"], None)

    need = hbl.hbl_kv_cache_bytes(4, 64, 2, 128, 3)
    for kw in (dict(K=None), dict(V=None), dict(slots=None), dict(cache=None), dict(Q=None), dict(qo=None), dict(T=-1),
               dict(Hkv=0), dict(Hq=-1), dict(np=0), dict(ps=0), dict(cb=need - 1), dict(cache=FAKE + 8),
               dict(K=FAKE + 2), dict(ks=128), dict(ks=260), dict(vs=252), dict(qs=510), dict(qos=504),
               dict(theta=1.0), dict(theta=float("nan")), dict(pos=FAKE + 1), dict(slots=FAKE + 2),
               dict(qo=FAKE, qos=1024)):
        assert call(**kw) == hbl.HBL_EINVAL, kw
    for kw in (dict(D=96), dict(bits=5), dict(ps=24), dict(np=1 << 26, ps=64), dict(Hkv=70000)):
        assert call(**kw) == hbl.HBL_EUNSUPPORTED, kw
    assert call(T=0, K=None, V=None, Q=None, slots=None) == hbl.HBL_OK  # nothing to do


def test_kv_gather_refuses(L):
    need = hbl.hbl_kv_cache_bytes(4, 64, 2, 128, 3)
    ok = dict(cache=FAKE, cb=need, np=4, ps=64, slots=FAKE, T=5, Hkv=2, D=128, bits=3, K=FAKE, V=FAKE)

    def call(**kw):
        a = {**ok, **kw}
        return L.hbl_kv_gather(a["cache"], a["cb"], a["np"], a["ps"], a["slots"], a["T"], a["Hkv"], a["D"], a["bits"],
                               a["K"], a["V"], None)

    for kw in (dict(cache=None), dict(cb=need - 1), dict(slots=None), dict(T=-1), dict(K=None, V=None), dict(K=FAKE + 8),
               dict(Hkv=0), dict(slots=FAKE + 1)):
        assert call(**kw) == hbl.HBL_EINVAL, kw
    for kw in (dict(D=32), dict(bits=6), dict(ps=40, np=1)):
        assert call(**kw) == hbl.HBL_EUNSUPPORTED, kw
    assert call(T=0, slots=None) == hbl.HBL_OK


def test_attn_decode_refuses(L):
    need = hbl.hbl_kv_cache_bytes(4, 64, 2, 128, 3)
    ws = hbl.hbl_attn_decode_workspace(3, 8, 2, 128)
    ok = dict(Q=FAKE, qs=1024, cache=FAKE, cb=need, np=4, ps=64, tab=FAKE, w=2, lens=FAKE, B=3, Hq=8, Hkv=2, D=128,
              bits=3, scale=0.1, ws=FAKE, wb=ws, O=FAKE, lse=None)

    def call(**kw):
        a = {**ok, **kw}
        return L.hbl_attn_decode(a["Q"], a["qs"], a["cache"], a["cb"], a["np"], a["ps"], a["tab"], a["w"], a["lens"],
                                 a["B"], a["Hq"], a["Hkv"], a["D"], a["bits"], a["scale"], a["ws"], a["wb"], a["O"],
                                 a["lse"], None)

    for kw in (dict(Q=None), dict(qs=1000), dict(cache=None), dict(cb=need - 1), dict(tab=None), dict(w=0),
               dict(lens=None), dict(B=-1), dict(Hq=7), dict(Hq=0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(ws=None), dict(ws=FAKE + 16), dict(wb=ws - 1), dict(O=None), dict(O=FAKE + 8), dict(lse=FAKE + 2)):
        assert call(**kw) == hbl.HBL_EINVAL, kw
    for kw in (dict(B=4097, wb=BIG), dict(w=1 << 26), dict(D=80), dict(bits=1)):
        assert call(**kw) == hbl.HBL_EUNSUPPORTED, kw
    assert call(B=0, Q=None, tab=None, lens=None) == hbl.HBL_OK


def test_attn_prompt_refuses(L):
    ok = dict(Q=FAKE, qs=1024, K=FAKE, ks=256, V=FAKE, vs=256, cq=FAKE, ck=FAKE, B=2, tq=10, tk=12, mq=10, Hq=8, Hkv=2,
              D=128, scale=0.1, causal=1, O=FAKE, lse=None)

    def call(**kw):
        a = {**ok, **kw}
        return L.hbl_attn_prompt(a["Q"], a["qs"], a["K"], a["ks"], a["V"], a["vs"], a["cq"], a["ck"], a["B"], a["tq"],
                                 a["tk"], a["mq"], a["Hq"], a["Hkv"], a["D"], a["scale"], a["causal"], a["O"], a["lse"],
                                 None)

    for kw in (dict(Q=None), dict(K=None), dict(V=None), dict(qs=1016), dict(ks=128), dict(vs=260), dict(cq=None),
               dict(ck=None), dict(B=-1), dict(tq=-1), dict(tk=-1), dict(mq=-1), dict(Hq=9), dict(Hkv=0),
               dict(scale=float("nan")), dict(O=None), dict(O=FAKE + 4), dict(lse=FAKE + 1), dict(Q=FAKE + 8),
               dict(cq=FAKE + 1)):
        assert call(**kw) == hbl.HBL_EINVAL, kw
    for kw in (dict(D=96), dict(B=4097)):
        assert call(**kw) == hbl.HBL_EUNSUPPORTED, kw
    assert call(B=0, Q=None, cq=None) == hbl.HBL_OK
    assert call(tq=0, Q=None, O=None) == hbl.HBL_OK


def test_binding_refuses_before_any_call():
    bf = torch.zeros((4, 2, 64), dtype=torch.bfloat16)  # host tensors
    cache = torch.zeros(1 << 16, dtype=torch.uint8)
    i4 = torch.zeros(4, dtype=torch.int32)
    for f in (lambda: hbl.hbl_kv_append(bf, bf, i4, cache, 16),
              lambda: hbl.hbl_kv_append(bf.float(), bf, i4, cache, 16),
              lambda: hbl.hbl_kv_append(bf, bf[:3], i4, cache, 16),
              lambda: hbl.hbl_kv_gather(cache, i4, 2, 64, 16, K=bf[:3]),
              lambda: hbl.hbl_attn_decode(bf, cache, i4, i4, 2, 16),
              lambda: hbl.hbl_attn_prompt(bf, bf, bf[:, :, :32], i4, i4)):
        with pytest.raises(ValueError):
            f()


def test_library_call_with_null_stream_argument_types(L):
    # the C signatures as declared: sizes are 64-bit, a call with a size past 32 bits is checked as such
    assert L.hbl_kv_gather.argtypes[1] is ctypes.c_size_t
    assert L.hbl_attn_decode.argtypes[16] is ctypes.c_size_t


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
def test_a_masked_half_word_is_an_fp16_operand(bits):
    # u << p inside a half-word is the fp16 number u 2^(p - 24) as long as it stays below 2^11
    u = np.arange(1 << bits, dtype=np.uint16)
    p = 0
    while ((1 << bits) - 1) << p < 1 << 11:
        np.testing.assert_array_equal((u << p).astype(np.uint16).view(np.float16).astype(np.float64), u * 2.0 ** (p - 24))
        p += 1
    assert p > {2: 8, 3: 6, 4: 4, 8: 0}[bits]  # the highest place that the decode uses


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
def test_a_code_becomes_its_state_by_one_exact_multiply_add(bits):
    # the code at bit p >= 1 with the bits of 2^23 above it is 2^23 + u 2^p; times 2 / 2^p, less 2^24 / 2^p + L
    L = (1 << bits) - 1
    u = np.arange(L + 1, dtype=np.uint32)
    for p in range(1, 17 - bits + 1):
        f = ((u << p) | np.uint32(0x4B000000)).view(np.float32).astype(np.float64)
        a, b = 2.0 / 2 ** p, 2.0 ** 24 / 2 ** p + L
        assert float(np.float32(a)) == a and float(np.float32(b)) == b
        np.testing.assert_array_equal(f * a - b, 2.0 * u - L)
