"""The low-bit cache and the attention over it against 64-bit evaluations.

Bars. Codes: equal to the oracle's 64-bit evaluation, all of them. gamma: fp32, off by at most the
fp32 rotation's 2^-21. Read-back: half a bf16 step (2^-8 of the value) plus fp32 rounding. Attention:
attn_ref.check_close, with weights rounded to fp16 (decode, half a step 2^-11) or bf16 (prompt, 2^-8).
"""
import numpy as np
import pytest
import torch

import oracle
import hadamard_bit_quant_hbl_b200 as hbl
from hadamard_bit_quant_hbl_b200 import inputs
from attn_ref import attention, check_close, join_records, quantise, record_bytes, split_records, states

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)
    hbl.lib()
    yield
    assert hbl.hbl_device_status() == hbl.HBL_OK


def bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def i32(a):
    return torch.from_numpy(np.asarray(a, np.int32)).cuda()


def fused_states(T, Hq, Hkv, D, seed, pad=0):
    """One fused bf16 QKV buffer [T, (Hq + 2 Hkv) D + pad] and its three slices."""
    n = (Hq + 2 * Hkv) * D
    x = inputs.qkv_states(T, Hq + 2 * Hkv, D, seed=seed, row_stride=n + pad)
    X = bf16(x)
    cut = [0, Hq * D, (Hq + Hkv) * D, n]
    host = [x[:, a:b].reshape(T, -1, D) for a, b in zip(cut, cut[1:])]
    dev = [X[:, a:b].view(T, -1, D) if b > a else None for a, b in zip(cut, cut[1:])]
    return X, host, dev


# ------------------------------------------------------------------------------------ append, gather

APPEND = [
    # (T, Hq, Hkv, D, bits, page, rope, pad)
    (1, 4, 4, 128, 3, 16, True, 0),
    (17, 8, 2, 128, 3, 64, True, 0),
    (33, 6, 3, 64, 3, 32, True, 8),
    (16, 2, 1, 256, 3, 16, True, 0),
    (40, 5, 5, 128, 2, 48, True, 24),
    (21, 0, 2, 64, 2, 16, True, 0),
    (19, 3, 1, 256, 2, 128, True, 0),
    (50, 4, 2, 128, 4, 64, False, 0),
    (23, 4, 4, 64, 4, 16, True, 0),
    (18, 2, 2, 256, 4, 32, True, 0),
    (31, 4, 2, 128, 8, 64, True, 0),
    (35, 9, 3, 64, 8, 16, True, 16),
    (20, 4, 2, 256, 8, 16, False, 0),
    (300, 32, 8, 128, 3, 64, True, 0),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,bits,page,rope,pad", APPEND)
def test_append_and_gather(T, Hq, Hkv, D, bits, page, rope, pad):
    X, (q, k, v), (Q, K, V) = fused_states(T, Hq, Hkv, D, seed=T + D + bits, pad=pad)
    rng = np.random.default_rng(T)
    pos = rng.integers(0, 100000, T) if rope else None
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T]  # in no order: every token in a place of its own
    dropped = rng.random(T) < 0.1
    slots[dropped] = -1 - rng.integers(0, 5, dropped.sum())
    before = rng.integers(0, 256, hbl.hbl_kv_cache_bytes(pages, page, Hkv, D, bits)).astype(np.uint8)
    cache = torch.from_numpy(before).cuda()
    keep = X.clone()
    out = hbl.hbl_kv_append(K, V, i32(slots), cache, page, bits, pos=None if pos is None else i32(pos), rope_theta=5e5,
                            Q=Q)
    assert torch.equal(X.view(torch.int16), keep.view(torch.int16))
    uk, uv, gk, gv = split_records(cache.cpu().numpy(), Hkv, D, bits, page)
    old = split_records(before, Hkv, D, bits, page)
    live = ~dropped
    for u, g, x, p in ((uk, gk, k, pos), (uv, gv, v, None)):
        ru, rg = quantise(x, p, bits, 5e5)
        np.testing.assert_array_equal(u[slots[live]], ru[live])
        np.testing.assert_allclose(g[slots[live]], rg[live], rtol=2.0 ** -21)
    others = np.setdiff1d(np.arange(pages * page), slots[live])
    for a, b in zip((uk, uv, gk, gv), old):
        np.testing.assert_array_equal(a[others], b[others])  # every other token as it was (NaNs alike)
    if Q is not None:
        rq = oracle.bf16_to_f64(q) if pos is None else oracle.rope(oracle.bf16_to_f64(q), pos, 5e5)
        d = np.abs(out.float().cpu().numpy() - rq)
        big = np.abs(rq).max(-1, keepdims=True)
        assert np.all(d <= 2.0 ** -8 * np.abs(rq) + 2.0 ** -21 * big)
    else:
        assert out is None
    # read back, in another order, twice the same token, some rows left alone
    order = np.concatenate([rng.permutation(slots[live]), slots[live][:3], [-1, -7]])
    gK = torch.full((len(order), Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    gV = torch.full_like(gK, -3.0)
    hbl.hbl_kv_gather(cache, i32(order), Hkv, D, page, bits, K=gK, V=gV)
    for y, u, g, kept in ((gK, uk, gk, 7.0), (gV, uv, gv, -3.0)):
        y = y.float().cpu().numpy()
        r = states(u, g, bits)[order[:-2]]
        np.testing.assert_allclose(y[:-2], r, rtol=2.0 ** -8 + 2.0 ** -20, atol=1e-30)
        assert np.all(y[-2:] == kept)
    assert hbl.hbl_device_status() == hbl.HBL_OK


def test_append_in_place_and_far_positions():
    T, Hq, Hkv, D, bits, page = 37, 4, 2, 128, 8, 16
    _, (q, k, v), (Q, K, V) = fused_states(T, Hq, Hkv, D, seed=3)
    pos = np.random.default_rng(0).integers(2 ** 30, 2 ** 31 - 1, T)
    cache = torch.zeros(hbl.hbl_kv_cache_bytes(3, page, Hkv, D, bits), dtype=torch.uint8, device="cuda")
    got = hbl.hbl_kv_append(K, V, i32(np.arange(T)), cache, page, bits, pos=i32(pos), Q=Q, q_out=Q)
    assert got is Q
    rq = oracle.rope(oracle.bf16_to_f64(q), pos)
    big = np.abs(rq).max(-1, keepdims=True)
    # the angle is below 2^31 in fp64: half a step of it, 2^-22, is what the reduction can lose
    assert np.all(np.abs(Q.float().cpu().numpy() - rq) <= 2.0 ** -8 * np.abs(rq) + 2.0 ** -19 * big)
    uk, uv, _, _ = split_records(cache.cpu().numpy(), Hkv, D, bits, page)
    ru, _ = quantise(v, None, bits)
    np.testing.assert_array_equal(uv[:T], ru)
    rk, _ = quantise(k, pos, bits)
    d = np.abs(uk[:T] - rk.astype(np.int64))
    assert d.max() <= 1 and np.count_nonzero(d) <= 1e-3 * d.size


def test_append_degenerate_heads():
    D, page = 128, 16
    x = np.zeros((16, 2 * 2 * D), np.float32)
    x[1, 7] = -2.5
    x[2, :D] = 1.0
    x[3, 2 * D:3 * D] = np.linspace(-3, 3, D)
    x[4, 2 * D:2 * D + 6] = [1.5625, 0.625, -0.625, 1.25, -1.25, 0.0]  # exact .5 ties at 8 bits in V
    x[5] = 1e-38
    x[6] = 3e38
    b = inputs.f32_to_bf16_bits(x).reshape(16, 4, D)
    X = bf16(b)
    for bits in (2, 3, 4, 8):
        cache = torch.zeros(hbl.hbl_kv_cache_bytes(1, page, 2, D, bits), dtype=torch.uint8, device="cuda")
        hbl.hbl_kv_append(X[:, :2], X[:, 2:], i32(np.arange(16)), cache, page, bits)
        uk, uv, gk, gv = split_records(cache.cpu().numpy(), 2, D, bits, page)
        for u, g, xs in ((uk, gk, b[:, :2]), (uv, gv, b[:, 2:])):
            ru, rg = quantise(xs, None, bits)
            np.testing.assert_array_equal(u, ru)
            np.testing.assert_array_equal(g, rg)


def test_append_and_gather_flag_slots_out_of_range():
    T, H, D, bits, page = 5, 2, 64, 4, 16
    _, _, (_, K, V) = fused_states(T, 0, H, D, seed=1)
    cache = torch.zeros(hbl.hbl_kv_cache_bytes(2, page, H, D, bits), dtype=torch.uint8, device="cuda")
    slots = i32([3, 32, 31, 2 ** 31 - 1, 0])
    hbl.hbl_kv_append(K, V, slots, cache, page, bits)
    assert hbl.hbl_device_status() == hbl.HBL_EINVAL
    assert hbl.hbl_device_status() == hbl.HBL_OK
    k = torch.full((T, H, D), 5.0, dtype=torch.bfloat16, device="cuda")
    hbl.hbl_kv_gather(cache, slots, H, D, page, bits, K=k)
    assert hbl.hbl_device_status() == hbl.HBL_EINVAL
    assert (k[[1, 3]] == 5).all() and (k[[0, 2, 4]] != 5).any()


def test_append_matches_the_state_quantiser():
    # the same heads through hbl_qkv_quant: its codes may differ where the decision is within fp32
    # rounding of a border (its documented behaviour), and nowhere else
    T, H, D, bits = 64, 4, 128, 3
    _, (_, k, _), (_, K, V) = fused_states(T, 0, H, D, seed=9)
    pos = np.arange(T)
    cache = torch.zeros(hbl.hbl_kv_cache_bytes(4, 16, H, D, bits), dtype=torch.uint8, device="cuda")
    hbl.hbl_kv_append(K, V, i32(pos), cache, 16, bits, pos=i32(pos))
    codes, gamma = hbl.hbl_qkv_quant(K.contiguous(), H, D, bits, pos=i32(pos))
    y = hbl.hbl_qkv_dequant(codes, gamma, D, bits)
    got, _ = hbl.hbl_kv_gather(cache, i32(pos), H, D, 16, bits)
    assert int((got != y).sum()) <= max(1, int(1e-4 * y.numel()))


# ------------------------------------------------------------------------------------------- decode

def random_cache(rng, pages, page, Hkv, D, bits, k_scale=1.0, v_scale=1.0):
    T = pages * page
    uk, uv = rng.integers(0, 1 << bits, (2, T, Hkv, D))
    gk = (k_scale * rng.uniform(0.5, 3, (T, Hkv))).astype(np.float32)
    gv = (v_scale * rng.uniform(0.1, 3, (T, Hkv))).astype(np.float32)
    return uk, uv, gk, gv


def tables_for(rng, lens, page, pages, width=None):
    need = [-(-n // page) for n in lens]
    perm = rng.permutation(pages)[:sum(need)]
    # entries past a sequence's pages are never read: fill them with numbers that are no page
    t = np.full((len(lens), max(1, max(need)) if width is None else width), 2 ** 31 - 1, np.int64)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = perm[at:at + n]
        at += n
    return t


def decode_case(lens, Hq, Hkv, D, bits, page, seed, q_scale=1.0, k_scale=1.0, gv=None, scale=None, q_pad=0, dirty=True):
    rng = np.random.default_rng(seed)
    need = sum(-(-n // page) for n in lens)
    pages = need + 2
    parts = list(random_cache(rng, pages, page, Hkv, D, bits, k_scale))
    if gv is not None:
        parts[3] = gv(rng, parts[3])
    t = tables_for(rng, lens, page, pages)
    clean = [p.copy() for p in parts]
    if dirty:  # whatever lies behind a sequence's last token must not matter
        used = np.zeros(pages * page, bool)
        for b, n in enumerate(lens):
            for j in range(n):
                used[t[b, j // page] * page + j % page] = True
        for g in parts[2:]:
            g[~used] = np.where(rng.random(g[~used].shape) < 0.5, np.nan, np.inf)
    cache = torch.from_numpy(join_records(*parts, bits, page)).cuda()
    B = len(lens)
    qb = inputs.f32_to_bf16_bits((q_scale * rng.standard_normal((B, Hq * D + q_pad))).astype(np.float32))
    Q = bf16(qb)[:, :Hq * D].view(B, Hq, D)
    scale = D ** -0.5 if scale is None else scale
    return dict(Q=Q, cache=cache, t=i32(t), lens=i32(lens), lens_host=list(lens), parts=clean, tables=t, Hq=Hq, Hkv=Hkv,
                D=D, bits=bits, page=page, scale=scale)


def run_decode(c, **kw):
    B = c["Q"].shape[0]
    lse = torch.full((B, c["Hq"]), 77.0, dtype=torch.float32, device="cuda")
    o = hbl.hbl_attn_decode(c["Q"], c["cache"], c["t"], c["lens"], c["Hkv"], c["page"], c["bits"], scale=c["scale"],
                            lse=lse, **kw)
    return o, lse


def decode_ref(c, b):
    n, page = c["lens_host"][b], c["page"]
    rows = np.array([c["tables"][b, j // page] * page + j % page for j in range(n)], np.int64)
    uk, uv, gk, gv = c["parts"]
    k = torch.from_numpy(states(uk[rows], gk[rows], c["bits"])).cuda()
    v = torch.from_numpy(states(uv[rows], gv[rows], c["bits"])).cuda()
    return k, v, attention(c["Q"][b:b + 1].double(), k, v, torch.tensor([n], device="cuda"), c["scale"])


def check_decode(c, o, lse):
    for b, n in enumerate(c["lens_host"]):
        k, v, ref = decode_ref(c, b)
        score_err, extra = 0.0, 0.0
        if n:
            # sums of D products in fp32 (16 at a time, each sum off by 2^-23 of the partial sums), of
            # codes up to L against q, then minus L sum q: together at most 3 sum|q| gamma
            q1 = c["Q"][b].double().abs().sum(-1).max()
            gmax = float(c["parts"][2][np.unique(
                [c["tables"][b, j // c["page"]] * c["page"] + j % c["page"] for j in range(n)])].max())
            score_err = float(3 * q1 * gmax * abs(c["scale"]) * (c["D"] / 16 + 4) * 2.0 ** -23)
            # weights below 2^-14 of the largest product p gamma are rounded to 2^-25 of its scale
            G = c["Hq"] // c["Hkv"]
            vm = v.abs().amax(2).amax(0).repeat_interleave(G)[None, :, None]
            extra = n * 2.0 ** -24 * vm * ref[3][..., None]
        check_close(o[b:b + 1], lse[b:b + 1], ref, 2.0 ** -11, score_err, extra)


DECODE = [
    # (lens, Hq, Hkv, D, bits, page)
    ([1], 1, 1, 64, 3, 16),
    ([0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65], 4, 4, 128, 3, 16),
    ([100, 0, 257], 8, 2, 128, 3, 32),
    ([500], 32, 32, 128, 3, 64),
    ([129, 70], 12, 4, 64, 3, 48),
    ([200, 33], 6, 2, 256, 3, 64),
    ([90, 1000], 8, 1, 128, 2, 64),
    ([77], 5, 1, 64, 2, 16),
    ([65, 300], 3, 3, 256, 2, 16),
    ([640, 12], 16, 1, 128, 4, 64),
    ([333], 24, 2, 64, 4, 128),
    ([50, 51], 4, 4, 256, 4, 32),
    ([1111], 20, 1, 128, 8, 64),
    ([48, 0], 2, 1, 64, 8, 16),
    ([260], 12, 1, 256, 8, 64),
    ([5000, 17, 2500], 8, 8, 128, 3, 64),
    ([0, 0], 4, 2, 128, 4, 16),
]


@pytest.mark.parametrize("lens,Hq,Hkv,D,bits,page", DECODE)
def test_decode_matches(lens, Hq, Hkv, D, bits, page):
    c = decode_case(lens, Hq, Hkv, D, bits, page, seed=sum(lens) + D + bits, q_pad=8 * (D == 64))
    o, lse = run_decode(c)
    check_decode(c, o, lse)
    o2, lse2 = run_decode(c)  # the same sums in the same order
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("lens,Hq,Hkv,D,bits", [([40000], 4, 2, 128, 3), ([131072], 8, 1, 128, 4),
                                               ([7] * 300, 4, 2, 64, 3), ([9000, 1] * 20, 2, 1, 256, 2)])
def test_decode_long_and_many(lens, Hq, Hkv, D, bits):
    c = decode_case(lens, Hq, Hkv, D, bits, 64, seed=5, dirty=False)
    o, lse = run_decode(c)
    check_decode(c, o, lse)


def test_decode_extreme_scales():
    def zeros(rng, g):
        g = g.copy()
        g[rng.random(g.shape) < 0.3] = 0.0
        return g

    def outliers(rng, g):
        return np.where(rng.random(g.shape) < 0.02, 1e4 * g, g).astype(np.float32)

    for name, gv in (("zeros", zeros), ("outliers", outliers), ("tiny", lambda r, g: 1e-20 * g),
                     ("huge", lambda r, g: 1e20 * g), ("all zero", lambda r, g: 0 * g),
                     ("rising", lambda r, g: np.exp2(np.linspace(-20, 20, g.size)).reshape(g.shape).astype(np.float32))):
        c = decode_case([300, 40], 4, 2, 128, 3, 16, seed=3, gv=gv)
        o, lse = run_decode(c)
        check_decode(c, o, lse)
    # sharp softmax, rising and falling scores, negative scale, zero and huge queries
    for kw in (dict(q_scale=8.0), dict(k_scale=30.0), dict(scale=-0.1), dict(q_scale=0.0), dict(q_scale=1e30, scale=1e-31),
               dict(q_scale=1e-30, scale=1e29), dict(scale=0.0)):
        c = decode_case([700, 33], 4, 2, 128, 3, 16, seed=4, **kw)
        o, lse = run_decode(c)
        check_decode(c, o, lse)


def test_decode_flags_bad_pages_and_lengths():
    c = decode_case([100, 50], 4, 2, 128, 3, 16, seed=6, dirty=False)
    assert hbl.hbl_device_status() == hbl.HBL_OK
    bad = c["t"].clone()
    bad[0, 2] = -1      # 16 tokens of sequence 0 are left out
    o = hbl.hbl_attn_decode(c["Q"], c["cache"], bad, c["lens"], 2, 16, 3)
    assert hbl.hbl_device_status() == hbl.HBL_EINVAL
    k, v, _ = decode_ref(c, 0)
    rows = torch.cat([torch.arange(32), torch.arange(48, 100)]).cuda()
    ref = attention(c["Q"][:1].double(), k[rows], v[rows], torch.tensor([84], device="cuda"), c["scale"])
    assert float((o[:1].double() - ref[0]).norm() / ref[0].norm()) < 2.0 ** -8
    width = c["t"].shape[1]
    for n in (-5, width * 16 + 1, 2 ** 31 - 1):
        lens = c["lens"].clone()
        lens[1] = n
        t = c["t"].clamp(max=c["cache"].numel() // (2 * record_bytes(128, 3)) - 1)
        o = hbl.hbl_attn_decode(c["Q"], c["cache"], t, lens, 2, 16, 3)
        assert hbl.hbl_device_status() == hbl.HBL_EINVAL, n
        if n < 0:
            assert (o[1] == 0).all()


def test_decode_captured_and_replayed_with_other_lengths():
    c = decode_case([700, 33, 250], 8, 2, 128, 3, 64, seed=8, dirty=False)
    ws = torch.empty(hbl.hbl_attn_decode_workspace(3, 8, 2, 128), dtype=torch.uint8, device="cuda").fill_(255)
    O = torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    run_decode(c, workspace=ws, O=O)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lse = torch.empty((3, 8), dtype=torch.float32, device="cuda")
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    O2, lse2 = torch.empty_like(O), torch.empty_like(lse)
    for g, o, e in ((g1, O, lse), (g2, O2, lse2)):  # two graphs on one workspace, replayed one after the other
        with torch.cuda.graph(g, stream=s):
            hbl.hbl_attn_decode(c["Q"], c["cache"], c["t"], c["lens"], 2, 64, 3, scale=c["scale"], workspace=ws, O=o,
                                lse=e)
    for lens in ([700, 33, 250], [1, 0, 249], [640, 20, 3]):
        c["lens"].copy_(i32(lens))
        c["lens_host"] = lens
        ws.random_(0, 256)
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        check_decode(c, O, lse)
        assert torch.equal(O.view(torch.int16), O2.view(torch.int16)) and torch.equal(lse, lse2)


def test_decode_on_two_streams():
    cs = [decode_case([3000, 100 + i], 8, 4, 128, 3, 64, seed=20 + i, dirty=False) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cs]
    outs = []
    torch.cuda.synchronize()
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            outs.append(run_decode(c))
    torch.cuda.synchronize()
    for c, (o, lse) in zip(cs, outs):
        check_decode(c, o, lse)


# ------------------------------------------------------------------------------------------- prompt

def prompt_case(nq, nk, Hq, Hkv, D, seed, causal=True, gap=0, q_scale=1.0, pad=0, dirty=False):
    rng = np.random.default_rng(seed)
    cq = np.cumsum([gap] + list(nq))
    ck = np.cumsum([gap] + list(nk))
    Tq, Tk = int(cq[-1]) + gap, int(ck[-1]) + gap

    def rows(T, H, scale=1.0):
        x = (scale * rng.standard_normal((T, H * D + pad))).astype(np.float32)
        return bf16(inputs.f32_to_bf16_bits(x))[:, :H * D].unflatten(1, (H, D))

    Q, K, V = rows(Tq, Hq, q_scale), rows(Tk, Hkv), rows(Tk, Hkv)
    if dirty:  # rows of no sequence
        for x, cu in ((Q, cq), (K, ck), (V, ck)):
            x[:cu[0]] = float("nan")
            x[cu[-1]:] = float("inf")
    return dict(Q=Q, K=K, V=V, cq=cq, ck=ck, causal=causal, scale=D ** -0.5, D=D)


def run_prompt(c, **kw):
    O = torch.full(c["Q"].shape, 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(c["Q"].shape[:2], 9.0, dtype=torch.float32, device="cuda")
    hbl.hbl_attn_prompt(c["Q"], c["K"], c["V"], i32(c["cq"]), i32(c["ck"]), scale=c["scale"], causal=c["causal"], O=O,
                        lse=lse, **kw)
    return O, lse


def check_prompt(c, O, lse, only=None):
    for b in range(len(c["cq"]) - 1) if only is None else only:
        q = c["Q"][c["cq"][b]:c["cq"][b + 1]].double()
        k, v = (x[c["ck"][b]:c["ck"][b + 1]].double() for x in (c["K"], c["V"]))
        nq, nk = q.shape[0], k.shape[0]
        seen = torch.arange(nq, device="cuda") + 1 + nk - nq if c["causal"] else torch.full((nq,), nk, device="cuda")
        ref = attention(q, k, v, seen.clamp(0, nk), c["scale"])
        err = 0.0
        if nq and nk:
            err = float((q.abs().sum(-1).max() * k.abs().max()) * abs(c["scale"]) * (c["D"] / 16 + 4) * 2.0 ** -23)
        sl = slice(int(c["cq"][b]), int(c["cq"][b + 1]))
        check_close(O[sl], lse[sl], ref, 2.0 ** -8, err)
    for sl in (slice(0, int(c["cq"][0])), slice(int(c["cq"][-1]), None)):  # rows of no sequence
        assert (O[sl] == 9).all() and (lse[sl] == 9).all()
    assert hbl.hbl_device_status() == hbl.HBL_OK


PROMPT = [
    # (nq, nk (None: the same), Hq, Hkv, D, causal)
    ([1], None, 1, 1, 64, True),
    ([1, 2, 3], None, 4, 2, 128, True),
    ([127, 128, 129], None, 4, 4, 128, True),
    ([17, 120, 64], None, 32, 8, 128, True),
    ([255, 256, 257], None, 3, 1, 64, True),
    ([300], None, 2, 2, 256, True),
    ([130, 5, 260], None, 6, 2, 256, True),
    ([1000, 1, 513], None, 4, 1, 128, True),
    ([385], None, 5, 5, 128, True),
    ([64, 1, 100], [300, 700, 100], 8, 2, 128, True),    # cached prefixes
    ([1, 1, 1, 1], [1, 129, 400, 64], 8, 8, 128, True),  # single queries
    ([40, 200], [513, 1025], 4, 2, 64, True),
    ([33, 140], [290, 700], 2, 1, 256, True),
    ([50, 200], [20, 0], 4, 2, 128, True),               # more queries than keys: rows that see nothing
    ([5, 0, 9], [0, 30, 9], 2, 2, 64, True),
    ([300, 20], [7, 3], 2, 1, 256, True),
    ([100, 300], None, 4, 2, 128, False),
    ([10, 129], [200, 77], 4, 4, 64, False),
    ([3, 150], [0, 130], 2, 2, 256, False),
    ([3, 7, 0, 1, 2, 40] * 9, None, 4, 2, 128, True),
]


@pytest.mark.parametrize("nq,nk,Hq,Hkv,D,causal", PROMPT)
def test_prompt_matches(nq, nk, Hq, Hkv, D, causal):
    c = prompt_case(nq, nq if nk is None else nk, Hq, Hkv, D, seed=sum(nq) + D, causal=causal, gap=5, dirty=True,
                    pad=8 * (len(nq) % 2))
    O, lse = run_prompt(c, max_q=max(nq))
    check_prompt(c, O, lse)
    O2, lse2 = run_prompt(c)  # the default bound, and the same sums
    assert torch.equal(O.view(torch.int16), O2.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("D,Hq,Hkv,n", [(128, 4, 1, 4096), (64, 3, 3, 3001), (256, 2, 1, 2500)])
def test_prompt_long(D, Hq, Hkv, n):
    c = prompt_case([n], [n + 333], Hq, Hkv, D, seed=n)
    check_prompt(c, *run_prompt(c))


def test_prompt_neighbours_do_not_leak():
    # NaN and infinities everywhere in one sequence's states: the others' results as without it
    nq, nk = [70, 90, 110], [130, 200, 110]
    c = prompt_case(nq, nk, 4, 2, 128, seed=1)
    for x, cu in ((c["Q"], c["cq"]), (c["K"], c["ck"]), (c["V"], c["ck"])):
        x[cu[1]:cu[2]] = float("nan")
        x[cu[1]] = float("inf")
    O, lse = run_prompt(c)
    check_prompt(c, O, lse, only=[0, 2])


def test_prompt_scales():
    for kw, scale in ((dict(q_scale=8.0), None), (dict(q_scale=100.0), None), (dict(q_scale=0.0), None),
                      (dict(), -0.2), (dict(), 0.0)):
        c = prompt_case([200, 31], [333, 31], 4, 2, 128, seed=2, **kw)
        if scale is not None:
            c["scale"] = scale
        check_prompt(c, *run_prompt(c))


def test_prompt_flags_bad_borders_and_bounds():
    c = prompt_case([100, 100], [100, 100], 2, 1, 128, seed=7)
    for name, cu in (("cq", [0, 100, 250]), ("ck", [0, 100, 201]), ("ck", [0, 150, 100]), ("cq", [-4, 100, 200]),
                     ("cq", [0, 120, 100])):
        d = dict(c)
        d[name] = np.array(cu)
        run_prompt(d)
        assert hbl.hbl_device_status() == hbl.HBL_EINVAL, (name, cu)
    O, lse = run_prompt(c, max_q=64)  # queries past the bound are left out
    assert hbl.hbl_device_status() == hbl.HBL_EINVAL
    assert (O[64:100] == 9).all() and (O[:64] != 9).any()


def test_prompt_captured_and_replayed():
    c = prompt_case([150, 90], [150, 190], 4, 2, 128, seed=9)
    cq, ck = i32(c["cq"]), i32(c["ck"])
    O = torch.full(c["Q"].shape, 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(c["Q"].shape[:2], 9.0, dtype=torch.float32, device="cuda")
    run_prompt(c)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hbl.hbl_attn_prompt(c["Q"], c["K"], c["V"], cq, ck, scale=c["scale"], O=O, lse=lse)
    for bq, bk in (([0, 150, 240], [0, 150, 340]), ([0, 10, 240], [0, 100, 340]), ([0, 240, 240], [0, 340, 340])):
        c["cq"], c["ck"] = np.array(bq), np.array(bk)
        cq.copy_(i32(bq))
        ck.copy_(i32(bk))
        g.replay()
        torch.cuda.synchronize()
        check_prompt(c, O, lse)


# ----------------------------------------------------------------------------------- all of them together

@pytest.mark.parametrize("bits,Hq,Hkv,D", [(3, 4, 4, 128), (4, 8, 2, 64), (2, 2, 1, 256)])
def test_a_block_from_qkv_to_wo(bits, Hq, Hkv, D):
    """Prompts, then new tokens one by one, through the projections, the cache and the attention: each
    step's attention against 64 bits on the same projections, its cache rows against the oracle."""
    rng = np.random.default_rng(bits)
    hidden, page = 512, 16
    nqkv = (Hq + 2 * Hkv) * D
    wqkv, a1 = hbl.hbl_pack_weights(torch.from_numpy(rng.standard_normal((hidden, nqkv)).astype(np.float32)).cuda())
    wo, a2 = hbl.hbl_pack_weights(torch.from_numpy(rng.standard_normal((Hq * D, hidden)).astype(np.float32)).cuda())
    lens = [37, 5, 64]
    steps = 20
    width = max(-(-(n + steps) // page) for n in lens)
    tables = rng.permutation(len(lens) * width + 1)[:len(lens) * width].reshape(len(lens), width)
    cache = torch.empty(hbl.hbl_kv_cache_bytes(len(lens) * width + 1, page, Hkv, D, bits), dtype=torch.uint8,
                        device="cuda").fill_(255)
    past = [[] for _ in lens]  # the oracle's K~, V~ of each sequence

    def project(x):
        y = hbl.hbl_forward(x, wqkv, a1, nqkv, had_block=1, out_dtype=hbl.HBL_OUT_BF16)
        q, k, v = y[:, :Hq * D], y[:, Hq * D:(Hq + Hkv) * D], y[:, (Hq + Hkv) * D:]
        return [z.unflatten(1, (-1, D)) for z in (q, k, v)]

    def remember(b, k, v, pos):
        for x, p in ((k, pos), (v, None)):
            u, g = quantise(x, p, bits)
            yield states(u, g.astype(np.float32), bits)

    def to_bits(t):
        return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)

    def step(q_lens, start):
        T = sum(q_lens)
        x = bf16(inputs.f32_to_bf16_bits(rng.standard_normal((T, hidden)).astype(np.float32)))
        Q, K, V = project(x)
        pos = np.concatenate([np.arange(s, s + n) for s, n in zip(start, q_lens)])
        seq = np.repeat(np.arange(len(lens)), q_lens)
        slots = tables[seq, pos // page] * page + pos % page
        Qr = hbl.hbl_kv_append(K, V, i32(slots), cache, page, bits, pos=i32(pos), Q=Q)
        if max(q_lens) > 1:
            Kd, Vd = hbl.hbl_kv_gather(cache, i32(slots), Hkv, D, page, bits)
            cu = i32(np.cumsum([0] + q_lens))
            lse = torch.empty((T, Hq), dtype=torch.float32, device="cuda")
            O = hbl.hbl_attn_prompt(Qr, Kd, Vd, cu, cu, max_q=max(q_lens), lse=lse)
        else:
            lse = torch.empty((T, Hq), dtype=torch.float32, device="cuda")
            O = hbl.hbl_attn_decode(Qr, cache, i32(tables), i32(np.array(start) + 1), Hkv, page, bits, lse=lse)
        kb, vb = to_bits(K), to_bits(V)
        at = 0
        for b, (n, s) in enumerate(zip(q_lens, start)):
            past[b].append(list(remember(b, kb[at:at + n], vb[at:at + n], pos[at:at + n])))
            k, v = (torch.from_numpy(np.concatenate([p[i] for p in past[b]])).cuda() for i in (0, 1))
            q = Qr[at:at + n].double()
            prompt = max(q_lens) > 1
            if prompt:
                # the attention reads K~ and V~ as bf16. gamma's 2^-21 can move a value to the other side of
                # a bf16 boundary, a whole step, so the 64-bit attention takes the bf16 values that were read
                # back, and those are held to the states by themselves
                for x, y in ((k, Kd[at:at + n].double()), (v, Vd[at:at + n].double())):
                    far = (x - y).abs() > (2.0 ** -8 + 2.0 ** -20) * x.abs() + 1e-30
                    assert not far.any(), (int(far.sum()), x[far][:4].tolist(), y[far][:4].tolist(), far.nonzero()[:4].tolist())
                k, v = Kd[at:at + n].double(), Vd[at:at + n].double()
            ref = attention(q, k, v, torch.arange(s, s + n, device="cuda") + 1, D ** -0.5)
            # gamma is off by 2^-21 at most; sums as in check_decode
            most = float(q.abs().sum(-1).max() * k.abs().max()) * D ** -0.5
            err = most * (3 * (D / 16 + 4) * 2.0 ** -23 + 2.0 ** -20)
            extra = (s + n) * 2.0 ** -24 * v.abs().max() * ref[3].max()
            check_close(O[at:at + n], lse[at:at + n], ref, 2.0 ** -8 if prompt else 2.0 ** -11, err, float(extra))
            at += n
        Y = hbl.hbl_forward(O.view(T, Hq * D), wo, a2, hidden, out_dtype=hbl.HBL_OUT_BF16)
        assert torch.isfinite(Y.float()).all()

    step(lens, [0] * len(lens))
    for i in range(steps):
        step([1] * len(lens), [n + i for n in lens])
    assert hbl.hbl_device_status() == hbl.HBL_OK


# ------------------------------------------------------------------------- corners of the fast paths

@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("rope", [True, False])
def test_append_borders_and_zeros(bits, rope):
    """Heads whose values lie on the codes' borders, just beside them, or are all zero: with a largest value
    7 * 15 * 255 / 2^k-like, every multiple of gamma / L is a bf16 number."""
    D, page, T, H = 128, 16, 64, 2
    L = (1 << bits) - 1
    rng = np.random.default_rng(bits)
    x = np.zeros((T, 2 * H, D), np.float32)
    for t in range(T):
        for h in range(2 * H):
            unit = 2.0 ** rng.integers(-3, 4)
            if t % 4 == 0:      # borders: x = gamma m / L, gamma = L unit
                x[t, h] = unit * rng.integers(-L, L + 1, D)
            elif t % 4 == 1:    # one bf16 step beside them
                x[t, h] = unit * rng.integers(-L, L + 1, D) * (1 + rng.choice([-1, 1], D) * 2.0 ** -8)
            elif t % 4 == 2:    # next to the middle border
                x[t, h] = unit * rng.choice([-1, 1], D) * 2.0 ** rng.integers(-40, 0, D)
            if t % 4 != 3:
                x[t, h, rng.integers(D)] = L * unit * (1 if t % 8 < 4 else -1)
    b = inputs.f32_to_bf16_bits(x.reshape(T, -1)).reshape(T, 2 * H, D)
    X = bf16(b)
    pos = np.where(rng.random(T) < 0.5, 0, rng.integers(0, 5000, T)) if rope else None
    cache = torch.zeros(hbl.hbl_kv_cache_bytes(T // page, page, H, D, bits), dtype=torch.uint8, device="cuda")
    hbl.hbl_kv_append(X[:, :H], X[:, H:], i32(np.arange(T)), cache, page, bits, pos=None if pos is None else i32(pos))
    uk, uv, gk, gv = split_records(cache.cpu().numpy(), H, D, bits, page)
    for u, g, xs, p in ((uk, gk, b[:, :H], pos), (uv, gv, b[:, H:], None)):
        ru, rg = quantise(xs, p, bits)
        np.testing.assert_array_equal(u, ru)
        np.testing.assert_allclose(g, rg, rtol=2.0 ** -21)


def test_cache_past_4_gib():
    # the same tokens in the last pages of a cache of more than 4 GiB and in a small one
    Hkv, D, bits, page, n = 8, 128, 8, 64, 150
    need = -(-n // page)
    pages = (5 << 30) // hbl.hbl_kv_cache_bytes(1, page, Hkv, D, bits)
    big = torch.empty(hbl.hbl_kv_cache_bytes(pages, page, Hkv, D, bits), dtype=torch.uint8, device="cuda")
    small = torch.empty(hbl.hbl_kv_cache_bytes(need, page, Hkv, D, bits), dtype=torch.uint8, device="cuda")
    assert big.numel() > 1 << 32
    _, _, (Q, K, V) = fused_states(n, 16, Hkv, D, seed=2)
    out = []
    for cache, first in ((big, pages - need), (small, 0)):
        slots = i32(first * page + np.arange(n))
        hbl.hbl_kv_append(K, V, slots, cache, page, bits, pos=i32(np.arange(n)))
        table = i32(first + np.arange(need)[None])
        lse = torch.empty((1, 16), dtype=torch.float32, device="cuda")
        o = hbl.hbl_attn_decode(Q[:1], cache, table, i32([n]), Hkv, page, bits, lse=lse)
        out.append((*hbl.hbl_kv_gather(cache, slots, Hkv, D, page, bits), o, lse))
    for a, b in zip(*out):
        assert torch.equal(a, b) and torch.isfinite(a.float()).all()
    assert hbl.hbl_device_status() == hbl.HBL_OK


def test_decode_wide_range_of_v_scales():
    def mixed(low, high):
        return lambda rng, g: np.where(rng.random(g.shape) < 0.3, high * g, low * g).astype(np.float32)

    for low, high in ((1.0, 1e25), (1e-12, 1e12), (1e-35, 1e-30), (1e30, 1e36)):
        c = decode_case([500, 77], 8, 2, 128, 3, 32, seed=12, gv=mixed(low, high))
        check_decode(c, *run_decode(c))


@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 9, 16, 17, 40])
def test_decode_group_sizes(G):
    for D, bits in ((64, 4), (128, 3), (256, 2)):
        c = decode_case([333, 0, 64, 1], 2 * G, 2, D, bits, 64, seed=G)
        check_decode(c, *run_decode(c))


def test_outputs_at_16_byte_offsets():
    c = prompt_case([200, 31], [200, 231], 4, 2, 128, seed=5)
    ref, _ = run_prompt(c)
    O = torch.empty(ref.numel() + 8, dtype=torch.bfloat16, device="cuda")[8:].view(ref.shape)
    hbl.hbl_attn_prompt(c["Q"], c["K"], c["V"], i32(c["cq"]), i32(c["ck"]), O=O)
    assert torch.equal(O, ref)
    d = decode_case([70], 2, 1, 64, 4, 16, seed=5, dirty=False)
    K, V = hbl.hbl_kv_gather(d["cache"], i32(np.arange(48)), 1, 64, 16, 4)
    buf = torch.empty(2 * (K.numel() + 8), dtype=torch.bfloat16, device="cuda")
    k, v = buf[8:8 + K.numel()].view(K.shape), buf[K.numel() + 16:].view(K.shape)
    hbl.hbl_kv_gather(d["cache"], i32(np.arange(48)), 1, 64, 16, 4, K=k, V=v)
    assert torch.equal(k, K) and torch.equal(v, V)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompt_rising_and_falling_scores(D):
    # keys that grow from block to block move the running maximum again and again; shrinking ones never
    for order in (1, -1):
        c = prompt_case([140, 300], [1500, 300], 4, 2, D, seed=D)
        for b in range(2):
            n = int(c["ck"][b + 1] - c["ck"][b])
            ramp = torch.linspace(0.1, 30.0, n, device="cuda")[::1 if order > 0 else 1]
            ramp = ramp if order > 0 else ramp.flip(0)
            c["K"][c["ck"][b]:c["ck"][b + 1]] *= ramp[:, None, None].to(torch.bfloat16)
        check_prompt(c, *run_prompt(c))


def test_prompt_many_sequences():
    rng = np.random.default_rng(0)
    nq = rng.integers(0, 9, 700)
    nk = nq + rng.integers(0, 3, 700) * rng.integers(0, 40, 700)
    nq[300], nk[300] = 700, 900
    for causal in (True, False):
        c = prompt_case(nq, nk, 2, 1, 64, seed=3, causal=causal)
        check_prompt(c, *run_prompt(c))


def test_calls_on_several_streams_at_once():
    ps = [prompt_case([700 + i, 65], [900 + i, 65], 8, 2, 128, seed=30 + i) for i in range(3)]
    ds = [decode_case([2000 + i, 5], 8, 2, 128, 3, 64, seed=40 + i, dirty=False) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(5)]
    outs = []
    torch.cuda.synchronize()
    for _ in range(3):
        outs.clear()
        for c, s in zip(ps + ds, streams):
            with torch.cuda.stream(s):
                outs.append(run_prompt(c) if "cq" in c else run_decode(c))
    torch.cuda.synchronize()
    for c, (o, lse) in zip(ps + ds, outs):
        (check_prompt if "cq" in c else check_decode)(c, o, lse)


def test_calls_on_a_given_stream():
    c = decode_case([300], 4, 2, 128, 3, 64, seed=1, dirty=False)
    ref = run_decode(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(hbl.hbl_attn_decode_workspace(1, 4, 2, 128), dtype=torch.uint8, device="cuda")
    O = torch.empty((1, 4, 128), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        O.zero_()
        torch.cuda.synchronize()
        run_decode(c, O=O, workspace=ws, stream=stream)
        s.synchronize()
        assert torch.equal(O, ref[0])


def test_binding_refuses_mixed_tensors():
    c = decode_case([40], 4, 2, 128, 3, 16, seed=1, dirty=False)
    p = prompt_case([30], [30], 4, 2, 128, seed=1)
    cq, ck = i32(p["cq"]), i32(p["ck"])
    for f in (lambda: hbl.hbl_attn_decode(c["Q"], c["cache"].cpu(), c["t"], c["lens"], 2, 16, 3),
              lambda: hbl.hbl_attn_decode(c["Q"], c["cache"], c["t"].long(), c["lens"], 2, 16, 3),
              lambda: hbl.hbl_attn_decode(c["Q"], c["cache"], c["t"], c["lens"], 2, 16, 3, O=c["Q"].float()),
              lambda: hbl.hbl_attn_prompt(p["Q"], p["K"], p["V"], cq.cpu(), ck),
              lambda: hbl.hbl_attn_prompt(p["Q"], p["K"], p["V"], cq, ck[:1]),
              lambda: hbl.hbl_attn_prompt(p["Q"].transpose(0, 1), p["K"], p["V"], cq, ck)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(hbl.HblError):  # a workspace that is too small
        hbl.hbl_attn_decode(c["Q"], c["cache"], c["t"], c["lens"], 2, 16, 3,
                            workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_given_stream_owns_what_a_call_allocates():
    """Outputs and workspaces of calls on a given stream belong to it: work and allocations that follow at
    once on the current stream leave them alone."""
    c = decode_case([3000, 500], 8, 2, 128, 3, 64, seed=2, dirty=False)
    p = prompt_case([1500], [1500], 8, 2, 128, seed=2)
    ref_d, ref_p = run_decode(c)[0], run_prompt(p)[0]
    slots = i32(np.arange(64))
    ref_k, _ = hbl.hbl_kv_gather(c["cache"], slots, 2, 128, 64, 3)
    s = torch.cuda.Stream()
    cq, ck = i32(p["cq"]), i32(p["ck"])
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        for _ in range(5):
            o = hbl.hbl_attn_decode(c["Q"], c["cache"], c["t"], c["lens"], 2, 64, 3, scale=c["scale"], stream=stream)
            q = hbl.hbl_attn_prompt(p["Q"], p["K"], p["V"], cq, ck, stream=stream)
            k, _ = hbl.hbl_kv_gather(c["cache"], slots, 2, 128, 64, 3, stream=stream)
            for n in (hbl.hbl_attn_decode_workspace(2, 8, 2, 128), o.numel() * 2, q.numel() * 2):
                torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
            torch.cuda.synchronize()
            assert torch.equal(o, ref_d) and torch.equal(q, ref_p) and torch.equal(k, ref_k)
