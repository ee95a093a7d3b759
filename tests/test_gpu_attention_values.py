"""The low-bit cache and the attention over it at values where they can go wrong: NaN and infinities, a
dominant token beside very many small ones, far positions, equal tokens in calls of other sizes."""
import numpy as np
import pytest
import torch

import hadamard_bit_quant_hbl_b200 as hbl
from attn_check import check_rows
from attn_ref import attention, join_records, record_bytes, states
from test_gpu_attention import (bf16, decode_case, decode_ref, fused_states, i32, prompt_case, run_decode,  # noqa: F401
                                run_prompt, _gpu)

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


# ------------------------------------------------------------------------------------------- prompt

def prompt_rows(c, O, lse, b):
    """Sequence b of a prompt case against 64 bits, NaN and all."""
    q = c["Q"][c["cq"][b]:c["cq"][b + 1]].double()
    k, v = (x[c["ck"][b]:c["ck"][b + 1]].double() for x in (c["K"], c["V"]))
    nq, nk = q.shape[0], k.shape[0]
    seen = torch.arange(nq, device="cuda") + 1 + nk - nq if c["causal"] else torch.full((nq,), nk, device="cuda")
    ref = list(attention(q, k, v, seen.clamp(0, nk), c["scale"]))
    ref[1] = torch.where(torch.isposinf(ref[1]), NAN, ref[1])  # log sum exp(s - max) + max: inf - inf, as in the weights
    fin = lambda x: torch.where(torch.isfinite(x), x, 0.0).abs()
    err = 0.0
    if nq and nk:
        err = float(fin(q).sum(-1).max() * fin(k).max()) * abs(c["scale"]) * (c["D"] / 16 + 4) * 2.0 ** -23
    sl = slice(int(c["cq"][b]), int(c["cq"][b + 1]))
    check_rows(O[sl], lse[sl], ref, 2.0 ** -8, err)
    return ref


@pytest.mark.parametrize("D,Hq,Hkv,causal", [(64, 3, 3, True), (128, 4, 2, True), (256, 2, 1, True), (128, 8, 1, False),
                                             (64, 2, 1, False)])
def test_prompt_keeps_nan(D, Hq, Hkv, causal):
    """NaN in a query makes that query's head NaN; NaN in a key makes every query that sees it NaN. Neither
    looks like a query that sees no key, and no other row changes."""
    c = prompt_case([70, 200, 5], [70, 450, 0], Hq, Hkv, D, seed=D + Hq, causal=causal)
    a = int(c["cq"][1])
    c["Q"][3, 0, 5] = NAN
    c["Q"][a + 150, Hq - 1] = NAN
    c["K"][int(c["ck"][1]) + 300, Hkv - 1, 7] = NAN  # the queries from 50 on see it when causal
    O, lse = run_prompt(c)
    refs = [prompt_rows(c, O, lse, b) for b in range(3)]
    assert torch.isnan(refs[0][1]).sum() == 1 and torch.isnan(refs[1][1]).sum() >= 150
    assert torch.isneginf(refs[2][1]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompt_infinite_scores(D):
    """A score of +inf is NaN after the softmax (inf - inf), one of -inf a weight of 0."""
    c = prompt_case([150], [400], 2, 1, D, seed=D)
    c["Q"][:, :, 0] = c["Q"][:, :, 0].abs() + 0.5
    c["Q"][:, 1, 0] *= -1
    c["K"][290, 0, 0] = -INF  # the first head's queries from 40 on give it no weight, the second's are NaN
    O, lse = run_prompt(c)
    ref = prompt_rows(c, O, lse, 0)
    assert not torch.isnan(ref[1][:, 0]).any() and torch.isnan(ref[1][:, 1]).sum() == 110


# ------------------------------------------------------------------------------------------- decode

def decode_rows(c, o, lse, b):
    """Sequence b of a decode case against 64 bits, NaN and all."""
    n, page = c["lens_host"][b], c["page"]
    k, v, ref = decode_ref(c, b)
    fin = lambda x: torch.where(torch.isfinite(x), x, 0.0).abs()
    score_err, extra = 0.0, 0.0
    if n:
        # as in test_gpu_attention.check_decode: sums of D products of codes and q, then minus L sum q
        score_err = float(3 * fin(c["Q"][b].double()).sum(-1).max() * fin(k).max() * abs(c["scale"]) *
                          (c["D"] / 16 + 4) * 2.0 ** -23)
        # weights below fp16's normal range are off by half its smallest step, 2^-25 where the largest product
        # p gamma is 2^6 at least
        rows = [c["tables"][b, j // page] * page + j % page for j in range(n)]
        g = fin(torch.from_numpy(c["parts"][3][rows].astype(np.float64)).cuda()).amax(0)
        extra = n * 2.0 ** -31 * g.repeat_interleave(c["Hq"] // c["Hkv"])[None, :, None] * \
            torch.nan_to_num(ref[3][..., None], nan=0.0)
    # a lane adds the weights of its tokens, an eighth of a warp's, one after another: each sum is off by half a
    # step, 2^-24 of it (a dominant token's lane drops all that lies below)
    check_rows(o[b:b + 1], lse[b:b + 1], ref, 2.0 ** -11, score_err, extra, n / 8 * 2.0 ** -24)
    return ref


def with_records(c, change):
    """The case with its cache's codes and scales changed in place by change(uk, uv, gk, gv, rows of sequence b)."""
    page = c["page"]

    def rows(b):
        return np.array([c["tables"][b, j // page] * page + j % page for j in range(c["lens_host"][b])], np.int64)

    change(*c["parts"], rows)
    c["cache"] = torch.from_numpy(join_records(*c["parts"], c["bits"], page)).cuda()
    return c


@pytest.mark.parametrize("Hq,Hkv,D,bits", [(2, 2, 128, 3), (4, 2, 64, 2), (8, 2, 128, 4), (10, 2, 128, 8), (24, 2, 64, 3),
                                           (6, 2, 256, 3)])
@pytest.mark.parametrize("n", [40, 5000])
def test_decode_keeps_nan(Hq, Hkv, D, bits, n):
    """NaN in q, in a K scale or in a V scale: the same answer whether one warp holds the sequence or many."""
    c = decode_case([n, n, n, n], Hq, Hkv, D, bits, 16, seed=n + D, dirty=False)
    c["Q"][0, Hq - 1, 3] = NAN
    c["Q"][0, 0] = NAN

    def change(uk, uv, gk, gv, rows):
        gk[rows(1)[n // 2], Hkv - 1] = NAN
        gv[rows(2)[n // 3], 0] = NAN

    with_records(c, change)
    o, lse = run_decode(c)
    refs = [decode_rows(c, o, lse, b) for b in range(4)]
    G = Hq // Hkv
    assert torch.isnan(refs[0][1]).sum() == 2
    assert torch.isnan(refs[1][1]).sum() == G
    assert not torch.isnan(refs[2][1]).any() and torch.isnan(refs[2][0]).sum() == G * D
    assert hbl.hbl_device_status() == hbl.HBL_OK


@pytest.mark.parametrize("D,bits", [(128, 3), (64, 8), (128, 4)])
def test_decode_long_pieces(D, bits):
    """Sums over very many tokens: with as many sequences as warps, over the same pages, a warp holds 131072."""
    c = decode_case([131072], 1, 1, D, bits, 64, seed=D + bits, dirty=False)
    B = 1776
    many = dict(c, Q=c["Q"].expand(B, 1, D).contiguous(), t=c["t"].expand(B, -1).contiguous(),
                lens=c["lens"].expand(B).contiguous())
    o, lse = run_decode(many)
    for b in (0, 700, 1775):
        decode_rows(c, o[b:b + 1], lse[b:b + 1], 0)


def dominant_case(n, below, bits=8, copies=1776):
    """`copies` equal sequences over the same pages, so that a warp holds long pieces: n tokens whose weights are
    2^-below of one more token's, which has the middle code (1/L of gamma) in its V where the others have gamma."""
    D, page = 64, 64
    L = (1 << bits) - 1
    T = -(-(n + 1) // page) * page
    uk = np.full((T, 1, D), L, np.int64)
    uv = np.full((T, 1, D), L, np.int64)
    uv[0] = (L + 1) // 2
    gk = np.full((T, 1), 0.125, np.float32)
    gk[0] = 0.125 + below * np.log(2.0) / 8  # score = gammaK * 64 / 8 at q = 1
    gv = np.ones((T, 1), np.float32)
    table = np.repeat(np.arange(T // page)[None], copies, 0)
    Q = torch.ones((copies, 1, D), dtype=torch.bfloat16, device="cuda")
    return dict(Q=Q, cache=torch.from_numpy(join_records(uk, uv, gk, gv, bits, page)).cuda(), t=i32(table),
                lens=i32([n + 1] * copies), lens_host=[n + 1] * copies, parts=[uk, uv, gk, gv], tables=table, Hq=1, Hkv=1,
                D=D, bits=bits, page=page, scale=0.125)


@pytest.mark.parametrize("n,below", [(131071, 25.05), (131071, 24.8), (65535, 23.3), (131071, 20.0)])
def test_decode_small_weights_beside_a_dominant_one(n, below):
    """What very many small weights add up to: 2^-25 of the largest each, they come to as much as the
    dominant token's own output. A weight is off by 2^-31 of the largest at most."""
    c = dominant_case(n, below)
    o, lse = run_decode(c)
    assert (o == o[0]).all() or float((o - o[0]).abs().max()) < 2.0 ** -8 * float(o[0].abs().max())
    for b in (0, 1, 888, 1775):
        decode_rows(c, o, lse, b)


def test_decode_norms_at_scaled_values():
    """The norm of the error in the outputs' own scale, whatever V's."""
    for low, high in ((1e-20, 1e-20), (1e20, 1e20), (1.0, 1e25), (1e30, 1e36), (1e-12, 1e12)):
        c = decode_case([500, 77], 8, 2, 128, 3, 32, seed=14, dirty=False, gv=lambda rng, g: np.where(
            rng.random(g.shape) < 0.3, high * g, low * g).astype(np.float32))
        o, lse = run_decode(c)
        for b in range(2):
            decode_rows(c, o, lse, b)


# ------------------------------------------------------------------------------------------- append

def k_bytes(cache, Hkv, D, page):
    """K codes [tokens, Hkv, D] at eight bits (a byte each) and the scales [tokens, Hkv], in slot order."""
    rec = cache.view(-1, Hkv, page // 16, record_bytes(D, 8)).transpose(1, 2).reshape(-1, Hkv, record_bytes(D, 8))
    k = rec[:, :, :16 * D].view(-1, Hkv, 16, D).transpose(1, 2).reshape(-1, Hkv, D)
    g = rec[:, :, 32 * D:32 * D + 64].contiguous().view(torch.float32).transpose(1, 2).reshape(-1, Hkv)
    return k.cpu().numpy(), g.cpu().numpy()


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 5, 7), (128, 4, 8), (128, 3, 5), (256, 2, 2)])
@pytest.mark.parametrize("bits", [3, 8])
def test_append_does_not_depend_on_the_call(D, Hq, Hkv, bits):
    """A token's record is the same in one long prompt, in pieces of it and alone: heads share a warp with
    other heads there."""
    T, page = 2700, 16
    _, _, (Q, K, V) = fused_states(T, Hq, Hkv, D, seed=D + bits)
    pos = i32(np.random.default_rng(1).integers(0, 100000, T))
    slots = i32(np.arange(T))
    size = hbl.hbl_kv_cache_bytes(-(-T // page), page, Hkv, D, bits)
    caches = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(3)]
    hbl.hbl_kv_append(K, V, slots, caches[0], page, bits, pos=pos, Q=Q)
    for a in range(0, T, 90):
        hbl.hbl_kv_append(K[a:a + 90], V[a:a + 90], slots[a:a + 90], caches[1], page, bits, pos=pos[a:a + 90])
    for a in range(T):
        hbl.hbl_kv_append(K[a:a + 1], V[a:a + 1], slots[a:a + 1], caches[2], page, bits, pos=pos[a:a + 1], Q=Q[a:a + 1])
    for cache in caches[1:]:
        assert int((cache != caches[0]).sum()) == 0


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 3, 5), (128, 2, 3), (256, 1, 2)])
@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("rope", [True, False])
def test_append_marks_heads_that_are_not_finite(D, Hq, Hkv, bits, rope):
    """A head with a NaN or an infinity gets the scale NaN: it reads back as NaN and makes the attention over
    it NaN. The records of the heads around it are those without it."""
    T, page = 40, 16
    X, _, (Q, K, V) = fused_states(T, Hq, Hkv, D, seed=D + bits)
    pos = i32(np.arange(T) * 17) if rope else None
    size = hbl.hbl_kv_cache_bytes(3, page, Hkv, D, bits)
    want, got = (torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2))
    hbl.hbl_kv_append(K, V, i32(np.arange(T)), want, page, bits, pos=pos, Q=Q)
    bad = {}  # (which, token, head)
    for i, (t, value, where) in enumerate([(0, NAN, slice(3, 4)), (5, INF, slice(D - 1, D)), (15, -INF, slice(0, 1)),
                                           (16, NAN, slice(None)), (31, INF, slice(None)), (39, NAN, slice(D // 2, None))]):
        for x, which in ((K, 0), (V, 1)):
            h = (i + which) % Hkv
            x[t, h, where] = value
            bad[which, t, h] = True
    hbl.hbl_kv_append(K, V, i32(np.arange(T)), got, page, bits, pos=pos, Q=Q)
    back, ref = (hbl.hbl_kv_gather(c, i32(np.arange(T)), Hkv, D, page, bits) for c in (got, want))
    for which in (0, 1):
        nan = torch.zeros((T, Hkv), dtype=torch.bool, device="cuda")
        for w, t, h in bad:
            if w == which:
                nan[t, h] = True
        assert torch.isnan(back[which][nan]).all()
        assert torch.equal(back[which][~nan], ref[which][~nan])
        # the scales, as they lie: NaN there and nowhere else
        rec = got.view(-1, Hkv, 1, record_bytes(D, bits))[:, :, 0, 4 * D * bits + 64 * which:][:, :, :64]
        g = rec.contiguous().view(torch.float32).transpose(1, 2).reshape(-1, Hkv)[:T]
        assert torch.equal(torch.isnan(g), nan)
    table = i32(np.arange(3)[None].repeat(2, 0))
    q = torch.randn(2, Hkv, D, device="cuda").to(torch.bfloat16)
    o = hbl.hbl_attn_decode(q, got, table, i32([T, 0]), Hkv, page, bits)
    some = [any((w, t, h) in bad for w in (0, 1) for t in range(T)) for h in range(Hkv)]
    for h in range(Hkv):
        assert bool(torch.isnan(o[0, h]).all()) == some[h] and (o[1, h] == 0).all()
    assert hbl.hbl_device_status() == hbl.HBL_OK


def turned(x, pos, D, theta):
    """RoPE in extended precision (a significand of 64 bits) of x [T, H, D]."""
    half = D // 2
    inv = np.longdouble(theta) ** (-2 * np.arange(half).astype(np.longdouble) / D)
    ang = pos.astype(np.longdouble)[:, None] * inv
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = x[..., :half].astype(np.longdouble), x[..., half:].astype(np.longdouble)
    return np.concatenate([a * c - b * s, a * s + b * c], -1), ang.astype(np.float64)


def check_codes(u, g, x, pos, D, theta):
    """Eight-bit codes and scales of x [T, H, D]. The angle of pair f is off by a step of theta^(-2f/D) in 64 bits
    and half a step of its product, together 3/2 2^-52 of it (nothing at f = 0, where both are exact), and by
    2^-49 for its reduction; a state moves by 2 gamma times that, and so does gamma. A code is the nearest whole
    number unless a border lies within this distance."""
    y, ang = turned(x, pos, D, theta)
    L = 255
    gamma = np.abs(y).max(-1)
    t = (L * y + L * gamma[..., None]) / (2 * gamma[..., None])
    e = 1.5 * 2.0 ** -52 * np.abs(ang)
    e[:, 0] = 0
    e = np.concatenate([e, e], -1)[:, None] + 2.0 ** -49
    bound = L * (e + e.max(-1, keepdims=True)) + 2.0 ** -40
    frac = t - np.floor(t)
    near = np.abs(frac - 0.5) <= bound
    d = u - np.rint(t).astype(np.int64)
    tie = near | (x == 0)  # a zero is L/2 exactly, whose rounding the reference's gamma may tip
    assert np.all(d[~tie] == 0), (int((d[~tie] != 0).sum()), d.size)
    assert np.abs(d).max() <= 1
    np.testing.assert_allclose(g, gamma.astype(np.float64), rtol=2.0 ** -21)


def test_append_one_pair_at_far_positions():
    """The pair whose angle is the position itself, which 64 bits hold exactly: codes are exact up to 2^31."""
    T, H, D, page = 65536, 8, 64, 16
    rng = np.random.default_rng(4)
    x = np.zeros((T, H, D), np.float32)
    x[:, :, 0], x[:, :, D // 2] = rng.standard_normal((2, T, H))
    K = torch.from_numpy(x).cuda().to(torch.bfloat16)
    x = K.float().cpu().numpy()
    pos = rng.integers(2 ** 30, 2 ** 31, T)
    pos[::8] = np.exp2(rng.uniform(0, 31, T // 8)).astype(np.int64)
    pos[1::8] *= -1
    cache = torch.zeros(hbl.hbl_kv_cache_bytes(T // page, page, H, D, 8), dtype=torch.uint8, device="cuda")
    hbl.hbl_kv_append(K, K, i32(np.arange(T)), cache, page, 8, pos=i32(pos))
    u, g = k_bytes(cache, H, D, page)
    two = [0, D // 2]
    check_codes(u[:, :, two].astype(np.int64), g, x[:, :, two], pos, 2, 10000.0)


@pytest.mark.parametrize("low,high", [(0, 2 ** 17), (2 ** 24, 2 ** 25), (2 ** 27, 2 ** 28), (2 ** 30, 2 ** 31)])
def test_append_codes_over_positions(low, high):
    T, H, D, page = 2048, 4, 128, 16
    rng = np.random.default_rng(low % 97)
    K = torch.from_numpy(rng.standard_normal((T, H, D)).astype(np.float32)).cuda().to(torch.bfloat16)
    pos = rng.integers(low, high, T)
    cache = torch.zeros(hbl.hbl_kv_cache_bytes(T // page, page, H, D, 8), dtype=torch.uint8, device="cuda")
    hbl.hbl_kv_append(K, K, i32(np.arange(T)), cache, page, 8, pos=i32(pos), rope_theta=500000.0)
    u, g = k_bytes(cache, H, D, page)
    check_codes(u.astype(np.int64), g, K.float().cpu().numpy(), pos, D, 500000.0)


# ------------------------------------------------------------------------------------------- refusals

def test_prompt_without_room_for_queries_is_flagged():
    """A bound of no queries beside sequences that have some: flagged like any other bound that is too small."""
    c = prompt_case([3, 20], [3, 40], 2, 1, 128, seed=1)
    assert hbl.hbl_device_status() == hbl.HBL_OK
    O, lse = run_prompt(c, max_q=0)
    assert hbl.hbl_device_status() == hbl.HBL_EINVAL
    assert (O == 9).all() and (lse == 9).all()
    c["cq"] = np.zeros(3, np.int64)  # sequences without queries beside rows of none: nothing to leave out
    O, lse = run_prompt(c, max_q=0)
    assert hbl.hbl_device_status() == hbl.HBL_OK
    assert (O == 9).all() and (lse == 9).all()


def test_binding_refuses_one_wrong_argument():
    """Calls that differ from a valid one in a single argument, each refused for that argument."""
    d = decode_case([40, 17], 4, 2, 128, 3, 16, seed=1, dirty=False)
    p = prompt_case([30], [30], 4, 2, 128, seed=1)
    Q, K, V, cq, ck = p["Q"], p["K"], p["V"], i32(p["cq"]), i32(p["ck"])
    T = K.shape[0]
    slots, cache, t, lens = i32(np.arange(T)), d["cache"], d["t"], d["lens"]

    def append(K=K, V=V, slots=slots, cache=cache, Q=Q, pos=None, q_out=None):
        hbl.hbl_kv_append(K, V, slots, cache, 16, 3, pos=pos, Q=Q, q_out=q_out)

    def gather(cache=cache, slots=slots, K=None, V=None):
        hbl.hbl_kv_gather(cache, slots, 2, 128, 16, 3, K=K, V=V)

    def decode(Q=d["Q"], cache=cache, t=t, lens=lens, O=None, lse=None):
        hbl.hbl_attn_decode(Q, cache, t, lens, 2, 16, 3, O=O, lse=lse)

    def prompt(Q=Q, K=K, V=V, cq=cq, ck=ck, O=None, lse=None):
        hbl.hbl_attn_prompt(Q, K, V, cq, ck, O=O, lse=lse)

    for f in (append, gather, decode, prompt):
        f()
    f32 = torch.zeros((2, 4), device="cuda")
    for f, kw, why in (
            (append, dict(K=K.float()), "bf16 K"), (append, dict(V=V.half()), "bf16 V"), (append, dict(Q=Q.float()), "bf16 Q"),
            (append, dict(V=V[:-1]), "one shape"), (append, dict(K=K[:, :, ::2], V=V[:, :, ::2]), "dense heads in K"),
            (append, dict(V=V[:, :, :64]), "dense heads in V"), (append, dict(Q=Q[:-1]), "tokens and the head size"),
            (append, dict(q_out=Q[:, :2]), "shape of Q"), (append, dict(slots=slots[:-1]), "slots of"),
            (append, dict(slots=slots.long()), "slots"), (append, dict(pos=slots[:-1]), "pos of"),
            (append, dict(cache=cache.view(torch.int8)), "cache"), (append, dict(cache=cache[::2]), "cache"),
            (append, dict(slots=slots.cpu()), "CUDA"), (append, dict(K=K.view(T, -1)), "tokens, heads, D"),
            (gather, dict(K=K[:-1].contiguous()), "K of shape"), (gather, dict(V=V.float()), "contiguous"),
            (gather, dict(slots=slots.long()), "slots"), (gather, dict(cache=cache.view(torch.int32)), "cache"),
            (decode, dict(Q=d["Q"].float()), "bf16 Q"), (decode, dict(t=t[:1]), "tables"), (decode, dict(t=t[0]), "tables"),
            (decode, dict(t=t.long()), "tables"), (decode, dict(lens=lens[:1]), "lens"), (decode, dict(lens=lens.float()), "lens"),
            (decode, dict(O=d["Q"][:1].contiguous()), "O of shape"), (decode, dict(lse=f32.double()), "lse"),
            (decode, dict(lse=f32[:1]), "lse of shape"), (decode, dict(lens=lens.cpu()), "CUDA"),
            (prompt, dict(K=K[:-1]), "one shape"), (prompt, dict(K=K[:, :, :64], V=V[:, :, :64]), "dense heads in K"),
            (prompt, dict(K=K[:, :, :64].contiguous(), V=V[:, :, :64].contiguous()), "head size of Q"),
            (prompt, dict(ck=ck[:1]), "cu_k of"), (prompt, dict(cq=cq.long()), "cu_q"), (prompt, dict(O=Q[:-1].contiguous()), "O of shape"),
            (prompt, dict(lse=f32), "lse of shape"), (prompt, dict(V=V.cpu()), "CUDA")):
        with pytest.raises(ValueError, match=why):
            f(**kw)
    assert hbl.hbl_device_status() == hbl.HBL_OK
