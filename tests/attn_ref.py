"""Plain 64-bit attention and the documented cache layout, for the tests of the cache and attention
operators. The layout is read bit by bit from the description in include/hbl.h; nothing here is
shared with the CUDA path."""
import numpy as np
import torch

import oracle


def record_bytes(D, bits):
    return 4 * D * bits + 128


def k_bit(d, i, bits):
    """Bit index inside a K row of bit i of code d."""
    if bits != 3:
        return bits * d + i
    g, c = divmod(d, 32)
    if c < 30:
        return 96 * g + 16 * (c // 5) + 3 * (c % 5) + i
    return 96 * g + 16 * (2 * i + c - 30) + 15


def v_bit(d, i, bits):
    """(unit, bit of the unit) of bit i of code d of V."""
    if bits != 3:
        return divmod(bits * d + i, 16)
    g, c = divmod(d, 16)
    return (3 * g + c // 5, 3 * (c % 5) + i) if c < 15 else (3 * g + i, 15)


def split_records(cache, Hkv, D, bits, page):
    """uint8 cache -> codes uK, uV [tokens, Hkv, D] (int64) and gammas [tokens, Hkv] (float64), tokens
    in slot order."""
    rec = np.ascontiguousarray(cache).reshape(-1, Hkv, page // 16, record_bytes(D, bits))
    rec = rec.transpose(0, 2, 1, 3).reshape(-1, Hkv, rec.shape[-1])  # [chunks, Hkv, bytes]
    n = 2 * D * bits
    kb = np.unpackbits(rec[:, :, :n].reshape(-1, 16, D * bits // 8), axis=-1, bitorder="little")
    vb = np.unpackbits(rec[:, :, n:2 * n].reshape(-1, D * bits // 16, 16, 2), axis=-1, bitorder="little")
    vb = vb.reshape(-1, D * bits // 16, 16, 16)
    uk = np.zeros((kb.shape[0], 16, D), np.int64)
    uv = np.zeros((kb.shape[0], 16, D), np.int64)
    for d in range(D):
        for i in range(bits):
            uk[:, :, d] |= kb[:, :, k_bit(d, i, bits)].astype(np.int64) << i
            unit, bit = v_bit(d, i, bits)
            uv[:, :, d] |= vb[:, unit, :, bit].astype(np.int64) << i
    g = rec[:, :, 2 * n:].copy().view(np.float32).astype(np.float64).reshape(-1, Hkv, 2, 16)

    def tokens(u):
        return u.reshape(-1, Hkv, 16, D).transpose(0, 2, 1, 3).reshape(-1, Hkv, D)

    return tokens(uk), tokens(uv), g[:, :, 0].transpose(0, 2, 1).reshape(-1, Hkv), \
        g[:, :, 1].transpose(0, 2, 1).reshape(-1, Hkv)


def join_records(uk, uv, gk, gv, bits, page):
    """The inverse of split_records: a uint8 cache of whole pages."""
    T, Hkv, D = uk.shape
    n = 2 * D * bits

    def chunks(u):
        return u.reshape(T // 16, 16, Hkv, D).transpose(0, 2, 1, 3).reshape(-1, 16, D)

    uk, uv = chunks(np.asarray(uk)), chunks(np.asarray(uv))
    kb = np.zeros((uk.shape[0], 16, D * bits), np.uint8)
    vb = np.zeros((uk.shape[0], D * bits // 16, 16, 16), np.uint8)
    for d in range(D):
        for i in range(bits):
            kb[:, :, k_bit(d, i, bits)] = (uk[:, :, d] >> i) & 1
            unit, bit = v_bit(d, i, bits)
            vb[:, unit, :, bit] = (uv[:, :, d] >> i) & 1
    parts = [np.packbits(kb, axis=-1, bitorder="little").reshape(-1, n),
             np.packbits(vb, axis=-1, bitorder="little").reshape(-1, n)]
    for g in (gk, gv):
        g = np.asarray(g, np.float32).reshape(T // 16, 16, Hkv).transpose(0, 2, 1)
        parts.append(np.ascontiguousarray(g).reshape(-1, 16).view(np.uint8))
    rec = np.concatenate(parts, axis=1)
    return np.ascontiguousarray(rec.reshape(T // page, page // 16, Hkv, -1).transpose(0, 2, 1, 3)).reshape(-1)


def quantise(x, pos, bits, theta=10000.0):
    """The oracle's quantiser, with zeros at the code nearest to the middle that is even: a state that
    is 0 is L gamma / (2 gamma) = L/2 exactly, a tie, but where gamma comes from a rotation the rounding
    of L gamma in float64 can take the oracle's quotient to either side of it."""
    u, g = oracle.qkv_quant(x, pos, bits, theta)
    xr = oracle.bf16_to_f64(x) if x.dtype == np.uint16 else np.asarray(x, np.float64)
    if pos is not None:
        xr = oracle.rope(xr, pos, theta)
    return np.where(xr == 0, np.uint8(np.rint(((1 << bits) - 1) / 2)), u), g


def states(u, g, bits):
    return oracle.dequantize_unsigned(u, g, bits)


def attention(q, k, v, seen, scale):
    """softmax(scale q k^T) v of queries [n, H, D], keys and values [m, Hkv, D] (float64 CUDA or CPU
    tensors), query i seeing its first seen[i] keys. Returns o [n, H, D], lse [n, H], and for the error
    bounds A = sum p |v| [n, H, D], the largest weight's place in it: pmax [n, H]."""
    n, H, D = q.shape
    m, Hkv, _ = k.shape
    o = torch.zeros_like(q)
    A = torch.zeros_like(q)
    lse = torch.full((n, H), -np.inf, dtype=torch.float64, device=q.device)
    pmax = torch.zeros((n, H), dtype=torch.float64, device=q.device)
    if m == 0 or n == 0:
        return o, lse, A, pmax
    hide = torch.arange(m, device=q.device)[None] >= seen[:, None]
    some = (seen > 0)[:, None]
    for h in range(H):
        s = (q[:, h] @ k[:, h // (H // Hkv)].T) * scale
        s = s.masked_fill(hide, -np.inf)
        e = torch.logsumexp(s, 1, keepdim=True)
        p = torch.where(some, torch.exp(s - torch.where(some, e, 0.0)), 0.0)
        vv = torch.where(hide.all(0)[:, None], 0.0, v[:, h // (H // Hkv)])  # keys nobody sees have no say
        o[:, h], A[:, h] = p @ vv, p @ vv.abs()
        lse[:, h], pmax[:, h] = e[:, 0], p.amax(1)
    return o, lse, A, pmax


def check_close(o, lse, ref, weight_step, score_err, extra=0.0):
    """Element by element and in the norm.

    The output is rounded once to bf16 (half a step: 2^-8 of the value) from sum p v, whose weights are
    rounded to a type with half a step of `weight_step` (so at most that share of A = sum p |v|) and
    come from scores that are off by at most score_err (a factor e^(2 score_err) at most after the
    normalisation). `extra` [like A] covers weights below the type's normal range. In the norm the two
    roundings are independent, each with a mean square of a third of its half step's square."""
    ro, rlse, A, _ = ref
    o, lse = o.double(), lse.double()
    assert torch.isfinite(o).all()
    tol = 2.0 ** -8 * ro.abs() * 1.01 + (weight_step + 2.5 * score_err + 2.0 ** -18) * A + extra + 1e-30
    bad = (o - ro).abs() > tol
    assert not bad.any(), ("elements", int(bad.sum()), float(((o - ro).abs() / tol).max()))
    if ro.numel() and float(ro.norm()) > 0:
        rel = float((o - ro).norm() / ro.norm())
        assert rel <= (2.0 ** -16 + weight_step ** 2) ** 0.5 + 3 * score_err + float(torch.as_tensor(extra).max()), rel
    empty = torch.isinf(rlse)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    assert (o[empty] == 0).all()
    d = (lse - rlse)[~empty].abs()
    if d.numel():
        lim = score_err + 2.0 ** -17 + 2.0 ** -21 * rlse[~empty].abs()
        assert (d <= lim).all(), float((d / lim).max())
