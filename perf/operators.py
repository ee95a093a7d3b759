"""The attention operators around the low-bit key-value cache: what is measured, and their plain forms.

Four operators, as a serving program calls them between the fused QKV projection and the output
projection Wo:

  append  RoPE on the query and key states, and quantisation of the key and value states per head
          into a paged cache, then the read-back of the tokens just written (the states that the
          attention over a prompt sees)
  gather  the read-back of whole cached sequences as bf16
  decode  attention of one new token per sequence over the paged low-bit cache
  prompt  attention over packed prompts with grouped heads, causal, with or without a cached prefix

The cache is one byte buffer of [pages][KV heads][page size / 16] records of 4 D b + 128 bytes, each
holding 16 tokens of one head: K codes (16 rows of D b / 8 bytes), V codes (D b / 16 units of 16 bits,
each for the 16 tokens in turn), then the fp32 scales of K and of V. Codes are little-endian bit
strings, except that three-bit codes go five to a half-word, at bits 0, 3, ... 12, with the codes
left over in the spare bits 15: in K, codes 30 and 31 of each 32 in those of the even and of the odd
half-words of the group; in V, code 15 of each 16 in those of the group's three units.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a batch of 64 sequences: latency, a few hundred KB
        dict(name="append_step_64", op="append", T=64, Hq=32, Hkv=8, D=128, bits=3, page=64, theta=10000.0, first=1900),
        # an odd piece of a prompt, small heads, four bits, odd positions, small pages
        dict(name="append_odd_333", op="append", T=333, Hq=12, Hkv=4, D=64, bits=4, page=16, theta=500000.0, first=70001),
        # a whole 8192-token prompt of the 7B-like block (fused QKV 4096 -> 12288, 32 heads of 128)
        dict(name="append_prompt_8192", op="append", T=8192, Hq=32, Hkv=32, D=128, bits=3, page=64, theta=10000.0, first=0),
        # a short prefix with wide heads at eight bits
        dict(name="gather_77_d256", op="gather", B=1, low=77, high=77, Hkv=2, D=256, bits=8, page=32),
        # the cached prefixes of five ragged sequences
        dict(name="gather_ragged_5", op="gather", B=5, low=700, high=4096, Hkv=32, D=128, bits=3, page=64),
        # one sequence, short cache: the latency of a single request
        dict(name="decode_one_500", op="decode", B=1, low=500, high=500, Hq=32, Hkv=32, D=128, bits=3, page=64),
        # one request over a very long cache: split over the length
        dict(name="decode_one_131072", op="decode", B=1, low=131072, high=131072, Hq=32, Hkv=8, D=128, bits=4, page=64),
        # a ragged batch with grouped heads, an empty sequence now and then
        dict(name="decode_ragged_64", op="decode", B=64, low=0, high=8192, Hq=32, Hkv=8, D=128, bits=3, page=64),
        # the largest: a full batch of the 7B-like block, one KV head to each query head
        dict(name="decode_full_64", op="decode", B=64, low=3500, high=4096, Hq=32, Hkv=32, D=128, bits=3, page=64),
        # three short prompts packed together: latency
        dict(name="prompt_three_short", op="prompt", B=3, low=17, high=120, prefix=0, Hq=32, Hkv=8, D=128),
        # packed ragged prompts with grouped heads
        dict(name="prompt_packed_12", op="prompt", B=12, low=100, high=2400, prefix=0, Hq=32, Hkv=8, D=128),
        # one 8192-token prompt of the 7B-like block
        dict(name="prompt_one_8192", op="prompt", B=1, low=8192, high=8192, prefix=0, Hq=32, Hkv=32, D=128),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append", "gather", "decode", "decode", "prompt", "prompt"])
    D = rng.choice([64, 128, 128, 256])
    bits = rng.choice([2, 3, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    G = rng.choice([1, 2, 3, 4, 8, 12])
    if op == "append":
        T = _log_int(rng, 1, 4096)
        return dict(op=op, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, bits=bits, page=page,
                    theta=rng.choice([10000.0, 500000.0]), first=rng.randrange(0, 100000))
    if op == "gather":
        high = _log_int(rng, 1, 4096)
        return dict(op=op, B=rng.randint(1, 9), low=max(0, high // rng.choice([1, 3, 50])), high=high, Hkv=Hkv, D=D,
                    bits=bits, page=page)
    if op == "decode":
        high = _log_int(rng, 1, 40000)
        most = max(1, min(96, 400000 // high))
        return dict(op=op, B=_log_int(rng, 1, most), low=max(0, high // rng.choice([1, 2, 20])), high=high, Hq=Hkv * G,
                    Hkv=Hkv, D=D, bits=bits, page=page)
    high = _log_int(rng, 1, 4000)
    prefix = rng.choice([0, 0, _log_int(rng, 1, 6000)])
    Hq = min(32, Hkv * G) // Hkv * Hkv
    if Hq * D * high * (high + prefix) > 1.3e11:  # no more products than the largest listed case
        prefix = 0
    most = 1.3e11 / (Hq * D * high * (high + prefix))
    return dict(op=op, B=_log_int(rng, 1, max(1, min(16, int(most)))), low=max(1, high // rng.choice([1, 2, 20])),
                high=high, prefix=prefix, Hq=Hq, Hkv=Hkv, D=D)


def _lengths(case):
    """The sequences' lengths: a matter of the case, not of the inputs' seed."""
    rng = random.Random("%d %d %d" % (case["B"], case["low"], case["high"]))
    return [case["high"]] + [rng.randint(case["low"], case["high"]) for _ in range(case["B"] - 1)]


def _prefixes(case):
    """Cached tokens before each prompt (ragged, up to case["prefix"])."""
    rng = random.Random("prefix %d %d" % (case["B"], case["prefix"]))
    return [rng.randint(case["prefix"] // 2, case["prefix"]) for _ in range(case["B"])]


def work(case):
    D = case["D"]
    if case["op"] == "prompt":
        nq = _lengths(case)
        nk = [a + b for a, b in zip(nq, _prefixes(case))]
        pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(nq, nk))
        return {"bytes": sum(nq) * case["Hq"] * (4 * D + 4) + sum(nk) * case["Hkv"] * 4 * D,
                "flops": 4 * case["Hq"] * D * pairs}
    token = case["Hkv"] * (4 * D * case["bits"] + 128) / 16  # bytes of one cached token
    if case["op"] == "append":  # Q, K, V in; Q out, the cache, K and V read back
        return {"bytes": case["T"] * (2 * D * (2 * case["Hq"] + 4 * case["Hkv"]) + token), "flops": 0}
    total = sum(_lengths(case))
    if case["op"] == "gather":
        return {"bytes": total * (token + 4 * D * case["Hkv"]), "flops": 0}
    return {"bytes": total * token + case["B"] * case["Hq"] * (4 * D + 4), "flops": 4 * case["Hq"] * D * total}


# ------------------------------------------------------------------------------- inputs and cache

def _record_bytes(D, bits):
    return 4 * D * bits + 128


def _halves(u, bits, group):
    """Codes [..., D] as 16-bit half-words (int32) [..., D * bits / 16]; groups of three-bit codes
    hold `group` codes (32 in K, 16 in V)."""
    D = u.shape[-1]
    if bits != 3:
        per = 16 // bits
        sh = torch.arange(per, device=u.device, dtype=torch.int32) * bits
        return (u.view(*u.shape[:-1], D // per, per) << sh).sum(-1, dtype=torch.int32)
    n = group * 3 // 16
    g = u.view(*u.shape[:-1], D // group, group)
    sh = torch.arange(5, device=u.device, dtype=torch.int32) * 3
    h = (g[..., :5 * n].reshape(*g.shape[:-1], n, 5) << sh).sum(-1, dtype=torch.int32)
    if group == 16:
        spare = torch.stack([(g[..., 15] >> j) & 1 for j in range(3)], -1)
    else:
        spare = torch.stack([(g[..., 30 + j % 2] >> (j // 2)) & 1 for j in range(6)], -1)
    return (h | (spare << 15)).reshape(*u.shape[:-1], D // group * n)


def _pack(k, v, bits):
    """Quantises K and V [records, 16, D] (fp32) and lays them out as records (uint8)."""
    L = (1 << bits) - 1
    parts, scales = [], []
    for x, group in ((k, 32), (v, 16)):
        g = x.abs().amax(-1, keepdim=True)
        u = ((L * x + L * g) / (2 * g)).round().clamp(0, L).to(torch.int32)
        h = _halves(u, bits, group).to(torch.int16)
        h = h if group == 32 else h.transpose(1, 2)
        parts.append(h.contiguous().view(h.shape[0], -1).view(torch.uint8))
        scales.append(g.view(-1, 16).view(torch.uint8))
    return torch.cat(parts + scales, 1)


def _filled_cache(pages, case, gen):
    """A cache whose every token holds quantised states: normal keys and values of varying size."""
    Hkv, D, bits = case["Hkv"], case["D"], case["bits"]
    n = pages * Hkv * case["page"] // 16
    cache = torch.empty(n, _record_bytes(D, bits), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (16 * D))
    for i in range(0, n, step):
        m = min(step, n - i)
        k = torch.randn(m, 16, D, generator=gen, device="cuda") * (0.5 + torch.rand(m, 16, 1, generator=gen, device="cuda"))
        v = torch.randn(m, 16, D, generator=gen, device="cuda") * (0.1 + torch.rand(m, 16, 1, generator=gen, device="cuda"))
        cache[i:i + m] = _pack(k, v, bits)
    return cache.view(-1)


def _tables(lengths, page, gen):
    """Pages of each sequence, in no order, and the number of pages in the pool (some unused)."""
    need = [-(-n // page) for n in lengths]
    width = max(1, max(need))
    pages = sum(need) + 3
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).cpu()
    table = torch.zeros(len(lengths), width, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table.cuda(), pages


def _cu(lengths):
    return torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    D = case["D"]
    s = dict(case)
    if case["op"] == "append":
        T, Hq, Hkv, page = case["T"], case["Hq"], case["Hkv"], case["page"]
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen, device="cuda").to(torch.bfloat16)
        pages = -(-T // page) + 2
        table = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(T, device="cuda")
        s["Q"] = qkv[:, :Hq * D].view(T, Hq, D)
        s["K"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        s["V"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        s["pos"] = (at + case["first"]).to(torch.int32)
        s["slots"] = (table[at // page] * page + at % page).to(torch.int32)
        s["cache"] = torch.zeros(pages * Hkv * page // 16 * _record_bytes(D, case["bits"]), dtype=torch.uint8, device="cuda")
        return s
    lengths = _lengths(case)
    if case["op"] == "prompt":
        nk = [a + b for a, b in zip(lengths, _prefixes(case))]
        s["Q"] = torch.randn(sum(lengths), case["Hq"], D, generator=gen, device="cuda").to(torch.bfloat16)
        s["K"] = torch.randn(sum(nk), case["Hkv"], D, generator=gen, device="cuda").to(torch.bfloat16)
        s["V"] = torch.randn(sum(nk), case["Hkv"], D, generator=gen, device="cuda").to(torch.bfloat16)
        s["cu_q"], s["cu_k"], s["max_q"] = _cu(lengths), _cu(nk), max(lengths)
        s["lse"] = torch.empty(sum(lengths), case["Hq"], dtype=torch.float32, device="cuda")
        return s
    s["table"], pages = _tables(lengths, case["page"], gen)
    s["cache"] = _filled_cache(pages, case, gen)
    s["lens"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if case["op"] == "gather":
        page = case["page"]
        slots = [s["table"][i, torch.arange(n, device="cuda") // page] * page + torch.arange(n, device="cuda") % page
                 for i, n in enumerate(lengths)]
        s["slots"] = torch.cat(slots).to(torch.int32)
    else:
        s["Q"] = torch.randn(case["B"], case["Hq"], D, generator=gen, device="cuda").to(torch.bfloat16)
        s["lse"] = torch.empty(case["B"], case["Hq"], dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------------------------ plain forms

def _turn(x, pos, theta):
    """RoPE in 64 bits: positions reach far, and the quantiser's borders are sharp."""
    D = x.shape[-1]
    f = torch.arange(D // 2, device=x.device, dtype=torch.float64)
    ang = pos.double()[:, None, None] * torch.exp(-2.0 * f / D * math.log(theta))
    c, s = torch.cos(ang), torch.sin(ang)
    a, b = x.double().chunk(2, -1)
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def _quantised(x, bits):
    """The values that the stored codes and scales stand for, of x in 64 bits."""
    L = (1 << bits) - 1
    g = x.abs().amax(-1, keepdim=True)
    u = torch.where(g > 0, (L * x + L * g) / torch.where(g > 0, 2 * g, 1.0), 0.5 * L).round().clamp(0, L)
    return (2 * u.float() - L) * g.float() / L


def _codes(h, bits, group):
    """Half-words (int32, 16 bits used) [..., D * bits / 16] as codes [..., D]."""
    mask = (1 << bits) - 1
    if bits != 3:
        sh = torch.arange(16 // bits, device=h.device, dtype=torch.int32) * bits
        return ((h[..., None] >> sh) & mask).flatten(-2)
    n = group * 3 // 16
    g = h.view(*h.shape[:-1], h.shape[-1] // n, n)
    sh = torch.arange(5, device=h.device, dtype=torch.int32) * 3
    most = ((g[..., None] >> sh) & mask).flatten(-2)
    spare = (g >> 15) & 1
    if group == 16:
        left = (spare[..., 0] | (spare[..., 1] << 1) | (spare[..., 2] << 2))[..., None]
    else:
        left = spare[..., 0:2] | (spare[..., 2:4] << 1) | (spare[..., 4:6] << 2)
    return torch.cat([most, left], -1).flatten(-2)


def _states(records, D, bits, which):
    """K (0) or V (1) of records [..., 4 D b + 128] as fp32 [..., 16, D]."""
    L, n = (1 << bits) - 1, 2 * D * bits
    h = records[..., which * n:(which + 1) * n].contiguous().view(torch.int16).to(torch.int32) & 0xffff
    if which == 0:
        u = _codes(h.view(*h.shape[:-1], 16, D * bits // 16), bits, 32)
    else:
        u = _codes(h.view(*h.shape[:-1], D * bits // 16, 16).transpose(-1, -2).contiguous(), bits, 16)
    g = records[..., 2 * n + 64 * which:2 * n + 64 * (which + 1)].contiguous().view(torch.float32)
    return (2 * u.float() - L) * (g / L)[..., None]


def _soft(scores, visible):
    """Weights and the log of their sum; a row that sees nothing has weights 0 and -inf."""
    scores = scores.masked_fill(~visible, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    w = torch.exp(scores - top)
    total = w.sum(-1, keepdim=True)
    return w / torch.where(total > 0, total, 1.0), (total.log() + top).squeeze(-1)


def _plain(s):
    D = s["D"]
    if s["op"] == "append":
        q = _turn(s["Q"], s["pos"], s["theta"]).to(torch.bfloat16)
        k = _quantised(_turn(s["K"], s["pos"], s["theta"]), s["bits"]).to(torch.bfloat16)
        return q, k, _quantised(s["V"].double(), s["bits"]).to(torch.bfloat16)
    if s["op"] == "prompt":
        G = s["Hq"] // s["Hkv"]
        iq, ik = (torch.arange(x.shape[0], device="cuda") for x in (s["Q"], s["K"]))
        bq, bk = (torch.searchsorted(c[1:].long(), i, right=True) for c, i in ((s["cu_q"], iq), (s["cu_k"], ik)))
        # query i sits as far from its sequence's end as its own key does
        last = s["cu_k"][1:].long()[bq] - (s["cu_q"][1:].long()[bq] - iq)
        visible = (bq[:, None] == bk[None, :]) & (ik[None, :] <= last[:, None])
        o, lse = [], []
        for h in range(s["Hkv"]):  # one KV head at a time: the scores of all would not fit
            q = s["Q"][:, h * G:(h + 1) * G].transpose(0, 1).float()
            w, e = _soft(q @ s["K"][:, h].float().T / math.sqrt(D), visible)
            o.append(w @ s["V"][:, h].float())
            lse.append(e)
        return torch.cat(o).transpose(0, 1).to(torch.bfloat16), torch.cat(lse).T
    bits, page, Hkv = s["bits"], s["page"], s["Hkv"]
    rec = s["cache"].view(-1, Hkv, page // 16, _record_bytes(D, bits))
    if s["op"] == "gather":
        t = s["slots"].long()
        at = rec.transpose(1, 2).reshape(-1, Hkv, rec.shape[-1])[t // 16]
        i = (t % 16)[:, None, None, None].expand(-1, Hkv, 1, D)
        return tuple(_states(at, D, bits, w).gather(2, i).squeeze(2).to(torch.bfloat16) for w in (0, 1))
    B, G = s["Q"].shape[0], s["Hq"] // Hkv
    at = rec[s["table"].long()].transpose(1, 2)  # [B, Hkv, pages, page / 16, record]
    q = s["Q"].float().view(B, Hkv, G, D)
    sc = q @ _states(at, D, bits, 0).view(B, Hkv, -1, D).transpose(-1, -2) / math.sqrt(D)
    visible = torch.arange(sc.shape[-1], device="cuda") < s["lens"].view(B, 1, 1, 1)
    w, lse = _soft(sc, visible)
    o = w @ _states(at, D, bits, 1).view(B, Hkv, -1, D)
    return o.view(B, s["Hq"], D).to(torch.bfloat16), lse.view(B, s["Hq"])


def _calls(s):
    """The same through the framework."""
    import hadamard_bit_quant_hbl_b200 as hbl

    if s["op"] == "append":
        q = hbl.hbl_kv_append(s["K"], s["V"], s["slots"], s["cache"], s["page"], s["bits"], pos=s["pos"],
                              rope_theta=s["theta"], Q=s["Q"])
        k, v = hbl.hbl_kv_gather(s["cache"], s["slots"], s["Hkv"], s["D"], s["page"], s["bits"])
        return q, k, v
    if s["op"] == "gather":
        return hbl.hbl_kv_gather(s["cache"], s["slots"], s["Hkv"], s["D"], s["page"], s["bits"])
    if s["op"] == "decode":
        if "workspace" not in s:  # a serving program keeps one
            n = hbl.hbl_attn_decode_workspace(s["B"], s["Hq"], s["Hkv"], s["D"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return hbl.hbl_attn_decode(s["Q"], s["cache"], s["table"], s["lens"], s["Hkv"], s["page"], s["bits"],
                                   workspace=s["workspace"], lse=s["lse"]), s["lse"]
    return hbl.hbl_attn_prompt(s["Q"], s["K"], s["V"], s["cu_q"], s["cu_k"], max_q=s["max_q"], lse=s["lse"]), s["lse"]


def run(state):
    if own:
        return _calls(state)
    return _plain(state)


# ---------------------------------------------------------------------------- 64 bits, from the definition

def _bits_to_codes(bit, bits, group):
    """Single bits [..., 16 n] of half-words as codes, by the layout's definition."""
    if bits != 3:
        w = torch.tensor([1 << i for i in range(bits)], dtype=torch.float64, device=bit.device)
        return bit.reshape(*bit.shape[:-1], -1, bits).double() @ w
    n = group * 3 // 16
    place = torch.zeros(16 * n, group, dtype=torch.float64)
    for c in range(group):
        for i in range(3):
            if c < 5 * n:
                place[16 * (c // 5) + 3 * (c % 5) + i, c] = 1 << i
            elif group == 16:
                place[16 * i + 15, c] = 1 << i
            else:
                place[16 * (2 * i + c - 30) + 15, c] = 1 << i
    return (bit.reshape(*bit.shape[:-1], -1, 16 * n).double() @ place.to(bit.device)).flatten(-2)


def _token(records, D, bits):
    """K and V [n, D] in 64 bits of records [m, bytes] whose 16 tokens follow one another."""
    L, n = (1 << bits) - 1, 2 * D * bits
    eight = torch.arange(8, device=records.device, dtype=torch.uint8)
    bit = (records[:, :2 * n, None] >> eight) & 1
    k = _bits_to_codes(bit[:, :n].reshape(-1, 16, D * bits), bits, 32)
    v = _bits_to_codes(bit[:, n:].reshape(-1, D * bits // 16, 16, 16).transpose(1, 2).reshape(-1, 16, D * bits), bits, 16)
    g = records[:, 2 * n:].contiguous().view(torch.float32).double()
    return [((2 * u - L) / L * c[..., None]).view(-1, D) for u, c in ((k, g[:, :16]), (v, g[:, 16:]))]


def _row_exact(q, k, v, seen):
    """softmax(q k^T / sqrt(D)) v of queries [n, D], the i-th seeing its first seen[i] keys."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.full(q.shape[:1], -math.inf, dtype=torch.float64, device=q.device)
    s = (q @ k.T) * q.shape[-1] ** -0.5
    hidden = torch.arange(k.shape[0], device=q.device)[None, :] >= seen[:, None]
    lse = torch.logsumexp(s.masked_fill_(hidden, -math.inf), 1)
    p = torch.exp(s - torch.where(seen > 0, lse, 0.0)[:, None])
    return p @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    D = case["D"]
    if case["op"] == "append":
        L = 2 ** case["bits"] - 1
        f = np.arange(D // 2)
        ang = s["pos"].cpu().numpy().astype(np.float64)[:, None] * np.float64(case["theta"]) ** (-2.0 * f / D)
        turn = torch.polar(torch.ones(ang.shape, dtype=torch.float64), torch.from_numpy(ang)).cuda()[:, None]
        out = []
        for x, pos in ((s["Q"], True), (s["K"], True), (s["V"], False)):
            x = x.double()
            if pos:
                z = torch.complex(x[..., :D // 2].contiguous(), x[..., D // 2:].contiguous()) * turn
                x = torch.cat([z.real, z.imag], -1)
            out.append(x)
        for i in (1, 2):
            x = out[i]
            g = x.abs().max(-1, keepdim=True).values
            out[i] = torch.round(L * (x + g) / (2 * g)) * (2 * g / L) - g
        return tuple(out)
    lengths = _lengths(case)
    Hq = case.get("Hq", 0)
    if case["op"] == "prompt":
        G = Hq // case["Hkv"]
        o = torch.empty(sum(lengths), Hq, D, dtype=torch.float64, device="cuda")
        lse = torch.empty(sum(lengths), Hq, dtype=torch.float64, device="cuda")
        cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
        for b in range(case["B"]):
            nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
            seen = torch.arange(nq, device="cuda") + 1 + nk - nq
            for h in range(Hq):
                o[cq[b]:cq[b + 1], h], lse[cq[b]:cq[b + 1], h] = _row_exact(
                    s["Q"][cq[b]:cq[b + 1], h].double(), s["K"][ck[b]:ck[b + 1], h // G].double(),
                    s["V"][ck[b]:ck[b + 1], h // G].double(), seen)
        return o, lse
    Hkv, bits, page = case["Hkv"], case["bits"], case["page"]
    rec = s["cache"].view(-1, Hkv, page // 16, _record_bytes(D, bits))
    table = s["table"].long()
    if case["op"] == "gather":
        k = torch.empty(sum(lengths), Hkv, D, dtype=torch.float64, device="cuda")
        v = torch.empty_like(k)
    else:
        o = torch.zeros(case["B"], Hq, D, dtype=torch.float64, device="cuda")
        lse = torch.full((case["B"], Hq), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, n in enumerate(lengths):
        for h in range(Hkv):
            if n == 0:
                continue
            K, V = _token(rec[table[b, :-(-n // page)], h].reshape(-1, rec.shape[-1])[:-(-n // 16)], D, bits)
            if case["op"] == "gather":
                k[at:at + n, h], v[at:at + n, h] = K[:n], V[:n]
            else:
                G = Hq // Hkv
                seen = torch.full((G,), n, device="cuda")
                o[b, h * G:(h + 1) * G], lse[b, h * G:(h + 1) * G] = _row_exact(
                    s["Q"][b, h * G:(h + 1) * G].double(), K[:n], V[:n], seen)
        at += n
    return (k, v) if case["op"] == "gather" else (o, lse)
