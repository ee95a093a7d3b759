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
