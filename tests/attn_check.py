"""Checks of attention results that may hold NaN, with bounds in the outputs' own scale."""
import torch


def check_rows(o, lse, ref, weight_step, score_err, extra=0.0, sum_err=0.0):
    """o [n, H, D] and lse [n, H] against attn_ref.attention's result.

    NaN and -inf have to stand exactly where the 64-bit evaluation has them, and a row of lse = -inf is zero.
    Elsewhere an output is rounded once to bf16 (half a step: 2^-8 of the value) from sums whose weights are
    rounded to a type of half a step `weight_step` (of A = sum p |v|) and come from scores off by `score_err`
    (a factor of e^(2 score_err) after the normalisation); `extra`, in the outputs' scale, covers weights below
    the type's normal range. In the norm the two roundings are independent, each with a third of its half step's
    square, and `extra` enters as the share of its own norm. `sum_err` is what the sum of the weights can be off
    by, of itself."""
    ro, rlse, A, _ = ref
    o, lse = o.double(), lse.double()
    assert torch.equal(torch.isnan(o), torch.isnan(ro)), (int(torch.isnan(o).sum()), int(torch.isnan(ro).sum()))
    assert torch.equal(torch.isnan(lse), torch.isnan(rlse)), (int(torch.isnan(lse).sum()), int(torch.isnan(rlse).sum()))
    empty = torch.isneginf(rlse)
    assert torch.equal(torch.isneginf(lse), empty)
    assert (o[empty] == 0).all()
    ex = torch.as_tensor(extra, dtype=torch.float64, device=o.device).expand_as(ro)
    good = torch.isfinite(ro)
    err, big = (o - ro).abs()[good], ro.abs()[good]
    tol = 2.0 ** -8 * 1.01 * big + (weight_step + 2.5 * score_err + 2.0 ** -18) * A[good] + ex[good] + 1e-30
    assert (err <= tol).all(), ("elements", int((err > tol).sum()), float((err / tol).max()))
    if big.numel() and float(big.norm()) > 0:
        rel = float(err.norm() / big.norm())
        assert rel <= (2.0 ** -16 + weight_step ** 2) ** 0.5 + 3 * score_err + float(ex[good].norm() / big.norm()), rel
    fine = torch.isfinite(rlse)
    d = (lse - rlse)[fine].abs()
    if d.numel():
        lim = score_err + sum_err + 2.0 ** -17 + 2.0 ** -21 * rlse[fine].abs()
        assert (d <= lim).all(), float((d / lim).max())
