"""Tolerances of the attention block's GPU tests, from the arithmetic (u = half a bf16 step = 2^-8).

Scores: exact bf16 products summed in fp32 over dh terms, each addition off by at most 2^-23 relative
to the sum of absolute values M, then one rounding by the scale: |dS| <= s = (dh + 2) 2^-23 M.  exp2
and log2 are good to 2^-21 relative.  A sum of n terms in fp32, one after the other, with the running sum
rescaled before each addition, has two roundings of 2^-24 per term, all of them of non-negative partial
sums (or bounded by the sum of absolute values A): it is off by at most n 2^-23 relative.  Together
e = 2^-20 + n 2^-23.

forward   p off by at most 2 s + 2 e relative (numerator and sum), p rounded to bf16 (u), out rounded (u):
          |out - ref| <= (u + (1 + u)(2 s + 2 e)) (1 + u) A + u |ref|, A = sum_j p_j |v_j|
          |lse - ref| <= s + e + 2^-23 |ref|
backward  (from the forward's out and lse as stored) P off by s + e relative, rounded to bf16 for dv
          (u); dS = scale P (dP - D) off by (s + e) |dS| and by the fp32 sums in dP and D,
          (dh + 2) 2^-23 of their sums of absolute values ("wide"), and rounded to bf16 (u).  Where D is the sum
          of P dP, with P off by s + e, it is off by (s + e) sum P |dP| more, and |dP| is at most its sum of
          absolute values: (s + e) of the part of "wide" that stands for D."""
import numpy as np

from oracle import caat_oracle as O

U = 2.0 ** -8


def _e(n):
    return 2.0 ** -20 + n * 2.0 ** -23


def _check(got, ref, bound, what):
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {err.size} out of bound, "
                           f"max err/bound {np.nanmax(err / bound):.3f}, first at {np.argwhere(bad)[0].tolist()}")


def _s(M, dh):
    return (dh + 2) * 2.0 ** -23 * M


def check_out(got, ref, what=""):
    """got [P,T,hq*dh] against the oracle's dict; rows with NaN in the reference are skipped."""
    o, dh = ref["out"], ref["out"].shape[-1]
    got = O._f64(got).reshape(o.shape)
    M = ref["M"] if ref["M"].shape == o.shape[:3] else ref["M"].transpose(0, 2, 1)
    s = _s(M, dh)[..., None]
    bound = (U + (1 + U) * (2 * s + 2 * _e(ref["n"]))) * (1 + U) * ref["A"] + U * np.abs(o) + 1e-30
    rows = ~np.isnan(o).any(axis=(0, 2, 3))
    _check(got[:, rows], o[:, rows], bound[:, rows], f"out {what}")


def check_lse(got, ref, dh, what=""):
    got, l = O._f64(got), ref["lse"]
    rows = ~np.isnan(l).any(axis=(0, 1))
    g, r, M = got[..., rows], l[..., rows], ref["M"][..., rows]
    empty = np.isneginf(r)
    assert np.array_equal(np.isneginf(g), empty), f"lse {what}: empty rows"
    _check(g[~empty], r[~empty], (_s(M, dh) + _e(ref["n"]) + 2.0 ** -23 * np.abs(r))[~empty], f"lse {what}")


def check_grads(got, ref, M, dh, what=""):
    """got {"dq","dk","dv"} against oracle.attention_backward; M: the largest score sum."""
    s = _s(float(np.nanmax(M)) if M.size else 0.0, dh)
    for name in ("dq", "dk", "dv"):
        g, r = O._f64(got[name]), ref[name]
        bound = (U + (1 + U) * (s + _e(ref["n"]))) * ref[name + "_abs"] + U * np.abs(r) + 1e-30
        if name != "dv":
            bound = bound + (1 + U) * ((dh + 2) * 2.0 ** -22 + s + _e(ref["n"])) * ref[name + "_wide"]
        rows = ~np.isnan(r).any(axis=(0, 2, 3))
        _check(g[:, rows], r[:, rows], bound[:, rows], f"{name} {what}")
