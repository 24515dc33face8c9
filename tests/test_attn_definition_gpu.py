"""The gradients against the formula itself in 64 bits: probabilities, out and D = rowsum(dout out) are the
exact ones, nothing of the forward's stored results is taken over, and no tile size is known.

Tolerance, in the terms of attn_util (u, s, e): the stored lse is off by s + e + 2^-23 |lse| and the
recomputed scores and exponentials by s + e, so P is off by r = 2 s + 2 e + 2^-23 max |lse| relative.  The stored
out is off by b A with b = (u + (1 + u)(2 s + 2 e))(1 + u) + u and A = sum_j p_j |v_j|, so D by b |dout| A; where
D is the sum of P dP, it is off by r sum_j P |dout| |v|, the same |dout| A.  With W = scale P (|dout| |v|^T + |dout| A),
which is what the oracle calls "wide" when it is given A for out:

  |dv - ref| <= (u + (1 + u) r) sum P |dout| + u |ref|
  |dq - ref| <= (u + (1 + u) r) sum |dS| |k| + u |ref| + (1 + u)(1 + r)((dh + 2) 2^-22 + b + r) sum W |k|, dk likewise"""
import numpy as np
import pytest

from oracle import attn_oracle as A
from oracle import caat_oracle as O

from attn_util import U, _check, _e, _s
from gpu_util import ensure_built
from test_attn_gpu import backward, forward, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("P,hq,hk,dh,lens,klens", [
    (2, 4, 2, 64, [300, 1, 77], None),
    (1, 4, 1, 64, [100, 28], [128, 129]),     # tiles that see 128 keys at most, and 129
    (2, 3, 1, 128, [257, 64], None),
    (1, 2, 2, 96, [130, 5], [400, 3]),
    (16, 4, 4, 128, [300, 128], None),
    (1, 2, 1, 8, [90], [60]),
])
def test_gradients_match_the_formula(P, hq, hk, dh, lens, klens):
    d = make(P, hq, hk, dh, lens, klens, seed=50 + dh)
    out, lse = forward(d)
    got = backward(d, out, lse)
    f = A.attention(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"])
    given = [d["q"], d["k"], d["v"]], [d["dout"], d["cu_q"], d["cu_k"]]
    ref = A.attention_backward(*given[0], f["out"], f["lse"], *given[1])
    wide = A.attention_backward(*given[0], f["A"], f["lse"], *given[1])
    s, e = _s(float(f["M"].max()), dh), _e(ref["n"])
    r = 2 * s + 2 * e + 2.0 ** -23 * float(np.abs(f["lse"][np.isfinite(f["lse"])]).max())
    b = (U + (1 + U) * (2 * s + 2 * e)) * (1 + U) + U
    for name in ("dq", "dk", "dv"):
        bound = (U + (1 + U) * r) * ref[name + "_abs"] + U * np.abs(ref[name]) + 1e-30
        if name != "dv":
            bound = bound + (1 + U) * (1 + r) * ((dh + 2) * 2.0 ** -22 + b + r) * wide[name + "_wide"]
        _check(O._f64(got[name].cpu()), ref[name], bound, name)
