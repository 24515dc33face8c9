"""Float64 definitions of the attention block's operators (test infrastructure; NumPy).

Rotary positions, causal attention over packed sequences with grouped heads, its gradients and
decoding against a cache, for P ranks side by side.  Shares nothing with the CUDA path.  Each
attention function also returns the sums of absolute values that bound rounding errors.
"""
from __future__ import annotations

import math

import numpy as np

from .caat_oracle import _f64


def rope_frequencies(rot, theta=10000.0, scaling="none", factor=1.0, trained_length=4096.0):
    """(rotation per position of pair j = 0..rot/2-1, factor on the vectors)."""
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = np.array([theta ** (-2.0 * j / rot) for j in range(rot // 2)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        out = []
        for x in f:
            turns = trained_length * x / (2 * math.pi)
            keep = 0.0 if turns < 1 else 1.0 if turns > 32 else (turns - 1) / 31
            out.append((1 - keep) * x / factor + keep * x)
        return np.array(out), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rope(x, positions, freq, interleaved=False, backward=False, mscale=1.0):
    """x [P, T, heads, dh] with the first 2 len(freq) elements of every head turned."""
    y = _f64(x).copy()
    rot = 2 * len(freq)
    first = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    second = first + 1 if interleaved else first + rot // 2
    w = np.outer(np.asarray(positions, dtype=np.float64), freq)[None, :, None, :]
    z = (y[..., first] + 1j * y[..., second]) * mscale * np.exp(-1j * w if backward else 1j * w)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _visible(n, m):
    """[n, m] truth: query i sees key j (the last query sees the last key)."""
    return np.arange(m)[None, :] < np.arange(n)[:, None] + 1 + (m - n)


def _sequences(cu_q, cu_k):
    cu_k = cu_q if cu_k is None else cu_k
    for i in range(len(cu_q) - 1):
        yield cu_q[i], cu_q[i + 1], cu_k[i], cu_k[i + 1]


def attention(q, k, v, cu_q, cu_k=None, scale=None):
    """dict: out [P,Tq,hq,dh], lse [P,hq,Tq], A = sum_j p_j |v_j|, M [P,hq,Tq] = the largest
    visible scale sum_d |q_d k_d| and n, the most terms a sum has.  Rows outside every sequence are NaN."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    P, Tq, hq, dh = q.shape
    group = hq // k.shape[2]
    scale = dh ** -0.5 if scale is None else scale
    out, A = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse, M = np.full((P, hq, Tq), np.nan), np.full((P, hq, Tq), np.nan)
    for a, b, c, d in _sequences(cu_q, cu_k):
        see = _visible(b - a, d - c)
        some = see.any(1)
        for r in range(P):
            for h in range(hq):
                K, V = k[r, c:d, h // group], v[r, c:d, h // group]
                S = np.where(see, scale * (q[r, a:b, h] @ K.T), -np.inf)
                top = np.where(some, S.max(1, initial=-np.inf), 0.0)
                E = np.exp(S - top[:, None])
                Z = E.sum(1)
                with np.errstate(divide="ignore", invalid="ignore"):
                    W = np.where(some[:, None], E / Z[:, None], 0.0)
                    lse[r, h, a:b] = np.where(some, top + np.log(Z), -np.inf)
                out[r, a:b, h], A[r, a:b, h] = W @ V, W @ np.abs(V)
                M[r, h, a:b] = np.where(see, scale * (np.abs(q[r, a:b, h]) @ np.abs(K).T), 0).max(1, initial=0.0)
    return {"out": out, "lse": lse, "A": A, "M": M, "n": k.shape[1]}


def attention_backward(q, k, v, out, lse, dout, cu_q, cu_k=None, scale=None):
    """Gradients from the forward's out and lse as given: dict dq, dk, dv with, for each, `*_abs`
    (the sum of the absolute values of its terms) and for dq, dk `*_wide` (the same with
    |dP| and |D| replaced by their sums of absolute values, which bounds cancellation).

    D = rowsum(dout out).  Of a sequence's queries, taken 128 at a time, those that all see 128 keys at most
    have the sum of P dP instead, for which the former stands: the stored out has it rounded."""
    q, k, v, out, lse, dout = (_f64(x) for x in (q, k, v, out, lse, dout))
    P, Tq, hq, dh = q.shape
    out, dout = out.reshape(q.shape), dout.reshape(q.shape)
    group = hq // k.shape[2]
    scale = dh ** -0.5 if scale is None else scale
    g = {n: np.full(q.shape, np.nan) for n in ("dq", "dq_abs", "dq_wide")}
    g.update({n: np.full(k.shape, np.nan) for n in ("dk", "dk_abs", "dk_wide", "dv", "dv_abs")})
    for a, b, c, d in _sequences(cu_q, cu_k):
        see = _visible(b - a, d - c)
        for n in ("dk", "dk_abs", "dk_wide", "dv", "dv_abs"):
            g[n][:, c:d] = 0.0
        for r in range(P):
            for h in range(hq):
                kv = h // group
                Q, K, V, G = q[r, a:b, h], k[r, c:d, kv], v[r, c:d, kv], dout[r, a:b, h]
                L = np.where(np.isfinite(lse[r, h, a:b]), lse[r, h, a:b], 0.0)[:, None]
                W = np.exp(np.where(see, scale * (Q @ K.T) - L, -np.inf))
                dP, wide_P = G @ V.T, np.abs(G) @ np.abs(V).T
                D = (G * out[r, a:b, h]).sum(1, keepdims=True)
                wide_D = (np.abs(G) * np.abs(out[r, a:b, h])).sum(1, keepdims=True)
                for i in range(0, b - a, 128):
                    e = min(i + 128, b - a)
                    if e + (d - c) - (b - a) <= 128:
                        D[i:e] = (W[i:e] * dP[i:e]).sum(1, keepdims=True)
                        wide_D[i:e] = (W[i:e] * wide_P[i:e]).sum(1, keepdims=True)
                dS = scale * W * (dP - D)
                wide = scale * W * (wide_P + wide_D)
                g["dq"][r, a:b, h], g["dq_abs"][r, a:b, h] = dS @ K, np.abs(dS) @ np.abs(K)
                g["dq_wide"][r, a:b, h] = wide @ np.abs(K)
                g["dk"][r, c:d, kv] += dS.T @ Q
                g["dk_abs"][r, c:d, kv] += np.abs(dS).T @ np.abs(Q)
                g["dk_wide"][r, c:d, kv] += wide.T @ np.abs(Q)
                g["dv"][r, c:d, kv] += W.T @ G
                g["dv_abs"][r, c:d, kv] += W.T @ np.abs(G)
    g["n"] = max(group * Tq, k.shape[1])
    return g


def decode(q, k_cache, v_cache, lens, scale=None):
    """dict out [P,B,hq,dh], A, M: one query per sequence over the first lens[b] rows of its slab."""
    P, B, hq, dh = q.shape
    o = {"out": np.zeros(q.shape), "A": np.zeros(q.shape), "M": np.zeros((P, B, hq)), "n": k_cache.shape[2]}
    for b, n in enumerate(lens):
        if n == 0:
            continue
        x = attention(q[:, b:b + 1], k_cache[:, b, :n], v_cache[:, b, :n], [0, 1], [0, n], scale)
        o["out"][:, b], o["A"][:, b], o["M"][:, b] = x["out"][:, 0], x["A"][:, 0], x["M"][:, :, 0]
    return o
