"""Layouts of the attention block's tensors, as the binding hands them to the library, and what the library
refuses of them before any device work."""
import ctypes

import numpy as np
import pytest
import torch

from partial_activation_sync_caat_b200 import build as B
from partial_activation_sync_caat_b200 import caat as C


def heads4(t):
    return C._heads4(t, "q", torch.bfloat16, -1)[1:]


@pytest.mark.parametrize("shape,to", [((1, 1, 4, 64), (2, 100, 4, 64)), ((4, 64), (1, 100, 4, 64)), ((3, 1, 4, 64), (3, 100, 4, 64)),
                                      ((1, 1, 1, 64), (1, 2, 1, 64)), ((1, 1, 1, 64), (8, 16, 1, 64))])
def test_expanded_tokens_are_refused(shape, to):
    """Strides (0, 0) mean a contiguous tensor to the library, which an expanded one is not."""
    x = torch.zeros(shape, dtype=torch.bfloat16).expand(to)
    assert not x.is_contiguous()
    with pytest.raises(ValueError, match="share memory"):
        heads4(x)


def test_tokens_that_overlap_are_refused():
    x = torch.zeros(4096, dtype=torch.bfloat16).as_strided((2, 4, 2, 64), (1024, 64, 64, 1))
    with pytest.raises(ValueError, match="share memory"):
        heads4(x)


def test_strides_that_are_passed_on():
    x = torch.zeros(2, 5, 4, 64, dtype=torch.bfloat16)
    assert heads4(x) == (0, 0)
    assert heads4(x[:, :, :2]) == (5 * 256, 256)
    assert heads4(x[:, ::2]) == (5 * 256, 512)
    # one token, or one rank: that dimension has no stride to speak of
    assert heads4(x[:1].expand(1, 5, 4, 64)) == (0, 0)
    assert heads4(x[:, :1]) == (5 * 256, 256)
    assert heads4(x[:1, :, 1:]) == (5 * 256, 256)
    assert heads4(torch.zeros(0, 5, 4, 64, dtype=torch.bfloat16)) == (0, 0)


@pytest.fixture(scope="module")
def L():
    B.build()
    return C.lib()


# Positions at an odd address are refused behind the checks of what overlaps: a call that gets as far is one
# whose layout was accepted, and still launches nothing.
ACCEPTED, REFUSED = C.CAAT_ERR_UNSUPPORTED, C.CAAT_ERR_INVALID_ARG


def turned(L, P, T, dh=64, **tensors):
    """caat_rope on tensors given as (first element, heads, rank stride, token stride, in place) in one buffer."""
    base, f = 1 << 32, np.ones(dh // 2)
    a = C.RopeArgs(inv_freq=f.ctypes.data, positions=0x8002, T=T, P=P, dh=dh, rot=dh, mscale=1.0)
    for name, (at, heads, rank, token, in_place) in tensors.items():
        p = base + 2 * at
        setattr(a, name, p)
        setattr(a, "heads_" + name, heads)
        setattr(a, name + "_stride_rank", rank)
        setattr(a, name + "_stride_token", token)
        setattr(a, name + "_out", p if in_place else (1 << 40) + (ord(name) << 34))
    return L.caat_rope(ctypes.byref(a))


def shares(P, T, *tensors):
    """Whether any two rows of the tensors ((first element, row length, rank stride, token stride)) share an
    element, found by marking them."""
    marked = set()
    for at, row, rank, token in tensors:
        for r in range(P):
            for t in range(T):
                cells = set(range(at + r * rank + t * token, at + r * rank + t * token + row))
                if marked & cells:
                    return True
                marked |= cells
    return False


def test_rotated_in_place_ranks_inside_a_token(L):
    S = 2 * 64
    for T in (2, 5):
        # [T, 4, heads, dh]: q is ranks 0 and 1, k ranks 1 and 2 (k of rank 0 is q of rank 1), or 2 and 3
        q = (0, 2, S, 4 * S, True)
        assert turned(L, 2, T, q=q, k=(S, 2, S, 4 * S, True)) == REFUSED
        assert turned(L, 2, T, q=q, k=(S, 2, S, 4 * S, False)) == REFUSED
        assert turned(L, 2, T, q=q, k=(2 * S, 2, S, 4 * S, True)) == ACCEPTED
        # ranks two apart, the other tensor's between them; and one that reaches into the next token
        assert turned(L, 2, T, q=(0, 2, 2 * S, 4 * S, True), k=(S, 2, 2 * S, 4 * S, True)) == ACCEPTED
        assert turned(L, 2, T, q=(0, 2, 2 * S, 4 * S, True), k=(2 * S, 2, 2 * S, 4 * S, True)) == REFUSED
        assert turned(L, 2, T, q=(0, 2, 3 * S, 4 * S, True), k=(S, 2, 3 * S, 4 * S, True)) == REFUSED


@pytest.mark.parametrize("seed", range(4))
def test_rotated_in_place_against_marked_elements(L, seed):
    """Random layouts of two tensors: refused exactly where elements are shared (with strides in common)."""
    rng = np.random.default_rng(seed)
    counts = {ACCEPTED: 0, REFUSED: 0}
    for _ in range(400):
        P, T = int(rng.integers(1, 4)), int(rng.integers(2, 5))
        hq, hk = int(rng.integers(1, 3)), int(rng.integers(1, 3))
        dh = 16
        rank, token = (dh * int(rng.integers(2, 13)) for _ in range(2))
        q, k = (0, hq * dh, rank, token), (8 * int(rng.integers(-30, 90)), hk * dh, rank, token)
        shared = shares(P, T, q, k)
        code = turned(L, P, T, dh, q=(q[0], hq, rank, token, True), k=(k[0], hk, rank, token, True))
        assert code == (REFUSED if shared else ACCEPTED), (P, T, q, k)
        counts[code] += 1
    assert min(counts.values()) > 40


def test_one_token_turned_in_place(L):
    """A single token has no token stride: slices of one projection [P, 1, all] are apart by their rank stride,
    whatever the call gives for the other one."""
    hq, hk, dh, P = 4, 2, 64, 3
    every, k0 = (hq + 2 * hk) * dh, hq * dh
    for token_q, token_k in ((every, every), (hq * dh, hk * dh)):
        q, k = (0, hq, every, token_q, True), (k0, hk, every, token_k, True)
        assert turned(L, P, 1, q=q, k=k) == ACCEPTED
        assert turned(L, P, 1, q=q, k=(*k[:4], False)) == ACCEPTED
        assert turned(L, 1, 1, q=q, k=k) == ACCEPTED
        assert turned(L, P, 1, q=q, k=(k0 - 8, hk, every, token_k, True)) == REFUSED
        assert turned(L, P, 1, q=q, k=(every + 8, hk, every, token_k, True)) == REFUSED
        assert turned(L, P, 1, q=q, k=(k0, hk, every + 8, token_k, True)) == REFUSED  # (strides of its own)
