"""The prompt attention's CTAs with two tiles of 128 queries (heads wider than 64, more tiles than SMs): two heads
of a group on the same rows where the group is even, 256 rows of one head where it is odd.  What the other tests
show at sizes that take one tile a CTA, here with both tiles in use."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as A
from oracle import caat_oracle as O

from attn_util import check_grads, check_lse, check_out
from gpu_util import ensure_built
from test_attn_gpu import backward, forward, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def two(P, hq, hk, dh, lens, klens=None, **kw):
    """Inputs of a call that takes two tiles a CTA: its tiles of 128 queries outnumber the SMs."""
    tiles = sum((n + 127) // 128 for n in lens) * P * hq
    assert dh > 64 and tiles > torch.cuda.get_device_properties(0).multi_processor_count
    return make(P, hq, hk, dh, lens, klens, **kw)


EVEN, ODD = (4, 2), (3, 1)  # heads of queries and keys
BOTH = pytest.mark.parametrize("hq,hk", [EVEN, ODD], ids=["two heads", "256 rows"])


@pytest.mark.parametrize("P,hq,hk,dh,lens,klens", [
    (4, 6, 2, 128, [1100, 130, 1], None),      # rows: 256 of one head, more than eight blocks of keys
    (4, 4, 1, 96, [1030, 257], None),          # heads in pairs
    (4, 4, 2, 128, [700, 257, 40], [1300, 257, 41]),
    (8, 5, 5, 72, [500, 129], [1025, 700]),
    (16, 3, 1, 128, [300, 200], [100, 30]),    # first tiles that see no key, or part of one
    (16, 4, 2, 128, [300, 200], [100, 0]),
    (64, 3, 3, 80, [129, 1, 256, 255, 127], None),
    (64, 2, 1, 128, [129, 1, 256, 255, 127], None),
])
def test_matches_oracle(P, hq, hk, dh, lens, klens):
    d = two(P, hq, hk, dh, lens, klens, seed=40 + dh)
    out, lse = forward(d)
    ref = A.attention(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"])
    check_out(out.cpu(), ref)
    check_lse(lse.cpu(), ref, dh)
    again, lse2 = forward(d)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    got = {n: t.cpu() for n, t in backward(d, out, lse).items()}
    g = A.attention_backward(d["q"], d["k"], d["v"], out.cpu(), lse.cpu(), d["dout"], d["cu_q"], d["cu_k"])
    check_grads(got, g, ref["M"], dh)


@BOTH
@pytest.mark.parametrize("std,scale", [(3.0, None), (8.0, None), (1.0, 0.7), (0.01, 1e-3)])
def test_scores_of_every_size(hq, hk, std, scale):
    d = two(20, hq, hk, 128, [300], [513], seed=41, std=std)
    out, lse = forward(d, scale)
    ref = A.attention(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"], scale)
    check_out(out.cpu(), ref)
    check_lse(lse.cpu(), ref, 128)


@BOTH
def test_rising_scores_along_the_keys(hq, hk):
    """Every block moves the maximum, of the ranks with odd numbers late: only from key 600 on."""
    d = two(8, hq, hk, 128, [900], seed=42)
    at = torch.arange(900)[None, :, None, None].expand(8, 900, hk, 128) / 32.0
    late = torch.where(at * 32 < 600, torch.zeros_like(at), at)
    ramp = torch.where((torch.arange(8) % 2 == 1)[:, None, None, None], late, at)
    d["q"] = torch.ones_like(d["q"])
    d["k"] = (d["k"].float() * 0.1 + ramp).to(torch.bfloat16)
    out, lse = forward(d)
    ref = A.attention(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"])
    check_out(out.cpu(), ref)
    check_lse(lse.cpu(), ref, 128)


@BOTH
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -3.0e38])
def test_rows_outside_the_sequences(hq, hk, junk):
    P, first = 30, 3
    d = two(P, hq, hk, 128, [130, 77], [150, 90], seed=43, extra=150)
    for name, end in (("q", d["cu_q"][-1]), ("k", d["cu_k"][-1]), ("v", d["cu_k"][-1])):
        d[name][:, :first] = junk
        d[name][:, first + end:] = junk
    d["cu_q"] = [first + x for x in d["cu_q"]]
    d["cu_k"] = [first + x for x in d["cu_k"]]
    out, lse = forward(d)
    ref = A.attention(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"])
    check_out(out.cpu(), ref)
    check_lse(lse.cpu(), ref, 128)
    assert bool((out[:, :first] == 7).all()) and bool((out[:, d["cu_q"][-1]:] == 7).all())
    assert bool((lse[..., :first] == 7).all()) and bool((lse[..., d["cu_q"][-1]:] == 7).all())


@BOTH
def test_other_sequences_do_not_reach_a_row(hq, hk):
    d = two(30, hq, hk, 128, [70, 40, 90], seed=44)
    out, lse = forward(d)
    e = {n: (x.clone() if torch.is_tensor(x) else x) for n, x in d.items()}
    for name in ("q", "k", "v"):
        e[name][:, 70:110] = float("nan") if name != "v" else float("inf")
    out2, lse2 = forward(e)
    assert torch.equal(out[:, :70], out2[:, :70]) and torch.equal(out[:, 110:], out2[:, 110:])
    assert torch.equal(lse[..., :70], lse2[..., :70]) and torch.equal(lse[..., 110:], lse2[..., 110:])


@BOTH
def test_later_tokens_do_not_reach_earlier_rows(hq, hk):
    """NaN, +inf and -inf in v of single tokens, in the blocks that only some rows of a job see whole, at places
    that differ from rank to rank: each column is what it was up to its token and that value from there on."""
    P, T = 20, 600
    d = two(P, hq, hk, 128, [T], seed=45)
    out, _ = forward(d)
    e = {n: (x.clone() if torch.is_tensor(x) else x) for n, x in d.items()}
    rng = np.random.default_rng(4)
    odd = []
    for r in range(P):
        for g in range(hk):
            cols = rng.choice(128, 6, replace=False)
            for i, col in enumerate(cols):
                at, value = int(rng.integers(0, T)), [np.nan, np.inf, -np.inf][i % 3]
                e["v"][r, at, g, col] = value
                odd.append((r, g, int(col), at, value))
    out2, _ = forward(e)
    want, got = (O._f64(x.cpu()).reshape(P, T, hq, 128) for x in (out, out2))
    for r, g, col, at, value in odd:
        want[r, at:, g * (hq // hk):(g + 1) * (hq // hk), col] = value
    np.testing.assert_array_equal(got, want)


@BOTH
def test_values_that_are_not_finite_in_many_sequences(hq, hk):
    """Several units a CTA; each sequence has its own odd token, and nothing of it is left for the next."""
    rng = np.random.default_rng(5)
    P, lens = 2, rng.integers(20, 400, 90).tolist()
    d = two(P, hq, hk, 128, lens, seed=46)
    out, _ = forward(d)
    e = {n: (x.clone() if torch.is_tensor(x) else x) for n, x in d.items()}
    odd = []
    for i, n in enumerate(lens):
        at, col, value = int(rng.integers(0, n)), int(rng.integers(0, 128)), [np.nan, np.inf, -np.inf, None][i % 4]
        odd.append((at, col, value))
        if value is not None:
            e["v"][:, d["cu_k"][i] + at, :, col] = value
    out2, _ = forward(e)
    a, b = (O._f64(x.cpu()).reshape(P, -1, hq, 128) for x in (out, out2))
    for i, (at, col, value) in enumerate(odd):
        if value is not None:
            a[:, d["cu_q"][i] + at:d["cu_q"][i + 1], :, col] = value
    np.testing.assert_array_equal(b, a)
