"""GPU parity of the packed causal attention and its gradients with the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as A
from partial_activation_sync_caat_b200 import caat as C

from attn_util import check_grads, check_lse, check_out
from gpu_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def cumulative(lens):
    return [0] + np.cumsum(lens).tolist()


def make(P, hq, hk, dh, lens, klens=None, seed=0, extra=0, std=1.0):
    """q, k, v, dout on the CPU for packed sequences, with `extra` rows behind the last one."""
    g = torch.Generator().manual_seed(seed)
    cu_q, cu_k = cumulative(lens), cumulative(lens if klens is None else klens)
    Tq, Tk = cu_q[-1] + extra, cu_k[-1] + extra

    def draw(*shape):
        return (std * torch.randn(*shape, generator=g)).to(torch.bfloat16)

    return {"q": draw(P, Tq, hq, dh), "k": draw(P, Tk, hk, dh), "v": draw(P, Tk, hk, dh), "dout": draw(P, Tq, hq * dh),
            "cu_q": cu_q, "cu_k": cu_k}


def forward(d, scale=None, **kw):
    q, k, v = d["q"].cuda(), d["k"].cuda(), d["v"].cuda()
    P, Tq, hq, dh = q.shape
    out = torch.full((P, Tq, hq * dh), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((P, hq, Tq), 7.0, dtype=torch.float32, device="cuda")
    C.caat_attn_forward(q, k, v, d["cu_q"], out, cu_k=d["cu_k"], lse=lse, scale=scale, **kw)
    torch.cuda.synchronize()
    assert C.caat_get_device_status() == 0
    return out, lse


def backward(d, out, lse, scale=None, **kw):
    q, k, v = d["q"].cuda(), d["k"].cuda(), d["v"].cuda()
    dq, dk, dv = (torch.full_like(x, 7.0) for x in (q, k, v))
    C.caat_attn_backward(q, k, v, out, lse, d["dout"].cuda(), d["cu_q"], dq, dk, dv, cu_k=d["cu_k"], scale=scale, **kw)
    torch.cuda.synchronize()
    assert C.caat_get_device_status() == 0
    return {"dq": dq, "dk": dk, "dv": dv}


CASES = [
    # P, hq, hk, dh, query lengths, key lengths (None: the same)
    (1, 1, 1, 128, [1], None),
    (2, 2, 2, 128, [128], None),
    (1, 2, 2, 128, [129, 127], None),
    (2, 4, 2, 128, [257, 1, 64], None),
    (1, 4, 1, 64, [300, 0, 5, 513], None),
    (1, 3, 3, 64, [255, 256], None),
    (1, 3, 1, 64, [130, 31], None),
    (1, 2, 1, 96, [200, 33], None),
    (1, 2, 2, 8, [70], None),
    (1, 2, 2, 72, [140], None),
    (1, 2, 1, 128, [1, 130, 7], [300, 131, 129]),
    (1, 2, 2, 64, [200, 3], [64, 0]),
    (1, 8, 1, 128, [385], [600]),
    (3, 2, 2, 128, [640], None),
    (1, 2, 2, 64, [0, 0, 17], None),
    (1, 1, 1, 128, [5], [0]),
    (1, 16, 2, 64, [90, 260], [400, 261]),
    # more work items than SMs, several to a CTA
    (8, 4, 4, 128, [300, 1, 129, 260], None),
    (4, 8, 2, 128, [140, 70, 257, 3, 128], [150, 70, 300, 2, 128]),
    (64, 1, 1, 16, [65, 64, 63], None),
    # tiles that see 64, 65, 128 or 129 keys: where blocks, and the pass for D, end
    (2, 2, 1, 64, [64, 65, 128, 129], None),
    (2, 2, 1, 64, [100, 28, 1], [128, 129, 64]),
    (1, 3, 1, 128, [100, 28, 129], [128, 129, 130]),
    # a key tile's queries shared by CTAs
    (1, 8, 1, 64, [1500], None),
    (1, 4, 2, 96, [700, 20], [721, 20]),
]


@pytest.mark.parametrize("P,hq,hk,dh,lens,klens", CASES)
def test_forward_matches_oracle(P, hq, hk, dh, lens, klens):
    d = make(P, hq, hk, dh, lens, klens, seed=sum(lens))
    out, lse = forward(d)
    ref = A.attention(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"])
    check_out(out.cpu(), ref)
    check_lse(lse.cpu(), ref, dh)


@pytest.mark.parametrize("P,hq,hk,dh,lens,klens", CASES)
def test_backward_matches_oracle(P, hq, hk, dh, lens, klens):
    d = make(P, hq, hk, dh, lens, klens, seed=1 + sum(lens))
    out, lse = forward(d)
    got = {n: t.cpu() for n, t in backward(d, out, lse).items()}
    M = A.attention(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"])["M"]
    ref = A.attention_backward(d["q"], d["k"], d["v"], out.cpu(), lse.cpu(), d["dout"], d["cu_q"], d["cu_k"])
    check_grads(got, ref, M, dh)


@pytest.mark.parametrize("std,scale", [(3.0, None), (8.0, None), (1.0, 0.7), (0.01, 1e-3)])
def test_scores_of_every_size(std, scale):
    """Large scores (one key takes nearly everything, the running maximum moves by far) and tiny ones."""
    d = make(1, 2, 1, 64, [300], [513], seed=5, std=std)
    out, lse = forward(d, scale)
    ref = A.attention(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"], scale)
    check_out(out.cpu(), ref)
    check_lse(lse.cpu(), ref, 64)
    got = {n: t.cpu() for n, t in backward(d, out, lse, scale).items()}
    g = A.attention_backward(d["q"], d["k"], d["v"], out.cpu(), lse.cpu(), d["dout"], d["cu_q"], d["cu_k"], scale)
    check_grads(got, g, ref["M"], 64)


def test_rising_scores_along_the_keys():
    """Scores that grow from key block to key block: every block moves the maximum."""
    d = make(1, 1, 1, 64, [640], seed=6)
    ramp = torch.arange(640)[None, :, None, None] / 16.0
    d["q"] = torch.ones_like(d["q"])
    d["k"] = (d["k"].float() * 0.1 + ramp).to(torch.bfloat16)
    out, lse = forward(d)
    ref = A.attention(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"])
    check_out(out.cpu(), ref)
    check_lse(lse.cpu(), ref, 64)


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -3.0e38])
def test_rows_outside_the_sequences(junk):
    """Whatever stands before the first and behind the last sequence is neither used nor overwritten."""
    d = make(1, 4, 2, 128, [130, 77], [150, 90], seed=8, extra=150)
    first = 3  # the sequences start behind three rows of junk
    for name, end in (("q", d["cu_q"][-1]), ("k", d["cu_k"][-1]), ("v", d["cu_k"][-1]), ("dout", d["cu_q"][-1])):
        d[name][:, :first] = junk
        d[name][:, first + end:] = junk
    d["cu_q"] = [first + x for x in d["cu_q"]]
    d["cu_k"] = [first + x for x in d["cu_k"]]
    out, lse = forward(d)
    ref = A.attention(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"])
    check_out(out.cpu(), ref)
    check_lse(lse.cpu(), ref, 128)
    grads = backward(d, out, lse)
    g = A.attention_backward(d["q"], d["k"], d["v"], out.cpu(), lse.cpu(), d["dout"], d["cu_q"], d["cu_k"])
    check_grads({n: t.cpu() for n, t in grads.items()}, g, ref["M"], 128)
    for t, cu in ((out, d["cu_q"]), (grads["dq"], d["cu_q"]), (grads["dk"], d["cu_k"]), (grads["dv"], d["cu_k"])):
        assert bool((t[:, :first] == 7).all()) and bool((t[:, cu[-1]:] == 7).all())
    assert bool((lse[..., :first] == 7).all()) and bool((lse[..., d["cu_q"][-1]:] == 7).all())


def test_other_sequences_do_not_reach_a_row():
    """NaN and infinities in one packed sequence leave its neighbours' results as they are, bit for bit."""
    d = make(1, 2, 1, 64, [70, 40, 90], seed=9)
    out, lse = forward(d)
    grads = backward(d, out, lse)
    e = {n: (x.clone() if torch.is_tensor(x) else x) for n, x in d.items()}
    for name in ("q", "k", "v", "dout"):
        e[name][:, 70:110] = float("nan") if name != "v" else float("inf")
    out2, lse2 = forward(e)
    grads2 = backward(e, out2, lse2)
    for a, b in ((out, out2), *((grads[n], grads2[n]) for n in grads)):
        assert torch.equal(a[:, :70], b[:, :70]) and torch.equal(a[:, 110:], b[:, 110:])
    assert torch.equal(lse[..., :70], lse2[..., :70]) and torch.equal(lse[..., 110:], lse2[..., 110:])


def test_later_tokens_do_not_reach_earlier_rows():
    """Causality for values that are not finite: NaN, +inf and -inf in v (and k) of one token leave the
    rows before it as they are."""
    d = make(1, 2, 1, 64, [200], seed=10)
    out, lse = forward(d)
    e = {n: (x.clone() if torch.is_tensor(x) else x) for n, x in d.items()}
    e["v"][0, 150, 0, 3], e["v"][0, 160, 0, 5], e["v"][0, 40, 0, 7] = float("nan"), float("inf"), -float("inf")
    e["k"][0, 180, 0, 1] = float("nan")
    out2, lse2 = forward(e)
    assert torch.equal(lse[..., :180], lse2[..., :180])
    o, o2 = out.view(1, 200, 2, 64), out2.view(1, 200, 2, 64)
    assert torch.equal(o[:, :40], o2[:, :40])
    keep = [c for c in range(64) if c not in (3, 5, 7)]
    assert torch.equal(o[:, :180, :, keep], o2[:, :180, :, keep])
    assert torch.equal(o[:, :150, :, 3], o2[:, :150, :, 3]) and bool(o2[:, 150:, :, 3].isnan().all())
    assert torch.equal(o[:, :160, :, 5], o2[:, :160, :, 5]) and bool((o2[:, 160:180, :, 5] == float("inf")).all())
    assert bool((o2[:, 40:180, :, 7] == -float("inf")).all())


def fused(d):
    """q, k, v as slices of one projection [P, T, (hq + 2 hk) dh]."""
    P, T, hq, dh = d["q"].shape
    hk = d["k"].shape[2]
    qkv = torch.cat([d[n].flatten(2) for n in ("q", "k", "v")], -1).cuda()
    q, k, v = qkv.split([hq * dh, hk * dh, hk * dh], -1)
    return q.unflatten(-1, (hq, dh)), k.unflatten(-1, (hk, dh)), v.unflatten(-1, (hk, dh))


def test_slices_of_a_fused_projection():
    d = make(2, 4, 2, 64, [150, 33], seed=11)
    out, lse = forward(d)
    grads = backward(d, out, lse)
    q, k, v = fused(d)
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    C.caat_attn_forward(q, k, v, d["cu_q"], out2, lse=lse2)
    dq, dk, dv = (torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (q, k, v))
    C.caat_attn_backward(q, k, v, out2, lse2, d["dout"].cuda(), d["cu_q"], dq, dk, dv)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        assert torch.equal(grads[n], t), n


def test_many_sequences():
    """More work items than a launch carries in its arguments."""
    lens = [(7 * i) % 23 for i in range(700)]
    d = make(1, 2, 1, 64, lens, seed=12)
    out, lse = forward(d)
    ref = A.attention(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"])
    check_out(out.cpu(), ref)
    check_lse(lse.cpu(), ref, 64)
    got = {n: t.cpu() for n, t in backward(d, out, lse).items()}
    check_grads(got, A.attention_backward(d["q"], d["k"], d["v"], out.cpu(), lse.cpu(), d["dout"], d["cu_q"]), ref["M"], 64)


def test_deterministic_and_lse_optional():
    d = make(1, 4, 2, 128, [300, 200], seed=13)
    a, lse = forward(d)
    b, _ = forward(d)
    assert torch.equal(a, b)
    c = torch.empty_like(a)
    C.caat_attn_forward(d["q"].cuda(), d["k"].cuda(), d["v"].cuda(), d["cu_q"], c)
    assert torch.equal(a, c)
    g, h = backward(d, a, lse), backward(d, a, lse)
    assert all(torch.equal(g[n], h[n]) for n in g)


def test_captured_and_on_another_stream():
    d = make(1, 2, 2, 64, [200, 57], seed=14)
    out, lse = forward(d)
    grads = backward(d, out, lse)
    q, k, v, dout = (d[n].cuda() for n in ("q", "k", "v", "dout"))
    o, l = torch.zeros_like(out), torch.zeros_like(lse)
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))
    ws = [C.alloc_workspace(C.caat_attn_workspace_size(257, 257, 2, 1, 2, 2, 64, n))
          for n in (C.CAAT_VARIANT_ATTN, C.CAAT_VARIANT_ATTN_BWD)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def both():
        C.caat_attn_forward(q, k, v, d["cu_q"], o, lse=l, workspace=ws[0], stream=side)
        C.caat_attn_backward(q, k, v, o, l, dout, d["cu_q"], dq, dk, dv, workspace=ws[1], stream=side)

    both()
    side.synchronize()
    assert torch.equal(out, o) and torch.equal(lse, l) and torch.equal(grads["dk"], dk)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both()
    for t in (o, l, dq, dk, dv):
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o) and torch.equal(lse, l)
    assert torch.equal(grads["dq"], dq) and torch.equal(grads["dk"], dk) and torch.equal(grads["dv"], dv)


def test_gradient_against_differences():
    """Directional differences of the float64 forward at the same point."""
    d = make(1, 2, 1, 64, [60, 20], [80, 20], seed=15)
    out, lse = forward(d)
    got = backward(d, out, lse)
    g = torch.Generator().manual_seed(1)
    for name in ("q", "k", "v"):
        u = torch.randn(d[name].shape, generator=g, dtype=torch.float64).numpy()
        h = 1e-4
        x = d[name].double().numpy()
        ends = []
        for s in (h, -h):
            e = {n: d[n].double().numpy() for n in ("q", "k", "v")}
            e[name] = x + s * u
            o = A.attention(e["q"], e["k"], e["v"], d["cu_q"], d["cu_k"])["out"]
            ends.append((o.reshape(1, -1, 128) * d["dout"].double().numpy()).sum())
        slope = (ends[0] - ends[1]) / (2 * h)
        t = got["d" + name].double().cpu().numpy()
        # each of the n elements is off by a few bf16 steps at most, with a sign of its own; u ~ N(0, 1):
        # 6 standard deviations of the sum of n independent errors of 3 u |element|, and the O(h^2) difference
        assert abs((t * u).sum() - slope) <= 6 * 3 * 2.0 ** -8 * np.sqrt((t * t).sum()) + 1e-4 * abs(slope)


def test_values_that_are_not_finite_in_many_sequences():
    """As above with several work items per CTA: each sequence has its own odd token (NaN, +inf, -inf or
    none), and nothing of it is left for the next."""
    rng = np.random.default_rng(3)
    lens = rng.integers(20, 150, 250).tolist()
    d = make(1, 2, 1, 64, lens, seed=16)
    out, _ = forward(d)
    e = {n: (x.clone() if torch.is_tensor(x) else x) for n, x in d.items()}
    odd = []
    for i, n in enumerate(lens):
        at, col, value = int(rng.integers(0, n)), int(rng.integers(0, 64)), [np.nan, np.inf, -np.inf, None][i % 4]
        odd.append((at, col, value))
        if value is not None:
            e["v"][0, d["cu_k"][i] + at, 0, col] = value
    out2, _ = forward(e)
    a, b = (x.view(-1, 2, 64).float().cpu().numpy() for x in (out, out2))
    for i, (at, col, value) in enumerate(odd):
        q0, q1 = d["cu_q"][i], d["cu_q"][i + 1]
        want = a[q0:q1].copy()
        if value is not None:
            want[at:, :, col] = value
        np.testing.assert_array_equal(b[q0:q1], want)


def test_two_streams_at_once():
    """Calls that overlap on the GPU, each with its own workspace, give what they give alone."""
    many = make(1, 2, 1, 64, [(5 * i) % 31 for i in range(600)], seed=17)
    long = make(2, 2, 2, 128, [900], seed=18)
    want = [forward(x) for x in (many, long)]
    grads = [backward(x, *w) for x, w in zip((many, long), want)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for x, w, st in zip((many, long), want, streams):
        with torch.cuda.stream(st):
            t = {n: x[n].cuda() for n in ("q", "k", "v", "dout")}
            o, l = torch.empty_like(w[0]), torch.empty_like(w[1])
            g = [torch.empty_like(t[n]) for n in ("q", "k", "v")]
            for _ in range(5):
                C.caat_attn_forward(t["q"], t["k"], t["v"], x["cu_q"], o, lse=l)
                C.caat_attn_backward(t["q"], t["k"], t["v"], o, l, t["dout"], x["cu_q"], *g)
            got.append((o, l, g, t))
    torch.cuda.synchronize()
    assert C.caat_get_device_status() == 0
    for (o, l, g, _), w, h in zip(got, want, grads):
        assert torch.equal(o, w[0]) and torch.equal(l, w[1])
        assert all(torch.equal(x, h[n]) for x, n in zip(g, ("dq", "dk", "dv")))


def test_rows_past_two_to_the_31_elements():
    """Rows whose element offset does not fit in 32 bits: the last tokens of a buffer of 2.2 10^9 elements
    (those before the only sequence are never touched, and never read)."""
    hq, hk, dh, n = 16, 1, 128, 200
    T = (1 << 31) // (hq * dh) + 30000
    small = make(1, hq, hk, dh, [n], seed=19)
    want, lse_w = forward(small)
    q = torch.empty(1, T, hq, dh, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.empty(1, T, hk, dh, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out, dout = (torch.empty(1, T, hq * dh, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse = torch.empty(1, hq, T, dtype=torch.float32, device="cuda")
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (dout, "dout")):
        t[:, T - n:] = small[name].cuda()
    cu = [T - n, T]
    C.caat_attn_forward(q, k, v, cu, out, lse=lse)
    assert torch.equal(out[:, T - n:], want) and torch.equal(lse[..., T - n:], lse_w)
    dq, dk, dv = (torch.empty_like(x) for x in (q, k, v))
    C.caat_attn_backward(q, k, v, out, lse, dout, cu, dq, dk, dv)
    # a longer buffer's key sums are split differently, so these go against the oracle, not bit for bit
    M = A.attention(small["q"], small["k"], small["v"], [0, n])["M"]
    ref = A.attention_backward(small["q"], small["k"], small["v"], want.cpu(), lse_w.cpu(), small["dout"], [0, n])
    check_grads({"dq": dq[:, T - n:].cpu(), "dk": dk[:, T - n:].cpu(), "dv": dv[:, T - n:].cpu()}, ref, M, dh)
    assert C.caat_get_device_status() == 0
