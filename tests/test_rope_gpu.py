"""GPU parity of the rotary positions (and of the append to a cache) with the float64 oracle.

Tolerance: the angle's fraction of a turn is exact to about 1e-9 and cos, sin come from fp32 (2^-22
with the scaling), so y = mscale (a cos - b sin) is off by at most 2^-21 mscale (|a| + |b|) before its one
rounding to bf16 (2^-8 relative)."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as A
from oracle import caat_oracle as O
from partial_activation_sync_caat_b200 import caat as C

from gpu_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def draw(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def check(got, x, positions, freq, inter, backward, mscale, what):
    ref = A.rope(x, positions, freq, inter, backward, mscale)
    size = A.rope(np.abs(O._f64(x)), np.zeros(len(positions)), freq, inter, False, mscale)
    rot = 2 * len(freq)
    first = np.arange(0, rot, 2) if inter else np.arange(rot // 2)
    second = first + 1 if inter else first + rot // 2
    size[..., first] = size[..., second] = size[..., first] + size[..., second]
    err = np.abs(O._f64(got) - ref)
    bound = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * 2.0 ** -21 * size
    bound[..., rot:] = 0.0
    assert (err <= bound).all(), f"{what}: max err {err.max():.3e}"


@pytest.mark.parametrize("P,T,hq,hk,dh,rot,inter,scaling,backward", [
    (1, 1, 1, 1, 128, 128, False, "none", False), (2, 5, 4, 2, 64, 64, True, "none", False),
    (8, 3, 4, 4, 128, 64, False, "linear", False), (1, 300, 3, 1, 96, 48, False, "yarn", True),
    (2, 129, 6, 2, 96, 96, True, "ntk", True), (1, 17, 1, 1, 8, 8, True, "none", False),
    (1, 9, 2, 1, 256, 256, False, "yarn", False), (1, 1025, 2, 2, 72, 16, False, "none", False),
    (3, 70, 5, 1, 80, 8, True, "linear", True)])
def test_matches_oracle(P, T, hq, hk, dh, rot, inter, scaling, backward):
    q, k = draw(1, P, T, hq, dh), draw(2, P, T, hk, dh)
    freq, mscale = C.caat_rope_frequencies(rot, 10000.0, scaling, 4.0)
    rng = np.random.default_rng(T)
    pos = rng.integers(0, 200000, T).astype(np.int32)
    qo, ko = torch.zeros_like(q).cuda(), torch.zeros_like(k).cuda()
    C.caat_rope(q.cuda(), k.cuda(), torch.tensor(pos).cuda(), freq, q_out=qo, k_out=ko, interleaved=inter,
                backward=backward, mscale=mscale)
    check(qo.cpu(), q, pos, freq, inter, backward, mscale, "q")
    check(ko.cpu(), k, pos, freq, inter, backward, mscale, "k")


def test_far_and_negative_positions():
    pos = np.array([2**31 - 1, -(2**31), 10**9 + 7, -1, 0, 123456789], dtype=np.int32)
    q = draw(3, 1, len(pos), 2, 128)
    freq, _ = C.caat_rope_frequencies(128)
    qo = torch.empty_like(q).cuda()
    C.caat_rope(q.cuda(), None, torch.tensor(pos).cuda(), freq, q_out=qo, k_out=None)
    # the oracle's own angle, position times frequency in float64, is off by up to 2^31 2^-53: under 2^-21
    check(qo.cpu(), q, pos, freq, False, False, 1.0, "far")


def test_in_place_default_positions_and_strides():
    P, T, hq, hk, dh = 2, 37, 4, 2, 64
    freq, _ = C.caat_rope_frequencies(64)
    qkv = draw(4, P, T, (hq + 2 * hk) * dh).cuda()
    q, k, v = (x.unflatten(-1, (-1, dh)) for x in qkv.split([hq * dh, hk * dh, hk * dh], -1))
    q0, k0, v0 = q.cpu().clone(), k.cpu().clone(), v.cpu().clone()
    qo, ko = torch.empty(P, T, hq, dh, dtype=torch.bfloat16, device="cuda"), torch.empty(P, T, hk, dh, dtype=torch.bfloat16, device="cuda")
    C.caat_rope(q, k, None, freq, q_out=qo, k_out=ko)
    C.caat_rope(q, k, None, freq, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v.cpu(), v0)
    check(q.cpu(), q0, np.arange(T), freq, False, False, 1.0, "q")
    check(k.cpu(), k0, np.arange(T), freq, False, False, 1.0, "k")


def test_append_to_a_cache():
    P, T, hq, hk, dh, B, cap = 2, 6, 4, 2, 96, 3, 11
    q, k, v = draw(5, P, T, hq, dh), draw(6, P, T, hk, dh), draw(7, P, T, hk, dh)
    kc, vc = draw(8, P, B, cap, hk, dh), draw(9, P, B, cap, hk, dh)
    freq, _ = C.caat_rope_frequencies(32)
    pos = np.array([0, 4, 10, 3, 2, 9], dtype=np.int32)
    slots = np.array([0, cap + 4, 2 * cap + 10, -1, 2, 9], dtype=np.int64)
    kd, vd, qo = kc.cuda(), vc.cuda(), torch.empty_like(q).cuda()
    C.caat_rope_append(q.cuda(), k.cuda(), v.cuda(), torch.tensor(pos).cuda(), torch.tensor(slots).cuda(), freq, kd, vd, q_out=qo)
    assert C.caat_get_device_status() == 0
    check(qo.cpu(), q, pos, freq, False, False, 1.0, "q")
    kept = np.ones(B * cap, bool)
    kept[slots[slots >= 0]] = False
    kf, vf = kd.cpu().view(P, B * cap, hk, dh), vd.cpu().view(P, B * cap, hk, dh)
    assert torch.equal(kf[:, kept], kc.view(P, -1, hk, dh)[:, kept]) and torch.equal(vf[:, kept], vc.view(P, -1, hk, dh)[:, kept])
    on = slots >= 0
    assert torch.equal(vf[:, slots[on]], v[:, on])
    check(kf[:, slots[on]], k[:, on], pos[on], freq, False, False, 1.0, "k cache")


def test_slots_outside_the_cache_are_reported_and_skipped():
    k, v = draw(1, 1, 3, 1, 64), draw(2, 1, 3, 1, 64)
    freq, _ = C.caat_rope_frequencies(64)
    kc = torch.full((1, 4, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    slots = torch.tensor([4, 1, -7], device="cuda")
    C.caat_rope_append(None, k.cuda(), v.cuda(), None, slots, freq, kc, vc)
    assert C.caat_get_device_status() & 0xFF == C.CAAT_ERR_INVALID_ARG
    assert C.caat_get_device_status() == 0
    assert torch.equal(vc[0, 1].cpu(), v[0, 1]) and bool((kc[0, [0, 2, 3]] == 5).all()) and bool((vc[0, [0, 2, 3]] == 5).all())


def test_backward_is_the_transpose():
    """<R x, y> = <x, R^T y>, each side rounded once per element: 2^-8 relative on sums of absolute values."""
    x, y = draw(11, 1, 50, 2, 64), draw(12, 1, 50, 2, 64)
    freq, mscale = C.caat_rope_frequencies(48, 10000.0, "yarn", 8.0)
    a, b = torch.empty_like(x).cuda(), torch.empty_like(y).cuda()
    for inter in (False, True):
        C.caat_rope(x.cuda(), None, None, freq, q_out=a, k_out=None, interleaved=inter, mscale=mscale)
        C.caat_rope(y.cuda(), None, None, freq, q_out=b, k_out=None, interleaved=inter, mscale=mscale, backward=True)
        l, r = a.double().cpu() * y.double(), x.double() * b.double().cpu()
        assert abs(float(l.sum() - r.sum())) <= 2.0 ** -8 * float(l.abs().sum() + r.abs().sum())


def test_captured():
    q = draw(13, 1, 20, 2, 64).cuda()
    freq, _ = C.caat_rope_frequencies(64)
    pos = torch.arange(20, dtype=torch.int32, device="cuda")
    out, ref = torch.empty_like(q), torch.empty_like(q)
    C.caat_rope(q, None, pos, freq, q_out=out, k_out=None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        C.caat_rope(q, None, pos, freq, q_out=out, k_out=None)
    pos += 100
    graph.replay()
    C.caat_rope(q, None, pos, freq, q_out=ref, k_out=None)
    assert torch.equal(out, ref)
