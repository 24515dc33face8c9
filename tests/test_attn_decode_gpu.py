"""GPU parity of decoding against a cache with the float64 oracle, and the attention block as a user
runs it: rotation, attention, the partially synchronized output projection, and back."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as A
from oracle import caat_oracle as O
from partial_activation_sync_caat_b200 import caat as C

from attn_util import check_out
from gpu_util import assert_out_close, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def draw(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def slab(x, capacity):
    """The cache with more rows behind, of NaN (or as it is)."""
    if not capacity:
        return x.cuda()
    P, B, cap, hk, dh = x.shape
    y = torch.full((P, B, capacity, hk, dh), float("nan"), dtype=x.dtype, device="cuda")
    y[:, :, :cap] = x.cuda()
    return y


DEAL = 16500  # a capacity whose tiles are dealt to the CTAs; smaller ones have a cluster per segment


def decode(q, kc, vc, lens, **kw):
    P, B, hq, dh = q.shape
    out = torch.full((P, B, hq * dh), 7.0, dtype=torch.bfloat16, device="cuda")
    C.caat_attn_decode(q.cuda(), kc.cuda(), vc.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), out, **kw)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("P,hq,hk,dh,cap,lens", [
    (1, 1, 1, 128, 1, [1]), (1, 1, 1, 128, 64, [64]), (2, 4, 4, 128, 300, [300, 1, 65, 0, 127]),
    (1, 8, 1, 64, 1000, [1000, 64, 63, 129]), (1, 6, 2, 96, 130, [130, 3]), (1, 2, 2, 8, 77, [77, 50]),
    (1, 16, 1, 128, 200, [199, 17]), (1, 20, 1, 64, 150, [150, 2]), (1, 48, 2, 72, 90, [88, 1, 90]),
    (8, 4, 4, 128, 2000, [1999]), (1, 2, 1, 128, 9000, [8193, 9000]), (1, 3, 1, 120, 70, [0, 0, 70]),
    (4, 8, 1, 64, 40, [1 + (7 * i) % 40 for i in range(70)]),
    # clusters of 8, 4, 2 and 1 CTAs per segment, of narrow and wide heads, more than 16 query heads to a key head
    (8, 4, 4, 64, 1500, [0, 1, 1500, 127, 129]), (8, 48, 2, 72, 700, [700, 1, 0, 350, 128, 64]),
    (16, 2, 2, 128, 130, [130, 64, 65, 1, 0, 129]), (16, 17, 1, 128, 60, [60, 0, 1, 33] * 4), (19, 1, 1, 128, 1024, [1024])])
@pytest.mark.parametrize("capacity", [None, DEAL])
def test_matches_oracle(P, hq, hk, dh, cap, lens, capacity):
    B = len(lens)
    q, kc, vc = draw(1, P, B, hq, dh), draw(2, P, B, cap, hk, dh), draw(3, P, B, cap, hk, dh)
    need = C.caat_attn_workspace_size(B, capacity or cap, 0, P, hq, hk, dh, C.CAAT_VARIANT_ATTN_DECODE)
    assert need > 0 or not capacity
    out = decode(q, slab(kc, capacity), slab(vc, capacity), lens)
    assert C.caat_get_device_status() == 0
    check_out(out.cpu(), A.decode(q, kc, vc, lens))


@pytest.mark.parametrize("P", [1, 20])
@pytest.mark.parametrize("capacity", [140, DEAL])
@pytest.mark.parametrize("junk", [float("nan"), float("inf")])
def test_rows_behind_a_length_are_never_used(junk, capacity, P):
    lens = [70, 5, 128, 0]
    q = draw(4, P, 4, 4, 64)
    kc, vc = slab(draw(5, P, 4, 140, 2, 64), capacity), slab(draw(6, P, 4, 140, 2, 64), capacity)
    for b, n in enumerate(lens):
        kc[:, b, n:] = 1
        vc[:, b, n:] = 1
    a = decode(q, kc, vc, lens)
    for b, n in enumerate(lens):
        kc[:, b, n:] = junk
        vc[:, b, n:] = junk
    assert torch.equal(a, decode(q, kc, vc, lens))


@pytest.mark.parametrize("P", [1, 60])
@pytest.mark.parametrize("capacity", [10, DEAL])
def test_lengths_outside_the_cache_are_reported(P, capacity):
    q, kc, vc = draw(7, P, 3, 2, 64), draw(8, P, 3, 10, 1, 64), draw(9, P, 3, 10, 1, 64)
    out = decode(q, slab(kc, capacity), slab(vc, capacity), [capacity + 1, 10, -1])
    assert C.caat_get_device_status() & 0xFF == C.CAAT_ERR_INVALID_ARG
    assert C.caat_get_device_status() == 0
    assert bool((out[:, [0, 2]] == 0).all())
    check_out(out[:, 1:2].cpu(), A.decode(q[:, 1:2], kc[:, 1:2], vc[:, 1:2], [10]))


@pytest.mark.parametrize("P", [2, 16])
@pytest.mark.parametrize("capacity", [None, DEAL])
def test_same_bits_every_time_and_from_a_fused_projection(P, capacity):
    """The parts of a cut sequence are joined in a fixed order, whichever CTA finishes last; q may be a
    slice of a fused projection."""
    B, hq, hk, dh, cap = 5, 8, 2, 64, 3000
    lens = [3000, 1, 777, 2999, 64]
    qkv = draw(30, P, B, (hq + 2 * hk) * dh).cuda()
    q = qkv[..., :hq * dh].unflatten(-1, (hq, dh))
    kc, vc = slab(draw(31, P, B, cap, hk, dh), capacity), slab(draw(32, P, B, cap, hk, dh), capacity)
    first = decode(q.contiguous(), kc, vc, lens)
    for _ in range(10):
        assert torch.equal(first, decode(q, kc, vc, lens))


def test_cache_past_two_to_the_31_elements():
    """Append to and decode from rows whose element offset does not fit in 32 bits."""
    B, cap, hk, hq, dh = 16, 140000, 8, 8, 128
    k = torch.empty(1, B, cap, hk, dh, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() > 1 << 31
    n = 300
    small_k, small_v, q = draw(33, 1, n, hk, dh).cuda(), draw(34, 1, n, hk, dh).cuda(), draw(35, 1, B, hq, dh).cuda()
    freq, _ = C.caat_rope_frequencies(dh)
    slots = torch.arange((B - 1) * cap, (B - 1) * cap + n, device="cuda")
    C.caat_rope_append(None, small_k, small_v, None, slots, freq, k, v)
    kr = torch.empty_like(small_k)
    C.caat_rope(small_k, None, None, freq, q_out=kr, k_out=None)
    assert torch.equal(k[0, -1, :n], kr[0]) and torch.equal(v[0, -1, :n], small_v[0])
    lens = [0] * (B - 1) + [n]
    out = decode(q, k, v, lens)
    assert C.caat_get_device_status() == 0
    want = decode(q[:, -1:], kr.view(1, 1, n, hk, dh), small_v.view(1, 1, n, hk, dh), [n])
    ref = A.decode(q[:, -1:].cpu(), kr.view(1, 1, n, hk, dh).cpu(), small_v.view(1, 1, n, hk, dh).cpu(), [n])
    check_out(out[:, -1:].cpu(), ref)
    check_out(want.cpu(), ref)
    assert bool((out[:, :-1] == 0).all())


def test_large_scores():
    q, kc, vc = 8 * draw(10, 1, 2, 4, 128), 4 * draw(11, 1, 2, 500, 2, 128), draw(12, 1, 2, 500, 2, 128)
    check_out(decode(q, kc, vc, [500, 300]).cpu(), A.decode(q, kc, vc, [500, 300]))


@pytest.mark.parametrize("cap", [200, DEAL])
def test_captured_step_follows_the_lengths(cap):
    """A captured step (append, decode) replayed over a growing context equals separate calls."""
    P, B, hq, hk, dh = 2, 3, 4, 2, 64
    freq, _ = C.caat_rope_frequencies(dh)
    kc, vc = draw(13, P, B, cap, hk, dh).cuda(), draw(14, P, B, cap, hk, dh).cuda()
    kc2, vc2 = kc.clone(), vc.clone()
    q, k, v = draw(15, P, B, hq, dh).cuda(), draw(16, P, B, hk, dh).cuda(), draw(17, P, B, hk, dh).cuda()
    lens = torch.tensor([60, 1, 130], dtype=torch.int32, device="cuda")
    pos, slots, base = lens - 1, (lens - 1).long() + cap * torch.arange(B, device="cuda"), None
    out, qr = torch.empty(P, B, hq * dh, dtype=torch.bfloat16, device="cuda"), torch.empty_like(q)
    need = C.caat_attn_workspace_size(B, cap, 0, P, hq, hk, dh, C.CAAT_VARIANT_ATTN_DECODE)
    assert (need == 0) == (cap == 200)  # both kernels
    ws = C.alloc_workspace(need)

    def step(kc, vc, out):
        C.caat_rope_append(q, k, v, pos, slots, freq, kc, vc, q_out=qr)
        C.caat_attn_decode(qr, kc, vc, lens, out, workspace=ws)

    start = lens.clone()
    step(kc2.clone(), vc2.clone(), out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(kc, vc, out)
        lens += 1
        pos += 1
        slots += 1
    results = []
    for _ in range(5):
        graph.replay()
        results.append(out.clone())
    lens.copy_(start)
    pos.copy_(start - 1)
    slots.copy_((start - 1).long() + cap * torch.arange(B, device="cuda"))
    for r in results:
        step(kc2, vc2, out)
        assert torch.equal(r, out)
        lens += 1
        pos += 1
        slots += 1
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_decode_continues_a_prompt():
    """The last row of a prompt's attention equals the decode of that token over the cache the prompt
    filled (both within the tolerance of the same reference), through rotation and append."""
    P, T, hq, hk, dh, cap = 2, 150, 4, 2, 64, 160
    freq, _ = C.caat_rope_frequencies(dh)
    q, k, v = draw(18, P, T, hq, dh), draw(19, P, T, hk, dh), draw(20, P, T, hk, dh)
    qr, kr = torch.empty_like(q).cuda(), torch.empty_like(k).cuda()
    C.caat_rope(q.cuda(), k.cuda(), None, freq, q_out=qr, k_out=kr)
    kc = torch.full((P, 1, cap, hk, dh), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc, qo = kc.clone(), torch.empty_like(qr)
    C.caat_rope_append(q.cuda(), k.cuda(), v.cuda(), None, torch.arange(T, device="cuda"), freq, kc, vc, q_out=qo)
    assert torch.equal(qo, qr) and torch.equal(kc[:, 0, :T], kr)
    out = torch.empty(P, T, hq * dh, dtype=torch.bfloat16, device="cuda")
    C.caat_attn_forward(qr, kr, v.cuda(), [0, T], out)
    one = torch.empty(P, 1, hq * dh, dtype=torch.bfloat16, device="cuda")
    C.caat_attn_decode(qr[:, T - 1:], kc, vc, torch.tensor([T], dtype=torch.int32, device="cuda"), one)
    ref = A.attention(qr.cpu(), kr.cpu(), v, [0, T])
    check_out(out.cpu(), ref)
    last = {"out": ref["out"][:, -1:], "A": ref["A"][:, -1:], "M": ref["M"][:, :, -1:], "n": T}
    check_out(one.cpu(), last)


@pytest.mark.parametrize("T", [5, 200])
def test_attention_block_and_its_gradients(T):
    """Rotation, attention and the partially synchronized output projection, then the projection's
    backward, the attention's and the rotation's: every stage against the oracle on the stage's own
    inputs."""
    P, hq, hk, dh, H, p = 2, 4, 2, 64, 256, 0.5
    K = P * hq * dh
    lens = [T - T // 3, T // 3]
    cu = [0, lens[0], T]
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)
    freq, _ = C.caat_rope_frequencies(dh)
    q, k, v = draw(21, P, T, hq, dh), draw(22, P, T, hk, dh), draw(23, P, T, hk, dh)
    W, R, gamma = (0.05 * draw(24, P, H, hq * dh).float()).to(torch.bfloat16), draw(25, P, T, H), draw(26, H)
    qr, kr = torch.empty_like(q).cuda(), torch.empty_like(k).cuda()
    vd = v.cuda()
    C.caat_rope(q.cuda(), k.cuda(), pos.cuda(), freq, q_out=qr, k_out=kr)
    X = torch.empty(P, T, hq * dh, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(P, hq, T, dtype=torch.float32, device="cuda")
    C.caat_attn_forward(qr, kr, vd, cu, X, lse=lse)
    out, h = torch.empty(P, T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(P, T, H, dtype=torch.bfloat16, device="cuda")
    C.caat_rowpar_forward(X, W.cuda(), R.cuda(), gamma.cuda(), None, P, p, out, h_out=h)
    check_out(X.cpu(), A.attention(qr.cpu(), kr.cpu(), v, cu))
    assert_out_close(out.cpu(), O.rowpar_forward(X.cpu(), W, R, gamma, P, p))
    dout = draw(27, P, T, H)
    dX, dW = torch.empty_like(X), torch.empty_like(W).cuda()
    dgamma = torch.empty(H, dtype=torch.float32, device="cuda")
    C.caat_rowpar_backward(X, W.cuda(), h, gamma.cuda(), dout.cuda(), None, P, p, dX, dW, dgamma)
    dq, dk, dv = torch.empty_like(qr), torch.empty_like(kr), torch.empty_like(vd)
    C.caat_attn_backward(qr, kr, vd, X, lse, dX, cu, dq, dk, dv)
    from attn_util import check_grads
    M = A.attention(qr.cpu(), kr.cpu(), v, cu)["M"]
    ref = A.attention_backward(qr.cpu(), kr.cpu(), v, X.cpu(), lse.cpu(), dX.cpu(), cu)
    check_grads({"dq": dq.cpu(), "dk": dk.cpu(), "dv": dv.cpu()}, ref, M, dh)
    dq0 = torch.empty_like(dq)
    C.caat_rope(dq, None, pos.cuda(), freq, q_out=dq0, k_out=None, backward=True)
    err = np.abs(O._f64(dq0.cpu()) - A.rope(dq.cpu(), pos.numpy(), freq, backward=True))
    size = np.abs(O._f64(dq.cpu()))
    assert (err <= 2.0 ** -8 * np.abs(O._f64(dq0.cpu())) * 1.01 + 2.0 ** -20 * (size + np.roll(size, dh // 2, -1))).all()
    assert C.caat_get_device_status() == 0
