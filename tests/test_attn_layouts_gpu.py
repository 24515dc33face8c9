"""Layouts of the attention block's tensors on the GPU: what is refused before any launch, and layouts of the
ranks and tokens that other tests do not have."""
import numpy as np
import pytest
import torch

from partial_activation_sync_caat_b200 import caat as C

from gpu_util import ensure_built

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.fixture(params=["compiled", "interpreted"])
def marshalling(request, monkeypatch):
    """Both halves of the binding."""
    if request.param == "compiled":
        assert C._fast() is not None
    else:
        monkeypatch.setattr(C, "_marshal", None)
        monkeypatch.setattr(C, "_fast", lambda: None)


@pytest.mark.parametrize("P,T", [(8, 16), (1, 16), (2, 2)])
def test_expanded_tensors_are_refused(marshalling, P, T):
    one = torch.ones(4, 64, dtype=BF, device="cuda")
    wide = one.expand(P, T, 4, 64)
    full = torch.zeros(P, T, 4, 64, dtype=BF, device="cuda")
    out, lse = torch.zeros(P, T, 256, dtype=BF, device="cuda"), torch.zeros(P, 4, T, device="cuda")
    freq, _ = C.caat_rope_frequencies(64)
    cache = [torch.zeros(P, T, 4, 64, dtype=BF, device="cuda") for _ in range(2)]
    slots = torch.arange(T, device="cuda")
    grads = [torch.zeros_like(full) for _ in range(3)]
    slab = torch.zeros(P, T, 8, 4, 64, dtype=BF, device="cuda")
    lens = torch.ones(T, dtype=torch.int32, device="cuda")
    calls = [lambda: C.caat_rope(wide, None, None, freq, q_out=wide, k_out=None),
             lambda: C.caat_rope(wide, None, None, freq, q_out=full, k_out=None),
             lambda: C.caat_rope(full, wide, None, freq, q_out=full, k_out=wide),
             lambda: C.caat_rope_append(None, wide, full, None, slots, freq, *cache),
             lambda: C.caat_rope_append(None, full, wide, None, slots, freq, *cache),
             lambda: C.caat_attn_decode(wide, slab, slab, lens, out)]
    for i in range(3):
        qkv = [full, full, full]
        qkv[i] = wide
        calls.append(lambda qkv=qkv: C.caat_attn_forward(*qkv, [0, T], out))
        calls.append(lambda qkv=qkv: C.caat_attn_backward(*qkv, out, lse, out, [0, T], *grads))
    for call in calls:
        with pytest.raises(ValueError, match="share memory"):
            call()
    torch.cuda.synchronize()
    assert bool((one == 1).all()) and not any(bool(x.any()) for x in (full, out, *cache, *grads))
    assert C.caat_get_device_status() == 0


def turned_alike(q, k, T, **kw):
    """In place, against contiguous outputs: the same bits, and nothing else touched."""
    freq, _ = C.caat_rope_frequencies(64)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 7
    want = [torch.empty(x.shape, dtype=BF, device="cuda") for x in (q, k)]
    C.caat_rope(q, k, pos, freq, q_out=want[0], k_out=want[1], **kw)
    C.caat_rope(q, k, pos, freq, q_out=q, k_out=k, **kw)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert C.caat_get_device_status() == 0


@pytest.mark.parametrize("T", [2, 33])
def test_rotated_in_place_ranks_inside_a_token(marshalling, T):
    torch.manual_seed(T)
    buf = torch.randn(T, 5, 2, 64, device="cuda").to(BF)
    rest = buf[:, 4].clone()
    turned_alike(buf[:, 0:2].transpose(0, 1), buf[:, 2:4].transpose(0, 1), T)
    turned_alike(buf[:, 0:4:2].transpose(0, 1), buf[:, 1:4:2].transpose(0, 1), T, interleaved=True)
    assert torch.equal(buf[:, 4], rest)
    freq, _ = C.caat_rope_frequencies(64)
    before = buf.clone()
    with pytest.raises(C.CaatError) as e:  # k of rank 0 is q of rank 1
        q, k = buf[:, 0:2].transpose(0, 1), buf[:, 1:3].transpose(0, 1)
        C.caat_rope(q, k, None, freq, q_out=q, k_out=k)
    assert e.value.code == C.CAAT_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.equal(buf, before)


@pytest.mark.parametrize("P,hq,hk", [(2, 4, 4), (3, 4, 1), (1, 4, 2)])
def test_one_token_of_a_fused_projection(marshalling, P, hq, hk):
    """A decoding step of one sequence, its q, k and v slices of one projection: q and k in place, and q in
    place with k and v into a cache."""
    dh = 64
    torch.manual_seed(P)
    qkv = torch.randn(P, 1, (hq + 2 * hk) * dh, device="cuda").to(BF)
    q, k, v = (x.unflatten(-1, (-1, dh)) for x in qkv.split([hq * dh, hk * dh, hk * dh], -1))
    v0 = v.clone()
    turned_alike(q, k, 1)
    freq, _ = C.caat_rope_frequencies(dh)
    pos, slots = torch.tensor([3], dtype=torch.int32, device="cuda"), torch.tensor([3], device="cuda")
    want = [torch.empty(x.shape, dtype=BF, device="cuda") for x in (q, k)]
    C.caat_rope(q, k, pos, freq, q_out=want[0], k_out=want[1])
    cache = [torch.zeros(P, 1, 9, hk, dh, dtype=BF, device="cuda") for _ in range(2)]
    C.caat_rope_append(q, k, v, pos, slots, freq, *cache, q_out=q)
    assert torch.equal(q, want[0]) and torch.equal(cache[0][:, 0, 3], want[1][:, 0]) and torch.equal(cache[1][:, 0, 3], v0[:, 0])
    assert torch.equal(v, v0)
    for c in cache:
        c[:, 0, 3] = 0
        assert not bool(c.any())
    assert C.caat_get_device_status() == 0


def test_workspaces_with_gaps_are_refused(marshalling):
    """A workspace is taken for as long as its elements are many: one that is not contiguous is not."""
    n = 64
    q, k = (torch.zeros(1, n, h, 64, dtype=BF, device="cuda") for h in (2, 1))
    out, lse = torch.zeros(1, n, 128, dtype=BF, device="cuda"), torch.zeros(1, 2, n, device="cuda")
    grads = [torch.zeros_like(x) for x in (q, k, k)]
    need = C.caat_attn_workspace_size(n, n, 1, 1, 2, 1, 64, C.CAAT_VARIANT_ATTN_BWD)
    byte = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for ws in (byte.expand(need // 256 + 1, 256), C.alloc_workspace(2 * need)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            C.caat_attn_backward(q, k, k, out, lse, out, [0, n], *grads, workspace=ws)
        with pytest.raises(ValueError, match="contiguous"):
            C.caat_attn_forward(q, k, k, [0, n], out, workspace=ws)
    torch.cuda.synchronize()
    assert not bool(byte.any()) and C.caat_get_device_status() == 0
