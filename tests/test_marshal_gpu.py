"""The compiled marshalling of the attention block's calls against the binding's own: the same results
for the arguments both take, the same refusals for those that neither does."""
import numpy as np
import pytest
import torch

from partial_activation_sync_caat_b200 import caat as C
from gpu_util import ensure_built

pytestmark = pytest.mark.gpu

P, T, HQ, HK, DH = 2, 37, 4, 2, 64
LENS = [0, 20, 37]


def rand(*shape):
    return torch.randn(*shape, device="cuda").bfloat16()


@pytest.fixture(scope="module")
def fused():
    ensure_built()
    torch.manual_seed(0)
    return rand(P, T, (HQ + 2 * HK) * DH)


def slices(x):
    return [y.unflatten(-1, (-1, DH)) for y in x.split([HQ * DH, HK * DH, HK * DH], dim=-1)]


def calls(x, cu, freq):
    """Every call once on slices of one projection; all results."""
    q, k, v = slices(x.clone())
    C.caat_rope(q, k, None, freq, q_out=q, k_out=k)
    qt, kt = torch.empty(P, T, HQ, DH, device="cuda").bfloat16(), torch.empty(P, T, HK, DH, device="cuda").bfloat16()
    pos = torch.arange(T, device="cuda", dtype=torch.int32) + 5
    C.caat_rope(q, k, pos, freq, q_out=qt, k_out=kt, interleaved=True, backward=True, mscale=0.5)
    cache = [torch.zeros(P, 3, T, HK, DH, device="cuda").bfloat16() for _ in range(2)]
    slots = torch.arange(T, device="cuda") * 2
    qa = torch.empty_like(qt)
    C.caat_rope_append(q, k, v, pos, slots, freq, *cache, q_out=qa)
    out = torch.empty(P, T, HQ * DH, device="cuda").bfloat16()
    lse = torch.empty(P, HQ, T, device="cuda")
    C.caat_attn_forward(q, k, v, cu, out, lse=lse)
    grads = [torch.empty(y.shape, device="cuda").bfloat16() for y in (q, k, v)]
    C.caat_attn_backward(q, k, v, out, lse, out, cu, *grads, cu_k=cu)
    o = torch.empty(P, 3, HQ * DH, device="cuda").bfloat16()
    lens = torch.tensor([T, 0, 3], device="cuda", dtype=torch.int32)
    C.caat_attn_decode(q[:, :3], *cache, lens, o, scale=0.25)
    torch.cuda.synchronize()
    assert C.caat_get_device_status() == 0
    return [q, k, qt, kt, qa, *cache, out, lse, *grads, o]


@pytest.mark.parametrize("cu", [LENS, tuple(LENS), np.array(LENS, dtype=np.int32)], ids=["list", "tuple", "array"])
def test_both_ways_give_the_same(fused, cu, monkeypatch):
    freq, _ = C.caat_rope_frequencies(DH)
    C.lib()
    taken = []

    class Spy:
        def __getattr__(self, name):
            def call(*a):
                code = getattr(C_marshal, name)(*a)
                taken.append((name, code))
                return code
            return call

    C_marshal = C._marshal
    assert C_marshal is not None
    monkeypatch.setattr(C, "_marshal", Spy())
    compiled = calls(fused, cu, freq)
    assert [n for n, _ in taken] == ["rope"] * 3 + ["attn_forward", "attn_backward", "attn_decode"]
    assert all(code == 0 for _, code in taken)
    monkeypatch.setattr(C, "_marshal", None)
    monkeypatch.setattr(C, "_fast", lambda: None)
    for a, b in zip(compiled, calls(fused, cu, freq)):
        assert torch.equal(a, b)


def test_refusals_keep_their_names(fused):
    freq, _ = C.caat_rope_frequencies(DH)
    q, k, v = slices(fused.clone())
    out, lse = rand(P, T, HQ * DH), torch.empty(P, HQ, T, device="cuda")
    with pytest.raises(TypeError, match="q must be"):
        C.caat_attn_forward(q.float(), k, v, LENS, out)
    with pytest.raises(ValueError, match="out must have the shape"):
        C.caat_attn_forward(q, k, v, LENS, out[:, 1:])
    with pytest.raises(ValueError, match="out must be contiguous"):
        C.caat_attn_forward(q, k, v, LENS, rand(P, T, HQ * DH + 8)[..., :HQ * DH])
    with pytest.raises(ValueError, match="v is on|v must have"):
        C.caat_attn_forward(q, k, v.cpu(), LENS, out)
    with pytest.raises(ValueError, match="same length"):
        C.caat_attn_forward(q, k, v, LENS, out, cu_k=[0, 37])
    with pytest.raises(ValueError, match="one-dimensional"):
        C.caat_attn_forward(q, k, v, [0.0, 37.0], out)
    with pytest.raises(C.CaatError) as e:
        C.caat_attn_forward(q, k, v, [0, 38], out)
    assert e.value.code == C.CAAT_ERR_INVALID_ARG
    with pytest.raises(C.CaatError) as e:
        C.caat_attn_forward(q, k, v, [0, 2**31], out)
    assert e.value.code == C.CAAT_ERR_INVALID_ARG
    with pytest.raises(C.CaatError) as e:
        C.caat_attn_forward(q, k, v, LENS, out, lse=lse, scale=-1.0)
    assert e.value.code == C.CAAT_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="in place"):
        C.caat_rope(q, k, None, freq, q_out=q.transpose(0, 1), k_out=k)
    with pytest.raises(ValueError, match="positions must have the shape"):
        C.caat_rope(q, k, torch.zeros(T - 1, device="cuda", dtype=torch.int32), freq, q_out=q, k_out=k)
    with pytest.raises(TypeError, match="slots must be"):
        C.caat_rope_append(q, k, v, None, torch.zeros(T, device="cuda", dtype=torch.int32), freq, rand(P, 40, HK, DH),
                           rand(P, 40, HK, DH), q_out=q)
    with pytest.raises(ValueError, match="k_cache must be"):
        C.caat_attn_decode(q[:, :3], rand(P, 2, 9, HK, DH), rand(P, 2, 9, HK, DH), torch.zeros(3, device="cuda", dtype=torch.int32),
                           rand(P, 3, HQ * DH))
    torch.cuda.synchronize()
    assert C.caat_get_device_status() == 0


def test_workspace_of_the_call_and_of_the_caller(fused):
    """A work list too long for the launch's arguments, and decoding that deals its tiles."""
    n = 400
    q, k, v = rand(1, n, 2, DH), rand(1, n, 1, DH), rand(1, n, 1, DH)
    cu = list(range(n + 1))
    need = C.caat_attn_workspace_size(n, n, n, 1, 2, 1, DH)
    assert need > 0
    outs = [rand(1, n, 2 * DH) for _ in range(2)]
    C.caat_attn_forward(q, k, v, cu, outs[0])
    C.caat_attn_forward(q, k, v, cu, outs[1], workspace=C.alloc_workspace(need))
    assert torch.equal(*outs)
    # a sequence of one token answers with its value
    assert torch.equal(outs[0].view(1, n, 2, DH), v.expand(1, n, 2, DH))
    with pytest.raises(C.CaatError) as e:
        C.caat_attn_forward(q, k, v, cu, outs[1], workspace=C.alloc_workspace(256)[:16])
    assert e.value.code == C.CAAT_ERR_WORKSPACE
    cache = rand(1, 1, 20000, 1, DH), rand(1, 1, 20000, 1, DH)
    lens = torch.tensor([4999], device="cuda", dtype=torch.int32)
    need = C.caat_attn_workspace_size(1, 20000, 0, 1, 2, 1, DH, C.CAAT_VARIANT_ATTN_DECODE)
    assert need > 0
    outs = [rand(1, 1, 2 * DH) for _ in range(2)]
    C.caat_attn_decode(q[:, :1], *cache, lens, outs[0])
    C.caat_attn_decode(q[:, :1], *cache, lens, outs[1], workspace=C.alloc_workspace(need))
    assert torch.equal(*outs)
    torch.cuda.synchronize()
    assert C.caat_get_device_status() == 0
