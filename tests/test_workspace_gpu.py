"""Calls on another stream that bring no workspace leave alone what the current stream still works on."""
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


def rand(*shape):
    return torch.randn(*shape, device="cuda").to(BF)


def beside_work_on_the_current_stream(need, call, results, repeat=3):
    """`call(stream)` next to a buffer of `need` bytes that the current stream has queued a late copy of, and
    that has been given back already: the copy holds what was put there, the call's results are those of a
    call alone."""
    torch.cuda.synchronize()
    call(None)
    torch.cuda.synchronize()
    want = [r.clone() for r in results]
    side = torch.cuda.Stream()
    copy = torch.empty(need, dtype=torch.uint8, device="cuda")
    call(side)
    torch.cuda.synchronize()
    for _ in range(repeat):
        torch.cuda.empty_cache()
        for r in results:
            r.zero_()
        b = torch.full((need,), 173, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(40_000_000)  # about 20 ms
        copy.copy_(b)
        b.fill_(255)
        del b
        call(side)
        side.synchronize()
        torch.cuda.synchronize()
        assert bool((copy == 173).all())
        assert all(torch.equal(r, w) for r, w in zip(results, want))
    assert C.caat_get_device_status() == 0


@pytest.mark.parametrize("dh", [64, 128])
def test_gradients(dh):
    P, T, hq, hk = 2, 700, 4, 2
    torch.manual_seed(dh)
    q, k, v, dout = rand(P, T, hq, dh), rand(P, T, hk, dh), rand(P, T, hk, dh), rand(P, T, hq * dh)
    cu = [0, 300, 700]
    out, lse = torch.empty_like(dout), torch.empty(P, hq, T, device="cuda")
    C.caat_attn_forward(q, k, v, cu, out, lse=lse)
    grads = [torch.empty_like(x) for x in (q, k, v)]
    need = C.caat_attn_workspace_size(T, T, 2, P, hq, hk, dh, C.CAAT_VARIANT_ATTN_BWD)
    beside_work_on_the_current_stream(
        need, lambda st: C.caat_attn_backward(q, k, v, out, lse, dout, cu, *grads, stream=st), grads)


def test_forward_with_a_long_list():
    n = 4000
    q, k, v = rand(1, n, 2, 64), rand(1, n, 1, 64), rand(1, n, 1, 64)
    cu = np.arange(n + 1, dtype=np.int32)
    out = torch.empty(1, n, 128, dtype=BF, device="cuda")
    need = C.caat_attn_workspace_size(n, n, n, 1, 2, 1, 64)
    assert need > 0
    beside_work_on_the_current_stream(need, lambda st: C.caat_attn_forward(q, k, v, cu, out, stream=st), [out])


def test_decode_with_the_even_deal():
    cache = rand(1, 1, 20000, 1, 64), rand(1, 1, 20000, 1, 64)
    q, lens = rand(1, 1, 2, 64), torch.tensor([19999], device="cuda", dtype=torch.int32)
    out = torch.empty(1, 1, 128, dtype=BF, device="cuda")
    need = C.caat_attn_workspace_size(1, 20000, 0, 1, 2, 1, 64, C.CAAT_VARIANT_ATTN_DECODE)
    assert need > 0
    beside_work_on_the_current_stream(need, lambda st: C.caat_attn_decode(q, *cache, lens, out, stream=st), [out])


def test_row_parallel_layer_and_its_gradients():
    P, T, K, H, p = 2, 256, 768, 768, 0.5
    X, W, R, g, dout = rand(P, T, K // P), rand(P, H, K // P), rand(P, T, H), rand(H), rand(P, T, H)
    out, h = torch.empty_like(R), torch.empty_like(R)
    beside_work_on_the_current_stream(
        C.caat_workspace_size(T, K, H, P),
        lambda st: C.caat_rowpar_forward(X, W, R, g, None, P, p, out, h_out=h, stream=st), [out, h])
    dX, dW, dg = torch.empty_like(X), torch.empty_like(W), torch.empty(H, device="cuda")
    beside_work_on_the_current_stream(
        C.caat_workspace_size(T, K, H, P, C.CAAT_VARIANT_ROWPAR_BWD),
        lambda st: C.caat_rowpar_backward(X, W, h, g, dout, None, P, p, dX, dW, dg, stream=st), [dX, dW, dg])
