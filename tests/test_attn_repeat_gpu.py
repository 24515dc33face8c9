"""The gradients of the packed attention run after run: the warps of a CTA meet in another order each time, the
results must not show it.  The first run goes against the float64 oracle, the others against the first, bit for
bit; two states take turns, so that what one leaves in shared and tensor memory is wrong for the other, and memory
that is no longer in the cache delays single warps."""
import pytest
import torch

from oracle import attn_oracle as A
from partial_activation_sync_caat_b200 import caat as C

from attn_util import check_grads
from gpu_util import ensure_built
from test_attn_gpu import backward, forward, make

pytestmark = pytest.mark.gpu

RUNS = 150


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("P,hq,hk,dh,lens,klens", [
    (2, 8, 1, 64, [1027, 5, 300], None),
    (4, 4, 2, 64, [513, 65, 128], [700, 128, 129]),
    (2, 4, 2, 128, [1100, 257], None),
    (2, 4, 1, 96, [640, 31], [900, 40]),
    (16, 4, 4, 128, [100, 28, 129], [128, 129, 300]),  # tiles with and without the pass for D
])
def test_gradients_run_after_run(P, hq, hk, dh, lens, klens):
    states = []
    for seed in (31, 32):
        d = make(P, hq, hk, dh, lens, klens, seed=seed)
        out, lse = forward(d)
        x = {n: d[n].cuda() for n in ("q", "k", "v", "dout")}
        M = A.attention(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"])["M"]
        ref = A.attention_backward(d["q"], d["k"], d["v"], out.cpu(), lse.cpu(), d["dout"], d["cu_q"], d["cu_k"])
        states.append((d, x, out, lse, ref, M))
    flush = torch.empty(160 << 20, dtype=torch.uint8, device="cuda")
    first = [None, None]
    differ = torch.zeros(3, dtype=torch.int64, device="cuda")
    for run in range(RUNS):
        for s, (d, x, out, lse, ref, M) in enumerate(states):
            if run % 2:
                flush.zero_()
            g = [torch.full_like(x[n], 7.0) for n in ("q", "k", "v")]
            C.caat_attn_backward(x["q"], x["k"], x["v"], out, lse, x["dout"], d["cu_q"], *g, cu_k=d["cu_k"])
            if first[s] is None:
                first[s] = g
                check_grads({n: t.cpu() for n, t in zip(("dq", "dk", "dv"), g)}, ref, M, dh, f"state {s}")
            else:
                differ += torch.stack([(a != b).any() for a, b in zip(g, first[s])])
    torch.cuda.synchronize()
    assert C.caat_get_device_status() == 0
    assert differ.tolist() == [0, 0, 0], f"runs with another dq, dk, dv: {differ.tolist()}"


def test_long_work_lists_captured():
    """More work items than a launch carries in its arguments: the lists travel through the workspace, and a graph
    puts them there anew each time, whatever the workspace held."""
    lens = [(11 * i) % 29 for i in range(500)]
    d = make(1, 2, 1, 64, lens, seed=33)
    want, lse_w = forward(d)
    grads_w = backward(d, want, lse_w)
    x = {n: d[n].cuda() for n in ("q", "k", "v", "dout")}
    out, lse = torch.empty_like(want), torch.empty_like(lse_w)
    grads = [torch.empty_like(x[n]) for n in ("q", "k", "v")]
    T, n = d["cu_q"][-1], len(lens)
    need = [C.caat_attn_workspace_size(T, T, n, 1, 2, 1, 64, v) for v in (C.CAAT_VARIANT_ATTN, C.CAAT_VARIANT_ATTN_BWD)]
    assert need[0] > 0
    ws = [C.alloc_workspace(b) for b in need]

    def both():
        C.caat_attn_forward(x["q"], x["k"], x["v"], d["cu_q"], out, lse=lse, workspace=ws[0])
        C.caat_attn_backward(x["q"], x["k"], x["v"], out, lse, x["dout"], d["cu_q"], *grads, workspace=ws[1])

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(3):
        for t in (out, lse, *grads):
            t.zero_()
        for w in ws:
            w.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, lse_w)
        assert all(torch.equal(g, grads_w[n]) for g, n in zip(grads, ("dq", "dk", "dv")))
    assert C.caat_get_device_status() == 0
