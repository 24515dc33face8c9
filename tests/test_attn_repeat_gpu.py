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
from test_attn_gpu import forward, make

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
