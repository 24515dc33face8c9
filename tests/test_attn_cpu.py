"""The attention block without a GPU: the oracle against hand-worked values and differences, the
frequencies bit for bit, and the refusals of every call before any device work."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import attn_oracle as A
from partial_activation_sync_caat_b200 import build as B
from partial_activation_sync_caat_b200 import caat as C


@pytest.fixture(scope="module")
def L():
    B.build()
    return C.lib()


def test_oracle_attention_hand_values():
    # two tokens, scores 0: the second averages both values; a lone query over no key is empty
    q = np.zeros((1, 3, 1, 2))
    k = np.ones((1, 2, 1, 2))
    v = np.array([[[[1.0, 0.0]], [[0.0, 4.0]]]])
    r = A.attention(q, k, v, [0, 2, 3], [0, 2, 2])
    np.testing.assert_allclose(r["out"][0, :, 0], [[1, 0], [0.5, 2], [0, 0]])
    np.testing.assert_allclose(r["lse"][0, 0, :2], [0, np.log(2)])
    assert np.isneginf(r["lse"][0, 0, 2])
    # more queries than keys: the first sees none; fewer: each sees the prefix
    r = A.attention(q[:, :3], k, v, [0, 3], [0, 2])
    assert np.isneginf(r["lse"][0, 0, 0]) and r["lse"][0, 0, 1] == 0
    np.testing.assert_allclose(A.attention(q[:, :1], k, v, [0, 1], [0, 2])["out"][0, 0, 0], [0.5, 2])


@pytest.mark.parametrize("lens,klens", [([4, 3], None), ([3, 2], [5, 1])])
def test_oracle_gradients_against_differences(lens, klens):
    rng = np.random.default_rng(0)
    cu_q, cu_k = [0, *np.cumsum(lens)], [0, *np.cumsum(klens or lens)]
    x = {"q": rng.normal(size=(2, cu_q[-1], 4, 6)), "k": rng.normal(size=(2, cu_k[-1], 2, 6)),
         "v": rng.normal(size=(2, cu_k[-1], 2, 6))}
    g = rng.normal(size=x["q"].shape)
    f = A.attention(x["q"], x["k"], x["v"], cu_q, cu_k, 0.8)
    grads = A.attention_backward(x["q"], x["k"], x["v"], f["out"], f["lse"], g, cu_q, cu_k, 0.8)
    for name in x:
        u = rng.normal(size=x[name].shape)
        ends = []
        for s in (1e-6, -1e-6):
            y = dict(x)
            y[name] = x[name] + s * u
            ends.append((A.attention(y["q"], y["k"], y["v"], cu_q, cu_k, 0.8)["out"] * g).sum())
        assert abs((ends[0] - ends[1]) / 2e-6 - (grads["d" + name] * u).sum()) < 1e-6


def test_oracle_rotation_keeps_relative_positions():
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(1, 1, 1, 8)), rng.normal(size=(1, 1, 1, 8))
    f, _ = A.rope_frequencies(8)
    for inter in (False, True):
        dots = [float((A.rope(q, [a], f, inter) * A.rope(k, [b], f, inter)).sum()) for a, b in ((5, 2), (105, 102), (3, 0))]
        np.testing.assert_allclose(dots, dots[0], rtol=1e-12)
        np.testing.assert_allclose(A.rope(A.rope(q, [7], f, inter), [7], f, inter, backward=True), q, atol=1e-15)
    # one pair, a quarter turn
    np.testing.assert_allclose(A.rope(np.array([[[[1.0, 0.0]]]]), [1], np.array([np.pi / 2]))[0, 0, 0], [0, 1], atol=1e-15)


@pytest.mark.parametrize("rot", [2, 16, 64, 128, 256])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0)])
def test_frequencies(L, rot, scaling, factor):
    if scaling == "ntk" and rot < 4:
        pytest.skip("one pair has no slowest and fastest")
    f, m = C.caat_rope_frequencies(rot, 10000.0, scaling, factor, 2048.0)
    g, n = A.rope_frequencies(rot, 10000.0, scaling, factor, 2048.0)
    np.testing.assert_allclose(f, g, rtol=1e-14)
    assert m == np.float32(n)


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=7), dict(rot=258), dict(theta=1.0), dict(theta=float("nan")),
                                dict(scaling="linear", factor=0.5), dict(scaling="ntk", rot=2, factor=2.0),
                                dict(scaling="yarn", factor=2.0, trained_length=0.0),
                                dict(scaling="ntk", factor=float("inf"))])
def test_frequencies_refuse(L, kw):
    with pytest.raises(C.CaatError) as e:
        C.caat_rope_frequencies(**{"rot": 64, **kw})
    assert e.value.code == C.CAAT_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        C.caat_rope_frequencies(64, scaling="other")


def fill(a, **kw):
    for n, x in kw.items():
        setattr(a, n, x)
    return a


def rope(L, **kw):
    f = np.ones(64)
    a = fill(C.RopeArgs(), q=0x100000, k=0x200000, q_out=0x300000, k_out=0x400000, inv_freq=f.ctypes.data, T=10, P=2,
             heads_q=4, heads_k=2, dh=128, rot=128, mscale=1.0)
    return L.caat_rope(ctypes.byref(fill(a, **kw)))


def test_rope_refuses(L):
    bad = np.array([1.0, np.nan] + [1.0] * 62)
    assert L.caat_rope(None) == C.CAAT_ERR_INVALID_ARG
    for kw in (dict(P=0), dict(P=65), dict(T=-1), dict(heads_q=-1), dict(dh=0), dict(rot=0), dict(rot=130),
               dict(mscale=float("nan")), dict(flags=4), dict(inv_freq=None), dict(inv_freq=bad.ctypes.data), dict(q=None),
               dict(q_out=None), dict(k_out=None), dict(slots=0x8000, v=0x500000, v_out=None, cache_rows=4),
               dict(slots=0x8000, v=None, v_out=0x600000, cache_rows=4),
               dict(slots=0x8000, v=0x500000, v_out=0x600000, cache_rows=-1), dict(q_stride_token=8, q_stride_rank=1 << 20),
               dict(q_out=0x100010), dict(k_out=0x300000), dict(q_out=0x200000)):
        assert rope(L, **kw) == C.CAAT_ERR_INVALID_ARG, kw
    for kw in (dict(dh=132), dict(dh=264, rot=16), dict(rot=72), dict(rot=20, flags=1), dict(q=0x100008), dict(k_out=0x400002),
               dict(T=(1 << 30) + 1), dict(q_stride_token=516, q_stride_rank=516 * 10), dict(positions=0x8002),
               dict(slots=0x8004, v=0x500000, v_out=0x600000, cache_rows=4)):
        assert rope(L, **kw) == C.CAAT_ERR_UNSUPPORTED, kw
    assert rope(L, T=0, q=None, k=None) == C.CAAT_OK
    assert rope(L, heads_q=0, heads_k=0) == C.CAAT_OK


def test_rope_refuses_what_overlaps(L):
    # positions or slots inside an output
    assert rope(L, positions=0x300000) == C.CAAT_ERR_INVALID_ARG
    assert rope(L, q_out=0x100000, positions=0x100100) == C.CAAT_ERR_INVALID_ARG
    cache = dict(v=0x500000, v_out=0x600000, cache_rows=4)
    assert rope(L, slots=0x400008, **cache) == C.CAAT_ERR_INVALID_ARG
    # in place: q and k on one buffer, on each other's rows, with strides of their own
    assert rope(L, q_out=0x100000, k=0x100000, k_out=0x100000) == C.CAAT_ERR_INVALID_ARG
    assert rope(L, q_out=0x100000, k=0x100000) == C.CAAT_ERR_INVALID_ARG
    fused = dict(q_out=0x100000, q_stride_token=768, q_stride_rank=7680, k_stride_token=768, k_stride_rank=7680)
    for k in (0x100000 + 2 * 504, 0x100000 + 2 * 520, 0x100000 - 2 * 248):
        assert rope(L, k=k, k_out=k, **fused) == C.CAAT_ERR_INVALID_ARG, hex(k)
    k = 0x100000 + 2 * 512
    assert rope(L, k=k, k_out=k, **{**fused, "k_stride_token": 776, "k_stride_rank": 7760}) == C.CAAT_ERR_INVALID_ARG
    # ranks that share rows
    assert rope(L, q_out=0x100000, q_stride_token=512, q_stride_rank=512) == C.CAAT_ERR_INVALID_ARG
    # a cache beyond any memory
    assert rope(L, slots=0x8000, v=0x500000, v_out=0x600000, cache_rows=1 << 62) == C.CAAT_ERR_UNSUPPORTED


def attn(L, name="caat_attn_forward", **kw):
    cu = np.array([0, 100, 300], dtype=np.int32)
    a = fill(C.AttnArgs() if name == "caat_attn_forward" else C.AttnBwdArgs(), q=0x1000000, k=0x2000000, v=0x3000000,
             out=0x4000000, lse=0x5000000, cu_q=cu.ctypes.data, workspace=0x6000000, ws_bytes=1 << 30, Tq=300, Tk=300, n_seq=2,
             P=2, heads_q=4, heads_k=2, dh=128, scale=0.1)
    if name != "caat_attn_forward":
        fill(a, dout=0x7000000, dq=0x8000000, dk=0x9000000, dv=0xA000000)
    return getattr(L, name)(ctypes.byref(fill(a, **kw)))


@pytest.mark.parametrize("name", ["caat_attn_forward", "caat_attn_backward"])
def test_attention_refuses(L, name):
    down, far, neg = (np.array(x, dtype=np.int32) for x in ([0, 200, 100], [0, 100, 301], [-1, 100, 300]))
    assert getattr(L, name)(None) == C.CAAT_ERR_INVALID_ARG
    for kw in (dict(P=0), dict(P=65), dict(heads_q=0), dict(heads_k=0), dict(heads_k=3), dict(dh=0), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(Tq=-1), dict(n_seq=-1), dict(flags=1),
               dict(cu_q=None), dict(cu_q=down.ctypes.data), dict(cu_q=far.ctypes.data), dict(cu_q=neg.ctypes.data),
               dict(cu_k=down.ctypes.data), dict(cu_k=far.ctypes.data), dict(q=None), dict(k=None), dict(v=None),
               dict(out=None), dict(q_stride_token=8, q_stride_rank=1 << 20), dict(k_stride_rank=8, k_stride_token=256)):
        assert attn(L, name, **kw) == C.CAAT_ERR_INVALID_ARG, kw
    for kw in (dict(dh=132), dict(dh=136), dict(q=0x1000008), dict(out=0x4000002), dict(lse=0x5000002),
               dict(Tq=(1 << 30) + 1), dict(q_stride_token=516, q_stride_rank=516 * 300),
               dict(q_stride_token=(1 << 31) + 8, q_stride_rank=1 << 34)):
        assert attn(L, name, **kw) == C.CAAT_ERR_UNSUPPORTED, kw
    long = np.array([0, 1 << 25, (1 << 26) + 1], dtype=np.int32)
    big = dict(Tq=1 << 27, Tk=1 << 27, P=1, heads_q=1, heads_k=1, dh=8, k=1 << 40, v=1 << 41, out=1 << 42, lse=1 << 43)
    assert attn(L, name, cu_q=long.ctypes.data, **big) == C.CAAT_ERR_UNSUPPORTED
    assert attn(L, name, n_seq=0, q=None) == C.CAAT_OK
    if name == "caat_attn_forward":
        assert attn(L, out=0x1000100) == C.CAAT_ERR_INVALID_ARG   # out inside q
        assert attn(L, lse=0x4000000) == C.CAAT_ERR_INVALID_ARG   # lse on out
    else:
        for kw in (dict(dout=None), dict(lse=None), dict(dq=None), dict(dk=None), dict(dv=None), dict(dq=0x1000000),
                   dict(dk=0x9000000, dv=0x9000010), dict(dk=0x7000000), dict(dq=0x5000000)):
            assert attn(L, name, **kw) == C.CAAT_ERR_INVALID_ARG, kw
        assert attn(L, name, workspace=None) == C.CAAT_ERR_WORKSPACE
        assert attn(L, name, ws_bytes=256) == C.CAAT_ERR_WORKSPACE
        assert attn(L, name, workspace=0x6000010) == C.CAAT_ERR_WORKSPACE


def decode(L, **kw):
    a = fill(C.AttnDecodeArgs(), q=0x1000000, k_cache=0x10000000, v_cache=0x20000000, lens=0x3000000, out=0x4000000,
             workspace=0x6000000, ws_bytes=1 << 30, B=3, capacity=100, P=2, heads_q=4, heads_k=2, dh=128, scale=0.1)
    return L.caat_attn_decode(ctypes.byref(fill(a, **kw)))


def test_decode_refuses(L):
    assert L.caat_attn_decode(None) == C.CAAT_ERR_INVALID_ARG
    for kw in (dict(P=0), dict(heads_k=3), dict(scale=0.0), dict(B=-1), dict(capacity=-1), dict(flags=1), dict(q=None),
               dict(k_cache=None), dict(v_cache=None), dict(lens=None), dict(out=None), dict(out=0x1000000), dict(out=0x10000010)):
        assert decode(L, **kw) == C.CAAT_ERR_INVALID_ARG, kw
    for kw in (dict(dh=132), dict(dh=136), dict(k_cache=0x10000008), dict(lens=0x3000002), dict(B=65536),
               dict(capacity=(1 << 30) + 1), dict(B=4096, capacity=1 << 30)):
        assert decode(L, **kw) == C.CAAT_ERR_UNSUPPORTED, kw
    for kw in (dict(workspace=None), dict(ws_bytes=1024), dict(workspace=0x6000010)):
        assert decode(L, capacity=20000, **kw) == C.CAAT_ERR_WORKSPACE, kw
    assert decode(L, B=0, q=None) == C.CAAT_OK


def test_workspace_size_refuses(L):
    for args in ((-1, 1, 1, 1, 1, 1, 64, 0), (1, 1, 1, 0, 1, 1, 64, 0), (1, 1, 1, 1, 3, 2, 64, 0), (1, 1, 1, 1, 1, 1, 63, 0),
                 (1, 1, 1, 1, 1, 1, 64, 3), (1, 1, -1, 1, 1, 1, 64, 1)):
        with pytest.raises(C.CaatError):
            C.caat_attn_workspace_size(*args)


def test_packed_arguments_are_the_structures(L):
    """The packed form of each call's arguments lays every field where the structure has it."""
    for name, (packed, args) in C._PACKED.items():
        values = [i + 1 for i in range(len(args._fields_))]
        a = args.from_buffer_copy(packed.pack(*values))
        assert [getattr(a, f) for f, *_ in args._fields_] == values, name


def test_binding_refuses_cpu_tensors_and_odd_layouts(L):
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    freq, _ = C.caat_rope_frequencies(64)
    with pytest.raises(ValueError):
        C.caat_rope(q, q, None, freq, q_out=q, k_out=q)
    with pytest.raises(ValueError):
        C.caat_attn_forward(q, q, q, [0, 4], torch.zeros(1, 4, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        C.caat_rope(None, None, None, freq, q_out=None, k_out=None)
    with pytest.raises(ValueError):
        C._heads4(q.transpose(2, 3), "q", torch.bfloat16, -1)
    with pytest.raises(ValueError):
        C._heads4(q[..., ::2], "q", torch.bfloat16, -1)
    with pytest.raises(TypeError):
        C._heads4(q.float(), "q", torch.bfloat16, -1)
    assert C._heads4(q[:, 1:, :1], "q", torch.bfloat16, -1)[1:] == (4 * 128, 128)
    assert C._heads4(q, "q", torch.bfloat16, -1)[1:] == (0, 0)
    for good in ([0, 4], (0, 4), np.array([0, 4]), np.array([9, 0, 4, 7], dtype=np.int32)[1:3], torch.tensor([0, 4])):
        keep, ptr, n = C._offsets(good, "cu_q")
        assert n == 2 and list((ctypes.c_int32 * 2).from_address(ptr)) == [0, 4] and keep is not None
    for bad in ([[0, 1]], [0.0, 1.0], [], np.array([[0, 1]]), np.array([0.0, 1.0]), "01"):
        with pytest.raises(ValueError):
            C._offsets(bad, "cu_q")
    for big in ([0, 2**31], np.array([0, 2**31])):
        with pytest.raises(C.CaatError):
            C._offsets(big, "cu_q")


def test_compiled_marshalling_leaves_odd_arguments_alone(L):
    """Without a GPU no tensor is taken: every function hands the call back."""
    m = C._marshal
    assert m is not None
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    f = np.ones(32)
    for x in (q, None, 3, [q]):
        assert m.rope(x, q, None, None, None, f, q, q, None, False, False, 1.0) is None
        assert m.attn_forward(x, q, q, [0, 4], None, q, None, None, None) is None
        assert m.attn_backward(x, q, q, [0, 4], None, q, q, q, q, q, q, None, None) is None
        assert m.attn_decode(x, q, q, q, q, None, None) is None
    assert m.rope() is None and m.attn_decode(q) is None
    with pytest.raises(TypeError):
        m.bind(1)


def test_bench_counts_the_attention_blocks_work():
    import bench
    T, P, heads, dh, H = 3, 2, 2, 8, 16
    visible = sum(i + 1 for i in range(T)) * P * heads
    assert bench.attn_block_flops(T, P, heads, dh, H, False) == (4 * dh * visible, 2.0 * T * (P * heads * dh) * H)
    assert bench.attn_block_flops(T, P, heads, dh, H, True) == (10 * dh * visible, 4.0 * T * (P * heads * dh) * H)
