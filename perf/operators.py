"""Workloads of the attention block's operators beside the partially synchronized output projection.

Four operators, all on P tensor-parallel ranks side by side in one GPU's memory, bf16 tensors:

* rope     rotary positions of q [P, T, hq, dh] and k [P, T, hk, dh], optionally with the rotated k
           and v appended to a cache [P, rows, hk, dh];
* attn     causal attention over packed prompts with grouped heads, out [P, T, hq dh] and lse;
* attn_bwd its gradients dq, dk, dv;
* decode   one token per sequence against a cache [P, B, capacity, hk, dh].

The sizes are those of the 7B shape (32 heads of 128 over P = 8 ranks, T = 8192) and the 1.1B
shape (32 query heads and 4 key heads of 64 over P = 4 ranks, T = 4096), with generic ragged ones.
"""
import math

import torch

own = False

DEV = "cuda"


def _rope(name, T, P, hq, hk, dh, rot, *, layout="half", scaling="none", factor=1.0, origin=0, backward=False,
          append=False):
    return {"name": name, "op": "rope", "P": P, "T": T, "hq": hq, "hk": hk, "dh": dh, "rot": rot, "layout": layout,
            "scaling": scaling, "factor": factor, "origin": origin, "backward": backward, "append": append}


def _attn(name, lens, P, hq, hk, dh, *, prefix=0, backward=False):
    return {"name": name, "op": "attn_bwd" if backward else "attn", "P": P, "lens": lens, "prefix": prefix, "hq": hq,
            "hk": hk, "dh": dh}


def _decode(name, lens, capacity, P, hq, hk, dh):
    return {"name": name, "op": "decode", "P": P, "lens": lens, "capacity": capacity, "hq": hq, "hk": hk, "dh": dh}


def listed():
    return [
        # one decoding step of eight sequences of the 7B shape at far positions, k and v into the cache
        _rope("rope-step-8", 8, 8, 4, 4, 128, 128, scaling="linear", factor=4.0, origin=30000, append=True),
        # a whole prompt of the 7B shape
        _rope("rope-prompt-7b", 8192, 8, 4, 4, 128, 128),
        # an odd-sized packed batch, interleaved pairs, part of the head, scaled frequencies, in the gradient
        _rope("rope-gradient-odd", 4099, 2, 6, 2, 96, 64, layout="interleaved", scaling="yarn", factor=8.0,
              backward=True),
        # a chunk of a prompt of the 1.1B shape appended to its cache
        _rope("rope-append-1b", 3001, 4, 8, 1, 64, 64, scaling="ntk", factor=2.0, origin=5000, append=True),
        # short questions answered at once: latency counts
        _attn("attn-short", "37,1,90", 8, 4, 4, 128),
        # a whole prompt of the 7B shape, as its output projection takes it
        _attn("attn-prompt-7b", "8192", 8, 4, 4, 128),
        # packed prompts of the 1.1B shape behind cached prefixes of 100 keys
        _attn("attn-packed-1b", "1500,1,333,64,900,17,1281", 4, 8, 1, 64, prefix=100),
        # a long document of the 7B shape
        _attn("attn-long-7b", "16384", 8, 4, 4, 128),
        # a training sequence of the 7B shape
        _attn("attn-bwd-7b", "4096", 8, 4, 4, 128, backward=True),
        # packed training documents of the 1.1B shape
        _attn("attn-bwd-packed-1b", "1027,2048,5,640,376", 4, 8, 1, 64, backward=True),
        # one user of the 7B shape
        _decode("decode-1", "4001", 8192, 8, 4, 4, 128),
        # a full batch of the 1.1B shape with ragged contexts
        _decode("decode-64", ",".join(str(1 + (i * 2654435761 >> 7) % 8191) for i in range(64)), 8192, 4, 8, 1, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn_bwd", "decode"])
    P = rng.choice([1, 2, 4, 8])
    dh = rng.choice([64, 96, 128])
    hk = rng.choice([1, 2, 4])
    hq = hk * rng.choice([1, 2, 4, 8]) if hk < 4 else hk
    if op == "rope":
        T = _log(rng, 1, 8192)
        return _rope("drawn", T, P, hq, hk, dh, rng.choice([dh, dh // 2]), layout=rng.choice(["half", "interleaved"]),
                     scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=rng.choice([2.0, 4.0, 8.0]),
                     origin=rng.choice([0, _log(rng, 1, 100000)]), **rng.choice([{}, {"backward": True}, {"append": True}]))
    if op == "decode":
        capacity = _log(rng, 16, 8192)
        lens = ",".join(str(_log(rng, 1, capacity)) for _ in range(_log(rng, 1, min(64, 131072 // capacity))))
        return _decode("drawn", lens, capacity, P, hq, hk, dh)
    lens = ",".join(str(_log(rng, 1, 4096 if op == "attn" else 2048)) for _ in range(rng.randint(1, 4)))
    if op == "attn":
        return _attn("drawn", lens, P, hq, hk, dh, prefix=rng.choice([0, 0, _log(rng, 1, 1000)]))
    return _attn("drawn", lens, P, hq, hk, dh, backward=True)


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _pairs(lens, prefix):
    """Visible (query, key) pairs of one head."""
    return sum(n * (n + 1) // 2 + n * prefix for n in lens)


def work(case):
    P, hq, hk, dh = case["P"], case["hq"], case["hk"], case["dh"]
    if case["op"] == "rope":
        T = case["T"]
        rows = P * T * dh
        moved = 2 * (hq + hk) * rows + (2 * hk * rows if case["append"] else 0)
        return {"bytes": 2 * moved + 4 * T + (8 * T if case["append"] else 0), "flops": 3 * P * T * (hq + hk) * case["rot"]}
    lens = _lens(case)
    if case["op"] == "decode":
        n = sum(lens)
        return {"bytes": 2 * P * dh * (2 * hk * n + 2 * hq * len(lens)) + 4 * len(lens), "flops": 4 * P * hq * dh * n}
    tq = sum(lens)
    tk = tq + case["prefix"] * len(lens)
    pairs = P * hq * _pairs(lens, case["prefix"])
    if case["op"] == "attn":
        return {"bytes": 2 * P * dh * (2 * hq * tq + 2 * hk * tk) + 4 * P * hq * tq, "flops": 4 * dh * pairs}
    return {"bytes": 2 * P * dh * (4 * hq * tq + 4 * hk * tk) + 4 * P * hq * tq, "flops": 10 * dh * pairs}


def _frequencies(case):
    """Rotation per position of each pair, in 64 bits, and the factor on the rotated vectors.

    theta = 10000; "linear" divides every frequency by the factor (position interpolation); "ntk" raises theta so that
    the slowest pair is slowed by the factor; "yarn" slows the pairs that turn less than once over 4096 positions,
    keeps those that turn more than 32 times, blends between, and scales the vectors by 0.1 ln(factor) + 1.
    """
    rot, factor, theta = case["rot"], case["factor"], 10000.0
    if case["scaling"] == "ntk":
        theta *= factor ** (rot / (rot - 2))
    f = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "yarn":
        keep = ((4096 * f / (2 * math.pi) - 1) / (32 - 1)).clamp(0, 1)
        return f * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _random(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    P, hq, hk, dh = case["P"], case["hq"], case["hk"], case["dh"]
    s = {"case": case}
    if case["op"] == "rope":
        T = case["T"]
        s["q"], s["k"] = _random(g, P, T, hq, dh), _random(g, P, T, hk, dh)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        if T <= 64:  # a decoding step: every sequence at a position of its own
            shift = torch.randint(0, 1000, (T,), generator=g, device=DEV, dtype=torch.int64)
            s["positions"] = (case["origin"] + shift).to(torch.int32)
        else:  # packed prompts: positions start again in the middle
            at = torch.arange(T, device=DEV, dtype=torch.int32)
            s["positions"] = torch.where(at < (T + 1) // 2, at, at - (T + 1) // 2) + case["origin"]
        f, s["mscale"] = _frequencies(case)
        s["frequencies"], s["frequencies_gpu"] = f.numpy(), f.to(DEV)
        if case["append"]:
            rows = 2 * T + 5
            s["v"] = _random(g, P, T, hk, dh)
            s["k_cache"], s["v_cache"] = _random(g, P, rows, hk, dh), _random(g, P, rows, hk, dh)
            s["slots"] = torch.randperm(rows, generator=g, device=DEV)[:T]
        return s
    lens = _lens(case)
    if case["op"] == "decode":
        B, cap = len(lens), case["capacity"]
        s["q"] = _random(g, P, B, hq, dh)
        s["k_cache"], s["v_cache"] = _random(g, P, B, cap, hk, dh), _random(g, P, B, cap, hk, dh)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["out"] = torch.empty(P, B, hq * dh, dtype=torch.bfloat16, device=DEV)
        return s
    s["cu_q"] = _offsets(lens)
    s["cu_k"] = _offsets([n + case["prefix"] for n in lens])
    tq, tk = s["cu_q"][-1], s["cu_k"][-1]
    s["q"], s["k"], s["v"] = _random(g, P, tq, hq, dh), _random(g, P, tk, hk, dh), _random(g, P, tk, hk, dh)
    if case["op"] == "attn":
        s["out"] = torch.empty(P, tq, hq * dh, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(P, hq, tq, dtype=torch.float32, device=DEV)
    else:  # the forward pass that the gradients belong to
        s["out"], s["lse"] = _plain_attn(s)
        s["dout"] = _random(g, P, tq, hq * dh)
        s["dq"], s["dk"], s["dv"] = torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "attn": _own_attn, "attn_bwd": _own_attn_bwd, "decode": _own_decode}[op](state)
    return {"rope": _plain_rope, "attn": _plain_attn, "attn_bwd": _plain_attn_bwd, "decode": _plain_decode}[op](state)


# ------------------------------------------------------------------ the framework's calls

def _own_rope(s):
    from partial_activation_sync_caat_b200 import caat as C
    c = s["case"]
    kw = dict(q_out=s["q_out"], interleaved=c["layout"] == "interleaved", backward=c["backward"], mscale=s["mscale"])
    if c["append"]:
        C.caat_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["frequencies"], s["k_cache"],
                           s["v_cache"], **kw)
        return s["q_out"], s["k_cache"], s["v_cache"]
    C.caat_rope(s["q"], s["k"], s["positions"], s["frequencies"], k_out=s["k_out"], **kw)
    return s["q_out"], s["k_out"]


def _own_attn(s):
    from partial_activation_sync_caat_b200 import caat as C
    C.caat_attn_forward(s["q"], s["k"], s["v"], s["cu_q"], s["out"], cu_k=s["cu_k"], lse=s["lse"])
    return s["out"], s["lse"]


def _own_attn_bwd(s):
    from partial_activation_sync_caat_b200 import caat as C
    C.caat_attn_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["cu_q"], s["dq"], s["dk"], s["dv"],
                         cu_k=s["cu_k"])
    return s["dq"], s["dk"], s["dv"]


def _own_decode(s):
    from partial_activation_sync_caat_b200 import caat as C
    C.caat_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["lens"], s["out"])
    return s["out"]


# ------------------------------------------------------------------ plain forms

def _rotate(x, cos, sin, rot, interleaved):
    y = x.float()
    r = y[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., : rot // 2], r[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, y[..., rot:]), -1).to(x.dtype)


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["frequencies_gpu"]
    cos = (torch.cos(angle) * s["mscale"]).float()[:, None]
    sin = (torch.sin(angle) * s["mscale"]).float()[:, None]
    if c["backward"]:
        sin = -sin
    inter = c["layout"] == "interleaved"
    q, k = _rotate(s["q"], cos, sin, c["rot"], inter), _rotate(s["k"], cos, sin, c["rot"], inter)
    if not c["append"]:
        return q, k
    s["k_cache"][:, s["slots"]] = k
    s["v_cache"][:, s["slots"]] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _scores(q, k):
    """Masked scores [P, hk, group, n, m] of one sequence, the last query at the last key."""
    n, m = q.shape[-2], k.shape[-2]
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(q.shape[-1]))
    hidden = torch.ones(n, m, dtype=torch.bool, device=q.device).triu_(m - n + 1)
    return x.masked_fill_(hidden, -math.inf)


def _heads(x, a, b, hk):
    """Rows a..b of x [P, T, h, dh] as fp32 [P, hk, h / hk, b - a, dh]."""
    return x[:, a:b].float().permute(0, 2, 1, 3).unflatten(1, (hk, -1))


def _rows(x):
    """[P, hk, group, n, dh] as [P, n, hk group, dh]."""
    return x.flatten(1, 2).permute(0, 2, 1, 3)


def _plain_attn(s):
    hk = s["case"]["hk"]
    outs, lses = [], []
    for a, b, c, d in zip(s["cu_q"], s["cu_q"][1:], s["cu_k"], s["cu_k"][1:]):
        x = _scores(_heads(s["q"], a, b, hk), _heads(s["k"], c, d, hk))
        top = x.amax(-1, keepdim=True)
        x = x.sub_(top).exp_()
        total = x.sum(-1, keepdim=True)
        o = torch.matmul(x, _heads(s["v"], c, d, hk)) / total
        outs.append(_rows(o).flatten(2).to(torch.bfloat16))
        lses.append((top + total.log()).squeeze(-1).flatten(1, 2))
    return torch.cat(outs, 1), torch.cat(lses, -1)


def _plain_attn_bwd(s):
    hk, dh = s["case"]["hk"], s["case"]["dh"]
    found = []
    for a, b, c, d in zip(s["cu_q"], s["cu_q"][1:], s["cu_k"], s["cu_k"][1:]):
        q, k, v = _heads(s["q"], a, b, hk), _heads(s["k"], c, d, hk), _heads(s["v"], c, d, hk)
        do = _heads(s["dout"].unflatten(-1, (-1, dh)), a, b, hk)
        p = _scores(q, k)
        p = p.sub_(p.amax(-1, keepdim=True)).exp_()
        p = p.div_(p.sum(-1, keepdim=True))
        dv = torch.matmul(p.transpose(-1, -2), do).sum(2, keepdim=True)
        dp = torch.matmul(do, v.transpose(-1, -2))
        dp = dp.sub_(torch.matmul(p, v).mul_(do).sum(-1, keepdim=True)).mul_(p).mul_(1.0 / math.sqrt(dh))
        dk = torch.matmul(dp.transpose(-1, -2), q).sum(2, keepdim=True)
        found.append([_rows(x).to(torch.bfloat16) for x in (torch.matmul(dp, k), dk, dv)])
    return tuple(torch.cat(x, 1) for x in zip(*found))


def _plain_decode(s):
    q, k, v = s["q"], s["k_cache"], s["v_cache"]
    P, B, cap, hk, dh = k.shape
    x = torch.einsum("pbhgd,pbnhd->pbhgn", q.float().unflatten(2, (hk, -1)), k.float()) / math.sqrt(dh)
    hidden = torch.arange(cap, device=q.device) >= s["lens"][:, None]
    x = x.masked_fill_(hidden[:, None, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    x = x.div_(x.sum(-1, keepdim=True))
    return torch.einsum("pbhgn,pbnhd->pbhgd", x, v.float()).flatten(2).to(torch.bfloat16)


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attn": _exact_attn, "attn_bwd": _exact_attn, "decode": _exact_decode}[case["op"]](s)


def _exact_rope(s):
    # pair j is the complex number a_j + i b_j, multiplied by mscale e^(i position f_j)
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    first = range(0, rot, 2) if c["layout"] == "interleaved" else range(half)
    second = range(1, rot, 2) if c["layout"] == "interleaved" else range(half, rot)
    first, second = torch.tensor(first, device=DEV), torch.tensor(second, device=DEV)
    angle = torch.outer(s["positions"].double(), torch.as_tensor(s["frequencies"], device=DEV))
    turn = torch.polar(torch.full_like(angle, s["mscale"]), -angle if c["backward"] else angle)[None, :, None]

    def rotated(x):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q, k = rotated(s["q"]), rotated(s["k"])
    if not c["append"]:
        return q, k
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    k_cache.index_copy_(1, s["slots"], k)
    v_cache.index_copy_(1, s["slots"], s["v"].double())
    return q, k_cache, v_cache


def _exact_attn(s):
    # one rank, head and sequence at a time, queries in blocks of 1024
    c = s["case"]
    P, hq, hk, dh = c["P"], c["hq"], c["hk"], c["dh"]
    back = c["op"] == "attn_bwd"
    tq, tk = s["cu_q"][-1], s["cu_k"][-1]
    out = torch.empty(P, tq, hq, dh, dtype=torch.float64, device=DEV)
    lse = torch.empty(P, hq, tq, dtype=torch.float64, device=DEV)
    dk = torch.zeros(P, tk, hk, dh, dtype=torch.float64, device=DEV)
    dv = torch.zeros_like(dk)
    for r in range(P):
        for h in range(hq):
            kv = h // (hq // hk)
            for i in range(len(s["cu_q"]) - 1):
                q0, q1, k0, k1 = s["cu_q"][i], s["cu_q"][i + 1], s["cu_k"][i], s["cu_k"][i + 1]
                K, V = s["k"][r, k0:k1, kv].double(), s["v"][r, k0:k1, kv].double()
                for a in range(q0, q1, 1024):
                    b = min(a + 1024, q1)
                    Q = s["q"][r, a:b, h].double()
                    last = torch.arange(a, b, device=DEV) - q0 + (k1 - k0) - (q1 - q0)
                    n = int(last[-1]) + 1
                    S = Q @ K[:n].T / dh ** 0.5
                    S[torch.arange(n, device=DEV)[None] > last[:, None]] = -math.inf
                    L = torch.logsumexp(S, -1)
                    W = torch.exp(S - L[:, None])
                    if not back:
                        lse[r, h, a:b], out[r, a:b, h] = L, W @ V[:n]
                        continue
                    G = s["dout"][r, a:b, h * dh:(h + 1) * dh].double()
                    dW = G @ V[:n].T
                    dS = W * (dW - (W * dW).sum(-1, keepdim=True)) / dh ** 0.5
                    dv[r, k0:k0 + n, kv] += W.T @ G
                    dk[r, k0:k0 + n, kv] += dS.T @ Q
                    out[r, a:b, h] = dS @ K[:n]
    return (out, dk, dv) if back else (out.flatten(2), lse)


def _exact_decode(s):
    c = s["case"]
    P, hk, dh = c["P"], c["hk"], c["dh"]
    out = torch.empty_like(s["out"], dtype=torch.float64)
    for b, n in enumerate(_lens(c)):
        K, V = s["k_cache"][:, b, :n].double(), s["v_cache"][:, b, :n].double()
        Q = s["q"][:, b].double().view(P, hk, -1, dh)
        W = torch.softmax(torch.matmul(Q, K.permute(0, 2, 3, 1)) / dh ** 0.5, -1)
        out[:, b] = torch.matmul(W, V.permute(0, 2, 1, 3)).reshape(P, -1)
    return out
