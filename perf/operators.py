"""Cases of the operators around the quantised projections of a transformer layer:

  gemm  Y = act(X What^T + bias) (+ residual), the W4A16 product with its epilogue; with
        `gated`, packed rows come in alternating blocks of 8 gate and 8 up rows and
        Y = act(gate) * up;
  rope  rotary positions on the query and key heads of a fused qkv projection's output;
  attn  attention of a packed batch of prompts (or of their next tokens over earlier
        keys) with grouped heads, causal positions aligned at the sequences' ends.

`run` computes them in plain 32-bit torch, or through the package where `own` is true.
"""
import math
import random

import numpy as np
import torch

own = False

GROUP_ROWS = 8      # rows of one gate (or up) block in the packed order of gated weights
W_STD = 0.02


def _gemm(name, M, N, K, dtype, group=128, symmetric=False, bias=False, act="none", gated=False, residual=False):
    c = {"op": "gemm", "M": M, "N": N, "K": K, "dtype": dtype, "group": group, "symmetric": symmetric,
         "bias": bias, "act": act, "gated": gated, "residual": residual}
    return {"name": name, **c} if name else c


def _rope(name, T, heads, kv_heads, dim, rot, dtype, interleaved=False, start=0, theta=10000.0, factor=1.0, mscale=1.0):
    c = {"op": "rope", "T": T, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot, "dtype": dtype,
         "interleaved": interleaved, "start": start, "theta": theta, "factor": factor, "mscale": mscale}
    return {"name": name, **c} if name else c


def _attn(name, batch, tokens, heads, kv_heads, dim, dtype, causal=True, keys=0, shortest=0):
    """`batch` sequences of `tokens` query tokens together, of lengths that the seed draws
    (all `tokens` for one sequence); `keys`: earlier keys together, on top of the tokens;
    `shortest`: how many of the sequences have one token."""
    c = {"op": "attn", "batch": batch, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
         "dtype": dtype, "causal": causal, "keys": keys, "shortest": shortest}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one token through the 7B-shaped qkv projection with its bias
        _gemm("gemm_decode_qkv_bias", 1, 12288, 4096, "fp16", bias=True),
        # eight streams through the 7B-shaped gate and up projections, SwiGLU in the product
        _gemm("gemm_decode_swiglu", 8, 22016, 4096, "fp16", act="silu", gated=True),
        # a small batch through the 70B-shaped down projection, added to the residual stream
        _gemm("gemm_batch_down_residual", 32, 8192, 28672, "fp16", residual=True),
        # a prompt through the 8B-shaped gate and up projections, SwiGLU in the product
        _gemm("gemm_prompt_swiglu", 2048, 28672, 4096, "bf16", act="silu", gated=True),
        # an odd prompt through a plain MLP's first layer: bias and GELU, symmetric weights, small groups
        _gemm("gemm_prompt_gelu", 1037, 11008, 4096, "bf16", group=64, symmetric=True, bias=True, act="gelu_tanh"),
        # the next token's 8B-shaped query and key heads (32 + 8): latency
        _rope("rope_token", 1, 32, 8, 128, 128, "bf16", start=4095, theta=500000.0),
        # a long prompt's, with frequencies stretched for long contexts
        _rope("rope_prompt", 8192, 32, 8, 128, 128, "bf16", theta=500000.0, factor=8.0, mscale=1.2),
        # an odd prompt's 7B-shaped heads, half of each head rotated in interleaved pairs, far positions
        _rope("rope_partial_far", 1531, 32, 32, 128, 64, "fp16", interleaved=True, start=1000003),
        # one short prompt, 7B-shaped heads: latency
        _attn("attn_short", 1, 61, 32, 32, 128, "fp16"),
        # one long 8B-shaped prompt
        _attn("attn_prompt", 1, 8192, 32, 8, 128, "bf16"),
        # a packed batch of 70B-shaped prompts of many lengths, some of one token
        _attn("attn_packed", 24, 8192, 64, 8, 128, "bf16", shortest=4),
        # the next token of sixteen 70B-shaped sequences over their earlier keys
        _attn("attn_next_token", 16, 16, 64, 8, 128, "fp16", keys=65536, shortest=16),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm uniform."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


DRAW_FLOPS = 4.5e11   # a drawn case costs less than the largest listed ones


def draw(rng):
    op = rng.choice(["gemm", "gemm", "rope", "attn", "attn"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "gemm":
        group = rng.choice([32, 64, 128, 128])
        gated = rng.random() < 0.4
        N = 16 * _between(rng, 16, 1376)
        K = max(group, 64) * _between(rng, 4, 14336 // max(group, 64))
        act = rng.choice(["silu", "gelu_tanh"]) if gated else rng.choice(["none", "none", "relu", "gelu", "gelu_tanh", "silu"])
        M = _between(rng, 1, max(1, min(1500, int(DRAW_FLOPS / (2 * N * K)))))
        return _gemm(None, M, N, K, dtype, group, rng.random() < 0.3, rng.random() < 0.5, act, gated, rng.random() < 0.5)
    if op == "rope":
        dim = rng.choice([64, 96, 128])
        kv = _between(rng, 1, 8)
        return _rope(None, _between(rng, 1, 8192), kv * rng.choice([1, 2, 4, 5]), kv, dim, rng.choice([dim, dim, dim // 2]), dtype,
                     rng.random() < 0.5, rng.choice([0, 0, _between(rng, 1, 1 << 20)]), rng.choice([10000.0, 500000.0]),
                     rng.choice([1.0, 4.0, 8.0]), rng.choice([1.0, 1.1]))
    kv = _between(rng, 1, 8)
    heads = kv * rng.choice([1, 1, 2, 3, 4, 7, 8])
    dim = rng.choice([64, 80, 128, 128])
    batch = _between(rng, 1, 32)
    if rng.random() < 0.3:   # next tokens, or the next few of some sequences
        return _attn(None, batch, batch + rng.choice([0, 0, _between(rng, 1, 64)]), heads, kv, dim, dtype, True,
                     _between(rng, 16, 60000), 0)
    most = math.sqrt(DRAW_FLOPS / (4 * dim * heads))   # tokens of one sequence whose square costs that
    return _attn(None, batch, batch + _between(rng, 16, int(min(8000, 0.75 * most))), heads, kv, dim, dtype, rng.random() < 0.8,
                 rng.choice([0, 0, _between(rng, 16, int(min(2000, most / 2)))]), min(batch - 1, rng.choice([0, 2])))


# ---------------------------------------------------------------- inputs
def _dtype(case):
    return torch.float16 if case["dtype"] == "fp16" else torch.bfloat16


def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + salt)


def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _codes(case, seed):
    """(codes int32 [N,K] in 0..15, scales fp16 [G,N], zeros fp16 [G,N] or None)."""
    N, K = case["N"], case["K"]
    g = _gen(seed, 1)
    # rounded normals around the middle of the range, as a quantiser leaves them
    q = (torch.randn(N, K, generator=g, device="cuda") * 2.6 + 7.5).round_().clamp_(0, 15).to(torch.int32)
    G = K // case["group"]
    scales = (W_STD / 2.6 * (0.8 + 0.4 * torch.rand(G, N, generator=g, device="cuda"))).half()
    zeros = None if case["symmetric"] else torch.randint(6, 10, (G, N), generator=g, device="cuda").half()
    return q, scales, zeros


def _pack(q):
    """The device layout: 128-row bands, stored 64-column block by block, in 16 x 64 atoms of
    32 lanes x 4 words whose nibbles are (row half, column 8s, column 1s)."""
    N, K = q.shape
    T, A = N // 16, K // 64
    v = q.view(T, 2, 8, A, 4, 2, 4, 2)   # row half, row, block, step, column 8s, pair, column 1s
    words = torch.zeros(T, 8, A, 4, 4, dtype=torch.int32, device=q.device)
    for half in range(2):
        for hi in range(2):
            for lo in range(2):
                words |= v[:, half, :, :, :, hi, :, lo] << (4 * (half + 2 * hi + 4 * lo))
    atoms = words.permute(0, 2, 1, 4, 3).reshape(T, A, 128)
    full = T // 8 * 8
    parts = [atoms[:full].view(full // 8, 8, A, 128).permute(0, 2, 1, 3).reshape(-1)]
    if full < T:
        parts.append(atoms[full:].permute(1, 0, 2).reshape(-1))
    return torch.cat(parts).contiguous()


def _lengths(case, seed):
    """(query lengths, earlier keys) of the sequences, as numpy arrays."""
    r = np.random.default_rng([int(seed) % (1 << 32), 7])
    B, T = case["batch"], case["tokens"]
    ones = min(case["shortest"], B)
    if ones == B and T == B:
        lens = np.ones(B, np.int64)
    else:
        w = np.exp(r.normal(0.0, 0.8, B))
        w[r.permutation(B)[:ones]] = 0.0
        if w.sum() == 0:
            w[:] = 1.0
        lens = 1 + np.floor(w / w.sum() * (T - B)).astype(np.int64)
        lens[int(np.argmax(w))] += T - lens.sum()
    w = np.exp(r.normal(0.0, 0.5, B))
    past = np.floor(w / w.sum() * case["keys"]).astype(np.int64)
    past[0] += case["keys"] - past.sum()
    return lens, past


def prepare(case, seed):
    if case["op"] == "gemm":
        M, N, K, dt = case["M"], case["N"], case["K"], _dtype(case)
        q, scales, zeros = _codes(case, seed)
        g = _gen(seed, 2)
        X = _randn(g, M, K, dtype=dt)
        n_out = N // 2 if case["gated"] else N
        return {"case": case, "X": X, "qweight": _pack(q), "scales": scales, "zeros": zeros,
                "bias": _randn(g, N, dtype=dt) if case["bias"] else None,
                "residual": _randn(g, M, n_out, dtype=dt) if case["residual"] else None}
    if case["op"] == "rope":
        T, H, Hk, D = case["T"], case["heads"], case["kv_heads"], case["dim"]
        qkv = _randn(_gen(seed, 3), T, H + 2 * Hk, D, dtype=_dtype(case))   # a fused projection's output
        inv = case["theta"] ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        return {"case": case, "qkv": qkv, "inv_freq": inv / case["factor"],
                "positions": case["start"] + torch.arange(T, dtype=torch.int32, device="cuda")}
    H, Hk, D, dt = case["heads"], case["kv_heads"], case["dim"], _dtype(case)
    lens, past = _lengths(case, seed)
    cu_q = np.concatenate([[0], np.cumsum(lens)])
    cu_k = np.concatenate([[0], np.cumsum(lens + past)])
    Tq, Tk = int(cu_q[-1]), int(cu_k[-1])
    g = _gen(seed, 4)
    if case["keys"] == 0:   # whole prompts: slices of the fused projection's output
        qkv = _randn(g, Tq, H + 2 * Hk, D, dtype=dt)
        Q, K, V = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    else:
        Q, K, V = _randn(g, Tq, H, D, dtype=dt), _randn(g, Tk, Hk, D, dtype=dt), _randn(g, Tk, Hk, D, dtype=dt)
    as_gpu = lambda a: torch.from_numpy(a.astype(np.int32)).cuda()  # noqa: E731
    return {"case": case, "Q": Q, "K": K, "V": V, "cu_q": as_gpu(cu_q), "cu_k": as_gpu(cu_k) if case["keys"] else None}


# ---------------------------------------------------------------- one pass
def run(state):
    return {"gemm": _run_gemm, "rope": _run_rope, "attn": _run_attn}[state["case"]["op"]](state)


def _package():
    import bit_weight_only_w4_b200 as w4
    return w4


def _run_gemm(s):
    c = s["case"]
    if own:
        return _package().w4a16_gemm_epi(s["X"], s["qweight"], s["scales"], s["zeros"], c["group"], bias=s["bias"],
                                         activation=c["act"], gated=c["gated"], residual=s["residual"])
    return _plain_gemm(s)


def _plain_gemm(s):
    c = s["case"]
    N, K = c["N"], c["K"]
    T, A = N // 16, K // 64
    full = T // 8 * 8
    words, cut = s["qweight"], full * A * 128
    atoms = torch.cat([words[:cut].view(full // 8, A, 8, 128).permute(0, 2, 1, 3).reshape(full, A, 128),
                       words[cut:].view(A, T - full, 128).permute(1, 0, 2)])
    # bits of a word: 4 (row half + 2 column 8s + 4 column 1s)
    nib = (atoms.view(T, A, 8, 4, 4, 1) >> torch.arange(0, 32, 4, device=atoms.device, dtype=torch.int32)) & 15
    q = nib.view(T, A, 8, 4, 4, 2, 2, 2).permute(0, 7, 2, 1, 4, 6, 3, 5).reshape(N, K)
    scale = s["scales"].float().t().repeat_interleave(c["group"], 1)
    zero = 8.0 if s["zeros"] is None else s["zeros"].float().t().repeat_interleave(c["group"], 1)
    y = s["X"].float() @ ((q.float() - zero) * scale).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if c["gated"]:
        y = y.view(c["M"], N // 16, 2, GROUP_ROWS)
        y = _activate(y[:, :, 0], c["act"]).reshape(c["M"], N // 2) * y[:, :, 1].reshape(c["M"], N // 2)
    else:
        y = _activate(y, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["X"].dtype)


def _activate(x, name):
    if name == "silu":
        return x / (1 + torch.exp(-x))
    if name == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if name == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _run_rope(s):
    c = s["case"]
    X = s["qkv"][:, :c["heads"] + c["kv_heads"]]
    if own:
        return _package().w4_rope(X, s["positions"], s["inv_freq"], interleaved=c["interleaved"], mscale=c["mscale"])
    rot = c["rot"]
    # angles in 64 bits: 32 lose far positions' fractions of a turn
    angle = s["positions"].double()[:, None] * s["inv_freq"][None, :]
    cos = (torch.cos(angle) * c["mscale"]).float()[:, None]
    sin = (torch.sin(angle) * c["mscale"]).float()[:, None]
    x = X.float()
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1).to(X.dtype)


def _run_attn(s):
    c = s["case"]
    Q, K, V = s["Q"], s["K"], s["V"]
    if own:
        return _package().w4_prompt_attention(Q, K, V, s["cu_q"], s["cu_k"], causal=c["causal"], return_lse=True)
    cu_q, cu_k = s["cu_q"].long(), (s["cu_q"] if s["cu_k"] is None else s["cu_k"]).long()
    Tq, Tk, H, Hk, D = Q.shape[0], K.shape[0], c["heads"], c["kv_heads"], c["dim"]
    at_q, at_k = torch.arange(Tq, device=Q.device), torch.arange(Tk, device=Q.device)
    of_q, of_k = torch.searchsorted(cu_q, at_q, right=True) - 1, torch.searchsorted(cu_k, at_k, right=True) - 1
    seen = of_q[:, None] == of_k[None, :]
    if c["causal"]:   # distances from the sequences' ends
        seen &= (cu_q[of_q + 1] - at_q)[:, None] <= (cu_k[of_k + 1] - at_k)[None, :]
    q = Q.float().view(Tq, Hk, H // Hk, D).permute(1, 2, 0, 3).reshape(Hk, H // Hk * Tq, D)
    scores = (q @ K.float().permute(1, 2, 0)).view(H, Tq, Tk).mul_(1 / math.sqrt(D))
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_min_(torch.finfo(torch.float32).min)
    p = scores.sub_(top).exp_()
    total = p.sum(-1)
    o = (p.view(Hk, H // Hk * Tq, Tk) @ V.float().permute(1, 0, 2)).view(H, Tq, D)
    o = o / total[..., None].masked_fill(total[..., None] == 0, 1.0)
    lse = (top[..., 0] + total.log()).t().contiguous()
    return o.permute(1, 0, 2).to(Q.dtype).contiguous(), lse


# ---------------------------------------------------------------- costs
def work(case):
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        n_out = N // 2 if case["gated"] else N
        meta = (1 if case["symmetric"] else 2) * 2 * (K // case["group"]) * N
        b = N * K // 2 + meta + 2 * M * K + 2 * M * n_out * (2 if case["residual"] else 1) + (2 * N if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * M * N * K}
    if case["op"] == "rope":
        n = case["T"] * (case["heads"] + case["kv_heads"])
        return {"bytes": 4 * n * case["dim"] + 4 * case["T"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    lens, past = _lengths(case, 0)   # the pairs depend on the lengths; those of one seed stand for all
    pairs = lens * past + (lens * (lens + 1) / 2 if case["causal"] else lens * lens)
    Tq, Tk = int(lens.sum()), int((lens + past).sum())
    return {"bytes": 2 * D * (2 * Tq * H + 2 * Tk * Hk) + 4 * Tq * H, "flops": 4 * D * H * float(pairs.sum())}


# ---------------------------------------------------------------- the same in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemm":
        q, scales, zeros = _codes(case, seed)
        G, N, K = scales.shape[0], case["N"], case["K"]
        zero = torch.full_like(scales, 8.0) if zeros is None else zeros
        X = s["X"].double()
        y = torch.zeros(case["M"], N, dtype=torch.float64, device="cuda")
        del s["qweight"]
        for n0 in range(0, N, 4096):
            n1 = min(N, n0 + 4096)
            w = q[n0:n1].view(n1 - n0, G, K // G).double()
            w = (w - zero[:, n0:n1].t()[:, :, None].double()) * scales[:, n0:n1].t()[:, :, None].double()
            y[:, n0:n1] = torch.einsum("mk,nk->mn", X, w.reshape(n1 - n0, K))
        if s["bias"] is not None:
            y += s["bias"].double()
        fn = {"none": lambda t: t, "relu": torch.relu, "silu": lambda t: t * torch.sigmoid(t),
              "gelu": lambda t: t * torch.special.ndtr(t),
              "gelu_tanh": lambda t: t * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3))}[case["act"]]
        if case["gated"]:
            rows = torch.arange(N, device="cuda")
            gate, up = rows[rows // GROUP_ROWS % 2 == 0], rows[rows // GROUP_ROWS % 2 == 1]
            y = fn(y[:, gate]) * y[:, up]
        else:
            y = fn(y)
        return y if s["residual"] is None else y + s["residual"].double()
    if case["op"] == "rope":
        x = s["qkv"][:, :case["heads"] + case["kv_heads"]].double()
        rot, half = case["rot"], case["rot"] // 2
        i = torch.arange(half, device="cuda")
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        turn = torch.polar(torch.full((), case["mscale"], dtype=torch.float64, device="cuda").expand(case["T"], half).contiguous(),
                           s["positions"].double()[:, None] * s["inv_freq"])[:, None]
        z = torch.complex(x[..., first], x[..., second]) * turn
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y
    lens, past = _lengths(case, seed)
    H, D, rep = case["heads"], case["dim"], case["heads"] // case["kv_heads"]
    o = torch.zeros(s["Q"].shape[0], H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((s["Q"].shape[0], H), -math.inf, dtype=torch.float64, device="cuda")
    a = b = 0
    for n, m in zip(lens.tolist(), (lens + past).tolist()):
        K, V = s["K"][b:b + m].double(), s["V"][b:b + m].double()
        for h in range(0, H, rep):
            x = torch.einsum("qgd,kd->gqk", s["Q"][a:a + n, h:h + rep].double(), K[:, h // rep]) / D ** 0.5
            if case["causal"]:
                x += torch.full((n, m), -math.inf, dtype=torch.float64, device="cuda").triu(m - n + 1)
            lse[a:a + n, h:h + rep] = torch.logsumexp(x, -1).t()
            o[a:a + n, h:h + rep] = torch.einsum("gqk,kd->qgd", torch.softmax(x, -1), V[:, h // rep])
        a, b = a + n, b + m
    return o, lse


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(k)) for k in range(6)]:
        print(case, work(case))
