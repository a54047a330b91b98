"""The cases on which layer normalisation and windowed attention are measured.

Layer normalisation (forward with the residual sum, backward with the weight
gradients) and attention with a sliding window and first tokens that stay
visible (forward, backward, and single tokens against a cache).  Each case
runs in two forms on the same inputs: elementary torch operations in 32 bits
(`own` false), or the calls a user makes of the library (`own` true).

Sizes: 16384 tokens of width 768 with 12 heads of 64 (128 sequences of 128
tokens), 32768 tokens of width 1024 (64 sequences of 512), the 4096-wide and
the 64-wide layers are the ones of the library's benchmark; the others are
generic.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-5


# --------------------------------------------------------------------------
# Cases

def norm(op, T, N, dtype, res):
    return {"op": op, "T": T, "N": N, "dtype": dtype, "res": res}


def attn(op, B, lo, hi, heads, kv, dim, left, right, sinks, dtype, q=0, cap=0):
    """B sequences of lo..hi keys.  q == 0: every key's token is a query too
    (packed sequences).  q > 0: the last q tokens of each sequence are the
    queries, the keys lie in a cache of `cap` rows a sequence."""
    return {"op": op, "B": B, "lo": lo, "hi": hi, "heads": heads, "kv": kv, "dim": dim,
            "left": left, "right": right, "sinks": sinks, "dtype": dtype, "q": q, "cap": cap}


def listed():
    return [
        # one step of the smallest layer of the benchmark: latency
        dict(norm("norm_fwd", 16, 64, "f32", False), name="norm fwd 16x64 f32"),
        # between the attention output and the FFN pair of a 768-wide block
        dict(norm("norm_fwd", 16384, 768, "bf16", True), name="norm fwd 16384x768 bf16"),
        dict(norm("norm_bwd", 16384, 768, "bf16", True), name="norm bwd 16384x768 bf16"),
        # a width whose rows are not aligned, in full precision
        dict(norm("norm_bwd", 4095, 1023, "f32", False), name="norm bwd 4095x1023 f32"),
        # a wide layer's output at the largest token count of the benchmark
        dict(norm("norm_fwd", 32768, 4096, "bf16", False), name="norm fwd 32768x4096 bf16"),
        # an encoder's self-attention: 128 sequences of 128 tokens, local, first token global
        dict(attn("attn_fwd", 128, 128, 128, 12, 12, 64, 64, 64, 1, "bf16"),
             name="attn fwd 128x128 h12 d64"),
        dict(attn("attn_bwd", 128, 128, 128, 12, 12, 64, 64, 64, 1, "bf16"),
             name="attn bwd 128x128 h12 d64"),
        # a ragged batch of longer sequences, packed
        dict(attn("attn_fwd", 64, 257, 512, 16, 16, 64, 128, 128, 1, "bf16"),
             name="attn fwd 64x257-512 h16 d64"),
        dict(attn("attn_bwd", 64, 257, 512, 16, 16, 64, 128, 128, 1, "bf16"),
             name="attn bwd 64x257-512 h16 d64"),
        # one long causal sequence with shared key heads: training on long text
        dict(attn("attn_bwd", 1, 16384, 16384, 8, 2, 128, 1023, 0, 4, "bf16"),
             name="attn bwd 16384 causal h8/2 d128"),
        # full precision, ragged, a small model's heads
        dict(attn("attn_bwd", 32, 33, 97, 8, 8, 32, 24, 24, 2, "f32"),
             name="attn bwd 32x33-97 h8 d32 f32"),
        # one new token a sequence against a long cache: serving
        dict(attn("attn_fwd", 32, 3001, 8192, 16, 4, 128, 1023, 0, 4, "bf16", 1, 8192),
             name="attn decode 32x3001-8192 h16/4 d128"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    kind = rng.choice(["norm_fwd", "norm_bwd", "attn_fwd", "attn_bwd", "decode"])
    if kind.startswith("norm"):
        N = _log_int(rng, 48, 4200)
        N -= N % rng.choice([1, 2, 8, 64]) if N >= 128 else 0
        N += N == 3072
        T = _log_int(rng, 1, min(40000, 134000000 // N))
        return norm(kind, T, N, dtype, rng.random() < 0.5)
    kv = rng.choice([1, 2, 4, 12])
    heads = kv * rng.choice([1, 1, 2, 4])
    dim = rng.choice([32, 40, 64, 64, 80, 128]) if dtype == "bf16" else rng.choice([24, 32, 64])
    sinks = rng.choice([0, 1, 4, 17])
    if kind == "decode":
        hi = _log_int(rng, 64, 30000)
        lo = max(1, hi - _log_int(rng, 1, hi))
        B = _log_int(rng, 1, max(1, min(64, 200000 // hi)))
        left = rng.choice([-1, _log_int(rng, 16, 4000)])
        return attn("attn_fwd", B, lo, hi, heads, kv, dim, left, 0, sinks, dtype,
                    rng.choice([1, 1, 1, 2]), hi + rng.randrange(0, 100))
    hi = _log_int(rng, 16, 6000 if dtype == "bf16" else 1200)
    lo = max(1, hi - rng.choice([0, hi // 7, hi // 2]))
    # the padded score matrices stay under a sixth of the largest listed case's
    B = _log_int(rng, 1, max(1, min(64, 350000000 // (heads * hi * hi))))
    left = _log_int(rng, 8, 1200)
    right = rng.choice([0, left])
    return attn(kind, B, lo, hi, heads, kv, dim, left, right, sinks, dtype)


# --------------------------------------------------------------------------
# Inputs

def _lengths(c):
    span = c["hi"] - c["lo"] + 1
    return [c["lo"] + (b * 7919 + span - 1) % span for b in range(c["B"])]


def _visible(c):
    """(visible query-key pairs, distinct keys seen) of one head over the batch."""
    pairs = keys = 0
    for n in _lengths(c):
        lq = c["q"] or n
        lq = min(lq, n)
        i = torch.arange(n - lq, n, dtype=torch.int64)
        hi = torch.full_like(i, n - 1) if c["right"] < 0 else (i + c["right"]).clamp(max=n - 1)
        lo = torch.zeros_like(i) if c["left"] < 0 else (i - c["left"]).clamp(min=0)
        sunk = torch.minimum(lo, torch.full_like(i, c["sinks"]))
        sunk = torch.minimum(sunk, hi + 1).clamp(min=0)
        pairs += int((hi - lo + 1 + sunk).sum())
        keys += min(n, n - int(lo.min()) + min(c["sinks"], int(lo.min())))
    return pairs, keys


def prepare(case, seed):
    c = dict(case)
    dt = DTYPES[c["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    st = {"case": c}
    if c["op"].startswith("norm"):
        T, N = c["T"], c["N"]
        # activations with a feature-dependent offset and spread, as a trained block has
        x = torch.randn(T, N, generator=g, device="cuda")
        x = (x * (0.5 + torch.rand(N, generator=g, device="cuda")) +
             0.3 * torch.randn(N, generator=g, device="cuda")).to(dt)
        st["x"] = x
        st["gamma"] = 1.0 + 0.2 * torch.randn(N, generator=g, device="cuda")
        st["beta"] = 0.1 * torch.randn(N, generator=g, device="cuda")
        if c["op"] == "norm_fwd":
            st["res"] = randn(T, N) if c["res"] else None
        else:
            st["dy"] = randn(T, N, scale=0.1)
            st["dsum"] = randn(T, N, scale=0.1) if c["res"] else None
            st["stats"] = _plain_stats(x.float())
        return st
    B, H, KV, D = c["B"], c["heads"], c["kv"], c["dim"]
    lens = _lengths(c)
    lk = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if c["q"]:
        lq = torch.full_like(lk, c["q"]).minimum(lk)
        Tk = B * c["cap"]
        k_begin = torch.arange(B, dtype=torch.int32, device="cuda") * c["cap"]
        Tq, max_q = sum(min(c["q"], n) for n in lens), c["q"]
        q_end = torch.cumsum(lq, 0).to(torch.int32)
        st["k_begin"], st["k_end"] = k_begin, k_begin + lk
    else:
        lq, Tq, Tk, max_q = lk, sum(lens), sum(lens), c["hi"]
        q_end = torch.cumsum(lq, 0).to(torch.int32)
        st["k_begin"], st["k_end"] = q_end - lk, q_end
    st["q_begin"], st["q_end"] = q_end - lq, q_end
    st["max_q"], st["max_k"] = max_q, c["hi"]
    st["q"] = randn(Tq, H, D, scale=1.5)
    st["k"] = randn(Tk, KV, D)
    st["v"] = randn(Tk, KV, D)
    if c["op"] == "attn_bwd":
        st["do"] = randn(Tq, H, D)
        st["o"], st["lse"] = _plain_attn_fwd(st)
    return st


# --------------------------------------------------------------------------
# Plain forms

def _plain_stats(s):
    mean = s.mean(1, keepdim=True)
    var = (s - mean).square().mean(1, keepdim=True)
    return torch.cat([mean, (var + EPS).rsqrt()], 1)


def _plain_norm_fwd(st):
    s = st["x"].float()
    if st["res"] is not None:
        s = s + st["res"].float()
    stats = _plain_stats(s)
    y = (s - stats[:, :1]) * stats[:, 1:] * st["gamma"] + st["beta"]
    dt = st["x"].dtype
    return {"y": y.to(dt), "sum": s.to(dt) if st["res"] is not None else None, "stats": stats}


def _plain_norm_bwd(st):
    dy = st["dy"].float()
    mean, rstd = st["stats"][:, :1], st["stats"][:, 1:]
    xhat = (st["x"].float() - mean) * rstd
    g = dy * st["gamma"]
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if st["dsum"] is not None:
        dx = dx + st["dsum"].float()
    return {"dx": dx.to(st["x"].dtype), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}


def _rows(x, begin, end, most):
    """Each sequence's rows of x in 32 bits, (B, heads, most, dim), zero past its end."""
    i = torch.arange(most, device=x.device)
    valid = i < (end - begin)[:, None]
    at = torch.where(valid, begin[:, None] + i, 0)
    return (x[at].float() * valid[:, :, None, None]).transpose(1, 2)


def _packed(x, begin, end, rows):
    """The inverse of _rows: (B, heads, most, dim) to (rows, heads, dim), rows of no sequence zero."""
    t = torch.arange(rows, device=x.device)
    inside = (t[:, None] >= begin) & (t[:, None] < end)
    b = (inside * torch.arange(begin.shape[0], device=x.device)).sum(1)
    i = (t - begin[b]).clamp(0, x.shape[2] - 1)
    return x.transpose(1, 2)[b, i] * inside.any(1)[:, None, None]


def _plain_probs(st):
    """The padded operands, softmax weights (0 where masked) and row log-sums."""
    c = st["case"]
    B, KV, G, D = c["B"], c["kv"], c["heads"] // c["kv"], c["dim"]
    nq, nk = st["max_q"], st["max_k"]
    q = _rows(st["q"], st["q_begin"], st["q_end"], nq).reshape(B, KV, G * nq, D)
    k = _rows(st["k"], st["k_begin"], st["k_end"], nk)
    v = _rows(st["v"], st["k_begin"], st["k_end"], nk)
    lq, lk = st["q_end"] - st["q_begin"], st["k_end"] - st["k_begin"]
    t, j = torch.arange(nq, device="cuda"), torch.arange(nk, device="cuda")
    i = (t + (lk - lq)[:, None])[:, :, None]
    seen = (t < lq[:, None])[:, :, None] & (j < lk[:, None])[:, None, :]
    if c["right"] >= 0:
        seen = seen & (j <= i + c["right"])
    if c["left"] >= 0:
        seen = seen & ((j >= i - c["left"]) | (j < c["sinks"]))
    s = (q @ k.transpose(2, 3)).mul_(1 / math.sqrt(D)).reshape(B, KV, G, nq, nk)
    s = s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(4, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    z = p.sum(4, keepdim=True)
    p = p.div_(torch.where(z == 0, 1.0, z))
    return q, k, v, p.reshape(B, KV, G * nq, nk), (m + z.log()).reshape(B, KV * G, nq, 1)


def _plain_attn_fwd(st):
    c = st["case"]
    rows = st["q"].shape[0]
    q, k, v, p, lse = _plain_probs(st)
    o = (p @ v).reshape(c["B"], c["heads"], st["max_q"], c["dim"])
    o = _packed(o, st["q_begin"], st["q_end"], rows)
    lse = _packed(lse, st["q_begin"], st["q_end"], rows)[:, :, 0].t().contiguous()
    return o.to(st["q"].dtype), lse


def _plain_attn_bwd(st):
    c = st["case"]
    B, KV, H, D, nq = c["B"], c["kv"], c["heads"], c["dim"], st["max_q"]
    q, k, v, p, _ = _plain_probs(st)
    do = _rows(st["do"], st["q_begin"], st["q_end"], nq).reshape(B, KV, -1, D)
    dv = p.transpose(2, 3) @ do
    ds = do @ v.transpose(2, 3)
    ds = ds.sub_((ds * p).sum(3, keepdim=True)).mul_(p).mul_(1 / math.sqrt(D))
    dq = (ds @ k).reshape(B, H, nq, D)
    dk = ds.transpose(2, 3) @ q
    dt, Tq, Tk = st["q"].dtype, st["q"].shape[0], st["k"].shape[0]
    return {"dq": _packed(dq, st["q_begin"], st["q_end"], Tq).to(dt),
            "dk": _packed(dk, st["k_begin"], st["k_end"], Tk).to(dt),
            "dv": _packed(dv, st["k_begin"], st["k_end"], Tk).to(dt)}


# --------------------------------------------------------------------------
# One pass

def run(st):
    op = st["case"]["op"]
    if own:
        return _own(st, op)
    if op == "norm_fwd":
        return _plain_norm_fwd(st)
    if op == "norm_bwd":
        return _plain_norm_bwd(st)
    if op == "attn_fwd":
        o, lse = _plain_attn_fwd(st)
        return {"o": o, "lse": lse}
    return _plain_attn_bwd(st)


def _own(st, op):
    """The library's calls; the plan, output buffers and workspace are kept
    with the state, as a program that runs many steps keeps them."""
    c = st["case"]
    if op.startswith("norm"):
        if "plan" not in st:
            from tensor_train_compressed_tt_gb300.layer import TTNorm
            st["plan"] = TTNorm(c["N"], DTYPES[c["dtype"]], eps=EPS)
            st["ws"] = st["plan"].workspace(c["T"])
            st["out"] = torch.empty_like(st["x"])
            st["sum"] = torch.empty_like(st["x"]) if st.get("res") is not None else None
            st["new_stats"] = torch.empty(c["T"], 2, device="cuda")
            st["dgamma"], st["dbeta"] = torch.empty_like(st["gamma"]), torch.empty_like(st["beta"])
        if op == "norm_fwd":
            y, s, stats = st["plan"].forward(st["x"], st["gamma"], st["beta"], res=st["res"],
                                             y=st["out"], sum=st["sum"], stats=st["new_stats"])
            return {"y": y, "sum": s, "stats": stats}
        dx, dgamma, dbeta = st["plan"].backward(
            st["x"], st["dy"], st["gamma"], st["stats"], dsum=st["dsum"], dx=st["out"],
            dgamma=st["dgamma"], dbeta=st["dbeta"], ws=st["ws"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if "plan" not in st:
        from tensor_train_compressed_tt_gb300.layer import TTAttention, TTSeqs
        st["plan"] = TTAttention(c["heads"], c["dim"], kv_heads=c["kv"], dtype=DTYPES[c["dtype"]],
                                 left=c["left"], right=c["right"], sinks=c["sinks"])
        st["seqs"] = TTSeqs(st["q_begin"], st["q_end"], st["k_begin"], st["k_end"],
                            Tq=st["q"].shape[0], Tk=st["k"].shape[0],
                            max_q=st["max_q"], max_k=st["max_k"])
        st["ws"] = st["plan"].workspace(st["seqs"], backward=op == "attn_bwd")
        st["out"] = [torch.empty_like(st["q"]), torch.empty_like(st["k"]),
                     torch.empty_like(st["v"]),
                     torch.empty(c["heads"], st["q"].shape[0], device="cuda")]
    dq, dk, dv, lse = st["out"]
    if op == "attn_fwd":
        o, lse = st["plan"].forward(st["q"], st["k"], st["v"], st["seqs"], o=dq, lse=lse,
                                    ws=st["ws"])
        return {"o": o, "lse": lse}
    dq, dk, dv = st["plan"].backward(st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"],
                                     st["seqs"], dq=dq, dk=dk, dv=dv, ws=st["ws"])
    return {"dq": dq, "dk": dk, "dv": dv}


# --------------------------------------------------------------------------
# What a pass cannot do without

def work(case):
    c = case
    e = SIZE[c["dtype"]]
    if c["op"].startswith("norm"):
        x = c["T"] * c["N"]
        if c["op"] == "norm_fwd":
            return {"bytes": x * e * (4 if c["res"] else 2) + 8 * c["T"] + 8 * c["N"],
                    "flops": x * (9 if c["res"] else 8)}
        return {"bytes": x * e * (4 if c["res"] else 3) + 8 * c["T"] + 12 * c["N"],
                "flops": x * (15 if c["res"] else 14)}
    pairs, keys = _visible(c)
    rows = sum(min(c["q"] or n, n) for n in _lengths(c))
    q, k = rows * c["heads"] * c["dim"] * e, keys * c["kv"] * c["dim"] * e
    lse = 4 * rows * c["heads"]
    if c["op"] == "attn_fwd":
        return {"bytes": 2 * q + 2 * k + lse, "flops": 4 * pairs * c["heads"] * c["dim"]}
    return {"bytes": 4 * q + 4 * k + lse, "flops": 10 * pairs * c["heads"] * c["dim"]}


# --------------------------------------------------------------------------
# The definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, st)
    c = case
    scale = c["dim"] ** -0.5
    group = c["heads"] // c["kv"]
    grad = c["op"] == "attn_bwd"
    q, k, v = (st[n].double().requires_grad_(grad) for n in "qkv")
    o = torch.zeros_like(st["q"], dtype=torch.float64)
    lse = torch.full((c["heads"], q.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    grads = [torch.zeros_like(x, dtype=torch.float64) for x in (q, k, v)]
    ends = zip(*(st[n].tolist() for n in ("q_begin", "q_end", "k_begin", "k_end")))
    for q0, q1, k0, k1 in ends:
        for a in range(q0, q1, 512):
            b = min(q1, a + 512)
            pos = torch.arange(a - q0, b - q0, device="cuda") + (k1 - k0) - (q1 - q0)
            # the keys this block of queries may see: the first ones and a span around it
            first = 0 if c["left"] < 0 else max(0, int(pos[0]) - c["left"])
            last = k1 - k0 if c["right"] < 0 else min(k1 - k0, int(pos[-1]) + c["right"] + 1)
            j = torch.arange(k1 - k0, device="cuda")
            j = j[((j >= first) | (j < c["sinks"])) & (j < last)]
            far = pos[:, None] - j
            keep = torch.ones_like(far, dtype=torch.bool)
            if c["left"] >= 0:
                keep &= (far <= c["left"]) | (j < c["sinks"])
            if c["right"] >= 0:
                keep &= -far <= c["right"]
            bias = torch.zeros_like(far, dtype=torch.float64).masked_fill(~keep, -math.inf)
            kk = k[k0 + j].repeat_interleave(group, 1)
            vv = v[k0 + j].repeat_interleave(group, 1)
            score = torch.einsum("ihd,jhd->hij", q[a:b], kk) * scale + bias
            norm_ = torch.logsumexp(score, 2)
            w = torch.exp(score - norm_[:, :, None])
            out = torch.einsum("hij,jhd->ihd", w, vv)
            if grad:
                for acc, part in zip(grads, torch.autograd.grad(out, (q, k, v),
                                                                st["do"][a:b].double())):
                    acc += part
            else:
                o[a:b], lse[:, a:b] = out, norm_
    if grad:
        return {"dq": grads[0], "dk": grads[1], "dv": grads[2]}
    return {"o": o, "lse": lse}


def _exact_norm(c, st):
    x = st["x"].double().requires_grad_(True)
    gamma = st["gamma"].double().requires_grad_(True)
    beta = st["beta"].double().requires_grad_(True)
    s = x if st.get("res") is None else x + st["res"].double()
    mean = s.sum(1) / c["N"]
    var = (s * s).sum(1) / c["N"] - mean * mean
    inv = 1 / torch.sqrt(var + EPS)
    y = gamma * ((s - mean[:, None]) * inv[:, None]) + beta
    if c["op"] == "norm_fwd":
        return {"y": y.detach(), "sum": s.detach() if st["res"] is not None else None,
                "stats": torch.stack([mean, inv], 1).detach()}
    dx, dgamma, dbeta = torch.autograd.grad(y, (x, gamma, beta), st["dy"].double())
    if st["dsum"] is not None:
        dx = dx + st["dsum"].double()
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
