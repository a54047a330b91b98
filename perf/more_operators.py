"""The cases on which rotary positions, token log probabilities and dropout are
measured.

Three operators on the way from a block's projections to its loss: the norm of
queries and keys for each head with the rotation by position in the same pass
(forward, backward, and new tokens written into a cache); the log probabilities
of given tokens with entropy and top alternatives, their gradient, and both in
one pass; dropout from a counter-based generator, alone and in front of the
residual sum of layer normalisation.  Each case runs in two forms on the same
inputs: elementary torch operations in 32 bits (`own` false), or the calls a
user makes of the library (`own` true).

Sizes: 16384 tokens of width 768 with 12 heads of 64 and the 64-wide and
4096-wide rows are the ones of the library's benchmark; the others are generic.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-5
BASE = 10000.0


# --------------------------------------------------------------------------
# Cases

def rope(op, T, heads, kv, dim, rot, dtype, norm=True, inter=False, packed=False, far=0):
    """T tokens of heads + kv vectors of dim, the first rot of them rotated.
    packed: q, k and v are slices of one buffer.  far: the first position.
    op "rope_cache": the keys and values of T new tokens go to a cache."""
    return {"op": op, "T": T, "heads": heads, "kv": kv, "dim": dim, "rot": rot, "dtype": dtype,
            "norm": norm, "inter": inter, "packed": packed, "far": far}


def logp(op, T, V, dtype, top=0, entropy=False, scale=1.0, masked=0, ignored=0.0):
    """T rows of V logits.  masked: every masked-th logit is -infinity.
    ignored: the share of rows without a target."""
    return {"op": op, "T": T, "V": V, "dtype": dtype, "top": top, "entropy": entropy,
            "scale": scale, "masked": masked, "ignored": ignored}


def drop(op, T, N, dtype, p, res, site=0):
    return {"op": op, "T": T, "N": N, "dtype": dtype, "p": p, "res": res, "site": site}


def listed():
    return [
        # one new token for each of 16 sequences, into the cache: latency of serving
        dict(rope("rope_cache", 16, 12, 12, 64, 64, "bf16", far=1000),
             name="rope cache 16 h12 d64"),
        # between the projections and the attention of a 768-wide block in training
        dict(rope("rope_fwd", 16384, 12, 12, 64, 64, "bf16"), name="rope fwd 16384 h12 d64"),
        dict(rope("rope_bwd", 16384, 12, 12, 64, 64, "bf16"), name="rope bwd 16384 h12 d64"),
        # full precision, heads rotated in part, neighbours as pairs, far positions
        dict(rope("rope_bwd", 4099, 16, 4, 80, 32, "f32", inter=True, packed=True, far=1 << 20),
             name="rope bwd 4099 h16/4 d80 r32 f32"),
        # choosing the next token of 8 sequences: latency of serving
        dict(logp("logp_fwd", 8, 131072, "f32", top=20, entropy=True, scale=1.25, masked=11),
             name="logp top 20 of 8x131072 f32"),
        # scoring a text: rows that are not aligned
        dict(logp("logp_fwd", 4096, 50001, "bf16", top=4, entropy=True),
             name="logp top 4 of 4096x50001"),
        # the loss of a training step and its gradient in one pass
        dict(logp("logp_loss", 8192, 32000, "bf16", ignored=0.1), name="logp loss 8192x32000"),
        # the gradient of a policy's objective: log probabilities and entropy
        dict(logp("logp_bwd", 2048, 131072, "bf16", entropy=True), name="logp bwd 2048x131072"),
        # the residual branch of a 768-wide block in training
        dict(drop("dropnorm_fwd", 16384, 768, "bf16", 0.1, True, 1),
             name="dropout norm fwd 16384x768"),
        dict(drop("dropnorm_bwd", 16384, 768, "bf16", 0.1, True, 1),
             name="dropout norm bwd 16384x768"),
        # a wide layer's output at the largest token count of the benchmark
        dict(drop("drop", 32768, 4096, "bf16", 0.1, False), name="dropout 32768x4096"),
        # an odd width in full precision, with the residual sum
        dict(drop("drop", 4095, 1023, "f32", 0.25, True, 3), name="dropout 4095x1023 f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    kind = rng.choice(["rope_cache", "rope_fwd", "rope_bwd", "logp_fwd", "logp_fwd", "logp_bwd",
                       "logp_loss", "drop", "dropnorm_fwd", "dropnorm_bwd"])
    if kind.startswith("rope"):
        kv = rng.choice([1, 2, 4, 8, 12])
        heads = kv * rng.choice([1, 1, 2, 4])
        dim = rng.choice([24, 32, 40, 64, 64, 80, 96, 128, 128, 160, 256])
        rot = rng.choice([dim, dim, dim // 2, dim // 4, 0])
        rot -= rot % 2
        most = 100000000 // ((heads + kv) * dim)
        T = _log_int(rng, 1, 300 if kind == "rope_cache" else min(40000, most))
        return rope(kind, T, heads, kv, dim, rot, dtype, rng.random() < 0.75 or rot == 0,
                    rng.random() < 0.4, rng.random() < 0.4,
                    rng.choice([0, 0, _log_int(rng, 1, 100000000)]))
    if kind.startswith("logp"):
        V = _log_int(rng, 200, 140000)
        V -= V % rng.choice([1, 1, 2, 8, 64])
        T = _log_int(rng, 1, min(20000, 200000000 // V))
        return logp(kind, T, V, dtype, rng.choice([0, 0, 1, 5, 20]) if kind == "logp_fwd" else 0,
                    rng.random() < 0.5, rng.choice([1.0, 1.0, 0.7, 1.6]),
                    rng.choice([0, 0, 3, 17]), rng.choice([0.0, 0.0, 0.3]))
    N = _log_int(rng, 48, 4200)
    N -= N % rng.choice([1, 2, 8, 64]) if N >= 128 else 0
    T = _log_int(rng, 1, min(40000, 134000000 // N))
    return drop(kind, T, N, dtype, rng.choice([0.0, 0.1, 0.1, 0.25, 0.5]), rng.random() < 0.6,
                rng.choice([0, 1, 7, 65535]))


# --------------------------------------------------------------------------
# Inputs

def prepare(case, seed):
    c = dict(case)
    dt = DTYPES[c["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    st = {"case": c}
    if c["op"].startswith("rope"):
        _prepare_rope(st, c, g, randn)
    elif c["op"].startswith("logp"):
        _prepare_logp(st, c, g, randn)
    else:
        T, N = c["T"], c["N"]
        # the state of the generator: a seed, and the step's offset
        st["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device="cuda")
        st["x"] = randn(T, N)
        if c["res"]:
            st["res"] = randn(T, N)
        if c["op"] != "drop":
            st["gamma"] = 1.0 + 0.2 * torch.randn(N, generator=g, device="cuda")
            st["beta"] = 0.1 * torch.randn(N, generator=g, device="cuda")
        if c["op"] == "dropnorm_bwd":
            st["dy"] = randn(T, N, scale=0.1)
            st["dsum"] = randn(T, N, scale=0.1) if c["res"] else None
            st["stats"] = _row_stats(st["x"].float())
    return st


def _prepare_rope(st, c, g, randn):
    T, H, KV, D = c["T"], c["heads"], c["kv"], c["dim"]
    # activations with a spread of their own for each channel, as projections have
    spread = 0.5 + torch.rand(D, generator=g, device="cuda")

    def three(scale=1.0):
        if c["packed"]:
            x = randn(T, H + 2 * KV, D, scale=scale)
            return list(x.mul_(spread.to(x.dtype)).split([H, KV, KV], 1))
        return [randn(T, n, D, scale=scale).mul_(spread.to(DTYPES[c["dtype"]]))
                for n in (H, KV, KV)]

    st["q"], st["k"], st["v"] = three()
    st["gq"], st["gk"] = (1.0 + 0.2 * torch.randn(2, D, generator=g, device="cuda")
                          if c["norm"] else (None, None))
    if c["op"] == "rope_cache":
        # every token is the newest of a sequence, whose rows lie anywhere in the cache
        st["pos"] = (c["far"] + torch.randint(0, 4000, (T,), generator=g, device="cuda")).int()
        st["rows"] = torch.randperm(4 * T, generator=g, device="cuda")[:T].int()
        st["keys"], st["values"] = randn(4 * T, KV, D), randn(4 * T, KV, D)
        return
    # packed sequences of some length, each from its own first position
    n = max(1, min(T, 512))
    st["pos"] = (c["far"] + torch.arange(T, device="cuda") % n).int()
    if c["op"] == "rope_bwd":
        st["dq"], st["dk"], _ = three(0.1)


def _prepare_logp(st, c, g, randn):
    T, V = c["T"], c["V"]
    # logits around each token's own level, some rows sharper than others
    x = torch.randn(T, V, generator=g, device="cuda")
    x.mul_(1.0 + 2.0 * torch.rand(T, 1, generator=g, device="cuda"))
    x.add_(2.0 * torch.randn(V, generator=g, device="cuda"))
    if c["masked"]:
        x[:, c["masked"] - 1::c["masked"]] = -math.inf
    st["logits"] = x.to(DTYPES[c["dtype"]])
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    if c["masked"]:
        t = torch.where((t + 1) % c["masked"] == 0, t - 1, t)
    gone = torch.rand(T, generator=g, device="cuda") < c["ignored"]
    st["targets"] = torch.where(gone, -1, t).int()
    if c["op"] != "logp_fwd":
        # the gradients of the log probabilities (a mean loss) and of the entropies
        st["dlogp"] = -(0.5 + torch.rand(T, generator=g, device="cuda")) / T
        st["dent"] = -0.01 * torch.rand(T, generator=g, device="cuda") / T \
            if c["entropy"] else None
    if c["op"] == "logp_bwd":
        st["lse"], st["ent"] = _row_lse_entropy(st["logits"].float() * c["scale"])


# --------------------------------------------------------------------------
# Plain forms

def _pair_index(c):
    """The two channels of each rotated pair."""
    i = torch.arange(c["rot"] // 2, device="cuda")
    return (2 * i, 2 * i + 1) if c["inter"] else (i, i + c["rot"] // 2)


def _angles(st, c):
    """cos and sin of every token's angles, (T, 1, rot / 2): far positions need 64 bits."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
    a = st["pos"].double()[:, None, None] * BASE ** (-2.0 * i / max(1, c["rot"]))
    return a.cos().float(), a.sin().float()


def _turn(u, c, cos, sin):
    a, b = _pair_index(c)
    y = u.clone()
    y[..., a] = u[..., a] * cos - u[..., b] * sin
    y[..., b] = u[..., a] * sin + u[..., b] * cos
    return y


def _plain_rope(st):
    c = st["case"]
    cos, sin = _angles(st, c)
    out = []
    for x, w in ((st["q"], st["gq"]), (st["k"], st["gk"])):
        u = x.float()
        if c["norm"]:
            u = u * (u.square().mean(2, keepdim=True) + EPS).rsqrt() * w
        out.append(_turn(u, c, cos, sin).to(x.dtype))
    if c["op"] == "rope_fwd":
        return {"q": out[0], "k": out[1]}
    rows = st["rows"].long()
    st["keys"][rows] = out[1]
    st["values"][rows] = st["v"]
    return {"q": out[0], "keys": st["keys"], "values": st["values"]}


def _plain_rope_bwd(st):
    c = st["case"]
    cos, sin = _angles(st, c)
    out = {}
    for n, x, dy, w in (("q", st["q"], st["dq"], st["gq"]), ("k", st["k"], st["dk"], st["gk"])):
        du = _turn(dy.float(), c, cos, -sin)
        if c["norm"]:
            u = x.float()
            r = (u.square().mean(2, keepdim=True) + EPS).rsqrt()
            h = u * r
            out["dg" + n] = (du * h).sum((0, 1))
            gx = du * w
            du = r * (gx - h * (gx * h).mean(2, keepdim=True))
        out["d" + n] = du.to(x.dtype)
    return out


def _row_lse_entropy(z):
    m = z.amax(1, keepdim=True)
    e = (z - m).exp()
    s = e.sum(1, keepdim=True)
    ent = s.log() - (e * torch.where(e > 0, z - m, 0.0)).sum(1, keepdim=True) / s
    return (m + s.log())[:, 0], ent[:, 0]


def _plain_logp(st):
    c = st["case"]
    z = st["logits"].float() * c["scale"]
    lse, ent = _row_lse_entropy(z)
    t = st["targets"].long()
    picked = z.gather(1, t.clamp(min=0)[:, None])[:, 0] - lse
    out = {"logp": torch.where(t < 0, 0.0, picked), "lse": lse}
    if c["entropy"]:
        out["entropy"] = ent
    if c["top"]:
        # ties go to the lowest index: a stable sort of the logits themselves
        ids = st["logits"].sort(dim=1, descending=True, stable=True).indices[:, :c["top"]]
        out["top"], out["top_logp"] = ids.int(), z.gather(1, ids) - lse[:, None]
    return out


def _plain_logp_grad(st, z, lse, ent):
    c = st["case"]
    t = st["targets"].long()
    g = torch.where(t < 0, 0.0, st["dlogp"])[:, None]
    lp = z - lse[:, None]
    p = lp.exp()
    d = p * -g
    if st["dent"] is not None:
        d = d - p * torch.where(p > 0, lp + ent[:, None], 0.0) * st["dent"][:, None]
    d.scatter_add_(1, t.clamp(min=0)[:, None], g)
    return (d * c["scale"]).to(st["logits"].dtype)


def _plain_loss(st):
    c = st["case"]
    z = st["logits"].float() * c["scale"]
    lse, ent = _row_lse_entropy(z)
    t = st["targets"].long()
    picked = z.gather(1, t.clamp(min=0)[:, None])[:, 0] - lse
    out = {"logp": torch.where(t < 0, 0.0, picked), "lse": lse,
           "dlogits": _plain_logp_grad(st, z, lse, ent)}
    if c["entropy"]:
        out["entropy"] = ent
    return out


LOW = 0xFFFFFFFF


def _words(rng, groups, site):
    """Philox 4x32 with ten rounds (Salmon et al., 2011): four 32-bit words for each
    group of eight elements, (groups, 4).  Key: the seed.  Counter: the group, the
    site, the offset."""
    i = torch.arange(groups, dtype=torch.int64, device="cuda")
    seed, offset = rng[0], rng[1]
    k0, k1 = seed & LOW, (seed >> 32) & LOW
    x = [i & LOW, (i >> 32) + (site << 16), (offset & LOW).expand_as(i),
         ((offset >> 32) & LOW).expand_as(i)]
    for _ in range(10):
        a, b = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57  # modulo 2^64
        x = [((b >> 32) & LOW) ^ x[1] ^ k0, b & LOW, ((a >> 32) & LOW) ^ x[3] ^ k1, a & LOW]
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    return torch.stack(x, 1)


def _cut(p):
    """An element stays when its 16 random bits are not below this."""
    return int(math.floor(p * 65536 + 0.5))


def _dropped(x, st):
    c = st["case"]
    n, cut = x.numel(), _cut(c["p"])
    w = _words(st["rng"], (n + 7) // 8, c["site"])
    bits = torch.stack([w & 0xFFFF, w >> 16], 2).reshape(-1)[:n].reshape(x.shape)
    return torch.where(bits >= cut, x * (65536.0 / (65536 - cut)), 0.0)


def _row_stats(s):
    mean = s.mean(1, keepdim=True)
    var = (s - mean).square().mean(1, keepdim=True)
    return torch.cat([mean, (var + EPS).rsqrt()], 1)


def _plain_dropnorm_fwd(st):
    s = _dropped(st["x"].float(), st)
    if "res" in st:
        s = s + st["res"].float()
    stats = _row_stats(s)
    y = (s - stats[:, :1]) * stats[:, 1:] * st["gamma"] + st["beta"]
    dt = st["x"].dtype
    return {"y": y.to(dt), "sum": s.to(dt), "stats": stats}


def _plain_dropnorm_bwd(st):
    """x is what was normalised: the forward's sum."""
    dt, dy = st["x"].dtype, st["dy"].float()
    mean, rstd = st["stats"][:, :1], st["stats"][:, 1:]
    h = (st["x"].float() - mean) * rstd
    g = dy * st["gamma"]
    ds = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    if st["dsum"] is not None:
        ds = ds + st["dsum"].float()
    out = {"dx": _dropped(ds, st).to(dt), "dgamma": (dy * h).sum(0), "dbeta": dy.sum(0)}
    if st["case"]["res"]:
        out["dres"] = ds.to(dt)
    return out


# --------------------------------------------------------------------------
# One pass

def run(st):
    op = st["case"]["op"]
    if own:
        return _own(st, op)
    if op in ("rope_fwd", "rope_cache"):
        return _plain_rope(st)
    if op == "rope_bwd":
        return _plain_rope_bwd(st)
    if op == "logp_fwd":
        return _plain_logp(st)
    if op == "logp_bwd":
        z = st["logits"].float() * st["case"]["scale"]
        return {"dlogits": _plain_logp_grad(st, z, st["lse"], st["ent"])}
    if op == "logp_loss":
        return _plain_loss(st)
    if op == "dropnorm_fwd":
        return _plain_dropnorm_fwd(st)
    if op == "dropnorm_bwd":
        return _plain_dropnorm_bwd(st)
    y = _dropped(st["x"].float(), st)
    return {"y": (y + st["res"].float() if "res" in st else y).to(st["x"].dtype)}


def _own(st, op):
    """The library's calls; the plan, output buffers and workspace are kept
    with the state, as a program that runs many steps keeps them."""
    c = st["case"]
    if op.startswith("rope"):
        return _own_rope(st, c, op)
    if op.startswith("logp"):
        return _own_logp(st, c, op)
    if op == "drop":
        if "plan" not in st:
            from tensor_train_compressed_tt_gb300.layer import TTDropout
            st["plan"] = TTDropout(c["p"], DTYPES[c["dtype"]], site=c["site"])
            st["out"] = torch.empty_like(st["x"])
        return {"y": st["plan"].forward(st["x"], st["rng"], res=st.get("res"), y=st["out"])}
    if "plan" not in st:
        from tensor_train_compressed_tt_gb300.layer import TTDropNorm
        st["plan"] = TTDropNorm(c["N"], c["p"], DTYPES[c["dtype"]], eps=EPS, site=c["site"])
        st["ws"] = st["plan"].workspace(c["T"])
        st["out"], st["out2"] = torch.empty_like(st["x"]), torch.empty_like(st["x"])
        st["new_stats"] = torch.empty(c["T"], 2, device="cuda")
        st["dgamma"], st["dbeta"] = torch.empty_like(st["gamma"]), torch.empty_like(st["beta"])
    if op == "dropnorm_fwd":
        y, s, stats = st["plan"].forward(st["x"], st["rng"], st["gamma"], st["beta"],
                                         res=st.get("res"), y=st["out"], sum=st["out2"],
                                         stats=st["new_stats"])
        return {"y": y, "sum": s, "stats": stats}
    dx, dres, dgamma, dbeta = st["plan"].backward(
        st["x"], st["dy"], st["rng"], st["gamma"], st["stats"], dsum=st["dsum"], dx=st["out"],
        dres=st["out2"] if c["res"] else None, residual=c["res"], dgamma=st["dgamma"],
        dbeta=st["dbeta"], ws=st["ws"])
    out = {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if c["res"]:
        out["dres"] = dres
    return out


def _own_rope(st, c, op):
    if "plan" not in st:
        from tensor_train_compressed_tt_gb300.layer import TTRotary
        st["plan"] = TTRotary(c["heads"], c["dim"], kv_heads=c["kv"], dtype=DTYPES[c["dtype"]],
                              rot=c["rot"], base=BASE, interleaved=c["inter"], norm=c["norm"],
                              eps=EPS)
        shape = (c["T"], c["heads"], c["dim"]), (c["T"], c["kv"], c["dim"])
        st["out"] = [torch.empty(s, dtype=DTYPES[c["dtype"]], device="cuda") for s in shape]
        if op == "rope_bwd":
            st["ws"] = st["plan"].workspace(c["T"])
            st["dg"] = [torch.empty(c["dim"], device="cuda") if c["norm"] else None
                        for _ in range(2)]
    q, k = st["out"]
    if op == "rope_bwd":
        dq, dk, dgq, dgk = st["plan"].backward(
            st["dq"], st["dk"], st["pos"], st["q"] if c["norm"] else None,
            st["k"] if c["norm"] else None, st["gq"], st["gk"], dq_in=q, dk_in=k,
            dgq=st["dg"][0], dgk=st["dg"][1], ws=st["ws"])
        out = {"dq": dq, "dk": dk}
        if c["norm"]:
            out["dgq"], out["dgk"] = dgq, dgk
        return out
    if op == "rope_fwd":
        q, k = st["plan"].forward(st["q"], st["k"], st["pos"], st["gq"], st["gk"], q_out=q,
                                  k_out=k)
        return {"q": q, "k": k}
    q, keys, values = st["plan"].to_cache(st["q"], st["k"], st["v"], st["pos"], st["rows"],
                                          st["keys"], st["values"], st["gq"], st["gk"], q_out=q)
    return {"q": q, "keys": keys, "values": values}


def _own_logp(st, c, op):
    if "plan" not in st:
        from tensor_train_compressed_tt_gb300.layer import TTLogProbs
        st["plan"] = TTLogProbs(c["V"], DTYPES[c["dtype"]], scale=c["scale"], top=c["top"])
        T = c["T"]
        st["out"] = [torch.empty(T, device="cuda") for _ in range(3)]
        if op != "logp_fwd":
            st["grad"] = torch.empty_like(st["logits"])
        if c["top"]:
            st["ids"] = torch.empty(T, c["top"], dtype=torch.int32, device="cuda")
            st["tops"] = torch.empty(T, c["top"], device="cuda")
    logp_, lse, ent = st["out"]
    if not c["entropy"]:
        ent = None
    if op == "logp_bwd":
        return {"dlogits": st["plan"].backward(st["logits"], st["targets"], st["lse"],
                                               st["dlogp"], st["ent"], st["dent"],
                                               dlogits=st["grad"])}
    if op == "logp_loss":
        d = st["plan"].loss(st["logits"], st["targets"], st["dlogp"], st["dent"], logp=logp_,
                            lse=lse, entropy=ent, dlogits=st["grad"])
        out = {"logp": logp_, "lse": lse, "dlogits": d[3]}
    else:
        st["plan"].forward(st["logits"], st["targets"], logp=logp_, lse=lse, entropy=ent,
                           top=st.get("ids"), top_logp=st.get("tops"))
        out = {"logp": logp_, "lse": lse}
        if c["top"]:
            out["top"], out["top_logp"] = st["ids"], st["tops"]
    if c["entropy"]:
        out["entropy"] = ent
    return out


# --------------------------------------------------------------------------
# What a pass cannot do without

def work(case):
    c = case
    e = SIZE[c["dtype"]]
    if c["op"].startswith("rope"):
        T, x = c["T"], c["T"] * (c["heads"] + c["kv"]) * c["dim"]
        turned = 3 * c["T"] * (c["heads"] + c["kv"]) * c["rot"]
        if c["op"] == "rope_bwd":
            return {"bytes": x * e * (3 if c["norm"] else 2) + 4 * T + 16 * c["dim"] * c["norm"],
                    "flops": turned + x * 10 * c["norm"]}
        v = T * c["kv"] * c["dim"] if c["op"] == "rope_cache" else 0
        return {"bytes": 2 * (x + v) * e + 4 * T + (4 * T if v else 0) + 8 * c["dim"] * c["norm"],
                "flops": turned + x * 4 * c["norm"]}
    if c["op"].startswith("logp"):
        x = c["T"] * c["V"]
        if c["op"] == "logp_fwd":
            return {"bytes": x * e + c["T"] * (12 + 4 * c["entropy"] + 8 * c["top"]),
                    "flops": x * (5 + 2 * c["entropy"])}
        if c["op"] == "logp_bwd":
            return {"bytes": 2 * x * e + c["T"] * (12 + 8 * c["entropy"]),
                    "flops": x * (4 + 2 * c["entropy"])}
        return {"bytes": 2 * x * e + c["T"] * (16 + 8 * c["entropy"]),
                "flops": x * (7 + 4 * c["entropy"])}
    x = c["T"] * c["N"]
    if c["op"] == "drop":
        return {"bytes": x * e * (3 if c["res"] else 2) + 16, "flops": x * (2 if c["res"] else 1)}
    if c["op"] == "dropnorm_fwd":
        return {"bytes": x * e * (4 if c["res"] else 3) + 8 * c["T"] + 8 * c["N"], "flops": x * 10}
    return {"bytes": x * e * (5 if c["res"] else 3) + 8 * c["T"] + 12 * c["N"], "flops": x * 16}


# --------------------------------------------------------------------------
# The definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("rope"):
        return _exact_rope(case, st)
    if case["op"].startswith("logp"):
        return _exact_logp(case, st)
    return _exact_drop(case, st)


def _exact_heads(x, w, pos, c):
    """One tensor of heads: normalised, then multiplied by e^(i angle) as complex numbers."""
    if c["norm"]:
        x = x / torch.sqrt((x * x).sum(2, keepdim=True) / c["dim"] + EPS) * w
    half = c["rot"] // 2
    if not half:
        return x
    f = torch.tensor([math.pow(BASE, -2.0 * i / c["rot"]) for i in range(half)],
                     dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones_like(f).expand(len(pos), half), pos.double()[:, None] * f)
    head, tail = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["inter"]:
        pairs = head.reshape(*head.shape[:2], half, 2)
    else:
        pairs = torch.stack([head[..., :half], head[..., half:]], 3)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
    head = z.reshape(head.shape) if c["inter"] else torch.cat([z[..., 0], z[..., 1]], 2)
    return torch.cat([head, tail], 2)


def _exact_rope(c, st):
    grad = c["op"] == "rope_bwd"
    out = {}
    for n in "qk":
        x = st[n].double().requires_grad_(grad)
        w = None if st["g" + n] is None else st["g" + n].double().requires_grad_(grad)
        y = _exact_heads(x, w, st["pos"], c)
        if grad:
            got = torch.autograd.grad(y, [x] + ([w] if c["norm"] else []), st["d" + n].double())
            out["d" + n] = got[0]
            if c["norm"]:
                out["dg" + n] = got[1]
        else:
            out[n] = y
    if c["op"] != "rope_cache":
        return out
    keys, values = st["keys"].double(), st["values"].double()
    keys.index_copy_(0, st["rows"].long(), out["k"])
    values.index_copy_(0, st["rows"].long(), st["v"].double())
    return {"q": out["q"], "keys": keys, "values": values}


def _exact_logp(c, st):
    """Some rows at a time; the gradient from the derivatives of log p and of the entropy."""
    parts = []
    step = max(1, 60000000 // c["V"])
    for a in range(0, c["T"], step):
        b = min(c["T"], a + step)
        x, t = st["logits"][a:b], st["targets"][a:b].long()
        z = x.double() * c["scale"]
        lse = torch.logsumexp(z, 1)
        lp = z - lse[:, None]
        there = t >= 0
        one = torch.zeros_like(z)
        rows = torch.nonzero(there)[:, 0]
        one[rows, t[rows]] = 1.0
        out = {"logp": torch.where(there, lp[torch.arange(b - a, device="cuda"), t.clamp(min=0)],
                                   torch.zeros_like(lse)), "lse": lse}
        p = lp.exp()
        plp = torch.where(p > 0, p * lp, torch.zeros_like(p))
        if c["entropy"]:
            out["entropy"] = -plp.sum(1)
        if c["op"] != "logp_fwd":
            g = torch.where(there, st["dlogp"][a:b].double(), torch.zeros_like(lse))[:, None]
            d = g * (one - p)
            if st["dent"] is not None:
                # dH / dz_v = -(p log p)_v + p_v sum (p log p)
                d = d + st["dent"][a:b].double()[:, None] * (p * plp.sum(1, keepdim=True) - plp)
            out["dlogits"] = c["scale"] * d
        if c["top"]:
            # the largest again and again: each time the first of its value
            left, ids = x.float(), []
            for _ in range(c["top"]):
                best = left.amax(1, keepdim=True)
                at = (left == best).int().argmax(1, keepdim=True)
                ids.append(at)
                left = left.scatter(1, at, -math.inf)
            ids = torch.cat(ids, 1)
            out["top"], out["top_logp"] = ids.int(), lp.gather(1, ids)
        parts.append(out)
    whole = {k: torch.cat([q[k] for q in parts]) for k in parts[0]}
    if c["op"] == "logp_bwd":
        return {"dlogits": whole["dlogits"]}
    return whole


def _mul32(a, b):
    """High and low words of a 32 x 32 product from its 16-bit halves."""
    ah, al, bh, bl = a >> 16, a % 65536, b >> 16, b % 65536
    mid = ah * bl + (al * bl >> 16)
    more = al * bh + mid % 65536
    return ah * bh + (mid >> 16) + (more >> 16), (more % 65536) * 65536 + al * bl % 65536


def _exact_keep(c, rng, shape):
    n = shape[0] * shape[1]
    group = torch.arange((n + 7) // 8, device="cuda")
    seed, offset = rng.tolist()
    v = [group % 2 ** 32, group // 2 ** 32 + c["site"] * 65536,
         torch.full_like(group, offset % 2 ** 32), torch.full_like(group, offset // 2 ** 32)]
    key = [seed % 2 ** 32, seed // 2 ** 32]
    for _ in range(10):
        h0, l0 = _mul32(v[0], 0xD2511F53)
        h1, l1 = _mul32(v[2], 0xCD9E8D57)
        v = [h1 ^ v[1] ^ key[0], l1, h0 ^ v[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    keep = torch.empty(group.numel(), 8, dtype=torch.bool, device="cuda")
    for i, w in enumerate(v):
        keep[:, 2 * i] = w % 65536 >= _cut(c["p"])
        keep[:, 2 * i + 1] = w // 65536 >= _cut(c["p"])
    return keep.flatten()[:n].reshape(shape)


def _exact_drop(c, st):
    keep = _exact_keep(c, st["rng"], st["x"].shape).double() / (1 - _cut(c["p"]) / 65536)
    x = st["x"].double()
    if c["op"] == "dropnorm_bwd":
        x.requires_grad_(True)
        gamma = st["gamma"].double().requires_grad_(True)
        beta = torch.zeros_like(gamma).requires_grad_(True)
        y = _exact_norm(x, gamma, beta)[0]
        ds, dgamma, dbeta = torch.autograd.grad(y, (x, gamma, beta), st["dy"].double())
        if st["dsum"] is not None:
            ds = ds + st["dsum"].double()
        out = {"dx": ds * keep, "dgamma": dgamma, "dbeta": dbeta}
        if c["res"]:
            out["dres"] = ds
        return out
    s = x * keep
    if "res" in st:
        s = s + st["res"].double()
    if c["op"] == "drop":
        return {"y": s}
    y, stats = _exact_norm(s, st["gamma"].double(), st["beta"].double())
    return {"y": y, "sum": s, "stats": stats}


def _exact_norm(s, gamma, beta):
    n = s.shape[1]
    mean = s.sum(1) / n
    var = (s * s).sum(1) / n - mean * mean
    inv = 1 / torch.sqrt(var + EPS)
    return gamma * ((s - mean[:, None]) * inv[:, None]) + beta, torch.stack([mean, inv], 1)
