"""Cross attention to an encoder's states and layer norm: the calls a conditional diffusion transformer
makes of them, as measured cases.

The sizes come from pixel-token images (32 x 32 to 256 x 256 pixels, 6 or 16 heads) with encoder states of
1 to some ten thousand tokens.  ``own`` selects the library's calls; otherwise ``run`` computes the
definitions with elementary torch operations in fp32.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one 16 x 16 latent against a short prompt: latency of the smallest call of a sampling step
        dict(name="cross-small", op="cross", train=False, dtype="bf16", batch=1, heads=6, kv_heads=6, nq=256, nk=77,
             d=64, layout="bhnd", lengths="full"),
        # sampling at 128 x 128 pixels with long prompts, all of the longest length
        dict(name="cross-sample-px128", op="cross", train=False, dtype="bf16", batch=8, heads=6, kv_heads=6, nq=16384,
             nk=512, d=64, layout="bnhd", lengths="full"),
        # a training step at 256 x 256 pixels with prompts padded to 120 tokens
        dict(name="cross-train-px256", op="cross", train=True, dtype="bf16", batch=2, heads=6, kv_heads=6, nq=65536,
             nk=120, d=64, layout="bhnd", lengths="ragged"),
        # a training step with the odd head dimension of a 1152-wide model, padded prompts, one of them dropped
        dict(name="cross-train-d72", op="cross", train=True, dtype="bf16", batch=4, heads=16, kv_heads=16, nq=4096,
             nk=300, d=72, layout="bnhd", lengths="ragged"),
        # a training step with shared key heads, d = 128, two concatenated encoders that leave holes in the keys
        dict(name="cross-train-shared", op="cross", train=True, dtype="bf16", batch=2, heads=16, kv_heads=4, nq=4096,
             nk=589, d=128, layout="bnhd", lengths="holes"),
        # one token per image against long encoder states (attention pooling, one step of a decoder)
        dict(name="cross-token", op="cross", train=False, dtype="bf16", batch=8, heads=16, kv_heads=4, nq=1, nk=16384,
             d=128, layout="bhnd", lengths="ragged"),
        # a training step of the 32 x 32 pixel fp32 configuration
        dict(name="cross-train-fp32", op="cross", train=True, dtype="fp32", batch=2, heads=6, kv_heads=6, nq=1024,
             nk=77, d=64, layout="bhnd", lengths="ragged"),
        # one small activation: latency
        dict(name="norm-small", op="norm", train=False, dtype="bf16", params="fp32", batch=1, heads=1, n=256, c=384,
             layout="bhnd", per_batch=False),
        # queries of a 256 x 256 image normalised per head in the projection's token-major output, training
        dict(name="norm-heads-px256", op="norm", train=True, dtype="bf16", params="fp32", batch=2, heads=6, n=65536,
             c=64, layout="bnhd", per_batch=False),
        # a block's input at 128 x 128 pixels, modulated per image, training
        dict(name="norm-modulated-px128", op="norm", train=True, dtype="bf16", params="bf16", batch=8, heads=1, n=16384,
             c=384, layout="bhnd", per_batch=True),
        # an odd width in fp32, training
        dict(name="norm-odd-fp32", op="norm", train=True, dtype="fp32", params="fp32", batch=1, heads=1, n=5000, c=1001,
             layout="bhnd", per_batch=False),
        # wide encoder states, sampling
        dict(name="norm-wide", op="norm", train=False, dtype="bf16", params="bf16", batch=4, heads=1, n=4096, c=8192,
             layout="bhnd", per_batch=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.6:
        dtype = "bf16" if rng.random() < 0.75 else "fp32"
        kv_heads = rng.choice([1, 2, 4, 6, 16])
        group = rng.choice([1, 1, 2, 4]) if kv_heads < 16 else 1
        case = dict(op="cross", train=rng.random() < 0.6, dtype=dtype, batch=_spread(rng, 1, 8), heads=kv_heads * group,
                    kv_heads=kv_heads, nq=1 if rng.random() < 0.15 else _spread(rng, 2, 65536), nk=_spread(rng, 1, 16384),
                    d=8 * rng.randint(2, 16) if rng.random() < 0.5 else rng.choice([64, 128]),
                    layout=rng.choice(["bhnd", "bnhd"]), lengths=rng.choice(["full", "ragged", "holes"]))
        least = 2 if case["train"] else 1       # with one key the gradients of q and k are zero
        case["nk"] = max(least, case["nk"])
        most = (2.5e10 if dtype == "bf16" else 1.5e9) / (3.5 if case["train"] else 1)   # pairs x channels
        wide = 5e7 if dtype == "bf16" else 2.5e7                                        # values of one tensor
        while (case["batch"] * case["heads"] * case["nq"] * case["nk"] * case["d"] > most
               or case["batch"] * case["heads"] * max(case["nq"], case["nk"]) * case["d"] > wide):
            big = "nq" if case["nq"] > case["nk"] else "nk"
            case[big] = max(least, int(case[big] * rng.uniform(0.4, 0.9)))
        return case
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    case = dict(op="norm", train=rng.random() < 0.6, dtype=dtype, params=rng.choice([dtype, "fp32"]),
                batch=_spread(rng, 1, 8), heads=rng.choice([1, 1, 6, 16]), n=_spread(rng, 1, 65536),
                c=_spread(rng, 8, 8192), layout=rng.choice(["bhnd", "bnhd"]), per_batch=rng.random() < 0.4)
    while case["batch"] * case["heads"] * case["n"] * case["c"] > (5e7 if dtype == "bf16" else 2.5e7):
        big = "n" if case["n"] > case["c"] else "c"
        case[big] = max(1, int(case[big] * rng.uniform(0.4, 0.9)))
    return case


def _key_counts(case):
    """Valid keys of each batch row (before the seed permutes the rows): for "ragged", from full down to one dropped
    prompt; for "holes", of the two concatenated encoders, each padded to its own length."""
    b, nk = case["batch"], case["nk"]
    if case["lengths"] == "full":
        return [(nk, 0)] * b
    if case["lengths"] == "ragged":
        return [(nk - (nk * i) // b if i < 3 or i < b - 1 else 0, 0) for i in range(b)]
    first = nk // 4
    return [(first - (first * i) // (2 * b), (nk - first) - ((nk - first) * i) // (b + 1)) for i in range(b)]


def _tokens(gen, case, heads, n, d, dtype):
    """A [batch, heads, n, d] tensor in the case's layout; bnhd: a projection's output, heads inside the token."""
    b = case["batch"]
    shape = (b, heads, n, d) if case["layout"] == "bhnd" else (b, n, heads, d)
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return x if case["layout"] == "bhnd" else x.transpose(1, 2)




def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * seed + 17)
    dt = TYPES[case["dtype"]]
    if case["op"] == "norm":
        b, h, n, c = case["batch"], case["heads"], case["n"], case["c"]
        x = _tokens(gen, case, h, n, c, dt)
        # channels of unlike size and offset, as activations have
        x = x * (0.5 + torch.rand(c, generator=gen, device="cuda")) + torch.randn(c, generator=gen, device="cuda")
        wshape = (b, c) if case["per_batch"] else (c,)
        pt = TYPES[case["params"]]
        s = dict(case=dict(case), x=x.to(dt),
                 weight=(1 + 0.2 * torch.randn(wshape, generator=gen, device="cuda")).to(pt),
                 bias=(0.2 * torch.randn(wshape, generator=gen, device="cuda")).to(pt), eps=1e-6)
        if case["train"]:
            s["dy"] = _tokens(gen, case, h, n, c, dt).to(dt)
        return s
    b, h, hk, nq, nk, d = (case[k] for k in ("batch", "heads", "kv_heads", "nq", "nk", "d"))
    q = 1.5 * _tokens(gen, case, h, nq, d, dt)
    k = _tokens(gen, case, hk, nk, d, dt) + 0.25 * torch.randn(d, generator=gen, device="cuda")
    v = _tokens(gen, case, hk, nk, d, dt)
    s = dict(case=dict(case), q=q.to(dt), k=k.to(dt), v=v.to(dt), kv_len=None, key_mask=None)
    counts = _key_counts(case)
    order = torch.randperm(b, generator=torch.Generator().manual_seed(seed)).tolist()
    counts = [counts[i] for i in order]
    if case["lengths"] == "ragged":
        s["kv_len"] = torch.tensor([a for a, _ in counts], dtype=torch.int32, device="cuda")
    elif case["lengths"] == "holes":
        at = torch.arange(nk, device="cuda")
        first = nk // 4
        s["key_mask"] = torch.stack([(at < a) | ((at >= first) & (at < first + c)) for a, c in counts]).to(torch.uint8)
    if case["train"]:
        s["dO"] = _tokens(gen, case, h, nq, d, dt).to(dt)
    return s


def _valid(s):
    """[batch, 1, 1, nk]: the keys that take part."""
    c = s["case"]
    if s["kv_len"] is not None:
        return (torch.arange(c["nk"], device="cuda") < s["kv_len"][:, None])[:, None, None, :]
    if s["key_mask"] is not None:
        return (s["key_mask"] != 0)[:, None, None, :]
    return torch.ones(c["batch"], 1, 1, c["nk"], dtype=torch.bool, device="cuda")


def _plain_cross(s):
    c = s["case"]
    b, h, hk, nq, nk, d = (c[k] for k in ("batch", "heads", "kv_heads", "nq", "nk", "d"))
    dt = TYPES[c["dtype"]]
    scale = 1.0 / math.sqrt(d)
    # the query heads that share a key head stand below one another
    q = s["q"].float().reshape(b, hk, (h // hk) * nq, d)
    k, v = s["k"].float(), s["v"].float()
    z = (q @ k.transpose(-1, -2)) * scale
    z = z.masked_fill(~_valid(s), -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(z - m)
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    o = p @ v
    out = {"o": o.reshape(b, h, nq, d).to(dt), "lse": (m + torch.log(total)).reshape(b, h, nq)}
    if c["train"]:
        g = s["dO"].float().reshape(b, hk, (h // hk) * nq, d)
        dp = g @ v.transpose(-1, -2)
        ds = p * (dp - (g * o).sum(-1, keepdim=True)) * scale
        out["dq"] = (ds @ k).reshape(b, h, nq, d).to(dt)
        out["dk"] = (ds.transpose(-1, -2) @ q).to(dt)
        out["dv"] = (p.transpose(-1, -2) @ g).to(dt)
    return out


def _plain_norm(s):
    c = s["case"]
    dt, pt = TYPES[c["dtype"]], TYPES[c["params"]]
    x = s["x"].float()
    over = (c["batch"], 1, 1, c["c"]) if c["per_batch"] else (c["c"],)
    w, bias = s["weight"].float().reshape(over), s["bias"].float().reshape(over)
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + s["eps"])
    xhat = xc * rstd
    out = {"y": (xhat * w + bias).to(dt)}
    if c["train"]:
        dy = s["dy"].float()
        g = dy * w
        dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
        dims = (1, 2) if c["per_batch"] else (0, 1, 2)
        out["dx"] = dx.to(dt)
        out["dweight"] = (dy * xhat).sum(dims).to(pt)
        out["dbias"] = dy.sum(dims).to(pt)
    return out


def _own_cross(s):
    from hierarchical_top_sparse_b200 import llsa
    c = s["case"]
    op = s.get("operator")
    if op is None:
        p = llsa.CrossProblem(batch=c["batch"], heads=c["heads"], kv_heads=c["kv_heads"], nq=c["nq"], nk=c["nk"],
                              d=c["d"], dtype=llsa.BF16 if c["dtype"] == "bf16" else llsa.FP32)
        op = s["operator"] = llsa.CrossAttention(p, backward=c["train"], token_major=c["layout"] == "bnhd")
    o, lse = op.forward(s["q"], s["k"], s["v"], kv_len=s["kv_len"], key_mask=s["key_mask"])
    out = {"o": o, "lse": lse}
    if c["train"]:
        out["dq"], out["dk"], out["dv"] = op.backward_pass(s["q"], s["k"], s["v"], s["dO"], kv_len=s["kv_len"],
                                                           key_mask=s["key_mask"])
    return out


def _own_norm(s):
    from hierarchical_top_sparse_b200 import llsa
    c = s["case"]
    op = s.get("operator")
    if op is None:
        number = {"bf16": llsa.BF16, "fp32": llsa.FP32}
        p = llsa.NormProblem(batch=c["batch"], heads=c["heads"], n=c["n"], c=c["c"], eps=s["eps"],
                             dtype=number[c["dtype"]], param_dtype=number[c["params"]], per_batch=c["per_batch"])
        op = s["operator"] = llsa.LayerNorm(p, backward=c["train"], token_major=c["layout"] == "bnhd")
    out = {"y": op.forward(s["x"], s["weight"], s["bias"])}
    if c["train"]:
        out["dx"], out["dweight"], out["dbias"] = op.backward_pass(s["x"], s["weight"], s["dy"])
    return out


def run(state):
    if own:
        return _own_cross(state) if state["case"]["op"] == "cross" else _own_norm(state)
    return _plain_cross(state) if state["case"]["op"] == "cross" else _plain_norm(state)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        rows = case["batch"] * case["heads"] * case["n"]
        nbytes = rows * case["c"] * size * (4 if case["train"] else 2)      # x, y (and dy, dx)
        params = case["c"] * (case["batch"] if case["per_batch"] else 1) * (2 if case["params"] == "bf16" else 4)
        return {"bytes": nbytes + params * (4 if case["train"] else 2),
                "flops": rows * case["c"] * (20 if case["train"] else 8)}
    b, h, hk, nq, d = (case[k] for k in ("batch", "heads", "kv_heads", "nq", "d"))
    keys = sum(a + c for a, c in _key_counts(case))                         # over the batch
    queries = b * h * nq * d * size
    states = keys * hk * d * size
    lse = b * h * nq * 4
    nbytes = 2 * queries + 2 * states + lse                                 # q, o, k, v, lse
    pairs = keys * h * nq
    if case["train"]:
        nbytes += 2 * queries + 2 * b * hk * case["nk"] * d * size          # dO, dq, dk, dv
    return {"bytes": nbytes, "flops": pairs * d * (14 if case["train"] else 4)}


def exact(case, seed):
    """The definitions in 64 bits, each quantity by its own formula over one key head at a time."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        x = s["x"].double()
        shape = (case["batch"], 1, 1, case["c"]) if case["per_batch"] else (1, 1, 1, case["c"])
        w, bias = s["weight"].double().view(shape), s["bias"].double().view(shape)
        n = case["c"]
        mean = x.sum(-1, keepdim=True) / n
        std = torch.sqrt(((x - mean) ** 2).sum(-1, keepdim=True) / n + s["eps"])
        xhat = (x - mean) / std
        out = {"y": xhat * w + bias}
        if case["train"]:
            dy = s["dy"].double()
            gw = dy * w
            # the Jacobian of xhat applied to gw: (I - 1 1^T / n - xhat xhat^T / n) / std
            out["dx"] = (gw - gw.sum(-1, keepdim=True) / n - xhat * ((gw * xhat).sum(-1, keepdim=True) / n)) / std
            pattern = "bhnc->bc" if case["per_batch"] else "bhnc->c"
            out["dweight"] = torch.einsum(pattern.replace("bhnc", "bhnc,bhnc"), dy, xhat)
            out["dbias"] = torch.einsum(pattern, dy)
        return out
    b, h, hk, nq, nk, d = (case[k] for k in ("batch", "heads", "kv_heads", "nq", "nk", "d"))
    group = h // hk
    f64 = dict(dtype=torch.float64, device="cuda")
    out = {"o": torch.zeros(b, h, nq, d, **f64), "lse": torch.full((b, h, nq), -math.inf, **f64)}
    if case["train"]:
        out.update(dq=torch.zeros(b, h, nq, d, **f64), dk=torch.zeros(b, hk, nk, d, **f64),
                   dv=torch.zeros(b, hk, nk, d, **f64))
    for i in range(b):
        if s["kv_len"] is not None:
            at = torch.arange(int(s["kv_len"][i]), device="cuda")
        elif s["key_mask"] is not None:
            at = torch.nonzero(s["key_mask"][i]).flatten()
        else:
            at = torch.arange(nk, device="cuda")
        if at.numel() == 0:
            continue
        for j in range(h):
            q = s["q"][i, j].double()
            k, v = s["k"][i, j // group].double()[at], s["v"][i, j // group].double()[at]
            z = torch.einsum("nd,md->nm", q, k) / math.sqrt(d)
            lse = torch.logsumexp(z, dim=1)
            p = torch.exp(z - lse[:, None])
            o = torch.einsum("nm,md->nd", p, v)
            out["o"][i, j], out["lse"][i, j] = o, lse
            if case["train"]:
                g = s["dO"][i, j].double()
                dp = torch.einsum("nd,md->nm", g, v)
                dz = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(d)
                out["dq"][i, j] = torch.einsum("nm,md->nd", dz, k)
                out["dk"][i, j // group].index_add_(0, at, torch.einsum("nm,nd->md", dz, q))
                out["dv"][i, j // group].index_add_(0, at, torch.einsum("nm,nd->md", p, g))
    return out
