"""The operators around the joint attention that `perf` measures: the norm in front of a projection,
the projection with low-rank adapters that makes Q, K and V, and the cross attention of latent tokens
to a text encoder's states, each with its plain form.

With `own` false `run` computes the plain forms in float32; with `own` true it calls this
repository's kernels. `exact` restates each operator in float64.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
_EPS = 1e-6

# The joint sequences of this repository's layers: text + high-resolution + low-resolution tokens.
_JOINT_1K = 512 + 64 * 64 + 16 * 16          # 4,864
_JOINT_4K = 512 + 256 * 256 + 64 * 64        # 70,144


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # text rows of two prompts, modulated per sample: a call where latency counts
        dict(name="norm_fwd_text", op="norm", dir="fwd", dtype="bf16", wdtype="bf16", batch=2, rows=77,
             cols=1536, weight="sample", plus_one=True),
        # every token of a 4K layer, modulated per sample, statistics kept for training
        dict(name="norm_fwd_4k", op="norm", dir="fwd", dtype="bf16", wdtype="fp32", batch=1, rows=_JOINT_4K,
             cols=2048, weight="sample", plus_one=True),
        # a 1K training layer, two images, one learned weight and bias
        dict(name="norm_bwd_1k", op="norm", dir="bwd", dtype="bf16", wdtype="fp32", batch=2, rows=_JOINT_1K,
             cols=1536, weight="shared", plus_one=False),
        # an odd width in single precision, gradients of a modulation of each sample
        dict(name="norm_bwd_odd", op="norm", dir="bwd", dtype="fp32", wdtype="fp32", batch=3, rows=37 * 29,
             cols=1153, weight="sample", plus_one=True),
        # 4K latent tokens over 512 text states
        dict(name="cross_fwd_4k", op="cross", dir="fwd", dtype="bf16", batch=1, nq=256 * 256, ns=512, heads=24,
             kv_heads=24, dim=128, lens="full", mask=False),
        # one new token of each of 16 sequences over long encoder states, shared key/value heads
        dict(name="cross_fwd_token", op="cross", dir="fwd", dtype="fp16", batch=16, nq=1, ns=4096, heads=32,
             kv_heads=8, dim=128, lens="ragged", mask=False),
        # the ragged latent (256 x 135) of two prompts of odd, unequal length
        dict(name="cross_fwd_ragged", op="cross", dir="fwd", dtype="fp16", batch=2, nq=256 * 135, ns=333, heads=24,
             kv_heads=24, dim=64, lens="ragged", mask=False),
        # training at 1K: four prompts of which the last is empty
        dict(name="cross_bwd_1k", op="cross", dir="bwd", dtype="bf16", batch=4, nq=64 * 64, ns=512, heads=24,
             kv_heads=24, dim=128, lens="empty", mask=False),
        # training with shared key/value heads and states masked one by one
        dict(name="cross_bwd_shared", op="cross", dir="bwd", dtype="fp16", batch=1, nq=128 * 128, ns=1000, heads=16,
             kv_heads=4, dim=64, lens="full", mask=True),
        # one modulation or text token of each of eight requests, an adapter for each request
        dict(name="adapter_token", op="adapter", dtype="bf16", rows=8, k=2048, n=6144, rank=16, adapters=8,
             ids="each", bias=True),
        # Q, K and V of two 1K images: adapters on the low-resolution tokens alone
        dict(name="adapter_1k", op="adapter", dtype="bf16", rows=2 * _JOINT_1K, k=1536, n=3 * 1536, rank=16,
             adapters=2, ids="lowres", bias=True),
        # a 4K layer of four requests' tokens packed one after another, rank 32
        dict(name="adapter_4k", op="adapter", dtype="fp16", rows=_JOINT_4K, k=2048, n=2048, rank=32, adapters=4,
             ids="runs", bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "cross", "adapter"])
    if op == "norm":
        d = rng.choice(["bf16", "fp16", "fp32"])
        batch, cols = rng.randint(1, 4), _log(rng, 64, 8192)
        most = _JOINT_4K * 2048 * 2 // _SIZE[d] // (cols * batch)
        return dict(op="norm", dir=rng.choice(["fwd", "bwd"]), dtype=d, wdtype=rng.choice([d, "fp32"]), batch=batch,
                    rows=max(1, min(most, _log(rng, 1, _JOINT_4K))), cols=cols,
                    weight=rng.choice(["none", "shared", "sample"]), plus_one=rng.random() < 0.5)
    if op == "cross":
        way, dim = rng.choice(["fwd", "bwd"]), rng.choice([64, 128])
        kv_heads, group = rng.choice([1, 2, 4, 8, 12, 24]), rng.choice([1, 1, 2, 3, 4])
        batch, ns = rng.randint(1, 6), _log(rng, 1, 4096)
        # scores of the largest listed case of the direction bound the cost
        scores = 24 * 65536 * 512 * 128 // (dim * (1 if way == "fwd" else 4))
        most = scores // (batch * kv_heads * group * ns)
        return dict(op="cross", dir=way, dtype=rng.choice(["bf16", "fp16"]), batch=batch,
                    nq=max(1, min(most, _log(rng, 1, 65536))), ns=ns, heads=kv_heads * group, kv_heads=kv_heads,
                    dim=dim, lens=rng.choice(["full", "ragged", "empty"]), mask=rng.random() < 0.3)
    k, n = 8 * _log(rng, 8, 512), _log(rng, 64, 6144)
    most = _JOINT_4K * 2048 * 2048 // (k * n)
    return dict(op="adapter", dtype=rng.choice(["bf16", "fp16"]), rows=max(1, min(most, _log(rng, 1, _JOINT_4K))), k=k,
                n=n, rank=rng.choice([4, 8, 16, 32, 64]), adapters=rng.randint(1, 8),
                ids=rng.choice(["each", "lowres", "runs"]), bias=rng.random() < 0.5)


# ------------------------------------------------------------------------------- inputs
def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _lens(case):
    """Visible states of each sample (None: all of them)."""
    b, s = case["batch"], case["ns"]
    if case["lens"] == "full":
        return None
    lens = [s - (i * s * 3) // (5 * b) for i in range(b)]     # padded prompts, the first one full
    if case["lens"] == "empty":
        lens[-1] = 0
    return lens


def _kept(case):
    """Whether state j of sample b is visible, [batch, ns] on the CPU."""
    b, s = case["batch"], case["ns"]
    j = torch.arange(s)[None, :]
    keep = torch.ones(b, s, dtype=torch.bool)
    if case["mask"]:
        keep &= (j + torch.arange(b)[:, None]) % 4 != 0
    if _lens(case) is not None:
        keep &= j < torch.tensor(_lens(case))[:, None]
    return keep


def _ids(case):
    """The adapter of each row, -1 for none, on the CPU."""
    m, a = case["rows"], case["adapters"]
    r = torch.arange(m)
    if case["ids"] == "each":                                  # requests interleaved row by row
        return (r % a).to(torch.int32)
    if case["ids"] == "runs":                                  # requests one after another
        return (r * a // m).to(torch.int32)
    part = -(-m // a)                                          # images of which the last 1/19 has an adapter
    return torch.where(r % part >= part - max(1, part // 19), r // part, -1).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = _TYPES[case["dtype"]]
    s = dict(case=dict(case))
    if case["op"] == "norm":
        b, r, c = case["batch"], case["rows"], case["cols"]
        wt = _TYPES[case["wdtype"]]
        # channels of unequal scale and offset, as a residual stream's
        scale = 0.5 + torch.rand(c, generator=gen, device="cuda") * 2
        s["x"] = (torch.randn(b, r, c, generator=gen, device="cuda") * scale
                  + 0.3 * torch.randn(c, generator=gen, device="cuda")).to(t)
        shape = (b, c) if case["weight"] == "sample" else (c,)
        off = 0.0 if case["plus_one"] else 1.0
        s["weight"] = s["bias"] = None
        if case["weight"] != "none":
            s["weight"] = (off + 0.2 * torch.randn(shape, generator=gen, device="cuda")).to(wt)
            s["bias"] = _normal(gen, shape, wt, 0.2)
        x = s["x"].float()
        mean = x.mean(-1)
        if case["dir"] == "fwd":
            s["y"] = torch.empty_like(s["x"])
            s["mean"], s["rstd"] = torch.empty_like(mean), torch.empty_like(mean)
        else:
            s["mean"] = mean                                   # kept by the forward pass
            s["rstd"] = torch.rsqrt((x - mean[..., None]).square().mean(-1) + _EPS)
            s["dy"] = _normal(gen, (b, r, c), t)
            s["dx"] = torch.empty_like(s["x"])
            s["dweight"] = s["dbias"] = None
            if case["weight"] != "none":
                s["dweight"] = torch.empty(shape, device="cuda")
                s["dbias"] = torch.empty(shape, device="cuda")
        return s
    if case["op"] == "cross":
        b, n, m, h, g, d = (case[k] for k in ("batch", "nq", "ns", "heads", "kv_heads", "dim"))
        s["q"] = _normal(gen, (b, n, h, d), t, 1.3)
        s["k"] = _normal(gen, (b, m, g, d), t)
        s["v"] = _normal(gen, (b, m, g, d), t)
        s["lens"] = None if _lens(case) is None else torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
        s["mask"] = None
        if case["mask"]:
            keep = (torch.arange(m)[None, :] + torch.arange(b)[:, None]) % 4 != 0
            s["mask"] = keep.cuda()
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(b, h, n, device="cuda")
        if case["dir"] == "bwd":
            o, lse = _cross(s)                                 # kept by the forward pass
            s["o"].copy_(o)
            s["lse"].copy_(lse)
            s["do"] = _normal(gen, (b, n, h, d), t)
            s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[x]) for x in ("q", "k", "v"))
        return s
    m, k, n, r, a = (case[x] for x in ("rows", "k", "n", "rank", "adapters"))
    s["x"] = _normal(gen, (m, k), t)
    s["w"] = _normal(gen, (n, k), t, k ** -0.5)
    s["a"] = _normal(gen, (a, r, k), t, k ** -0.5)
    s["b"] = _normal(gen, (a, n, r), t, 0.5 * r ** -0.5)
    s["scales"] = 0.5 + torch.rand(a, generator=gen, device="cuda")
    s["bias"] = _normal(gen, (n,), t, 0.1) if case["bias"] else None
    s["ids"] = _ids(case).cuda()
    s["y"] = torch.empty(m, n, dtype=t, device="cuda")
    return s


# ------------------------------------------------------------------------------- plain forms
def _modulation(s, dtype):
    """Weight and bias, broadcast over a sample's rows."""
    c = s["case"]
    if s["weight"] is None:
        return 1.0, 0.0
    w, b = s["weight"].to(dtype), s["bias"].to(dtype)
    if c["plus_one"]:
        w = w + 1
    return (w[:, None], b[:, None]) if c["weight"] == "sample" else (w, b)


def _norm(s):
    x = s["x"].float()
    w, b = _modulation(s, torch.float32)
    mean = x.mean(-1)
    xc = x - mean[..., None]
    rstd = 1 / torch.sqrt(xc.square().mean(-1) + _EPS)
    return (xc * rstd[..., None] * w + b).to(s["x"].dtype), mean, rstd


def _norm_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    w, _ = _modulation(s, torch.float32)
    xh = (x - s["mean"][..., None]) * s["rstd"][..., None]
    g = dy * w
    dx = s["rstd"][..., None] * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    over = 1 if s["case"]["weight"] == "sample" else (0, 1)
    out = [dx.to(s["x"].dtype)]
    if s["weight"] is not None:
        out += [(dy * xh).sum(over), dy.sum(over)]
    return tuple(out)


def _split(t, kv_heads):
    """[B, N, H, D] -> float32 [B, kv_heads, (H / kv_heads) * N, D]."""
    b, n, h, d = t.shape
    return t.float().reshape(b, n, kv_heads, h // kv_heads, d).permute(0, 2, 3, 1, 4).reshape(b, kv_heads, -1, d)


def _join(t, like):
    """The inverse of _split, rounded to the type of `like`."""
    b, n, h, d = like.shape
    g = t.shape[1]
    return t.reshape(b, g, h // g, n, d).permute(0, 3, 1, 2, 4).reshape(b, n, h, d).to(like.dtype)


def _weights(s):
    """Softmax weights [B, kv_heads, rows, S] (zeros in an empty row) and their log-sum-exp."""
    c = s["case"]
    scores = _split(s["q"], c["kv_heads"]) @ _split(s["k"], c["kv_heads"]).transpose(-1, -2)
    scores = scores * c["dim"] ** -0.5
    if s["mask"] is not None:
        scores = scores.masked_fill(~s["mask"][:, None, None, :], -math.inf)
    if s["lens"] is not None:
        far = torch.arange(c["ns"], device="cuda")[None, :] >= s["lens"][:, None]
        scores = scores.masked_fill(far[:, None, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).reshape(c["batch"], c["heads"], c["nq"])
    return p / torch.where(total == 0, torch.ones_like(total), total), lse


def _cross(s):
    p, lse = _weights(s)
    return _join(p @ _split(s["v"], s["case"]["kv_heads"]), s["q"]), lse


def _cross_backward(s):
    c = s["case"]
    g = c["kv_heads"]
    p, _ = _weights(s)
    do, v = _split(s["do"], g), _split(s["v"], g)
    dv = p.transpose(-1, -2) @ do
    dp = do @ v.transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * c["dim"] ** -0.5
    dq = ds @ _split(s["k"], g)
    dk = ds.transpose(-1, -2) @ _split(s["q"], g)
    return _join(dq, s["q"]), _join(dk, s["k"]), _join(dv, s["v"])


def _adapter(s):
    c = s["case"]
    x = s["x"].float()
    # each row's products with every adapter, of which its own is kept
    pick = s["ids"][:, None] == torch.arange(c["adapters"], device="cuda", dtype=torch.int32)
    t = (x @ s["a"].float().flatten(0, 1).T).view(c["rows"], c["adapters"], c["rank"])
    t = t * (pick * s["scales"])[..., None]
    y = x @ s["w"].float().T + t.flatten(1) @ s["b"].float().transpose(1, 2).flatten(0, 1)
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype)


def run(state):
    s = state
    c = s["case"]
    if own:
        import diffusion_transformer_ultra_b200 as ug
        if c["op"] == "norm" and c["dir"] == "fwd":
            ug.layer_norm(s["x"], s["y"], s["weight"], s["bias"], eps=_EPS, plus_one=c["plus_one"],
                          mean=s["mean"], rstd=s["rstd"])
            return s["y"], s["mean"], s["rstd"]
        if c["op"] == "norm":
            ug.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["dx"], s["weight"],
                                   plus_one=c["plus_one"], dweight=s["dweight"], dbias=s["dbias"])
            return (s["dx"],) if s["weight"] is None else (s["dx"], s["dweight"], s["dbias"])
        if c["op"] == "cross" and c["dir"] == "fwd":
            ug.cross_attention(s["q"], s["k"], s["v"], s["o"], kv_lens=s["lens"], key_mask=s["mask"], lse=s["lse"])
            return s["o"], s["lse"]
        if c["op"] == "cross":
            ug.cross_attention_backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["dq"], s["dk"], s["dv"],
                                        kv_lens=s["lens"], key_mask=s["mask"])
            return s["dq"], s["dk"], s["dv"]
        return ug.adapter_project(s["x"], s["w"], s["y"], s["a"], s["b"], s["ids"], scales=s["scales"],
                                  bias=s["bias"])
    if c["op"] == "norm":
        return _norm(s) if c["dir"] == "fwd" else _norm_backward(s)
    if c["op"] == "cross":
        return _cross(s) if c["dir"] == "fwd" else _cross_backward(s)
    return _adapter(s)


# ------------------------------------------------------------------------------- work
def work(case):
    z = _SIZE[case["dtype"]]
    if case["op"] == "norm":
        b, r, c = case["batch"], case["rows"], case["cols"]
        per = {"none": 0, "shared": c, "sample": b * c}[case["weight"]]
        if case["dir"] == "fwd":
            return {"bytes": 2 * b * r * c * z + 8 * b * r + 2 * per * _SIZE[case["wdtype"]], "flops": 8 * b * r * c}
        return {"bytes": 3 * b * r * c * z + 8 * b * r + per * (_SIZE[case["wdtype"]] + 8), "flops": 14 * b * r * c}
    if case["op"] == "cross":
        b, n, m, h, g, d = (case[k] for k in ("batch", "nq", "ns", "heads", "kv_heads", "dim"))
        seen = int(_kept(case).sum())                          # visible states of all samples
        q, kv, pairs = b * n * h * d * z, seen * g * d * z, seen * n * h
        if case["dir"] == "fwd":
            return {"bytes": 2 * q + 2 * kv + 4 * b * h * n, "flops": 4 * pairs * d}
        # the gradients of all states are written, the hidden ones' as zeros
        return {"bytes": 4 * q + 2 * kv + 2 * b * m * g * d * z + 4 * b * h * n, "flops": 10 * pairs * d}
    m, k, n, r, a = (case[x] for x in ("rows", "k", "n", "rank", "adapters"))
    ids = _ids(case)
    rows, used = int((ids >= 0).sum()), int(torch.unique(ids[ids >= 0]).numel())
    return {"bytes": z * (m * k + n * k + m * n + used * r * (k + n) + (n if case["bias"] else 0)) + 4 * m,
            "flops": 2 * m * n * k + 2 * rows * r * (k + n)}


# ------------------------------------------------------------------------------- 64 bits
def _exact_norm(s):
    c = s["case"]
    x = s["x"].double()
    mu = x.sum(-1, keepdim=True) / c["cols"]
    sd = torch.sqrt(((x - mu) ** 2).sum(-1, keepdim=True) / c["cols"] + _EPS)
    w = torch.zeros((), dtype=torch.float64, device="cuda") if s["weight"] is None else s["weight"].double()
    w = w + (1.0 if c["plus_one"] or s["weight"] is None else 0.0)
    per_sample = c["weight"] == "sample"
    if per_sample:
        w = w.unsqueeze(1)
    if c["dir"] == "fwd":
        y = (x - mu) / sd * w
        if s["bias"] is not None:
            y = y + (s["bias"].double().unsqueeze(1) if per_sample else s["bias"].double())
        return y, mu.squeeze(-1), (1 / sd).squeeze(-1)
    dy = s["dy"].double()
    z = (x - mu) / sd
    u = dy * w
    dx = (u - u.sum(-1, keepdim=True) / c["cols"] - z * (u * z).sum(-1, keepdim=True) / c["cols"]) / sd
    if s["weight"] is None:
        return (dx,)
    dw, db = (dy * z).sum(1), dy.sum(1)
    return (dx, dw, db) if per_sample else (dx, dw.sum(0), db.sum(0))


def _exact_cross(s):
    c = s["case"]
    keep, back = _kept(c).cuda(), c["dir"] == "bwd"
    share, scale = c["heads"] // c["kv_heads"], 1 / math.sqrt(c["dim"])
    first = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")     # o, or dq
    lse = torch.full((c["batch"], c["heads"], c["nq"]), -math.inf, dtype=torch.float64, device="cuda")
    dk = torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)

    def head(b, h):
        seen = keep[b].nonzero().squeeze(1)
        if not seen.numel():
            return
        q = s["q"][b, :, h].double()
        k, v = s["k"][b, seen, h // share].double(), s["v"][b, seen, h // share].double()
        logits = scale * (q @ k.T)
        lse[b, h] = torch.logsumexp(logits, -1)
        p = torch.exp(logits - lse[b, h][:, None])
        del logits
        if not back:
            first[b, :, h] = p @ v
            return
        g = s["do"][b, :, h].double()
        mean = (g * (p @ v)).sum(-1, keepdim=True)
        dv[b].index_put_((seen, torch.tensor(h // share, device="cuda")), p.T @ g, accumulate=True)
        p *= g @ v.T - mean
        first[b, :, h] = scale * (p @ k)
        dk[b].index_put_((seen, torch.tensor(h // share, device="cuda")), scale * (p.T @ q), accumulate=True)

    list(map(lambda i: head(i // c["heads"], i % c["heads"]), range(c["batch"] * c["heads"])))
    return (first, dk, dv) if back else (first, lse)


def _exact_adapter(s):
    c = s["case"]
    x = s["x"].double()
    y = x @ s["w"].double().T
    if s["bias"] is not None:
        y += s["bias"].double()

    def add(i):
        rows = (s["ids"] == i).nonzero().squeeze(1)
        y[rows] += s["scales"][i].double() * ((x[rows] @ s["a"][i].double().T) @ s["b"][i].double().T)

    list(map(add, range(c["adapters"])))
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "cross": _exact_cross, "adapter": _exact_adapter}[case["op"]](s)
