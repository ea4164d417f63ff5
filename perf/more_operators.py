"""Cases of the operators around a distilled training step, their plain forms and the calls a
user makes of them.

Three operators beside the fused loss, the packed attention and the head norm:

  distill     divergence of the student's softmax from a teacher's top logits, of hidden
              states and the unembedding matrix, without the N x V logits; the backward
              returns the gradients of both
  layer_norm  layer norm or RMS norm of rows, with the residual sum before it; the backward
              returns the rows' and the weights' gradients
  rope        rotary positions of query and key heads, scaled for long contexts

A case with "train" set is one training pass (forward and backward), one without is the forward
alone.  `own` selects the framework's calls; otherwise the operators are computed in plain torch
operations in 32 bits (angles in 64) and rounded once at the end.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
NORM_EPS = 1e-5
# most work of a drawn case: no more than that of the largest listed ones
MOST_LOGITS = 8192 * 128256 * 4096
MOST_ROWS = 16384 * 4096
MOST_HEADS = 32768 * 32 * 128


def distill(name, tokens, hidden, vocab, top, temperature=1.0, teacher="fp32", ignored=0.0, short=False,
            tail=False, train=True):
    return {"name": name, "op": "distill", "tokens": tokens, "hidden": hidden, "vocab": vocab, "top": top,
            "temperature": temperature, "teacher": teacher, "ignored": ignored, "short": short, "tail": tail,
            "train": train}


def norm(name, rows, hidden, dtype="bf16", rms=False, bias=True, residual=False, train=False):
    return {"name": name, "op": "layer_norm", "rows": rows, "hidden": hidden, "dtype": dtype, "rms": rms,
            "bias": bias, "residual": residual, "train": train}


def rope(name, tokens, q_heads, kv_heads, head_dim, rot, dtype="bf16", style="half", scaling="none", start=0,
         train=False):
    return {"name": name, "op": "rope", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rot": rot, "dtype": dtype, "style": style, "scaling": scaling, "start": start,
            "train": train}


def listed():
    return [
        # the step of a small model: launch and call latency
        distill("distill_small", 256, 256, 4096, 16),
        # the validation loss of a ragged batch: forward alone, odd vocabulary, softened, bf16 teacher
        # whose log-sum-exp over its whole vocabulary came with it
        distill("distill_eval", 2001, 2304, 32003, 50, 2.0, "bf16", 0.06, True, True, train=False),
        # a distillation step of the Llama-3 shape: 8192 tokens, the teacher's 64 top logits
        distill("distill_step", 8192, 4096, 128256, 64, ignored=0.05),
        # a step of the Qwen-2.5 shape, softened, with more of the teacher's logits
        distill("distill_step_wide", 4096, 3584, 152064, 100, 1.5, "bf16", 0.1, True),
        # one token of an interactive call
        norm("norm_token", 1, 4096),
        # the norm in front of a projection with the residual stream's sum, a prompt of 16384 tokens
        norm("norm_residual", 16384, 4096, rms=True, bias=False, residual=True),
        # a training pass of the final norm before the loss, 8192 tokens
        norm("norm_step", 8192, 4096, train=True),
        # a small ragged batch in fp32 with the residual sum, the Gemma-2 width
        norm("norm_step_fp32", 3001, 2304, "fp32", rms=True, bias=False, residual=True, train=True),
        # one token far into a long context
        rope("rotary_token", 1, 32, 8, 128, 128, scaling="yarn", start=100001),
        # a long prompt past the trained length
        rope("rotary_long", 32768, 28, 4, 128, 128, scaling="yarn"),
        # a training pass of 8192 tokens
        rope("rotary_step", 8192, 32, 8, 128, 128, scaling="llama3", train=True),
        # part of an odd head turned, as interleaved pairs, in fp32
        rope("rotary_part_fp32", 1999, 14, 2, 80, 40, "fp32", "pairs", "linear", 3000, True),
    ]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    train = rng.random() < 0.6
    kind = rng.random()
    if kind < 0.4:
        hidden = 8 * spread(rng, 16, 512)
        vocab = spread(rng, 2000, 160000)
        tokens = spread(rng, 1, max(1, min(8192, MOST_LOGITS // (hidden * vocab))))
        c = distill("", tokens, hidden, vocab, spread(rng, 1, 128), rng.choice([1.0, 1.0, 1.5, 2.0, 4.0]),
                    rng.choice(["bf16", "fp32"]), rng.choice([0.0, 0.05, 0.3]), rng.random() < 0.5,
                    rng.random() < 0.3, train)
    elif kind < 0.7:
        hidden = 8 * spread(rng, 8, 2048)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        most = MOST_ROWS // (hidden * (2 if dtype == "fp32" else 1))
        c = norm("", spread(rng, 1, min(32768, most)), hidden, dtype, rng.random() < 0.5, rng.random() < 0.5,
                 rng.random() < 0.5, train)
    else:
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 7] if kv < 8 else [1, 4])
        dim = rng.choice([64, 80, 96, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        per = (kv + kv * group) * dim * (2 if dtype == "fp32" else 1) * (2 if train else 1)
        c = rope("", spread(rng, 1, min(32768, MOST_HEADS // per)), kv * group, kv, dim,
                 rng.choice([dim, dim // 16 * 8]), dtype, rng.choice(["half", "pairs"]),
                 rng.choice(["none", "linear", "yarn", "llama3"]), rng.choice([0, spread(rng, 1, 1000000)]), train)
    del c["name"]
    return c


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * (seed + 1))
    s = {"case": case, "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    {"distill": prepare_distill, "layer_norm": prepare_norm, "rope": prepare_rope}[case["op"]](s, case, gen)
    return s


def prepare_distill(s, c, gen):
    N, H, V, K, T = c["tokens"], c["hidden"], c["vocab"], c["top"], c["temperature"]

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    W = (randn(V, H) * 0.02).bfloat16()
    # the teacher's tokens of a row: ranks spread over the logarithm of a vocabulary's
    # frequencies, one out of each of K intervals, in the order of their logits
    flat = max(1.0, V / 257.0, 2.0 * K)
    part = (torch.arange(K, device="cuda") + rand(N, K)) / K
    rank = (flat * ((V / flat + 1.0) ** part.double() - 1.0)).long().clamp_(0, V - 1)
    token_of = torch.randperm(V, generator=gen, device="cuda")
    order = rand(N, K).argsort(-1)
    ids = token_of[rank.gather(1, order)]
    t = (12.0 - 1.5 * torch.log1p(torch.arange(K, device="cuda")) + 0.5 * randn(N, K)).sort(-1, descending=True).values
    # hidden states of a student early in its training: its logits at the teacher's first token
    # are about 6, at the second about 4; the others have a spread of 0.02 sqrt(H)
    X = randn(N, H)
    X /= X.square().mean(-1, keepdim=True).sqrt()
    X.addcmul_(W[ids[:, 0]].float(), torch.tensor(6.0 / (0.0004 * H), device="cuda"))
    if K > 1:
        X.addcmul_(W[ids[:, 1]].float(), torch.tensor(4.0 / (0.0004 * H), device="cuda"))
    # prompt tokens have no entries, some rows fewer than K
    if c["short"]:
        ids.masked_fill_(torch.arange(K, device="cuda") >= (K * (0.3 + rand(N, 1))).ceil().clamp_(max=K), -1)
    ids.masked_fill_(rand(N, 1) < c["ignored"], -1)
    t = t.to(DTYPES[c["teacher"]])
    s.update(X=X.bfloat16(), W=W, ids=ids, t=t, tail=None, grad=torch.ones(1, device="cuda"))
    if c["tail"]:  # the K entries hold 0.7 to 1 of the teacher's probability
        lse = torch.logsumexp((t.float() / T).masked_fill(ids < 0, -math.inf), -1).nan_to_num(0.0, neginf=0.0)
        s["tail"] = lse - torch.log(0.7 + 0.3 * rand(N))


def prepare_norm(s, c, gen):
    R, H, dt = c["rows"], c["hidden"], DTYPES[c["dtype"]]

    def randn(*shape, scale=1.0, offset=0.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale + offset).to(dt)

    # a residual stream: rows of different sizes, a few columns that stand out
    size = torch.rand(R, 1, generator=gen, device="cuda") * 3.0 + 0.5
    column = 1.0 + 9.0 * (torch.rand(H, generator=gen, device="cuda") < 0.01)
    x = torch.randn(R, H, generator=gen, device="cuda")
    s["x"] = ((x + 0.2) * size * column).to(dt)
    s["residual"] = randn(R, H) if c["residual"] else None
    s["w"] = randn(H, scale=0.1, offset=1.0)
    s["b"] = randn(H, scale=0.1) if c["bias"] else None
    if c["train"]:
        s["dy"] = randn(R, H)
        s["ds"] = randn(R, H) if c["residual"] else None


def frequencies(c):
    """(inverse frequencies in 64 bits, magnitude): base 10000 or 500000, scaled eightfold from a
    trained length of 8192."""
    half, L, factor = c["rot"] // 2, 8192.0, 8.0
    theta = 500000.0 if c["scaling"] == "llama3" else 10000.0
    inv = theta ** (-torch.arange(half, dtype=torch.float64) / half)
    turns = L * inv / (2.0 * math.pi)
    if c["scaling"] == "linear":
        return inv / factor, 1.0
    if c["scaling"] == "yarn":
        # as they are from 32 turns in the trained length on, divided up to one turn, a ramp between
        at = [half * math.log(L / (2.0 * math.pi * b)) / math.log(theta) for b in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), 2 * half - 1)
        ramp = ((torch.arange(half, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        return inv * (1.0 - ramp) + inv / factor * ramp, 0.1 * math.log(factor) + 1.0
    if c["scaling"] == "llama3":
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return inv * keep + inv / factor * (1.0 - keep), 1.0
    return inv, 1.0


def prepare_rope(s, c, gen):
    T, HQ, HK, D, dt = c["tokens"], c["q_heads"], c["kv_heads"], c["head_dim"], DTYPES[c["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(dt)

    # the output of one fused projection, of which q and k are strided views
    qkv = randn(T, HQ + 2 * HK, D)
    inv, magnitude = frequencies(c)
    offset = int(torch.randint(0, 64, (1,), generator=gen, device="cuda").item())
    s.update(q=qkv[:, :HQ], k=qkv[:, HQ:HQ + HK], inv=inv.cuda(), magnitude=magnitude,
             positions=torch.arange(T, device="cuda") + (c["start"] + offset))
    if c["train"]:
        s.update(dq=randn(T, HQ, D), dk=randn(T, HK, D))


def run(s):
    op = s["case"]["op"]
    if op == "distill":
        return own_distill(s) if own else plain_distill(s)
    if op == "layer_norm":
        return own_norm(s) if own else plain_norm(s)
    return own_rope(s) if own else plain_rope(s)


# ----------------------------------------------------------------------------
# the framework's calls
# ----------------------------------------------------------------------------
def own_distill(s):
    from linear_cross_entropy_logit_gb300 import binding as B
    c = s["case"]
    args = s["X"], s["W"], s["ids"], s["t"]
    loss, lse, logits, valid, _ = B.flce_distill_forward(*args, c["temperature"], teacher_lse=s["tail"],
                                                         err_word=s["err"])
    r = {"loss": loss, "lse": lse, "logits": logits, "valid": valid}
    if c["train"]:
        r["dX"], r["dW"], _ = B.flce_distill_backward(*args, lse, logits, valid, c["temperature"],
                                                      teacher_lse=s["tail"], grad_loss=s["grad"],
                                                      err_word=s["err"])
    return r


def own_norm(s):
    from linear_cross_entropy_logit_gb300 import binding as B
    c = s["case"]
    y, x, mean, rstd = B.flce_layer_norm_forward(s["x"], s["w"], s["b"], NORM_EPS, residual=s["residual"],
                                                 rms=c["rms"])
    r = {"y": y}
    if c["residual"]:
        r["sum"] = x
    if c["train"]:
        r["dx"], r["dw"], db = B.flce_layer_norm_backward(s["dy"], x, s["w"], mean, rstd, dsum=s["ds"],
                                                          rms=c["rms"], bias=c["bias"])
        if c["bias"]:
            r["db"] = db
    return r


def own_rope(s):
    from linear_cross_entropy_logit_gb300 import binding as B
    c = s["case"]
    how = {"magnitude": s["magnitude"], "interleaved": c["style"] == "pairs"}
    r = {}
    r["q"], r["k"] = B.flce_rope_forward(s["q"], s["k"], s["inv"], s["positions"], **how)
    if c["train"]:
        r["dq"], r["dk"] = B.flce_rope_backward(s["dq"], s["dk"], s["inv"], s["positions"], **how)
    return r


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------
def plain_distill(s):
    c, ids, T = s["case"], s["ids"], s["case"]["temperature"]
    X, W = s["X"].float(), s["W"].float()
    there = ids >= 0
    at = ids.clamp(min=0)
    t = (s["t"].float() / T).masked_fill(~there, -math.inf)
    if s["tail"] is None:
        top = t.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        tl = top[:, 0] + (t - top).exp().sum(-1).log()
        tl = torch.where(there.any(-1), tl, torch.zeros_like(tl))
    else:
        tl = s["tail"]
    q = (t - tl[:, None]).exp()
    Q = q.sum(-1)
    z = X @ W.T
    logits = z.gather(1, at).masked_fill(~there, 0.0)
    z.div_(T)
    m = z.amax(-1, keepdim=True)
    z.sub_(m).exp_()
    total = z.sum(-1, keepdim=True)
    lse = (m + total.log())[:, 0]
    rows = (q * (t - logits / T).masked_fill(~there, 0.0)).sum(-1) + Q * (lse - tl)
    valid = there.any(-1)
    count = valid.sum()
    rows = rows.masked_fill(~valid, 0.0)
    r = {"loss": (rows.double().sum() / count.clamp(min=1)).float()[None], "lse": lse, "logits": logits,
         "valid": count.int()[None]}
    if c["train"]:
        z.mul_(Q[:, None] / total)
        z.scatter_add_(1, at, -q)
        z.mul_(torch.where(valid, s["grad"] / (T * count.clamp(min=1)), torch.zeros_like(lse))[:, None])
        r["dX"] = (z @ W).to(s["X"].dtype)
        r["dW"] = (z.T @ X).to(s["W"].dtype)
    return r


def plain_norm(s):
    c, dt = s["case"], s["x"].dtype
    x = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dt)
    r = {} if s["residual"] is None else {"sum": x}
    x, w = x.float(), s["w"].float()
    if not c["rms"]:
        x = x - x.mean(-1, keepdim=True)
    rstd = ((x * x).mean(-1, keepdim=True) + NORM_EPS).rsqrt()
    n = x * rstd
    r["y"] = (n * w if s["b"] is None else n * w + s["b"].float()).to(dt)
    if c["train"]:
        g = s["dy"].float()
        gw = g * w
        dx = gw - n * (gw * n).mean(-1, keepdim=True)
        if not c["rms"]:
            dx = dx - gw.mean(-1, keepdim=True)
        dx = dx * rstd
        r["dx"] = (dx if s["ds"] is None else dx + s["ds"].float()).to(dt)
        r["dw"] = (g * n).sum(0)
        if c["bias"]:
            r["db"] = g.sum(0)
    return r


def turn(x, cos, sin, rot, pairs):
    """The first `rot` values of each head turned by the angles; the others as they are."""
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    head = torch.stack((u, v), -1).flatten(-2) if pairs else torch.cat((u, v), -1)
    return torch.cat((head, x[..., rot:]), -1)


def plain_rope(s):
    c, dt = s["case"], s["q"].dtype
    angle = s["positions"].double()[:, None, None] * s["inv"]
    cos, sin = (angle.cos() * s["magnitude"]).float(), (angle.sin() * s["magnitude"]).float()
    how = c["rot"], c["style"] == "pairs"
    r = {"q": turn(s["q"], cos, sin, *how).to(dt), "k": turn(s["k"], cos, sin, *how).to(dt)}
    if c["train"]:
        r["dq"], r["dk"] = (turn(s[n], cos, -sin, *how).to(dt) for n in ("dq", "dk"))
    return r


# ----------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# ----------------------------------------------------------------------------
def work(case):
    if case["op"] == "distill":
        N, H, V, K = case["tokens"], case["hidden"], case["vocab"], case["top"]
        used = N * (1.0 - case["ignored"])  # rows without entries need no gradient
        entries = N * K * (8 + (2 if case["teacher"] == "bf16" else 4) + 4) + 4 * N * (2 if case["tail"] else 1)
        moved = 2 * (N + V) * H * (2 if case["train"] else 1) + entries
        # a product for the softmax; backward it is needed again, and one for each gradient
        return {"bytes": moved, "flops": 2.0 * V * H * (N + (3.0 * used if case["train"] else 0.0))}
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "layer_norm":
        x, H = case["rows"] * case["hidden"], case["hidden"]
        both = 2 if case["residual"] else 1
        moved = size * x * 2 * both + size * H * (2 if case["bias"] else 1)
        if case["train"]:  # the rows are read once for both passes
            moved += size * x * (1 + both) + 4 * H * (2 if case["bias"] else 1)
        return {"bytes": moved, "flops": x * (25.0 if case["train"] else 8.0)}
    x = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * case["head_dim"]
    passes = 2 if case["train"] else 1
    return {"bytes": passes * 2 * size * x + 8 * case["tokens"], "flops": 4.0 * passes * x}


def exact(case, seed):
    s = prepare(case, seed)
    return {"distill": exact_distill, "layer_norm": exact_norm, "rope": exact_rope}[case["op"]](s, case)


def exact_distill(s, c):
    f, T, ids = torch.float64, c["temperature"], s["ids"]
    N, H, V, K = c["tokens"], c["hidden"], c["vocab"], c["top"]
    X = s["X"].to(f)
    logits = torch.zeros(N, K, dtype=f, device="cuda")
    for k in range(K):
        row = torch.nonzero(ids[:, k] >= 0)[:, 0]
        logits[row, k] = torch.einsum("nh,nh->n", X[row], s["W"][ids[row, k]].to(f))
    valid = (ids >= 0).sum(-1) > 0
    count = int(valid.sum())
    r = {"loss": None, "lse": None, "logits": logits, "valid": torch.tensor([count])}
    if c["train"]:
        r.update(dX=None, dW=None)
    if work(c)["flops"] > 6e12:
        return r
    # teacher's probabilities, each entry by itself
    weight = torch.where(ids >= 0, s["t"].to(f) / T, torch.full_like(logits, -math.inf))
    if s["tail"] is None:
        log_mass = torch.logsumexp(weight, -1)
    else:
        log_mass = s["tail"].to(f)
    q = torch.where(ids >= 0, torch.exp(weight - log_mass[:, None]), torch.zeros_like(logits))
    blocks = [(a, min(a + 4096, V)) for a in range(0, V, 4096)]
    lse = torch.stack([torch.logsumexp(X @ s["W"][a:b].to(f).mT / T, -1) for a, b in blocks], -1).logsumexp(-1)
    gap = torch.xlogy(q, q) - q * (logits / T - lse[:, None])
    r.update(loss=gap[valid].sum()[None] / max(count, 1), lse=lse)
    if c["train"]:
        dX, dW = torch.zeros_like(X), torch.empty(V, H, dtype=f, device="cuda")
        for a, b in blocks:
            Wb = s["W"][a:b].to(f)
            d = torch.exp(X @ Wb.mT / T - lse[:, None]) * q.sum(-1, keepdim=True)
            for k in range(K):
                row = torch.nonzero((ids[:, k] >= a) & (ids[:, k] < b))[:, 0]
                d[row, ids[row, k] - a] -= q[row, k]
            d[~valid] = 0.0
            d *= s["grad"].item() / (max(count, 1) * T)
            dX += d @ Wb
            dW[a:b] = d.mT @ X
        r.update(dX=dX, dW=dW)
    return r


def exact_norm(s, c):
    f = torch.float64
    x, r = s["x"].to(f), {}
    if c["residual"]:
        r["sum"] = x + s["residual"].to(f)
        x = r["sum"].to(s["x"].dtype).to(f)  # the operator norms the sum as it is stored
    mu = torch.zeros_like(x[:, :1]) if c["rms"] else x.mean(-1, keepdim=True)
    sd = torch.sqrt(((x - mu) ** 2).sum(-1, keepdim=True) / c["hidden"] + NORM_EPS)
    w = s["w"].to(f)
    r["y"] = (x - mu) / sd * w
    if c["bias"]:
        r["y"] += s["b"].to(f)
    if c["train"]:
        g = s["dy"].to(f)
        along = torch.einsum("rh,rh,h->r", g, x - mu, w)[:, None] / c["hidden"]
        r["dx"] = g * w / sd - (x - mu) * along / sd ** 3
        if not c["rms"]:
            r["dx"] -= (g @ w)[:, None] / (c["hidden"] * sd)
        if c["residual"]:
            r["dx"] += s["ds"].to(f)
        r["dw"] = torch.einsum("rh,rh->h", g, (x - mu) / sd)
        if c["bias"]:
            r["db"] = torch.einsum("rh->h", g)
    return r


def exact_rope(s, c):
    f, rot = torch.float64, c["rot"]
    half = rot // 2
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if c["style"] == "pairs" else (i, i + half)
    z = torch.polar(torch.full((c["tokens"], half), s["magnitude"], dtype=f, device="cuda"),
                    torch.outer(s["positions"].to(f), s["inv"])).unsqueeze(1)

    def rotated(x, by):
        y = x.to(f)
        t = torch.complex(y[..., first], y[..., second]) * by
        y[..., first], y[..., second] = t.real, t.imag
        return y

    r = {"q": rotated(s["q"], z), "k": rotated(s["k"], z)}
    if c["train"]:
        r.update(dq=rotated(s["dq"], z.conj()), dk=rotated(s["dk"], z.conj()))
    return r
