"""Cases of the attention operators, their plain forms and the calls a user makes of them.

Two operators that surround the fused loss in a training step on packed
sequences:

  qk_norm_rope  RMS norm of every query and key head, its weight, and the
                rotary position rotation of the result, in one pass; the
                backward returns the gradients of the heads and of both weights
  attention     causal softmax attention over packed sequences of different
                lengths with grouped key / value heads; the backward returns
                the gradients of q, k and v

A case with "train" set is one training pass (forward and backward), one
without is the forward alone.  `own` selects the framework's calls; otherwise
the operators are computed in plain torch operations in 32 bits and rounded
once at the end.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
THETA = 10000.0
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# The plain form of attention holds a few (heads, tokens, tokens) fp32 arrays;
# a drawn case has no more elements of them than the largest listed ones.
MOST_SCORES = {False: 32768 * 32768 * 8, True: 16384 * 16384 * 16}
MOST_HEAD_ROWS = 16384 * 32


def rope(name, tokens, q_heads, kv_heads, head_dim, rot, dtype="bf16", style="half", train=False):
    return {"name": name, "op": "qk_norm_rope", "tokens": tokens, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "rot": rot, "dtype": dtype,
            "style": style, "train": train}


def attn(name, tokens, seqs, q_heads, kv_heads, head_dim, lengths="even", tail=0, train=False):
    return {"name": name, "op": "attention", "tokens": tokens, "seqs": seqs, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "lengths": lengths, "tail": tail,
            "dtype": "bf16", "train": train}


def listed():
    return [
        # one token of an interactive call: launch and call latency
        rope("rope_token", 1, 32, 8, 128, 128),
        # the prompt or the forward of one training batch of 8192 tokens
        rope("rope_batch", 8192, 32, 8, 128, 128),
        # a small odd model in fp32: interleaved pairs, half of each head rotated
        rope("rope_step_odd_fp32", 1021, 14, 2, 80, 40, "fp32", "pairs", True),
        # a training pass over 16384 tokens with seven query heads to a key head
        rope("rope_step", 16384, 28, 4, 128, 128, train=True),
        # a few short prompts: latency counts
        attn("attn_short", 77, 3, 8, 2, 64, "ragged"),
        # one long prompt of 8192 tokens
        attn("attn_prompt", 8192, 1, 32, 8, 128),
        # a pack of prompts of very different lengths
        attn("attn_packed", 16384, 37, 28, 4, 128, "ragged"),
        # a long document with small heads
        attn("attn_long", 32768, 1, 8, 2, 64),
        # a small model's step, an odd head size, unused rows at the end of the pack
        attn("attn_step_small", 544, 4, 12, 12, 96, "ragged", 31, True),
        # a training pass over one sequence of 8192 tokens
        attn("attn_step", 8192, 1, 32, 8, 128, train=True),
        # an instruction-tuning batch: four sequences of 4096 tokens
        attn("attn_step_packed", 16384, 4, 16, 4, 128, train=True),
        # conversations of very different lengths, a key head for each query head, a padded tail
        attn("attn_step_ragged", 9999, 61, 16, 16, 64, "ragged", 255, True),
    ]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 7, 8])
    while kv * group > 32:
        group = rng.choice([1, 2, 4])
    train = rng.random() < 0.5
    if rng.random() < 0.35:
        dim = rng.choice([64, 80, 96, 128])
        heads = kv * (group + 1)
        c = rope("", spread(rng, 1, min(16384, MOST_HEAD_ROWS // heads)), kv * group, kv, dim,
                 rng.choice([dim, dim // 16 * 8]), rng.choice(["bf16", "bf16", "fp32"]),
                 rng.choice(["half", "pairs"]), train)
    else:
        tokens = spread(rng, 1, 16384 if train else 32768)
        most = MOST_SCORES[train] // (kv * group)
        tokens = min(tokens, math.isqrt(most))
        seqs = spread(rng, 1, max(1, min(64, tokens)))
        tail = rng.choice([0, 0, min(rng.randrange(256), tokens // 2)])
        c = attn("", tokens, seqs, kv * group, kv, rng.choice([64, 80, 96, 128]),
                 rng.choice(["even", "ragged"]), tail, train)
    del c["name"]
    return c


def sequence_starts(case):
    """The seqs + 1 offsets of the pack: even lengths, or lengths spread over their logarithm
    (some may be zero).  The rows after the last one are the unused tail."""
    used, n = case["tokens"] - case["tail"], case["seqs"]
    if case["lengths"] == "even":
        share = np.arange(n + 1) / n
    else:
        w = np.exp(np.random.RandomState(used * 97 + n).uniform(0.0, math.log(32.0), n))
        share = np.concatenate([[0.0], np.cumsum(w) / w.sum()])
    cu = np.floor(share * used + 0.5).astype(np.int64)
    cu[-1] = used
    return cu


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * (seed + 1))
    dt = DTYPES[case["dtype"]]
    T, HQ, HK, D = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]

    def normal(*shape, dtype=dt, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    s = {"case": case, "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    # the output of one fused projection, of which q, k and v are strided views
    qkv = normal(T, HQ + 2 * HK, D)
    q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:]
    if case["op"] == "qk_norm_rope":
        half = case["rot"] // 2
        # positions restart in every packed sequence
        offset = int(torch.randint(0, 64, (1,), generator=gen, device="cuda").item())
        s["positions"] = (torch.arange(T, device="cuda") + offset) % 8192
        freq = THETA ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        angle = torch.arange(8192, device="cuda", dtype=torch.float64)[:, None] * freq
        s.update(q=q, k=k, cos=angle.cos().float(), sin=angle.sin().float(),
                 wq=(1.0 + normal(D, dtype=torch.float32, scale=0.1)).to(dt),
                 wk=(1.0 + normal(D, dtype=torch.float32, scale=0.1)).to(dt))
        if case["train"]:
            s.update(dq=normal(T, HQ, D), dk=normal(T, HK, D))
    else:
        # after the norm and the rotation q and k are arrays of their own; v is still a view
        s.update(q=q.contiguous(), k=k.contiguous(), v=v, scale=1.0 / math.sqrt(D),
                 cu=torch.from_numpy(sequence_starts(case)).to("cuda", torch.int32))
        if case["train"]:
            s["dout"] = normal(T, HQ, D)
    return s


def run(s):
    if s["case"]["op"] == "qk_norm_rope":
        return own_rope(s) if own else plain_rope(s)
    return own_attention(s) if own else plain_attention(s)


# ----------------------------------------------------------------------------
# the framework's calls
# ----------------------------------------------------------------------------
def own_rope(s):
    from linear_cross_entropy_logit_gb300 import binding as B
    pairs = s["case"]["style"] == "pairs"
    q_out, k_out, _ = B.flce_qk_norm_rope_forward(
        s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["positions"], EPS,
        interleaved=pairs, err_word=s["err"])
    r = {"q": q_out, "k": k_out}
    if s["case"]["train"]:
        r["dq"], r["dk"], r["dwq"], r["dwk"], _ = B.flce_qk_norm_rope_backward(
            s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"],
            s["positions"], EPS, interleaved=pairs, err_word=s["err"])
    return r


def own_attention(s):
    from linear_cross_entropy_logit_gb300 import binding as B
    out, lse, _ = B.flce_attention_forward(s["q"], s["k"], s["v"], s["cu"], s["scale"],
                                           err_word=s["err"])
    r = {"out": out, "lse": lse}
    if s["case"]["train"]:
        r["dq"], r["dk"], r["dv"], _ = B.flce_attention_backward(
            s["dout"], s["q"], s["k"], s["v"], out, lse, s["cu"], s["scale"], err_word=s["err"])
    return r


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------
def turn(x, cos, sin, rot, pairs):
    """The first `rot` values of each head turned by the angles; the others as they are."""
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, w = a * cos - b * sin, b * cos + a * sin
    head = torch.stack((u, w), -1).flatten(-2) if pairs else torch.cat((u, w), -1)
    return torch.cat((head, x[..., rot:]), -1)


def plain_rope(s):
    c, dt = s["case"], s["q"].dtype
    rot, pairs = c["rot"], c["style"] == "pairs"
    cos, sin = (t[s["positions"]][:, None, :] for t in (s["cos"], s["sin"]))

    def forward(x, w):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        return turn(x * r * w.float(), cos, sin, rot, pairs).to(dt)

    def backward(dy, x, w):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        n = x * r
        g = turn(dy.float(), cos, -sin, rot, pairs)
        gw = g * w.float()
        return (r * (gw - n * (gw * n).mean(-1, keepdim=True))).to(dt), (g * n).sum((0, 1))

    r = {"q": forward(s["q"], s["wq"]), "k": forward(s["k"], s["wk"])}
    if c["train"]:
        r["dq"], r["dwq"] = backward(s["dq"], s["q"], s["wq"])
        r["dk"], r["dwk"] = backward(s["dk"], s["k"], s["wk"])
    return r


def plain_attention(s):
    c, cu, dt = s["case"], s["cu"], s["q"].dtype
    T, HQ, HK, D = c["tokens"], c["q_heads"], c["kv_heads"], c["head_dim"]
    G = HQ // HK
    at = torch.arange(T, device=cu.device)
    of = torch.searchsorted(cu.long(), at, right=True) - 1
    of = torch.where((of >= 0) & (at < cu[-1]), of, -1 - at)
    hidden = (of[:, None] != of[None, :]) | (at[:, None] < at[None, :]) | (of[:, None] < 0)
    heads = lambda x: x.float().transpose(0, 1).reshape(HK, -1, T, D)  # noqa: E731
    q, k, v = heads(s["q"]), heads(s["k"]), heads(s["v"])
    p = (q * s["scale"]) @ k.transpose(-1, -2)
    p.masked_fill_(hidden, -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (m + total.log()).reshape(HQ, T)
    p.div_(torch.where(total == 0, torch.ones_like(total), total))
    out = p @ v
    rows = lambda x: x.reshape(-1, T, D).transpose(0, 1).to(dt).contiguous()  # noqa: E731
    r = {"out": rows(out), "lse": lse}
    if c["train"]:
        do = heads(s["dout"])
        r["dv"] = rows((p.transpose(-1, -2) @ do).sum(1))
        dp = do @ v.transpose(-1, -2)
        dp.sub_((do * out).sum(-1, keepdim=True)).mul_(p)
        del p
        r["dq"] = rows((dp @ k) * s["scale"])
        r["dk"] = rows((dp.transpose(-1, -2) @ q).sum(1) * s["scale"])
    return r


# ----------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# ----------------------------------------------------------------------------
def work(case):
    T, HQ, HK, D = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
    size = 2 if case["dtype"] == "bf16" else 4
    q, k = T * HQ * D, T * HK * D
    if case["op"] == "qk_norm_rope":
        table = 4 * min(T, 8192) * case["rot"] + 8 * T + 2 * D * size
        # forward: heads in, heads out; backward: output gradients in, head gradients out
        # (the heads are read once for both), the weights' gradients in fp32
        moved = size * (2 * (q + k) + (2 * (q + k) if case["train"] else 0)) + table
        return {"bytes": moved + (8 * D if case["train"] else 0),
                "flops": (q + k) * (30 if case["train"] else 10)}
    cu = sequence_starts(case)
    n = (cu[1:] - cu[:-1]).astype(np.float64)
    pairs = float((n * (n + 1) / 2).sum())
    moved = size * (2 * q + 2 * k) + 4 * T * HQ + 4 * len(cu)
    if case["train"]:
        moved += size * (2 * q + 2 * k)
    # two products of each visible pair and head forward, five backward
    return {"bytes": moved, "flops": pairs * HQ * D * (14 if case["train"] else 4)}


def exact(case, seed):
    s = prepare(case, seed)
    return exact_rope(s) if case["op"] == "qk_norm_rope" else exact_attention(s)


def exact_rope(s):
    c = s["case"]
    rot, half, f = c["rot"], c["rot"] // 2, torch.float64
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if c["style"] == "pairs" else (i, i + half)
    z = torch.complex(s["cos"].to(f), s["sin"].to(f))[s["positions"]].unsqueeze(1)

    def rotated(x, by):
        y, t = x.clone(), torch.complex(x[..., first], x[..., second]) * by
        y[..., first], y[..., second] = t.real, t.imag
        return y

    r = {}
    for n in ("q", "k"):
        x, w = s[n].to(f), s["w" + n].to(f)
        inv = 1.0 / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)
        r[n] = rotated(x * inv * w, z)
        if c["train"]:
            g = rotated(s["d" + n].to(f), z.conj())
            r["dw" + n] = torch.einsum("thd,thd->d", g, x * inv)
            along = (g * w * x).sum(-1, keepdim=True)
            r["d" + n] = inv * (g * w) - inv.pow(3) * x * along / x.shape[-1]
    return r


def exact_attention(s):
    c, f = s["case"], torch.float64
    if work(c)["flops"] > 4e12:
        return None
    T, HQ, HK, D = c["tokens"], c["q_heads"], c["kv_heads"], c["head_dim"]
    q, k, v = (s[n].to(f).permute(1, 0, 2) for n in ("q", "k", "v"))
    own_kv = torch.arange(HQ, device="cuda") // (HQ // HK)
    out = torch.zeros(HQ, T, D, dtype=f, device="cuda")
    lse = torch.full((HQ, T), -math.inf, dtype=f, device="cuda")
    dq, dk, dv = torch.zeros_like(out), torch.zeros_like(out), torch.zeros_like(out)
    do = s["dout"].to(f).permute(1, 0, 2) if c["train"] else None
    cu = sequence_starts(c).tolist()
    for lo, hi in zip(cu, cu[1:]):
        for a in range(lo, hi, 1024):
            b = min(a + 1024, hi)
            seen = torch.arange(lo, b, device="cuda")[None] <= torch.arange(a, b, device="cuda")[:, None]
            kk, vv = k[own_kv, lo:b], v[own_kv, lo:b]
            z = torch.bmm(q[:, a:b], kk.mT) * s["scale"]
            lse[:, a:b] = torch.logsumexp(z.masked_fill(~seen, -math.inf), -1)
            p = torch.exp(z - lse[:, a:b, None]) * seen
            out[:, a:b] = torch.bmm(p, vv)
            if c["train"]:
                g = do[:, a:b]
                dv[:, lo:b] += torch.bmm(p.mT, g)
                t = torch.bmm(g, vv.mT)
                t = p * (t - (p * t).sum(-1, keepdim=True)) * s["scale"]
                dq[:, a:b] = torch.bmm(t, kk)
                dk[:, lo:b] += torch.bmm(t.mT, q[:, a:b])
    r = {"out": out.permute(1, 0, 2), "lse": lse}
    if c["train"]:
        shared = lambda x: x.view(HK, -1, T, D).sum(1).permute(1, 0, 2)  # noqa: E731
        r.update(dq=dq.permute(1, 0, 2), dk=shared(dk), dv=shared(dv))
    return r
