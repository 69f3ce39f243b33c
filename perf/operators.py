"""The operators of a transformer block over packed tokens: inputs, plain forms, exact values and work.

Three operators, as `flow_matching_dit_b200` offers them:

- linear:         out = act(x W^T + bias) + residual
- norm_residual:  h' = residual_scale h + gate * post(y);  u = pre(h') (1 + scale) + shift
- attention:      softmax(scale q k^T) v of packed sequences of different lengths, grouped heads, causal or not

Where `own` is false `run` computes them with elementary torch operations in 32 bits, rounded once at the end;
where it is true it calls the library.
"""

import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------------------- cases

def _linear(name, m, n, k, act, out, bias=True, residual=False):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "act": act, "out": out, "bias": bias,
            "residual": residual}


def _norm(name, rows, dim, stream, out, post, pre, gate, mod, groups, residual_scale=1.0):
    return {"name": name, "op": "norm", "rows": rows, "dim": dim, "stream": stream, "out": out, "post": post,
            "pre": pre, "gate": gate, "mod": mod, "groups": groups, "residual_scale": residual_scale}


def _attention(name, kind, batch, q, k, heads, kv_heads, dim, causal, spread, lens):
    return {"name": name, "op": "attention", "kind": kind, "batch": batch, "q": q, "k": k, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "causal": causal, "spread": spread, "lens": lens}


def listed():
    return [
        # one token through a block's first feed-forward product: weights are all there is to read
        _linear("linear one token", 1, 4096, 1024, "gelu", "bf16"),
        # eight samples of 17 tokens, the second feed-forward product added to the f32 residual stream
        _linear("linear 8 samples", 136, 1024, 4096, "none", "f32", residual=True),
        # a few prompts' tokens, a width that no tile divides, residual in bf16
        _linear("linear ragged prompts", 1237, 2056, 1096, "silu", "bf16", residual=True),
        # the tokens of 64 prompts through a wide feed-forward product
        _linear("linear many prompts", 16384, 8192, 2048, "gelu", "bf16"),
        # one sample's 17 tokens between two blocks: latency
        _norm("norm one sample", 17, 1024, "f32", "bf16", "none", "layer", "group", True, 1),
        # the action head's rows at 256 samples, each sample with its own modulation and gate
        _norm("norm 256 samples", 4352, 1024, "f32", "bf16", "none", "layer", "group", True, 256),
        # norms on both sides of a block, a width that no vector divides, everything in bf16
        _norm("norm odd width", 2999, 1337, "bf16", "bf16", "rms", "rms", "channel", False, 1, 0.70710678),
        # the tokens of 256 prompts between two blocks, sandwich norms on an f32 stream
        _norm("norm many prompts", 65536, 2048, "f32", "bf16", "rms", "rms", "none", False, 1),
        # 32 prompts of 200 to 600 tokens, packed, q, k and v slices of one product's output
        _attention("attention prompts", "prompt", 32, 600, 600, 16, 8, 128, True, 0.34, 1),
        # two long prompts
        _attention("attention long prompts", "prompt", 2, 8192, 8192, 16, 8, 128, True, 1.0, 2),
        # the next token of 48 sequences over slots of a cache
        _attention("attention next token", "token", 48, 1, 4096, 16, 4, 128, True, 0.1, 3),
        # image patches, every token sees every token of its image, a head width of 72
        _attention("attention images", "prompt", 24, 256, 256, 16, 16, 72, False, 0.5, 4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "norm", "attention"])
    if op == "linear":
        while True:
            m, n, k = _log(rng, 1, 16384), _log(rng, 16, 8192), 8 * _log(rng, 1, 1024)
            if m * n * k <= 16384 * 8192 * 2048:
                break
        c = _linear("", m, n, k, rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                    rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.7, rng.random() < 0.5)
    elif op == "norm":
        while True:
            rows, dim = _log(rng, 1, 65536), _log(rng, 8, 8192)
            if rows * dim <= 65536 * 2048:
                break
        groups = rng.choice([1, 1, min(rows, rng.randint(2, 256))])
        c = _norm("", rows, dim, rng.choice(["f32", "bf16"]), rng.choice(["bf16", "f32"]),
                  rng.choice(["none", "layer", "rms"]), rng.choice(["layer", "rms"]),
                  rng.choice(["none", "channel", "group"]), rng.random() < 0.5, groups,
                  rng.choice([1.0, rng.uniform(0.25, 1.5)]))
    else:
        kind = rng.choice(["prompt", "prompt", "chunk", "token"])
        while True:
            kv_heads = rng.choice([1, 2, 4, 8, 16])
            heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
            dim = rng.choice([32, 64, 64, 72, 80, 96, 128, 128, 128])
            batch, k = _log(rng, 1, 64), _log(rng, 1, 8192)
            q = k if kind == "prompt" else 1 if kind == "token" else _log(rng, 1, k)
            if heads <= 32 and batch * heads * q * k <= 2 * 16 * 8192 * 4096 and batch * k * kv_heads * dim <= 1 << 28:
                break
        c = _attention("", kind, batch, q, k, heads, kv_heads, dim, kind != "prompt" or rng.random() < 0.7,
                       rng.choice([0.0, 0.3, 0.9, 1.0]), rng.randint(0, 1 << 20))
    del c["name"]
    return c


def _lengths(case):
    """(query lengths, key lengths) of the sequences: between `spread` times the longest and the longest, the first one longest."""
    r = np.random.RandomState(case["lens"])
    b, most = case["batch"], case["k"]
    k = r.randint(int(case["spread"] * most), most + 1, b).astype(np.int64)
    k[0] = most
    if case["kind"] == "prompt":
        return k, k
    q = np.minimum(k, r.randint(int(case["spread"] * case["q"]), case["q"] + 1, b) if case["kind"] == "chunk" else 1)
    q[0] = case["q"]
    return q.astype(np.int64), k


# ---------------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEVICE, dtype=dtype).mul_(std)

    bf16 = torch.bfloat16
    if case["op"] == "linear":
        m, n, k, out = case["m"], case["n"], case["k"], DTYPES[case["out"]]
        return {"case": case, "x": normal(m, k, dtype=bf16), "w": normal(n, k, std=k ** -0.5, dtype=bf16),
                "bias": normal(n, std=0.1) if case["bias"] else None,
                "residual": normal(m, n, dtype=out) if case["residual"] else None}
    if case["op"] == "norm":
        rows, dim, groups = case["rows"], case["dim"], case["groups"]
        s = {"case": case, "h": normal(rows, dim, dtype=DTYPES[case["stream"]]) * 3 + 0.25,
             "y": normal(rows, dim, dtype=bf16), "post_gain": None, "post_bias": None, "gate": None, "scale": None,
             "shift": None, "row_group": None}
        if case["post"] != "none":
            s["post_gain"] = 1 + normal(dim, std=0.1)
            s["post_bias"] = normal(dim, std=0.1) if case["post"] == "layer" else None
        if case["gate"] != "none":
            s["gate"] = normal(*([groups] if case["gate"] == "group" else []), dim, std=0.5)
        if case["mod"]:
            s["scale"], s["shift"] = normal(groups, dim, std=0.2), normal(groups, dim, std=0.2)
        s["pre_gain"] = 1 + normal(dim, std=0.1)
        s["pre_bias"] = normal(dim, std=0.1) if case["pre"] == "layer" else None
        if groups > 1:   # rows of a sample are neighbours
            s["row_group"] = (torch.arange(rows, device=DEVICE) * groups // rows).to(torch.int32)
        return s
    ql, kl = _lengths(case)
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    s = {"case": case, "max_q": int(ql.max()), "max_k": int(kl.max()), "k_len": None}
    start = np.zeros(len(ql) + 1, np.int32)
    start[1:] = np.cumsum(ql)
    s["cu_q"] = torch.from_numpy(start).to(DEVICE)
    if case["kind"] == "prompt":   # slices of the output of one product
        qkv = normal(int(ql.sum()), heads + 2 * kv_heads, dim, dtype=bf16)
        s["q"], s["k"], s["v"] = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
        s["cu_k"] = s["cu_q"]
        return s
    # a cache with a slot of the longest length for each sequence
    slot, b = case["k"], len(kl)
    s["q"] = normal(int(ql.sum()), heads, dim, dtype=bf16)
    s["k"], s["v"] = normal(b * slot, kv_heads, dim, dtype=bf16), normal(b * slot, kv_heads, dim, dtype=bf16)
    s["cu_k"] = torch.arange(0, (b + 1) * slot, slot, dtype=torch.int32, device=DEVICE)
    s["k_len"] = torch.from_numpy(kl.astype(np.int32)).to(DEVICE)
    return s


# ---------------------------------------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    if own:
        return _call(c, s)
    return {"linear": _plain_linear, "norm": _plain_norm, "attention": _plain_attention}[c["op"]](c, s)


def _call(c, s):
    import flow_matching_dit_b200 as gdit
    if c["op"] == "linear":
        return gdit.linear(s["x"], s["w"], s["bias"], activation=c["act"], residual=s["residual"],
                           out_dtype=DTYPES[c["out"]])
    if c["op"] == "norm":
        return gdit.norm_residual(s["h"], s["y"], post=c["post"], post_gain=s["post_gain"], post_bias=s["post_bias"],
                                  gate=s["gate"], residual_scale=c["residual_scale"], pre=c["pre"],
                                  pre_gain=s["pre_gain"], pre_bias=s["pre_bias"], scale=s["scale"], shift=s["shift"],
                                  row_group=s["row_group"], eps=1e-5, u_dtype=DTYPES[c["out"]])
    return gdit.attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], max_q=s["max_q"], max_k=s["max_k"],
                          causal=c["causal"], k_len=s["k_len"], return_lse=True)


def _plain_linear(c, s):
    v = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        v = v + s["bias"]
    if c["act"] == "relu":
        v = v.clamp_min(0)
    elif c["act"] == "gelu":
        v = 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    elif c["act"] == "gelu_tanh":
        v = 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    elif c["act"] == "silu":
        v = v * torch.sigmoid(v)
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(DTYPES[c["out"]])


def _plain_normed(x, kind, gain, bias):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5) * gain
    return x if bias is None else x + bias


def _plain_norm(c, s):
    def rows_of(t):
        return t if t is None or t.dim() == 1 else t[0] if t.shape[0] == 1 else t[s["row_group"].long()]

    y = _plain_normed(s["y"].float(), c["post"], s["post_gain"], s["post_bias"])
    gate = rows_of(s["gate"])
    h = s["h"].float() * c["residual_scale"] + (y if gate is None else y * gate)
    u = _plain_normed(h, c["pre"], s["pre_gain"], s["pre_bias"])
    if s["scale"] is not None:
        u = u * (1 + rows_of(s["scale"])) + rows_of(s["shift"])
    return h.to(DTYPES[c["stream"]]), u.to(DTYPES[c["out"]])


def _plain_attention(c, s):
    """Every sequence padded to the longest, one batched product for the scores and one for the values."""
    q, k, v, cu_q, cu_k = s["q"], s["k"], s["v"], s["cu_q"].long(), s["cu_k"].long()
    kv_heads, group, dim = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"]
    q_len, k_len = cu_q[1:] - cu_q[:-1], s["k_len"].long() if s["k_len"] is not None else cu_k[1:] - cu_k[:-1]
    i = torch.arange(s["max_q"], device=q.device)
    j = torch.arange(s["max_k"], device=q.device)
    at_q = (cu_q[:-1, None] + i).clamp_max(q.shape[0] - 1)
    at_k = (cu_k[:-1, None] + j).clamp_max(k.shape[0] - 1)
    qp = q[at_q].float().reshape(len(q_len), s["max_q"], kv_heads, group, dim).permute(0, 2, 3, 1, 4)
    kp, vp = k[at_k].float().permute(0, 2, 3, 1), v[at_k].float().permute(0, 2, 1, 3)
    b = len(q_len)
    a = (qp.reshape(b, kv_heads, group * s["max_q"], dim) @ kp).mul_(dim ** -0.5)
    a = a.view(b, kv_heads, group, s["max_q"], s["max_k"])
    seen = (j < k_len[:, None])[:, None, :]
    if c["causal"]:   # the last query sees every key
        seen = seen & (j[None, None] <= (i[None, :] + (k_len - q_len)[:, None])[:, :, None])
    a.masked_fill_(~seen[:, None, None], -math.inf)
    top = a.amax(-1, keepdim=True).clamp_min(-3e38)
    a.sub_(top).exp_()
    total = a.sum(-1, keepdim=True)
    o = (a.view(b, kv_heads, group * s["max_q"], s["max_k"]) @ vp).view(b, kv_heads, group, s["max_q"], dim)
    o = torch.where(total > 0, o / total, 0)
    lse = torch.where(total > 0, torch.log(total) + top, -math.inf)[..., 0]
    there = (i < q_len[:, None]).reshape(-1).nonzero()[:, 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(b * s["max_q"], c["heads"], dim)[there]
    lse = lse.permute(0, 3, 1, 2).reshape(b * s["max_q"], c["heads"])[there]
    return o.to(torch.bfloat16), lse


# ---------------------------------------------------------------------------------------------- work

def work(case):
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        size = 4 if case["out"] == "f32" else 2
        return {"bytes": 2 * (m * k + n * k) + 4 * n * case["bias"] + size * m * n * (2 if case["residual"] else 1),
                "flops": 2 * m * n * k}
    if case["op"] == "norm":
        rows, dim, groups = case["rows"], case["dim"], case["groups"]
        size = {"f32": 4, "bf16": 2}
        vectors = (1 + (case["pre"] == "layer") + (case["post"] != "none") + (case["post"] == "layer")
                   + (case["gate"] == "channel") + groups * (case["gate"] == "group") + 2 * groups * case["mod"])
        return {"bytes": rows * dim * (2 * size[case["stream"]] + 2 + size[case["out"]]) + 4 * dim * vectors
                + 4 * rows * (groups > 1), "flops": 20 * rows * dim}
    q, k = _lengths(case)
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    if case["causal"]:   # query i of a sequence sees k - q + 1 + i keys
        low = np.maximum(k - q, 0)
        pairs = np.where(k >= q, q * low + q * (q + 1) // 2, k * (k + 1) // 2).sum()
    else:
        pairs = (q * k).sum()
    read = np.where(q > 0, k, 0).sum()
    return {"bytes": int(q.sum()) * heads * (2 * 2 * dim + 4) + int(read) * kv_heads * 2 * 2 * dim,
            "flops": 4 * dim * heads * int(pairs)}


# ---------------------------------------------------------------------------------------------- exact values

def exact(case, seed):
    """What run(prepare(case, seed)) returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_linear(case, s)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    return _exact_attention(case, s)


def _exact_linear(c, s):
    x, w = s["x"].double(), s["w"].double()
    z = torch.einsum("mk,nk->mn", x, w)
    if c["bias"]:
        z += s["bias"].double()
    if c["act"] == "relu":
        z = torch.where(z > 0, z, torch.zeros_like(z))
    elif c["act"] == "gelu":
        z = z * torch.erfc(-z / math.sqrt(2)) / 2
    elif c["act"] == "gelu_tanh":   # (1 + tanh a) / 2 = 1 / (1 + exp(-2 a))
        z = z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    elif c["act"] == "silu":
        z = z / (1 + torch.exp(-z))
    return z + s["residual"].double() if c["residual"] else z


def _exact_norm(c, s):
    def up(name):
        return None if s[name] is None else s[name].double()

    def norm(t, kind, gain, bias):
        if kind == "none":
            return t
        mean = t.sum(1, keepdim=True) / t.shape[1] if kind == "layer" else 0.0
        var = ((t - mean) ** 2).sum(1, keepdim=True) / t.shape[1]
        r = (t - mean) / torch.sqrt(var + 1e-5) * gain
        return r if bias is None else r + bias

    group = torch.zeros(c["rows"], dtype=torch.long, device=DEVICE) if s["row_group"] is None else s["row_group"].long()
    branch = norm(up("y"), c["post"], up("post_gain"), up("post_bias"))
    if c["gate"] == "channel":
        branch = branch * up("gate")
    elif c["gate"] == "group":
        branch = branch * up("gate").index_select(0, group)
    stream = c["residual_scale"] * up("h") + branch
    u = norm(stream, c["pre"], up("pre_gain"), up("pre_bias"))
    if c["mod"]:
        u = u + u * up("scale").index_select(0, group) + up("shift").index_select(0, group)
    return stream, u


def _exact_attention(c, s):
    ql, kl = _lengths(c)
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    group, width = c["heads"] // c["kv_heads"], c["dim"]
    outs = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    lses = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEVICE)
    for b, (nq, nk) in enumerate(zip(ql.tolist(), kl.tolist())):
        if nq == 0:
            continue
        rows = slice(cu_q[b], cu_q[b] + nq)
        if nk == 0:
            lses[rows] = -math.inf
            continue
        last = torch.arange(nq, device=DEVICE)[:, None] + (nk - nq)
        hidden = torch.arange(nk, device=DEVICE)[None, :] > last if c["causal"] else None
        for kv in range(c["kv_heads"]):
            keys = s["k"][cu_k[b]:cu_k[b] + nk, kv].double()
            values = s["v"][cu_k[b]:cu_k[b] + nk, kv].double()
            for h in range(kv * group, (kv + 1) * group):
                z = s["q"][rows, h].double() @ keys.T / math.sqrt(width)
                if hidden is not None:
                    z.masked_fill_(hidden, -math.inf)
                lse = torch.logsumexp(z, 1)
                p = torch.exp(z - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
                outs[rows, h] = p @ values
                lses[rows, h] = lse
    return outs, lses
