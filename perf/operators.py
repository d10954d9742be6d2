"""The operators that turn prompts into caption features, as a caller uses them one by one.

A caption reaches the image model as features of a causal transformer over its tokens.
Four operators of that transformer's layer are measured here:

  rope_table        cos / sin tables of scaled rotary positions
  qk_norm_rope      per-head RMSNorm of queries and keys and the rotation, in one pass
  prompt_attention  causal attention over packed sequences with grouped heads, over whole
                    prompts, over the new part of a kept prefix, and for single tokens
  linear            a . W^T with bias, activation and residual in the epilogue

`own` selects between the plain torch form of an operator (fp32, fp64 for angles) and the
library's call.
"""
import math
import random

import torch

own = False

# projections of a caption encoder: width 2560, 32 query and 8 key heads of 128, hidden 9728;
# of the image model: width 3840, hidden 10240
CAP_WIDTH, CAP_HIDDEN, WIDTH, HIDDEN = 2560, 9728, 3840, 10240


def listed():
    return [
        # ---- scaled rotary tables
        # a cond / uncond pair of captions, plain frequencies: latency
        dict(name="rope caption pair", op="rope_table", tokens=133, rotary_dim=128, theta=1e6, kind="none",
             factor=1.0, first=0),
        # a long document at positions far past the trained length, frequencies scaled by parts
        dict(name="rope long by parts", op="rope_table", tokens=32768, rotary_dim=128, theta=1e6, kind="yarn",
             factor=4.0, first=98304),
        # ---- query / key norm and rotation
        # the caption pair's projection rows in fp32, halves rotated
        dict(name="qk caption pair", op="qk_norm_rope", tokens=133, kv_heads=8, group=4, head_dim=128,
             rotary_dim=128, layout="half", src="fp32", norm=True),
        # a long prompt in bf16, a quarter of each head rotated in pairs, odd token count
        dict(name="qk long partial", op="qk_norm_rope", tokens=16381, kv_heads=8, group=4, head_dim=128,
             rotary_dim=32, layout="interleaved", src="bf16", norm=True),
        # ---- attention
        # cond caption and empty uncond caption: latency
        dict(name="attn caption pair", op="prompt_attention", kind="prompt", batch=2, tokens=133, longest=0,
             kv_heads=8, group=4, head_dim=128, causal=True, lens=3),
        # a batch of captions of very different lengths, packed
        dict(name="attn caption batch", op="prompt_attention", kind="prompt", batch=24, tokens=4237, longest=0,
             kv_heads=8, group=4, head_dim=128, causal=True, lens=5),
        # one long prompt
        dict(name="attn long prompt", op="prompt_attention", kind="prompt", batch=1, tokens=16384, longest=0,
             kv_heads=8, group=4, head_dim=128, causal=True, lens=1),
        # the prompt's own words after a kept instruction prefix: few rows, narrow heads, odd group
        dict(name="attn after prefix", op="prompt_attention", kind="suffix", batch=3, tokens=111, longest=4099,
             kv_heads=4, group=6, head_dim=64, causal=True, lens=7),
        # one new token for each of 8 sequences, caches of a few thousand rows
        dict(name="attn single tokens", op="prompt_attention", kind="decode", batch=8, tokens=8, longest=8191,
             kv_heads=8, group=4, head_dim=128, causal=True, lens=9),
        # ---- projections
        # one token of each of 5 sequences through the output projection onto the fp32 stream
        dict(name="linear few rows", op="linear", m=5, n=CAP_WIDTH, k=4096, act="none", bias=False,
             residual="fp32", out="fp32"),
        # a caption pair through the first feed-forward matrix
        dict(name="linear caption pair", op="linear", m=133, n=CAP_HIDDEN, k=CAP_WIDTH, act="silu", bias=True,
             residual="none", out="bf16"),
        # the image model's joint sequence through its down projection, bf16 residual
        dict(name="linear joint rows", op="linear", m=8351, n=WIDTH, k=HIDDEN, act="gelu_tanh", bias=True,
             residual="bf16", out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_table", "qk_norm_rope", "prompt_attention", "prompt_attention", "linear", "linear"])
    if op == "rope_table":
        return dict(op=op, tokens=_log_int(rng, 1, 32768), rotary_dim=rng.choice([32, 64, 96, 128]),
                    theta=rng.choice([1e4, 5e5, 1e6]), kind=rng.choice(["none", "linear", "ntk", "yarn"]),
                    factor=rng.choice([2.0, 4.0, 8.0]), first=rng.randrange(0, 100000))
    if op == "qk_norm_rope":
        hd = rng.choice([64, 80, 128, 256])
        kvh, g = rng.choice([(1, 8), (2, 7), (8, 4), (5, 3), (16, 1)])
        rot = rng.choice([hd, hd // 2, hd // 4])
        return dict(op=op, tokens=_log_int(rng, 1, 8192), kv_heads=kvh, group=g, head_dim=hd, rotary_dim=rot,
                    layout=rng.choice(["half", "interleaved"]), src=rng.choice(["fp32", "bf16"]),
                    norm=rng.random() < 0.75)
    if op == "prompt_attention":
        kind = rng.choice(["prompt", "suffix", "decode"])
        kvh, g = rng.choice([(8, 4), (4, 6), (2, 8), (1, 7), (8, 1), (4, 3)])
        c = dict(op=op, kind=kind, kv_heads=kvh, group=g, head_dim=rng.choice([64, 128]), causal=True,
                 lens=rng.randrange(1 << 20))
        if kind == "prompt":
            c.update(batch=_log_int(rng, 1, 32), longest=0, causal=rng.random() < 0.8)
            c["tokens"] = _log_int(rng, 2 * c["batch"], 12000)
        elif kind == "suffix":
            c.update(batch=rng.randint(1, 8), longest=_log_int(rng, 64, 12000))
            c["tokens"] = _log_int(rng, 2 * c["batch"], 700)
        else:
            c.update(batch=_log_int(rng, 1, 48), longest=_log_int(rng, 8, 16000))
            c["tokens"] = c["batch"]
        return c
    while True:
        c = dict(op=op, m=_log_int(rng, 1, 8192), n=_log_int(rng, 64, 10240), k=_log_int(rng, 64, 10240),
                 act=rng.choice(["none", "silu", "gelu", "gelu_tanh"]), bias=rng.random() < 0.5,
                 residual=rng.choice(["none", "fp32", "bf16"]), out=rng.choice(["fp32", "bf16"]))
        if c["m"] * c["n"] * c["k"] < 1.5e11:
            return c


# ------------------------------------------------------------------------------ lengths
def _lengths(case):
    """(q_len, kv_len) of a prompt_attention case: ragged, summing to `tokens` new rows."""
    r = random.Random(case["lens"])
    B, T = case["batch"], case["tokens"]
    if case["kind"] == "decode":
        q = [1] * B
    else:
        cuts = [r.expovariate(1.0) + 0.05 for _ in range(B)]
        q = [1 + int((T - B) * c / sum(cuts)) for c in cuts]
        q[0] += T - sum(q)
    if case["kind"] == "prompt":
        return q, list(q)
    kv = [max(n, int(case["longest"] * r.uniform(0.3, 1.0))) for n in q]
    kv[-1] = max(q[-1], case["longest"])
    return q, kv


def _rope_pairs(case):
    return case["rotary_dim"] // 2


ORIGINAL_LEN = 32768  # trained length that `yarn` scales from
BETA_FAST, BETA_SLOW = 32.0, 1.0


def _attn_scale(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["kind"] == "yarn" else 1.0


# ------------------------------------------------------------------------------ inputs
def _rand(gen, *shape, dtype=torch.bfloat16, scale=1.0):
    x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
    return x.mul_(scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op == "rope_table":
        T = case["tokens"]
        # positions of a batch of documents: runs of consecutive tokens, each from its own offset
        off = torch.randint(0, 4096, (1,), generator=gen, device="cuda")
        s["pos"] = (torch.arange(T, device="cuda") + case["first"] + off).to(torch.int32)
        s["cos"] = torch.empty(T, _rope_pairs(case), device="cuda")
        s["sin"] = torch.empty_like(s["cos"])
    elif op == "qk_norm_rope":
        T, kvh, hd = case["tokens"], case["kv_heads"], case["head_dim"]
        H = kvh * case["group"]
        dt = torch.float32 if case["src"] == "fp32" else torch.bfloat16
        # one row of the projection per token: q | k | v
        s["qkv"] = _rand(gen, T, (H + 2 * kvh) * hd, dtype=dt, scale=3.0)
        s["q"] = s["qkv"][:, :H * hd].view(T, H, hd)
        s["k"] = s["qkv"][:, H * hd:(H + kvh) * hd].view(T, kvh, hd)
        s["w_q"] = 1.0 + 0.2 * _rand(gen, hd, dtype=torch.float32) if case["norm"] else None
        s["w_k"] = 1.0 + 0.2 * _rand(gen, hd, dtype=torch.float32) if case["norm"] else None
        P = _rope_pairs(case)
        ang = torch.arange(T, device="cuda", dtype=torch.float64)[:, None] * 1e6 ** (
            -torch.arange(P, device="cuda", dtype=torch.float64) / P)
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        s["q_out"] = torch.empty(T, H, hd, device="cuda", dtype=torch.bfloat16)
        s["k_out"] = torch.empty(T, kvh, hd, device="cuda", dtype=torch.bfloat16)
    elif op == "prompt_attention":
        kvh, hd = case["kv_heads"], case["head_dim"]
        H = kvh * case["group"]
        q_len, kv_len = _lengths(case)
        T = sum(q_len)
        s["q_len"], s["kv_len"] = q_len, kv_len
        if case["kind"] == "prompt":
            # rows of the packed projection
            qkv = _rand(gen, T, (H + 2 * kvh) * hd)
            s["q"] = qkv[:, :H * hd].view(T, H, hd)
            s["k"] = qkv[:, H * hd:(H + kvh) * hd].view(T, kvh, hd)
            s["v"] = qkv[:, (H + kvh) * hd:].view(T, kvh, hd)
            s["kv_start"] = [sum(kv_len[:b]) for b in range(len(kv_len))]
            starts = None
        else:
            # a cache with one slot of fixed capacity per sequence
            cap = (max(kv_len) + 63) // 64 * 64
            s["q"] = _rand(gen, T, H, hd)
            s["k"] = _rand(gen, len(kv_len) * cap, kvh, hd)
            s["v"] = _rand(gen, len(kv_len) * cap, kvh, hd)
            s["kv_start"] = starts = [b * cap for b in range(len(kv_len))]
        s["o"] = torch.empty(T, H, hd, device="cuda", dtype=torch.bfloat16)
        if own:
            import stream_diffusion_transformer_s3_b200 as Z
            s["batch"] = Z.PromptBatch(q_len, None if case["kind"] == "prompt" else kv_len, starts)
            need = Z.prompt_attention_workspace_bytes(s["batch"], H, kvh, hd, causal=case["causal"])
            s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    else:
        m, n, k = case["m"], case["n"], case["k"]
        kp = (k + 7) // 8 * 8  # rows start at multiples of 16 bytes
        s["a"] = _rand(gen, m, kp)[:, :k]
        s["w"] = _rand(gen, n, kp, scale=1.0 / math.sqrt(k))[:, :k]
        s["bias"] = _rand(gen, n, dtype=torch.float32, scale=0.5) if case["bias"] else None
        dt = {"fp32": torch.float32, "bf16": torch.bfloat16}
        s["residual"] = _rand(gen, m, n, dtype=dt[case["residual"]], scale=4.0) if case["residual"] != "none" else None
        s["out"] = torch.empty(m, n, device="cuda", dtype=dt[case["out"]])
    return s


# ------------------------------------------------------------------------------ plain forms
def _plain_rope_table(s):
    c = s["case"]
    d, f = c["rotary_dim"], c["factor"]
    i = torch.arange(d // 2, device="cuda", dtype=torch.float64)
    base = c["theta"] * f ** (d / (d - 2)) if c["kind"] == "ntk" else c["theta"]
    w = base ** (-2.0 * i / d)
    if c["kind"] == "linear":
        w = w / f
    elif c["kind"] == "yarn":
        turns = ORIGINAL_LEN * w / (2 * math.pi)
        keep = ((turns - BETA_SLOW) / (BETA_FAST - BETA_SLOW)).clamp(0.0, 1.0)
        w = w * keep + w / f * (1 - keep)
    ang = s["pos"].double()[:, None] * w
    m = _attn_scale(c)
    return {"cos": (ang.cos() * m).float(), "sin": (ang.sin() * m).float()}


def _plain_norm_rotate(x, w, cos, sin, layout, rot, eps=1e-6):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w
    y = x.clone()
    cos, sin = cos[:, None, :], sin[:, None, :]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if layout == "interleaved" else (x[..., :rot // 2], x[..., rot // 2:rot])
    p, q = a * cos - b * sin, a * sin + b * cos
    if layout == "interleaved":
        y[..., 0:rot:2], y[..., 1:rot:2] = p, q
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = p, q
    return y.to(torch.bfloat16)


def _plain_attention(s):
    c = s["case"]
    kvh, g, hd = c["kv_heads"], c["group"], c["head_dim"]
    o, t0 = s["o"], 0
    for n, m, k0 in zip(s["q_len"], s["kv_len"], s["kv_start"]):
        k = s["k"][k0:k0 + m].float().permute(1, 2, 0)  # [kvh, hd, m]
        v = s["v"][k0:k0 + m].float().permute(1, 0, 2)  # [kvh, m, hd]
        key = torch.arange(m, device="cuda")
        for r0 in range(0, n, 2048):  # rows at a time, so that the scores fit
            r1 = min(n, r0 + 2048)
            q = s["q"][t0 + r0:t0 + r1].float().view(r1 - r0, kvh, g, hd).permute(1, 2, 0, 3)
            x = torch.matmul(q.reshape(kvh, -1, hd), k).view(kvh, g, r1 - r0, m).mul_(1.0 / math.sqrt(hd))
            if c["causal"]:
                last = torch.arange(r0, r1, device="cuda") + (m - n)
                x.masked_fill_(key[None, :] > last[:, None], -math.inf)
            x.sub_(x.amax(-1, keepdim=True)).exp_()
            y = torch.matmul(x.view(kvh, -1, m), v).view(kvh, g, r1 - r0, hd) / x.sum(-1, keepdim=True)
            o[t0 + r0:t0 + r1] = y.permute(2, 0, 1, 3).reshape(r1 - r0, kvh * g, hd).to(o.dtype)
        t0 += n
    return {"o": o}


def _plain_linear(s):
    c = s["case"]
    y = torch.matmul(s["a"].float(), s["w"].float().t())
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    elif c["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    elif c["act"] == "gelu_tanh":
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"out": y.to(s["out"].dtype)}


# ------------------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "rope_table":
            return _plain_rope_table(s)
        if op == "qk_norm_rope":
            return {"q": _plain_norm_rotate(s["q"], s["w_q"], s["cos"], s["sin"], c["layout"], c["rotary_dim"]),
                    "k": _plain_norm_rotate(s["k"], s["w_k"], s["cos"], s["sin"], c["layout"], c["rotary_dim"])}
        return _plain_attention(s) if op == "prompt_attention" else _plain_linear(s)
    import stream_diffusion_transformer_s3_b200 as Z
    if op == "rope_table":
        kind = {"none": Z.ROPE_SCALE_NONE, "linear": Z.ROPE_SCALE_LINEAR, "ntk": Z.ROPE_SCALE_NTK,
                "yarn": Z.ROPE_SCALE_YARN}[c["kind"]]
        Z.zdit_rope_table_scaled(s["pos"], c["rotary_dim"], c["theta"], s["cos"], s["sin"],
                                 Z.RopeScaling(kind, c["factor"], ORIGINAL_LEN, BETA_FAST, BETA_SLOW, _attn_scale(c)))
        return {"cos": s["cos"], "sin": s["sin"]}
    if op == "qk_norm_rope":
        layout = Z.ROPE_HALF if c["layout"] == "half" else Z.ROPE_INTERLEAVED
        Z.zdit_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["w_q"], s["w_k"], s["cos"], s["sin"],
                            c["rotary_dim"], layout, eps=1e-6)
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "prompt_attention":
        Z.zdit_prompt_attention(s["q"], s["k"], s["v"], s["o"], s["batch"], s["ws"], causal=c["causal"])
        return {"o": s["o"]}
    act = {"none": Z.ACT_NONE, "silu": Z.ACT_SILU, "gelu": Z.ACT_GELU, "gelu_tanh": Z.ACT_GELU_TANH}[c["act"]]
    Z.zdit_linear(s["a"], s["w"], s["out"], bias=s["bias"], act=act, residual=s["residual"])
    return {"out": s["out"]}


# ------------------------------------------------------------------------------ floors
def work(case):
    op = case["op"]
    if op == "rope_table":
        n = case["tokens"] * _rope_pairs(case)
        return {"bytes": 8.0 * n + 4.0 * case["tokens"], "flops": 10.0 * n}
    if op == "qk_norm_rope":
        rows = case["tokens"] * case["kv_heads"] * (case["group"] + 1)
        size = 4.0 if case["src"] == "fp32" else 2.0
        return {"bytes": rows * case["head_dim"] * (size + 2.0) + 8.0 * case["tokens"] * _rope_pairs(case),
                "flops": 7.0 * rows * case["head_dim"]}
    if op == "prompt_attention":
        q_len, kv_len = _lengths(case)
        H, hd = case["kv_heads"] * case["group"], case["head_dim"]
        if case["causal"]:
            pairs = sum(n * (m - n) + n * (n + 1) / 2 for n, m in zip(q_len, kv_len))
        else:
            pairs = sum(n * m for n, m in zip(q_len, kv_len))
        return {"bytes": 2.0 * hd * (2 * H * sum(q_len) + 2 * case["kv_heads"] * sum(kv_len)),
                "flops": 4.0 * hd * H * pairs}
    m, n, k = case["m"], case["n"], case["k"]
    size = {"fp32": 4.0, "bf16": 2.0, "none": 0.0}
    return {"bytes": 2.0 * k * (m + n) + m * n * (size[case["out"]] + size[case["residual"]]) + 4.0 * n * case["bias"],
            "flops": 2.0 * m * n * k}


# ------------------------------------------------------------------------------ definitions in 64 bits
def _exact_freq(case):
    d, w = case["rotary_dim"], []
    for i in range(d // 2):
        f = 1.0 / case["theta"] ** (2 * i / d)
        if case["kind"] == "linear":
            f /= case["factor"]
        if case["kind"] == "ntk":
            f = 1.0 / (case["theta"] * case["factor"] ** (d / (d - 2))) ** (2 * i / d)
        if case["kind"] == "yarn":
            length = 2 * math.pi / f  # wavelength in tokens
            ramp = min(1.0, max(0.0, (ORIGINAL_LEN / length - BETA_SLOW) / (BETA_FAST - BETA_SLOW)))
            f = (1.0 - ramp) * f / case["factor"] + ramp * f
        w.append(f)
    return torch.tensor(w, dtype=torch.float64, device="cuda")


def _exact_heads(x, w, cos, sin, case):
    x = x.to(torch.float64)
    if w is not None:
        x = x / x.square().mean(dim=2, keepdim=True).add(1e-6).sqrt() * w.to(torch.float64)
    rot = case["rotary_dim"]
    z = x[:, :, :rot].reshape(x.shape[0], x.shape[1], -1, 2) if case["layout"] == "interleaved" else \
        x[:, :, :rot].reshape(x.shape[0], x.shape[1], 2, -1).transpose(2, 3)
    turn = torch.complex(cos.to(torch.float64), sin.to(torch.float64)).unsqueeze(1)
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
    if case["layout"] != "interleaved":
        z = z.transpose(2, 3)
    return torch.cat([z.reshape(x.shape[0], x.shape[1], rot), x[:, :, rot:]], dim=2)


def _exact_attention(s):
    c = s["case"]
    g, hd = c["group"], c["head_dim"]
    out = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for n, m, start in zip(s["q_len"], s["kv_len"], s["kv_start"]):
        for h in range(out.shape[1]):
            q = s["q"][first:first + n, h].to(torch.float64)
            k = s["k"][start:start + m, h // g].to(torch.float64)
            v = s["v"][start:start + m, h // g].to(torch.float64)
            logits = (q @ k.T) / hd ** 0.5
            if c["causal"]:
                seen = torch.ones(n, m, dtype=torch.bool, device="cuda").tril(m - n)
                logits = torch.where(seen, logits, torch.full_like(logits, -math.inf))
            out[first:first + n, h] = torch.exp(logits - torch.logsumexp(logits, 1, keepdim=True)) @ v
        first += n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope_table":
        ang = torch.outer(s["pos"].to(torch.float64), _exact_freq(case))
        return {"cos": torch.cos(ang) * _attn_scale(case), "sin": torch.sin(ang) * _attn_scale(case)}
    if op == "qk_norm_rope":
        return {"q": _exact_heads(s["q"], s["w_q"], s["cos"], s["sin"], case),
                "k": _exact_heads(s["k"], s["w_k"], s["cos"], s["sin"], case)}
    if op == "prompt_attention":
        return {"o": _exact_attention(s)}
    y = s["a"].to(torch.float64) @ s["w"].to(torch.float64).T
    if s["bias"] is not None:
        y += s["bias"].to(torch.float64)
    if case["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif case["act"] == "gelu":
        y = y * 0.5 * torch.special.erfc(-y / 2 ** 0.5)
    elif case["act"] == "gelu_tanh":
        y = y * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (y + 0.044715 * y ** 3))
    if s["residual"] is not None:
        y = y + s["residual"].to(torch.float64)
    return {"out": y}
