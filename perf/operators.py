"""The operators of the paged 4-bit KV cache as cases that can be timed and compared: rotary positions,
appending rotated keys and values to the cache, reading it back, and attention over it.

`own` chooses the side: False runs the plain form (elementary torch operations in 32 bits, angles in
64), True makes the calls of `masked_block_diffusion_b200`. `exact` gives the definition in 64 bits.

The cache. A page holds `page` positions of one layer; per page, per K and V, per KV head and per
position it has head_dim / 2 code bytes and head_dim / 16 scale bytes:
  codes  uint8 [n_pages][2][n_kv_heads][page][head_dim / 2]
  scales uint8 [n_pages][2][n_kv_heads][page][head_dim / 16]
Sixteen consecutive dims share a scale byte s: five exponent and three mantissa bits, the upper bits
of a positive fp16 number. The value of a dim is scale * (code - 8). The eight codes of dims 8 w .. 8 w + 7
are one little-endian 32-bit word: dim 8 w + 2 j is nibble j, dim 8 w + 2 j + 1 is nibble j + 4.
"""

import math
import random

import torch

own = False

# The shapes are those of the repository's models: 16 query heads over 8 KV heads of 176 dims (the 26B
# MoE) and 16 over 4 of 64 dims (the small MoE), a 256-position canvas and a 4096-token prompt.


def listed():
    wide = {"heads": 16, "kv_heads": 8, "dim": 176, "page": 64}
    small = {"heads": 16, "kv_heads": 4, "dim": 64, "page": 32}
    return [
        # the queries of one token for each of 64 requests: latency counts
        {"name": "rope_64_tokens", "op": "rope", "tokens": 64, "heads": 16, "dim": 176, "rotary": 176, "layout": "half",
         "scaling": "none", "factor": 1.0, "far": 4352, "in": "f32", "out": "bf16", "transposed": False},
        # a long prompt's queries, half of each head rotated in the interleaved layout, positions beyond the
        # trained length
        {"name": "rope_long_prompt", "op": "rope", "tokens": 32768, "heads": 16, "dim": 64, "rotary": 32, "layout": "interleaved",
         "scaling": "yarn", "factor": 32.0, "far": 131072, "in": "bf16", "out": "bf16", "transposed": False},
        # one new token for each of 64 requests, out of a fused fp32 QKV projection
        {"name": "append_64_tokens", "op": "append", **wide, "batch": 64, "new": 1, "prefix": 4352, "pads": 0,
         "scaling": "none", "factor": 1.0, "in": "f32"},
        # three prompts of odd lengths, 4096 tokens the longest, with padding tokens between them
        {"name": "append_prompts", "op": "append", **wide, "batch": 3, "new": 4096, "prefix": 0, "pads": 37,
         "scaling": "none", "factor": 1.0, "in": "bf16"},
        # one canvas back as bf16
        {"name": "read_canvas", "op": "read", **small, "batch": 1, "length": 256},
        # the whole cache of 16 requests back as bf16, to hand it to another place
        {"name": "read_16_requests", "op": "read", **wide, "batch": 16, "length": 4352},
        # one token of one request over a prompt and a canvas
        {"name": "attend_token", "op": "attend", **wide, "batch": 1, "queries": 1, "keys": 4352, "causal": True},
        # one token for each of 64 requests of different lengths
        {"name": "attend_64_tokens", "op": "attend", **wide, "batch": 64, "queries": 1, "keys": 4352, "causal": True},
        # one token of two requests over a very long cache
        {"name": "attend_token_long", "op": "attend", **small, "batch": 2, "queries": 1, "keys": 131072, "causal": True},
        # one denoising pass's attention: a canvas that sees the prompt and itself
        {"name": "attend_canvas", "op": "attend", **wide, "batch": 1, "queries": 256, "keys": 4352, "causal": False},
        # the same for 16 requests with prompts of different lengths
        {"name": "attend_16_canvases", "op": "attend", **wide, "batch": 16, "queries": 256, "keys": 4352, "causal": False},
        # pieces of three prompts over what is cached of them
        {"name": "attend_prompt_pieces", "op": "attend", **small, "batch": 3, "queries": 1024, "keys": 4096, "causal": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attend", "attend", "attend"])
    kv = rng.choice([1, 2, 4, 8])
    shape = {"heads": kv * rng.choice([1, 2, 3, 4, 8] if kv < 8 else [1, 2, 4]), "kv_heads": kv, "dim": rng.choice([64, 128, 176]),
             "page": rng.choice([16, 32, 64, 128])}
    if op == "rope":
        dim = shape["dim"]
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return {"op": op, "tokens": _log(rng, 1, 16384), "heads": rng.randint(1, 16), "dim": dim, "rotary": rng.choice([dim, dim, dim // 2, 2 * rng.randint(2, dim // 2)]),
                "layout": rng.choice(["half", "interleaved"]), "scaling": scaling, "factor": 1.0 if scaling == "none" else float(rng.choice([2, 8, 32])),
                "far": _log(rng, 64, 1 << 20), "in": rng.choice(["f32", "bf16"]), "out": rng.choice(["f32", "bf16"]), "transposed": rng.random() < 0.25}
    if op == "append":
        new = _log(rng, 1, 4096)
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return {"op": op, **shape, "batch": _log(rng, 1, max(1, min(64, 8192 // new))), "new": new, "prefix": rng.choice([0, _log(rng, 1, 8192)]),
                "pads": rng.choice([0, rng.randint(1, 50)]), "scaling": scaling, "factor": 1.0 if scaling == "none" else 8.0,
                "in": rng.choice(["f32", "bf16"])}
    if op == "read":
        length = _log(rng, 1, 16384)
        return {"op": op, **shape, "batch": _log(rng, 1, max(1, min(64, 32768 // length))), "length": length}
    kind = rng.choice(["token", "canvas", "prompt"])
    if kind == "token":  # up to a few tokens at once, as a draft to verify has them
        keys = _log(rng, 1, 131072)
        return {"op": op, **shape, "batch": _log(rng, 1, max(1, min(64, 262144 // keys))), "queries": rng.choice([1, 1, 2, rng.randint(3, 8)]), "keys": keys, "causal": True}
    if kind == "canvas":
        keys = _log(rng, 256, 8192)
        return {"op": op, **shape, "batch": _log(rng, 1, max(1, min(16, 32768 // keys))), "queries": rng.choice([32, 256, 256]), "keys": keys, "causal": False}
    keys = _log(rng, 16, 4096)
    return {"op": op, **shape, "batch": rng.randint(1, 4), "queries": _log(rng, 9, 2048), "keys": keys, "causal": True}


def _lengths(case):
    """Queries and keys of each request, from the case alone: the first request is the longest, the others
    go down to half of it, and a piece of a prompt may be shorter than the longest."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = case["batch"]
    if case["op"] == "append":
        return [case["new"] if b == 0 else rng.randint((case["new"] + 1) // 2, case["new"]) for b in range(n)], \
               [case["prefix"] if b == 0 else rng.randint(case["prefix"] // 2, case["prefix"]) for b in range(n)]
    if case["op"] == "read":
        return None, [case["length"] if b == 0 else rng.randint((case["length"] + 1) // 2, case["length"]) for b in range(n)]
    keys = [case["keys"] if b == 0 else rng.randint((case["keys"] + 1) // 2, case["keys"]) for b in range(n)]
    pieces = case["queries"] > 8 and case["causal"]
    queries = [case["queries"] if b == 0 or not pieces else rng.randint((case["queries"] + 1) // 2, case["queries"]) for b in range(n)]
    return queries, keys


_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
_YARN = {"original_ctx": 4096, "beta_fast": 32.0, "beta_slow": 1.0}


def _rope_args(case):
    return {"rotary_dim": case.get("rotary", case["dim"]), "layout": case.get("layout", "half"), "theta": 10000.0,
            "scaling": case["scaling"], "factor": case["factor"], **(_YARN if case["scaling"] == "yarn" else {})}


def _table(lengths, page, g):
    """A page table over pages in random order, and how many pages the cache has (a few more than are used)."""
    per = [max(1, -(-n // page)) for n in lengths]
    total = sum(per) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    starts = torch.tensor([0] + per, device="cuda").cumsum(0)[:-1]
    at = torch.arange(max(per), device="cuda")
    idx = starts[:, None] + at[None, :]
    used = at[None, :] < torch.tensor(per, device="cuda")[:, None]
    return torch.where(used, order[idx.clamp(max=total - 1)], torch.zeros_like(idx, dtype=torch.int32)).to(torch.int32).contiguous(), total


def _cache(case, total, g, filled):
    """The packed arrays: for a filled cache, codes of normally distributed values and scales over two octaves."""
    codes_shape = (total, 2, case["kv_heads"], case["page"], case["dim"] // 2)
    scales_shape = (total, 2, case["kv_heads"], case["page"], case["dim"] // 16)
    if not filled:
        return torch.zeros(codes_shape, dtype=torch.uint8, device="cuda"), torch.zeros(scales_shape, dtype=torch.uint8, device="cuda")
    n = math.prod(codes_shape)
    codes = torch.empty(n, dtype=torch.uint8, device="cuda")
    step = 1 << 27
    for a in range(0, n, step):
        m = min(step, n - a)
        u = torch.empty((2, m), dtype=torch.float16, device="cuda").normal_(0.0, 2.5, generator=g).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
        codes[a:a + m] = u[0] | (u[1] << 4)
    scales = torch.randint(11 * 8, 13 * 8, scales_shape, dtype=torch.uint8, device="cuda", generator=g)
    return codes.view(codes_shape), scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dev = "cuda"
    op = case["op"]
    if op == "rope":
        s = {"case": case, "x": torch.randn((case["tokens"], case["heads"], case["dim"]), generator=g, device=dev).to(_DTYPE[case["in"]]),
             "pos": torch.randint(0, case["far"], (case["tokens"],), dtype=torch.int32, generator=g, device=dev)}
        s["rope_args"] = _rope_args(case)
    elif op == "append":
        new, prefix = _lengths(case)
        table, total = _table([a + b for a, b in zip(new, prefix)], case["page"], g)
        req, pos = [], []
        for b, (n, p) in enumerate(zip(new, prefix)):
            req += [b] * n + [-1] * case["pads"]
            pos += list(range(p, p + n)) + [0] * case["pads"]
        tokens = len(req)
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        qkv = torch.randn((tokens, h + 2 * hk, d), generator=g, device=dev)
        qkv *= torch.empty((h + 2 * hk, d), device=dev).log_normal_(0.0, 0.5, generator=g)  # channels differ in size
        codes, scales = _cache(case, total, g, False)
        s = {"case": case, "qkv": qkv.to(_DTYPE[case["in"]]), "req": torch.tensor(req, dtype=torch.int32, device=dev),
             "pos": torch.tensor(pos, dtype=torch.int32, device=dev), "table": table, "codes": codes, "scales": scales, "rope_args": _rope_args(case)}
    elif op == "read":
        _, lengths = _lengths(case)
        table, total = _table(lengths, case["page"], g)
        codes, scales = _cache(case, total, g, True)
        req = torch.repeat_interleave(torch.arange(len(lengths), device=dev), torch.tensor(lengths, device=dev)).to(torch.int32)
        pos = torch.cat([torch.arange(n, device=dev) for n in lengths]).to(torch.int32)
        s = {"case": case, "req": req, "pos": pos, "table": table, "codes": codes, "scales": scales}
    elif op == "attend":
        queries, keys = _lengths(case)
        table, total = _table(keys, case["page"], g)
        codes, scales = _cache(case, total, g, True)
        q_start = torch.tensor([0] + queries, device=dev).cumsum(0).to(torch.int32)
        s = {"case": case, "table": table, "codes": codes, "scales": scales, "q_start": q_start,
             "q": (3.0 * torch.randn((sum(queries), case["heads"], case["dim"]), generator=g, device=dev)).to(torch.bfloat16),
             "kv_len": torch.tensor(keys, dtype=torch.int32, device=dev)}
    # the plan and the handle that a program keeps, on either side
    if "rope_args" in s:
        s["frequencies"] = _frequencies(s["rope_args"], dev)
    if own:
        from masked_block_diffusion_b200 import KVCache4, Rope
        if "rope_args" in s:
            s["rope"] = Rope(**s["rope_args"])
        if "codes" in s:
            s["cache"] = KVCache4.from_tensors(s["codes"], s["scales"])
    return s


# ---------------------------------------------------------------- the plain form


def _frequencies(a, device):
    rd = a["rotary_dim"]
    i = torch.arange(rd // 2, dtype=torch.float64, device=device)
    theta, m = a["theta"], 1.0
    if a["scaling"] == "ntk":
        theta = theta * a["factor"] ** (rd / (rd - 2))
    f = theta ** (-2.0 * i / rd)
    if a["scaling"] == "linear":
        f = f / a["factor"]
    if a["scaling"] == "yarn":
        # pairs that turn more than beta_fast times over the trained length keep their frequency, those
        # under beta_slow turns have it divided, and a ramp lies between
        at = lambda turns: rd * math.log(a["original_ctx"] / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        low, high = max(math.floor(at(a["beta_fast"])), 0), min(math.ceil(at(a["beta_slow"])), rd - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / a["factor"] * ramp
        m = 0.1 * math.log(a["factor"]) + 1.0
    return f, m


def _rotate(x, pos, s, transposed=False):
    """x [T][H][d] in fp32, each product and sum rounded to fp32; cos and sin are 64-bit values rounded to fp32."""
    a, (f, m) = s["rope_args"], s["frequencies"]
    angle = pos.to(torch.float64)[:, None] * f
    cos = (m * angle.cos()).float()[:, None, :]
    sin = (m * angle.sin()).float()[:, None, :]
    if transposed:
        sin = -sin
    rd = a["rotary_dim"]
    rot, rest = x[..., :rd], x[..., rd:]
    if a["layout"] == "half":
        p, q = rot[..., :rd // 2], rot[..., rd // 2:]
        return torch.cat([p * cos - q * sin, q * cos + p * sin, rest], -1)
    p, q = rot[..., 0::2], rot[..., 1::2]
    return torch.cat([torch.stack([p * cos - q * sin, q * cos + p * sin], -1).flatten(-2), rest], -1)


def _scale_values(b):
    """What the scale bytes stand for, in fp32."""
    return (b.to(torch.int16) << 7).view(torch.float16).float()


def _quantise(x):
    """fp32 [..][d] -> code bytes [..][d / 2], scale bytes [..][d / 16]. The scale is the least one with 7 * scale >= the
    group's largest magnitude."""
    g = x.unflatten(-1, (-1, 16))
    top = g.abs().amax(-1)
    every = _scale_values(torch.arange(0, 211, dtype=torch.uint8, device=x.device))  # 210, which is 2560, is the largest one used
    byte = torch.searchsorted(7.0 * every, top.contiguous()).clamp(max=210)
    scale = every[byte][..., None]
    u = torch.where(scale > 0, g / scale, torch.zeros_like(g)).round().clamp(-7, 7).to(torch.int32) + 8
    u = u.flatten(-2).unflatten(-1, (-1, 4, 2))  # [..][word][j][dim 2 j or 2 j + 1]
    pair = u[..., 0::2, :] | (u[..., 1::2, :] << 4)  # nibbles j, j + 1 of a byte
    return torch.cat([pair[..., 0], pair[..., 1]], -1).to(torch.uint8).flatten(-2), byte.to(torch.uint8)


def _values(codes, scales):
    """Code and scale bytes -> fp32 values [..][d]."""
    b = codes.unflatten(-1, (-1, 2, 2)).to(torch.int32)  # [..][word][even or odd dims][byte]
    n = torch.stack([b & 15, b >> 4], -1).flatten(-2)  # [..][word][even or odd][j]
    v = (n - 8).transpose(-1, -2).flatten(-3).float()
    return (v.unflatten(-1, (-1, 16)) * _scale_values(scales)[..., None]).flatten(-2)


def _gather(s, req, pos):
    """Both arrays' rows of K and of V at (req, pos), [T][2][kv_heads][..]."""
    page = s["case"]["page"]
    at = s["table"][req, pos // page].long()
    return s["codes"][at, :, :, pos % page], s["scales"][at, :, :, pos % page]


def _attend_plain(s):
    case = s["case"]
    h, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    batch, most_q, most_k = case["batch"], case["queries"], case["keys"]
    q_start, kv_len = s["q_start"].long(), s["kv_len"].long()
    n_q = q_start[1:] - q_start[:-1]
    i = torch.arange(most_q, device=q_start.device)
    q = s["q"].float()[(q_start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)]  # [B][most_q][H][d]
    pages = s["table"].long()
    kv = _values(s["codes"][pages], s["scales"][pages])  # [B][pages][2][hk][page][d]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, batch, hk, -1, d)[:, :, :, :most_k]
    q = q.permute(0, 2, 1, 3).reshape(batch, hk, (h // hk) * most_q, d)
    w = (q @ kv[0].transpose(-1, -2)).view(batch, h, most_q, -1) * d ** -0.5
    key = torch.arange(w.shape[-1], device=w.device)
    seen = kv_len[:, None] if not case["causal"] else (kv_len - n_q)[:, None] + i[None, :] + 1
    w = w.masked_fill_((key >= torch.minimum(seen, kv_len[:, None])[..., None])[:, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = (w - top).exp_()
    total = w.sum(-1, keepdim=True)
    o = (w.view(batch, hk, -1, w.shape[-1]) @ kv[1]).view(batch, h, most_q, d) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log())[..., 0]
    t = torch.arange(s["q"].shape[0], device=w.device)
    b = torch.searchsorted(q_start, t, right=True) - 1
    at = t - q_start[b]
    return {"out": o[b, :, at].to(torch.bfloat16), "lse": lse[b, :, at]}


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "rope":
        if own:
            from masked_block_diffusion_b200 import rope
            return rope(s["x"], s["pos"], s["rope"], out_dtype=_DTYPE[case["out"]], transposed=case["transposed"])
        return _rotate(s["x"].float(), s["pos"], s, case["transposed"]).to(_DTYPE[case["out"]])
    if op == "append":
        # the new tokens' keys and values into the cache, and what the cache then holds for them
        h, hk = case["heads"], case["kv_heads"]
        k, v = s["qkv"][:, h:h + hk], s["qkv"][:, h + hk:]
        if own:
            s["cache"].append(k, v, s["req"], s["pos"], s["table"], rope=s["rope"])
            held = torch.zeros((2, *k.shape), dtype=torch.bfloat16, device=k.device)
            s["cache"].read(s["req"], s["pos"], s["table"], k_out=held[0], v_out=held[1])
            return held
        k = _rotate(k.float(), s["pos"], s)
        codes, scales = _quantise(torch.stack([k, v.float()], 1))
        real = (s["req"] >= 0).nonzero()[:, 0]
        req, pos = s["req"][real].long(), s["pos"][real].long()
        at = s["table"][req, pos // case["page"]].long()
        s["codes"][at, :, :, pos % case["page"]] = codes[real]
        s["scales"][at, :, :, pos % case["page"]] = scales[real]
        held = torch.zeros((2, *k.shape), dtype=torch.bfloat16, device=k.device)
        held[:, real] = _values(*_gather(s, req, pos)).transpose(0, 1).to(torch.bfloat16)
        return held
    if op == "read":
        if own:
            return list(s["cache"].read(s["req"], s["pos"], s["table"]))
        held = _values(*_gather(s, s["req"].long(), s["pos"].long())).to(torch.bfloat16)
        return [held[:, 0], held[:, 1]]
    if own:
        out, lse = s["cache"].attend(s["q"], s["q_start"], s["kv_len"], s["table"], max_q=case["queries"], max_kv=case["keys"],
                                     causal=case["causal"], return_lse=True)
        return {"out": out, "lse": lse}
    return _attend_plain(s)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    size = {"f32": 4, "bf16": 2}
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": n * case["dim"] * (size[case["in"]] + size[case["out"]]) + 4 * case["tokens"], "flops": 3 * n * case["rotary"]}
    hk, d = case["kv_heads"], case["dim"]
    packed = 2 * hk * (d // 2 + d // 16)  # of one position
    if op == "append":
        new, _ = _lengths(case)
        tokens = sum(new)
        # the new keys and values in, packed, and back as bf16
        return {"bytes": tokens * (2 * hk * d * size[case["in"]] + 2 * packed + 2 * hk * d * 2 + 16), "flops": tokens * 2 * hk * d * 8}
    queries, keys = _lengths(case)
    if op == "read":
        return {"bytes": sum(keys) * (packed + 2 * hk * d * 2 + 8), "flops": sum(keys) * 2 * hk * d}
    h = case["heads"]
    pairs = 0
    for n, k in zip(queries, keys):
        pairs += n * k if not case["causal"] else sum(max(0, k - n + i + 1) for i in range(n))
    return {"bytes": sum(keys) * packed + sum(queries) * h * (4 * d + 4) + 4 * sum(-(-k // case["page"]) for k in keys), "flops": 4 * pairs * h * d}


# ---------------------------------------------------------------- the definition in 64 bits


def _turn(x, pos, a, back=False):
    """The rotation pair by pair as a complex product, in 64 bits."""
    rd = a["rotary_dim"]
    base = a["theta"] if a["scaling"] != "ntk" else a["theta"] * a["factor"] ** (rd / (rd - 2.0))
    freq, size = [], 1.0
    for i in range(rd // 2):
        w = base ** (-2.0 * i / rd)
        if a["scaling"] == "linear":
            w /= a["factor"]
        elif a["scaling"] == "yarn":
            edge = [rd * math.log(a["original_ctx"] / (2.0 * math.pi * t)) / (2.0 * math.log(base)) for t in (a["beta_fast"], a["beta_slow"])]
            lo, hi = max(0, math.floor(edge[0])), min(rd - 1, math.ceil(edge[1]))
            share = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w = w * (1.0 - share) + w / a["factor"] * share
            size = 1.0 + 0.1 * math.log(a["factor"])
        freq.append(w)
    angle = torch.outer(pos.double(), torch.tensor(freq, dtype=torch.float64, device=x.device))
    unit = torch.polar(torch.full_like(angle, size), -angle if back else angle)[:, None]
    y = x.double().clone()
    half = a["layout"] == "half"
    first, second = (slice(0, rd // 2), slice(rd // 2, rd)) if half else (slice(0, rd, 2), slice(1, rd, 2))
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * unit
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _unpack64(codes, scales):
    """Packed rows to 64-bit values, word by word."""
    word = codes.contiguous().view(torch.int32).long()
    out = torch.empty((*codes.shape[:-1], codes.shape[-1] * 2), dtype=torch.float64, device=codes.device)
    for j in range(4):
        out[..., 2 * j::8] = ((word >> (4 * j)) & 15).double() - 8
        out[..., 2 * j + 1::8] = ((word >> (4 * j + 16)) & 15).double() - 8
    e, m = (scales >> 3).double(), (scales & 7).double()
    size = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 15), m / 8 * 2.0 ** -14)
    return out * torch.repeat_interleave(size, 16, -1)


def _held64(x):
    """What the cache holds for x [..][d] in 64 bits: the nearest multiple (ties to even) of the least sufficient scale."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    need = g.abs().amax(-1, keepdim=True) / 7
    _, e = torch.frexp(need)  # need = m 2^e, 0.5 <= m < 1
    grain = torch.exp2((e - 1).clamp(min=-14).double() - 3)  # the spacing of scales there
    size = (torch.ceil(need / grain) * grain).clamp(max=2560.0)
    return torch.where(size > 0, torch.round(g / size).clamp(-7, 7) * size, torch.zeros_like(g)).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _turn(s["x"], s["pos"], s["rope_args"], case["transposed"])
    if op == "append":
        h, hk = case["heads"], case["kv_heads"]
        held = torch.stack([_held64(_turn(s["qkv"][:, h:h + hk], s["pos"], s["rope_args"])), _held64(s["qkv"][:, h + hk:].double())])
        held[:, s["req"] < 0] = 0
        return held
    req_rows = s["table"].long()
    queries, keys = _lengths(case)
    if op == "read":
        found = [_unpack64(s["codes"][req_rows[b]], s["scales"][req_rows[b]]).permute(1, 0, 3, 2, 4).flatten(1, 2)[:, :n] for b, n in enumerate(keys)]
        return [torch.cat([f[i] for f in found]) for i in (0, 1)]
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    outs, lses, t = [], [], 0
    for b, (n, m) in enumerate(zip(queries, keys)):
        kv = _unpack64(s["codes"][req_rows[b]], s["scales"][req_rows[b]])
        out = torch.zeros((n, h, d), dtype=torch.float64, device=kv.device)
        lse = torch.full((n, h), -math.inf, dtype=torch.float64, device=kv.device)
        for j in range(h):
            k, v = (kv[:, i, j // (h // hk)].flatten(0, 1)[:m] for i in (0, 1))
            a = s["q"][t:t + n, j].double() @ k.T / math.sqrt(d)
            if case["causal"]:
                a[torch.ones_like(a, dtype=torch.bool).triu(m - n + 1)] = -math.inf
            lse[:, j] = torch.logsumexp(a, -1)
            out[:, j] = torch.softmax(a, -1).nan_to_num(0.0) @ v
        outs.append(out)
        lses.append(lse)
        t += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
