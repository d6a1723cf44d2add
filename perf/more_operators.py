"""Operators of decoder layers that take in text, images and video, as they are measured.

  block      the norm after a block, its gate and scales, the residual sum and the norm before the next block; BF16 out, or
             8 bits (e4m3) with a scale for each row
  rope       rotation of q and k by positions on several axes (time, height, width): alone, as in a vision tower, or with the
             append of k and v to the 4-bit paged cache, whose entries are then read back
  attention  attention over keys and values as they were projected: whole sequences of different lengths behind each other

Every sequence of a case has `new` tokens (its queries) and `kv` keys, for `rope` the tokens in the cache with the new ones
last: lists of numbers as text, since a case holds plain values.  The cache's layout is that of perf/operators.py.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of a generated answer: the norms around a block, launch and latency
        _block("block one token", 1, 4096, 16, post=True, gate="none"),
        # a decode batch with a gate for each channel, whose activations go to an 8-bit product of the caller's
        _block("block batch 8-bit", 257, 5120, 8, post=True, gate="channel"),
        # the rows of a packed batch of prompts
        _block("block prompts", 8191, 4096, 16, post=True, gate="channel"),
        # one token of one answer about a video: rotated, quantised, appended
        _rope("rope one token", 32, 8, 128, 16, [1], [1025], [16, 24, 24]),
        # a decode step of 64 answers of different lengths
        _rope("rope batch", 32, 8, 128, 16, [1] * 64, _ragged(64, 40, 8192), [16, 24, 24]),
        # four prompts of text around images, as they are first taken in
        _rope("rope prompts", 32, 8, 128, 64, [4096, 2047, 1, 1999], [4096, 2047, 700, 1999], [16, 24, 24]),
        # the patches of images in a vision tower: rows and columns, no cache
        _rope("rope patches", 16, 16, 64, 0, [4096, 1024, 2501, 999], [4096, 1024, 2501, 999], [16, 16]),
        # one short prompt: latency
        _attention("attention short", 32, 8, 128, [37]),
        # a packed batch of prompts of different lengths
        _attention("attention packed", 32, 8, 128, _ragged(21, 16, 3001)),
        # one long document
        _attention("attention long", 32, 8, 128, [16384]),
        # sliding windows, seven query heads to a kv head, one chunk that goes on from keys that are there already
        _attention("attention window", 28, 4, 128, [4099, 1, 2000], [4099, 333, 5001], window=1024),
        # the patches of images in a vision tower: every patch of an image sees all of it
        _attention("attention patches", 16, 16, 64, [4096, 1024, 2501, 999], causal=False),
    ]


def _block(name, rows, dim, bits, post, gate, residual_scale=1.0, block_scale=1.0, offset=0.0):
    return {"name": name, "op": "block", "rows": rows, "dim": dim, "bits": bits, "post": post, "gate": gate,
            "residual_scale": residual_scale, "block_scale": block_scale, "offset": offset}


def _rope(name, q_heads, kv_heads, dim, page, new, kv, sections, interleaved=False, mixed=False):
    """page 0: no cache.  sections: pairs of each axis; mixed: the axes take turns instead of following each other."""
    return {"name": name, "op": "rope", "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "new": _text(new), "kv": _text(kv), "sections": _text(sections), "interleaved": interleaved, "mixed": mixed}


def _attention(name, q_heads, kv_heads, dim, new, kv=None, causal=True, window=0):
    return {"name": name, "op": "attention", "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "new": _text(new),
            "kv": _text(kv or new), "causal": causal, "window": window}


def _text(numbers):
    return ",".join(map(str, numbers))


def _ragged(n, low, high):
    """n lengths from low to high, spread over their logarithm, in a mixed order."""
    at = [int(low * (high / low) ** (i / (n - 1))) for i in range(n)]
    return [at[i * 37 % n] for i in range(n)]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["block", "rope", "attention", "attention"])
    if op == "block":
        dim = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            dim = max(64, dim // 64 * 64)
        case = _block("", _log(rng, 1, max(1, min(8192, 8192 * 4096 // dim))), dim, rng.choice([16, 16, 8]),
                      rng.random() < 0.8, rng.choice(["none", "channel", "row"]), rng.choice([1.0, 0.5]),
                      rng.choice([1.0, 0.22]), rng.choice([0.0, 1.0]))
    else:
        dim = rng.choice([64, 128, 128])
        kv_heads = rng.choice([1, 2, 4, 8, 8])
        q_heads = kv_heads * rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
        if op == "rope":
            pairs = dim // 2 - 8 * rng.choice([0, 0, 0, 1])
            axes = rng.choice([1, 2, 3, 3, 4])
            cuts = sorted(rng.randint(0, pairs) for _ in range(axes - 1))
            sections = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
            kind = rng.choice(["one", "few", "prompt"])
            n = _log(rng, 1, 64) if kind == "one" else rng.randint(1, 6)
            new = [1 if kind == "one" else _log(rng, 2, 8 if kind == "few" else 8190 // n) for _ in range(n)]
            kv = [m + (0 if kind == "prompt" and rng.random() < 0.7 else _log(rng, 1, 8192)) for m in new]
            case = _rope("", q_heads, kv_heads, dim, rng.choice([0, 16, 32, 64, 128]), new, kv, sections,
                         rng.random() < 0.3, rng.random() < 0.4)
        else:
            n = _log(rng, 1, 24)
            most = 6000 if n == 1 else 6000 // n + 400
            new = [_log(rng, 1, most) for _ in range(n)]
            kv = [m + (0 if rng.random() < 0.8 else _log(rng, 1, 3000)) for m in new]
            case = _attention("", q_heads, kv_heads, dim, new, kv, rng.random() < 0.75,
                              _log(rng, 16, 4096) if rng.random() < 0.25 else 0)
    del case["name"]
    return case


def _lens(case, key):
    return [int(n) for n in case[key].split(",")]


def work(case):
    if case["op"] == "block":
        n, d = case["rows"], case["dim"]
        read = 2 * n * d * 2 + {"none": 0, "channel": d * 2, "row": n * d * 2}[case["gate"]] + d * (4 if case["post"] else 2)
        write = n * d * 2 + (n * d * 2 if case["bits"] == 16 else n * d + 4 * n)
        return {"bytes": read + write, "flops": n * d * (6 + 3 * case["post"] + (case["gate"] != "none"))}
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    new, kv = _lens(case, "new"), _lens(case, "kv")
    t = sum(new)
    if case["op"] == "rope":
        axes, pairs = len(_lens(case, "sections")), sum(_lens(case, "sections"))
        turned = 2 * t * (hq + hk) * d * 2 + t * axes * 4 + t * pairs * 8
        # and v in, the cache's entries and their values out, the entries read again
        cached = t * hk * d * 2 + 2 * t * 2 * hk * (d // 2 + 4) + 2 * t * hk * d * 2
        return {"bytes": turned + (cached if case["page"] else 0),
                "flops": t * (6 * pairs * (hq + hk) + (12 * hk * d if case["page"] else 0))}
    pairs = read = 0
    for n, m in zip(new, kv):
        lo = [max(0, m - n + i + 1 - case["window"]) if case["window"] else 0 for i in range(n)]
        hi = [m - n + i + 1 if case["causal"] else m for i in range(n)]
        pairs += sum(max(0, b - a) for a, b in zip(lo, hi))
        read += max(hi) - min(lo)
    return {"bytes": 2 * read * hk * d * 2 + 2 * t * hq * d * 2, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "block":
        n, d = case["rows"], case["dim"]
        x, r = normal(n, d) * (0.2 + normal(n, 1).abs()), normal(n, d) * 3
        r[:, ::97] *= 20  # the few large channels of a residual stream
        gate = {"none": None, "channel": normal(d) * 0.5, "row": normal(n, d) * 0.5}[case["gate"]]
        one = 1 - case["offset"]
        return {"case": case, "x": x.bfloat16(), "residual": r.bfloat16(), "eps": 1e-6,
                "weight": (one + 0.2 * normal(d)).bfloat16(),
                "post": (one + 0.2 * normal(d)).bfloat16() if case["post"] else None,
                "gate": None if gate is None else gate.bfloat16()}
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    new, kv = _lens(case, "new"), _lens(case, "kv")
    t = sum(new)

    def starts(lens):
        return torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()

    state = {"case": case, "start": starts(new)}
    if case["op"] == "attention":
        # a projection's rows: q beside k and v where they have the same tokens
        state["kv_start"] = None if new == kv else starts(kv)
        level = 0.5 + normal(1, hq + 2 * hk, 1).abs()
        if new == kv:
            qkv = (normal(t, hq + 2 * hk, d) * level).bfloat16()
            state["q"], state["k"], state["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        else:
            state["q"] = (normal(t, hq, d) * level[:, :hq]).bfloat16()
            state["k"] = (normal(sum(kv), hk, d) * level[:, hq:hq + hk]).bfloat16()
            state["v"] = (normal(sum(kv), hk, d) * level[:, hq + hk:]).bfloat16()
        return state
    sections = _lens(case, "sections")
    axes, pairs = len(sections), sum(sections)
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    if case["mixed"]:
        left, axis = list(sections), []
        while len(axis) < pairs:
            for a in range(axes):
                if left[a]:
                    left[a] -= 1
                    axis.append(a)
    state["axis"] = bytes(axis)
    state["pos"] = torch.cat([_positions(n, m, axes, case["page"] == 0) for n, m in zip(new, kv)], 1).int().cuda()
    width = max(kv) + 1
    angle = torch.arange(width, device="cuda").double()[:, None] * 10000.0 ** (
        -torch.arange(pairs, device="cuda").double() / pairs)
    state["cos"], state["sin"] = angle.cos().float(), angle.sin().float()
    state["qkv"] = (normal(t, hq + 2 * hk, d) * (0.3 + normal(1, hq + 2 * hk, d).abs())).bfloat16()
    page = case["page"]
    if page:
        state["length"] = torch.tensor(kv, dtype=torch.int32).cuda()
        counts = [-(-n // page) for n in kv]
        # pages in a mixed order, some of the pool in no sequence's table
        pool = sum(counts) + 3
        order = torch.randperm(pool, generator=g, device="cuda").int()
        table = torch.zeros(len(new), max(counts), dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(counts):
            table[i, :n] = order[at:at + n]
            at += n
        state["table"] = table
        state["pages"] = torch.randint(0, 256, (pool, hk, page * (d + 8)), dtype=torch.uint8, generator=g, device="cuda")
    return state


def _positions(n, m, axes, patches):
    """Positions [axes, n] of the last n of m tokens: text, where all axes go on together, around an image whose rows
    and columns are the last two axes; or patches alone."""
    at = torch.arange(m)
    if axes == 1:
        return at[None, m - n:]
    side = max(1, int(math.sqrt(m if patches else m // 2)))
    first = 0 if patches else m // 4
    image = m if patches else side * side
    pos = at.repeat(axes, 1)
    inside = at[first:first + image] - first
    pos[:, first:first + image] = first
    pos[-2, first:first + image] += inside // side
    pos[-1, first:first + image] += inside % side
    pos[:, first + image:] = first + side + torch.arange(max(0, m - first - image))
    return pos[:, m - n:].clamp(max=m)


# ------------------------------------------------------------------ the operators
def run(state):
    op = state["case"]["op"]
    if own:
        return {"block": _own_block, "rope": _own_rope, "attention": _own_attention}[op](state)
    return {"block": _plain_block, "rope": _plain_rope, "attention": _plain_attention}[op](state)


def _own_block(s):
    import lossless_bf16_weight_gb300 as uw

    c, x = s["case"], s["x"]
    h = torch.empty_like(x)
    scale = None
    if c["bits"] == 16:
        y = torch.empty_like(x)
    else:
        y = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
        scale = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    uw.block_norm(x, s["residual"], s["weight"], h, y, s["eps"], post_weight=s["post"], gate=s["gate"],
                  residual_scale=c["residual_scale"], block_scale=c["block_scale"], weight_offset=c["offset"], scale=scale)
    return {"y": y, "h": h} if scale is None else {"y": y, "scale": scale, "h": h}


def _own_rope(s):
    import lossless_bf16_weight_gb300 as uw

    c, qkv = s["case"], s["qkv"]
    hq, hk, t, d = c["q_heads"], c["kv_heads"], qkv.shape[0], c["dim"]
    if "ws" not in s:  # the workspace, and the cache's handle, which a program makes once and keeps
        if c["page"]:
            s["cache"] = uw.kv4_cache(s["pages"], s["table"], hk, d, c["page"])
        s["ws"] = torch.empty(256, dtype=torch.uint8, device="cuda")
        uw.workspace_init(s["ws"])
    q = torch.empty(t, hq, d, dtype=qkv.dtype, device=qkv.device)
    k = torch.empty(t, hk, d, dtype=qkv.dtype, device=qkv.device)
    if not c["page"]:
        uw.rope_axes(qkv[:, :hq], qkv[:, hq:hq + hk], s["pos"], s["axis"], q, k, s["cos"], s["sin"], s["ws"],
                     interleaved=c["interleaved"])
        return {"q": q, "k": k}
    uw.kv4_append_axes(s["cache"], s["start"], s["length"], s["pos"], s["axis"], qkv[:, :hq], qkv[:, hq:hq + hk],
                       qkv[:, hq + hk:], q, s["cos"], s["sin"], s["ws"], k_out=k, interleaved=c["interleaved"])
    held_k, held_v = torch.empty_like(k), torch.empty_like(k)
    uw.kv4_read(s["cache"], s["start"], s["length"], held_k, held_v, s["ws"])
    return {"q": q, "k": k, "held_k": held_k, "held_v": held_v}


def _own_attention(s):
    import lossless_bf16_weight_gb300 as uw

    c, q = s["case"], s["q"]
    if "ws" not in s:
        s["ws"] = torch.empty(uw.attention_workspace_size(c["dim"]), dtype=torch.uint8, device="cuda")
        uw.workspace_init(s["ws"])
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    uw.attention(q, s["k"], s["v"], out, s["start"], s["ws"], kv_start=s["kv_start"], causal=c["causal"],
                 window=c["window"], lse=lse)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ their plain forms
def _plain_block(s):
    c, x, w = s["case"], s["x"].float(), s["weight"].float() + s["case"]["offset"]
    if s["post"] is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * (s["post"].float() + c["offset"])
    if s["gate"] is not None:
        x = x * s["gate"].float()
    h = (c["residual_scale"] * s["residual"].float() + c["block_scale"] * x).bfloat16()
    f = h.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + s["eps"]) * w
    if c["bits"] == 16:
        return {"y": y.bfloat16(), "h": h}
    scale = (y.abs().amax(-1) / E4M3_MAX).clamp_min(TINY)
    return {"y": (y / scale[:, None]).to(torch.float8_e4m3fn), "scale": scale, "h": h}


def _regions(s):
    """The pages as K codes, V codes, K params, V params: views."""
    c, pages = s["case"], s["pages"]
    page, half = c["page"], c["dim"] // 2
    cut = page * half
    return (pages[..., :cut].unflatten(-1, (page, half)), pages[..., cut:2 * cut].unflatten(-1, (page, half)),
            pages[..., 2 * cut:2 * cut + 4 * page].unflatten(-1, (page, 4)),
            pages[..., 2 * cut + 4 * page:].unflatten(-1, (page, 4)))


def _values(code, par):
    """What packed codes [.., D/2] and their params [.., 4] stand for, in 32 bits."""
    par = par.contiguous().view(torch.bfloat16).float()
    c = torch.stack((code & 15, code >> 4), -1).flatten(-2).float()
    return par[..., 1:] + c * par[..., :1]


def _quantised(x):
    """Packed codes and params of the vectors x [.., D]."""
    x = x.float()
    hi, lo = x.amax(-1, keepdim=True), x.amin(-1, keepdim=True)
    scale = ((hi * 0.5 - lo * 0.5) / 7.5).bfloat16().float()
    code = ((x * 0.5 - lo * 0.5) / (scale * 0.5)).round().clamp(0, 15)
    code = torch.where(scale > 0, code, torch.zeros_like(code)).to(torch.uint8)
    par = torch.cat((scale, lo), -1).bfloat16().view(torch.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, par


def _plain_rope(s):
    c, qkv = s["case"], s["qkv"]
    hq, hk = c["q_heads"], c["kv_heads"]
    axis = torch.tensor(list(s["axis"]), device="cuda")
    pair = torch.arange(len(axis), device="cuda")
    at = s["pos"][axis].T.long()  # [token, pair]
    cos, sin = s["cos"][at, pair][:, None], s["sin"][at, pair][:, None]
    x, rest = qkv[:, :hq + hk, :2 * len(axis)].float(), qkv[:, :hq + hk, 2 * len(axis):]
    a, b = (x[..., 0::2], x[..., 1::2]) if c["interleaved"] else x.chunk(2, -1)
    a, b = a * cos - b * sin, b * cos + a * sin
    x = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
    x = torch.cat((x.bfloat16(), rest), -1)
    q, k = x[:, :hq].contiguous(), x[:, hq:].contiguous()
    if not c["page"]:
        return {"q": q, "k": k}
    token = torch.arange(len(qkv), device="cuda")
    seq = torch.searchsorted(s["start"][1:], token.int(), right=True)
    place = (s["length"][seq] - s["start"][seq + 1] + token).long()
    page, slot = s["table"][seq, place // c["page"]].long(), place % c["page"]
    kc, vc, kp, vp = _regions(s)
    kc[page, :, slot], kp[page, :, slot] = _quantised(k)
    vc[page, :, slot], vp[page, :, slot] = _quantised(qkv[:, hq + hk:])
    return {"q": q, "k": k, "held_k": _values(kc[page, :, slot], kp[page, :, slot]).bfloat16(),
            "held_v": _values(vc[page, :, slot], vp[page, :, slot]).bfloat16()}


def _plain_attention(s):
    c, q = s["case"], s["q"]
    hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
    start, kv_start = s["start"].long(), (s["start"] if s["kv_start"] is None else s["kv_start"]).long()
    n, m = max(_lens(c, "new")), max(_lens(c, "kv"))
    row, held = torch.arange(n, device="cuda"), torch.arange(m, device="cuda")
    count, length = (start[1:] - start[:-1])[:, None], (kv_start[1:] - kv_start[:-1])[:, None]
    # the rows of every sequence, as many as of the longest: [b, kv head, head of the group, row, dim] and [b, kv head, key, dim]
    rows = q[(start[:-1, None] + row).clamp_max(len(q) - 1)].float().unflatten(2, (hk, hq // hk)).permute(0, 2, 3, 1, 4)
    key = (kv_start[:-1, None] + held).clamp_max(len(s["k"]) - 1)
    k, v = s["k"][key].float().transpose(1, 2), s["v"][key].float().transpose(1, 2)
    pos = length - count + row
    seen = (held < length)[:, None] & (row < count)[:, :, None]
    if c["causal"]:
        seen = seen & (held <= pos[:, :, None])
    if c["window"]:
        seen = seen & (held > pos[:, :, None] - c["window"])
    score = (rows.flatten(2, 3) @ k.transpose(-1, -2)).unflatten(2, (hq // hk, n)).mul_(1 / math.sqrt(d))
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.flatten(2, 3) @ v).unflatten(2, (hq // hk, n)) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, total.log() + top, -math.inf)
    token = torch.arange(len(q), device="cuda")
    seq = torch.searchsorted(start[1:], token, right=True)
    at = token - start[seq]
    return {"out": out.permute(0, 3, 1, 2, 4).flatten(2, 3)[seq, at].bfloat16(),
            "lse": lse.squeeze(-1).permute(0, 3, 1, 2).flatten(2, 3)[seq, at]}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "block":
        z = s["x"].double()
        if case["post"]:
            z = z / torch.sqrt(torch.sum(z * z, 1) / z.shape[1] + s["eps"])[:, None] * (s["post"].double() + case["offset"])
        z = z * case["block_scale"] * (1.0 if s["gate"] is None else s["gate"].double())
        h = (z + s["residual"].double() * case["residual_scale"]).bfloat16().double()
        y = h / torch.sqrt(torch.sum(h * h, 1) / h.shape[1] + s["eps"])[:, None] * (s["weight"].double() + case["offset"])
        if case["bits"] == 16:
            return {"y": y, "h": h}
        scale = torch.maximum(torch.max(torch.abs(y), 1).values / E4M3_MAX, torch.tensor(TINY, device="cuda"))
        return {"y": (y / scale[:, None]).to(torch.float8_e4m3fn).double(), "scale": scale, "h": h}
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    new, kv = _lens(case, "new"), _lens(case, "kv")
    if case["op"] == "rope":
        x = s["qkv"].double()
        turned = x[:, :hq + hk].clone()
        pairs = len(s["axis"])
        for i, a in enumerate(s["axis"]):
            one, two = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + pairs)
            p = s["pos"][a].long()
            turn = torch.complex(s["cos"][p, i].double(), s["sin"][p, i].double())[:, None]
            z = torch.complex(x[:, :hq + hk, one].contiguous(), x[:, :hq + hk, two].contiguous()) * turn
            turned[:, :, one], turned[:, :, two] = z.real, z.imag
        turned = turned.bfloat16().double()
        out = {"q": turned[:, :hq], "k": turned[:, hq:]}
        if case["page"]:
            for name, u in (("held_k", out["k"]), ("held_v", x[:, hq + hk:])):
                lo = u.min(2, keepdim=True).values
                step = ((u.max(2, keepdim=True).values - lo) / 15).bfloat16().double()
                code = torch.clamp(torch.round((u - lo) / torch.where(step > 0, step, 1.0)), 0, 15)
                out[name] = lo + code * step
        return out
    out = torch.zeros(sum(new), hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(new), hq), -math.inf, dtype=torch.float64, device="cuda")
    at = key_at = 0
    for n, m in zip(new, kv):
        for a in range(0, n, 2048):
            e = min(n, a + 2048)
            pos = torch.arange(m - n + a, m - n + e, device="cuda")[:, None]
            first = max(0, m - n + a + 1 - case["window"]) if case["window"] else 0
            last = min(m, m - n + e) if case["causal"] else m
            held = torch.arange(first, last, device="cuda")
            seen = torch.ones(e - a, last - first, dtype=torch.bool, device="cuda")
            if case["causal"]:
                seen &= held <= pos
            if case["window"]:
                seen &= held > pos - case["window"]
            for head in range(hq):
                k = s["k"][key_at + first:key_at + last, head * hk // hq].double()
                v = s["v"][key_at + first:key_at + last, head * hk // hq].double()
                score = torch.where(seen, s["q"][at + a:at + e, head].double() @ k.T / d ** 0.5, -math.inf)
                total = torch.logsumexp(score, 1)
                lse[at + a:at + e, head] = total
                out[at + a:at + e, head] = torch.exp(score - torch.where(total > -math.inf, total, 0.0)[:, None]) @ v
        at, key_at = at + n, key_at + m
    return {"out": out, "lse": lse}
