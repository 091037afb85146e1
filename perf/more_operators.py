"""The operators of a 4-bit attention cache and what they are measured on.

An attention layer between the product that gives queries, keys and values and
the one that takes the heads' outputs, with keys and values held in MXFP4
(E2M1 codes, one power-of-two E8M0 scale per 32 channels of a token's head):

    mxfp4_cache_write            keys and values -> codes and scales in a paged cache
    norm_rope_mxfp4_cache_write  rows of q | k | v: norm of each query and key head, rotation,
                                 q out in bf16, keys and values into the cache
    mxfp4_cache_read             tokens of the cache by slot -> keys and values in bf16
    mxfp4_attention              grouped-head attention of packed query rows over the paged cache:
                                 causal, windowed or full, with or without a sink logit per head

The cache is four uint8 tensors: key codes [pages, kv_heads, page, d/2], key
scales [pages, kv_heads, page, d/32] and the same for values; slot = page number
* page + place in the page. A block's scale is 2^e with e = floor(log2(largest
magnitude)) - 2, an element the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 times that
(ties to the even code). What a writer left in the cache is returned as the
values it stands for, read back by slot.

`own` False: elementary torch operations. `own` True: the library's calls, into
outputs that the caller holds, as a serving loop makes them.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
MAX_POS = 131072


def listed():
    return [
        # one decode step of one sequence, keys rotated elsewhere: the smallest write
        dict(name="write_token", op="write", tokens=1, kv=8, d=128, page=16, dtype="bf16"),
        # fp32 rows of an odd number of prompt tokens, heads of 64 channels, a few tokens that are padding
        dict(name="write_prompt_f32", op="write", tokens=4097, kv=8, d=64, page=64, dtype="f32"),
        # one decode step of 64 sequences: the fused projection's rows, normed, rotated and written
        dict(name="rope_batch64", op="rope", tokens=64, heads=32, kv=8, d=128, rot=128, page=16, dtype="bf16", norm=True, interleaved=False),
        # a prompt of 8192 tokens
        dict(name="rope_prompt", op="rope", tokens=8192, heads=32, kv=8, d=128, rot=128, page=64, dtype="bf16", norm=True, interleaved=False),
        # the last words of a prompt, read back
        dict(name="read_few", op="read", tokens=130, kv=8, d=64, page=16),
        # a shared prefix of 16384 tokens read back for another kind of attention
        dict(name="read_prefix", op="read", tokens=16384, kv=8, d=128, page=64),
        # one decode step of one sequence of 777 tokens: latency
        dict(name="attn_token", op="attn", seqs=1, qmin=1, qmax=1, lmin=777, lmax=777, heads=32, kv=8, d=128, page=16, causal=True, window=0, sinks=False),
        # one decode step of 64 sequences of 512 to 8192 tokens: the cache's bytes bound it
        dict(name="attn_batch64", op="attn", seqs=64, qmin=1, qmax=1, lmin=512, lmax=8192, heads=32, kv=8, d=128, page=16, causal=True, window=0, sinks=False),
        # four drafted tokens after one context of 131072 tokens
        dict(name="attn_long_draft4", op="attn", seqs=1, qmin=4, qmax=4, lmin=131072, lmax=131072, heads=32, kv=8, d=128, page=64, causal=True, window=0, sinks=False),
        # 48 sequences with one to three tokens each, a window of 128 tokens and a sink per head, heads of 64 channels
        dict(name="attn_window_sinks", op="attn", seqs=48, qmin=1, qmax=3, lmin=1, lmax=4000, heads=64, kv=8, d=64, page=64, causal=True, window=128, sinks=True),
        # 512 new tokens of a prompt whose first 15872 are in the cache
        dict(name="attn_chunk512", op="attn", seqs=1, qmin=512, qmax=512, lmin=16384, lmax=16384, heads=32, kv=8, d=128, page=64, causal=True, window=0, sinks=False),
        # four packed prompts of 1 to 5000 tokens, all of them new
        dict(name="attn_prompts", op="attn", seqs=4, qmin=1, qmax=5000, lmin=0, lmax=0, heads=32, kv=8, d=128, page=64, causal=True, window=0, sinks=False),
    ]


def _spread(rng, lo, hi):
    """A whole number in lo..hi, spread over its logarithm."""
    return min(max(int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))), lo), hi)


def draw(rng):
    op = rng.choice(["write", "rope", "read", "attn", "attn", "attn"])
    kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 5, 8])
    d, page, dtype = rng.choice([64, 128]), rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "bf16", "f32"])
    if op in ("write", "read"):
        case = dict(op=op, tokens=_spread(rng, 1, 32768 // kv), kv=kv, d=d, page=page)
        return dict(case, dtype=dtype) if op == "write" else case
    if op == "rope":
        rot = rng.choice([d, d, d // 2, 32])
        return dict(op=op, tokens=_spread(rng, 1, 8192 // kv), heads=kv * group, kv=kv, d=d, rot=rot, page=page, dtype=dtype,
                    norm=rng.random() < 0.6, interleaved=rng.random() < 0.3)
    kind = rng.choice(["decode", "draft", "prompt", "long"])
    causal = kind != "prompt" or rng.random() < 0.8
    case = dict(op=op, heads=kv * group, kv=kv, d=d, page=page, causal=causal,
                window=_spread(rng, 16, 4096) if causal and rng.random() < 0.3 else 0, sinks=rng.random() < 0.3)
    if kind == "decode":
        return dict(case, seqs=_spread(rng, 1, 96), qmin=1, qmax=1, lmin=1, lmax=_spread(rng, 16, 6000))
    if kind == "draft":
        return dict(case, seqs=_spread(rng, 1, 24), qmin=0, qmax=_spread(rng, 2, 16), lmin=1, lmax=_spread(rng, 64, 8192))
    if kind == "long":
        return dict(case, seqs=_spread(rng, 1, 2), qmin=1, qmax=_spread(rng, 1, 64), lmin=8192, lmax=_spread(rng, 8192, 100000))
    return dict(case, seqs=_spread(rng, 1, 6), qmin=0, qmax=_spread(rng, 32, 2500), lmin=0, lmax=rng.choice([0, 0, 700]))


def _lengths(case):
    """(query tokens, cached tokens) of each sequence, spread evenly over the ranges, the first at the top; `lmax` 0: all that is
    cached is new, and otherwise the cached tokens hold the new ones where there are enough of them."""
    n, q, kv = case["seqs"], [], []
    for i in range(n):
        part = 1.0 if n == 1 else 1.0 - i / (n - 1)
        new = case["qmin"] + int(round((case["qmax"] - case["qmin"]) * part))
        other = 1.0 if n == 1 else ((i * 37 + n - 1) % n) / (n - 1)   # not in the order of the query lengths
        old = case["lmin"] + int(round((case["lmax"] - case["lmin"]) * other))
        q.append(new)
        kv.append(new if case["lmax"] == 0 else old)
    return q, kv


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(shape, dtype, g):
    """Normal rows of a size of their own, and a few channels of every head 8 times the rest, as keys have."""
    x = torch.randn(shape, device="cuda", generator=g)
    x *= torch.exp2(torch.randint(-3, 4, shape[:-1] + (1,), device="cuda", generator=g).float())
    x[..., torch.randint(0, shape[-1], (2,), device="cuda", generator=g)] *= 8.0
    return x.to(dtype)


def _filled(pages, kv, page, d, g):
    """A cache that holds quantized normal rows: codes and scales as bytes, made in pieces to bound the memory."""
    codes = torch.empty(pages, kv, page, d // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, kv, page, d // 32, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (kv * page * d))
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn(n, kv, page, d // 32, 32, device="cuda", generator=g)
        x[..., 0, 3] *= 6.0
        x *= torch.exp2(torch.randint(-2, 2, (n, kv, page, 1, 1), device="cuda", generator=g).float())
        e = (x.abs().amax(-1).view(torch.int32) >> 23) - 2
        c = torch.bucketize(x.abs() * ((254 - e) << 23).view(torch.float32).unsqueeze(-1), mids).to(torch.uint8) | ((x < 0).to(torch.uint8) << 3)
        c = c.view(n, kv, page, d // 2, 2)
        codes[p:p + n] = c[..., 0] | (c[..., 1] << 4)
        scales[p:p + n] = e.to(torch.uint8)
    return codes, scales


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    kv, d, page = case["kv"], case["d"], case["page"]
    if case["op"] == "attn":
        qs, ls = _lengths(case)
        need = [-(-n // page) for n in ls]
        width, pages = max(1, max(need)), sum(need) + 3
        order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
        table = torch.full((case["seqs"], width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        s["table"] = table
        s["lens"] = torch.tensor(ls, dtype=torch.int32, device="cuda")
        offsets = [0]
        for n in qs:
            offsets.append(offsets[-1] + n)
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        s["total"], s["most"] = offsets[-1], max(qs)
        s["q"] = (2.0 * torch.randn(s["total"], case["heads"], d, device="cuda", generator=g)).to(torch.bfloat16)
        s["cache"] = (*_filled(pages, kv, page, d, g), *_filled(pages, kv, page, d, g))
        s["sink"] = 2.0 * torch.randn(case["heads"], device="cuda", generator=g) if case["sinks"] else None
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = d ** -0.5
        return s
    tokens = case["tokens"]
    pages = -(-tokens // page) + 5
    s["slots"] = torch.randperm(pages * page, device="cuda", generator=g)[:tokens].contiguous()
    if tokens > 1000:
        s["slots"][torch.randint(0, tokens, (5,), device="cuda", generator=g)] = -1   # padding
    s["back"] = tuple(torch.empty(tokens, kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if case["op"] == "read":
        s["cache"] = (*_filled(pages, kv, page, d, g), *_filled(pages, kv, page, d, g))
        return s
    s["cache"] = tuple(torch.zeros(pages, kv, page, n, dtype=torch.uint8, device="cuda") for n in (d // 2, d // 32, d // 2, d // 32))
    dt = DT[case["dtype"]]
    if case["op"] == "write":
        s["k"], s["v"] = _rows((tokens, kv, d), dt, g), _rows((tokens, kv, d), dt, g)
        return s
    heads, rot = case["heads"], case["rot"]
    s["qkv"] = _rows((tokens, heads + 2 * kv, d), dt, g).view(tokens, -1)
    s["positions"] = torch.randint(0, MAX_POS, (tokens,), device="cuda", generator=g)
    angle = torch.arange(MAX_POS, device="cuda").double()[:, None] * 500000.0 ** (-torch.arange(0, rot, 2, device="cuda").double() / rot)
    s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    s["wq"], s["wk"] = ((1.0 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(dt) if case["norm"] else None for _ in range(2))
    s["q"] = torch.empty(tokens, heads, d, dtype=torch.bfloat16, device="cuda")
    return s


def _held(x, slots):
    """What the cache stands for after rows x [tokens, kv, d] (fp32) were written and read back."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    e = ((b.abs().amax(-1, keepdim=True).view(torch.int32) >> 23) - 2).clamp(min=1)
    unit, inverse = (e << 23).view(torch.float32), ((254 - e) << 23).view(torch.float32)
    a = b.abs() * inverse   # powers of two: exact, where a division on the GPU need not be
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    a = (torch.round(a * torch.where(a < 2.0, 2.0, torch.where(a < 4.0, 1.0, 0.5))) * step).clamp(max=6.0)
    y = (torch.sign(b) * a * unit).reshape(x.shape)
    return torch.where((slots >= 0)[:, None, None], y, torch.zeros_like(y)).to(torch.bfloat16)


def _values(codes, scales):
    """fp32 values of codes [..., d/2] and scales [..., d/32]."""
    mags = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    pairs = torch.cat([mags, -mags])
    pairs = torch.stack([pairs.repeat(16), pairs.repeat_interleave(16)], 1)     # byte -> (low, high nibble)
    x = pairs[codes.int()].view(*codes.shape[:-1], -1, 32)
    return (x * (scales.int() << 23).view(torch.float32).unsqueeze(-1)).view(*codes.shape[:-1], -1)


def _rotated(x, cos, sin, rot, interleaved):
    a, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        lo, hi = a[..., 0::2], a[..., 1::2]
        a = torch.stack([lo * cos - hi * sin, hi * cos + lo * sin], -1).flatten(-2)
    else:
        lo, hi = a[..., :rot // 2], a[..., rot // 2:]
        a = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)
    return torch.cat([a, rest], -1)


def _normed(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _attention(s):
    kv, d, page, heads = s["kv"], s["d"], s["page"], s["heads"]
    seqs, most, group = s["seqs"], s["most"], heads // kv
    table, total = s["table"].long().clamp(min=0), s["total"]
    parts = []
    for codes, scales in (s["cache"][:2], s["cache"][2:]):
        x = _values(codes[table].transpose(1, 2), scales[table].transpose(1, 2))   # [seqs, kv, pages, page, d]
        parts.append(x.reshape(seqs * kv, -1, d))
    k, v = parts
    width = k.shape[1]
    # the packed rows of each sequence side by side, those past its own repeated and left out at the end
    starts, stops = s["offsets"][:-1].long(), s["offsets"][1:].long()
    place = torch.arange(most, device="cuda")
    rows = (starts[:, None] + place).clamp(max=total - 1)
    q = s["q"].float()[rows].view(seqs, most, kv, group, d).permute(0, 2, 3, 1, 4).reshape(seqs * kv, group * most, d)
    scores = torch.bmm(q.contiguous(), k.transpose(1, 2).contiguous()).mul_(s["scale"]).view(seqs, kv, group, most, width)
    lens = s["lens"].long()
    at = torch.arange(width, device="cuda")
    seen = (at < lens[:, None]).unsqueeze(1)                                     # [seqs, 1, width]
    pos = (lens - (stops - starts))[:, None] + place                             # [seqs, most]
    if s["causal"]:
        seen = seen & (at <= pos[..., None])
        if s["window"]:
            seen = seen & (at > pos[..., None] - s["window"])
    else:
        seen = seen.expand(seqs, most, width)
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].view(1, kv, group, 1, 1)
        top = torch.maximum(top, sink)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total_p = p.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total_p = total_p + torch.exp(sink - top)
    out = torch.bmm(p.view(seqs * kv, group * most, width), v).view(seqs, kv, group, most, d)
    out = out / torch.where(total_p > 0, total_p, torch.ones_like(total_p))
    out = out.permute(0, 3, 1, 2, 4).reshape(seqs * most, heads, d)
    mine = (place < (stops - starts)[:, None]).view(-1)
    return out[torch.nonzero_static(mine, size=total)[:, 0]].to(torch.bfloat16)


def run(state):
    s = state
    if own:
        import gemm_e2m1_lut_amd as g
        if s["op"] == "attn":
            if "workspace" not in s:   # a serving loop holds one for its largest step
                size = g.mxfp4_attention_workspace_size(s["total"], s["seqs"], s["heads"], s["kv"], s["d"])
                s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
            return g.mxfp4_attention(s["q"], s["cache"], s["table"], s["lens"], s["offsets"], scale=s["scale"], causal=s["causal"],
                                     window=s["window"], sinks=s["sink"], out=s["out"], workspace=s["workspace"])
        if s["op"] == "write":
            g.mxfp4_cache_write(s["k"], s["v"], s["slots"], s["cache"])
        elif s["op"] == "rope":
            g.norm_rope_mxfp4_cache_write(s["qkv"], s["table"], s["positions"], s["slots"], s["cache"], q_weight=s["wq"],
                                          k_weight=s["wk"], eps=EPS, interleaved=s["interleaved"], out=s["q"])
        back = g.mxfp4_cache_read(s["cache"], s["slots"], out=s["back"])
        return (s["q"], *back) if s["op"] == "rope" else back
    if s["op"] == "attn":
        return _attention(s)
    if s["op"] == "write":
        return _held(s["k"].float(), s["slots"]), _held(s["v"].float(), s["slots"])
    kv, d = s["kv"], s["d"]
    if s["op"] == "read":
        slots = s["slots"].clamp(min=0)
        page, place = slots // s["page"], slots % s["page"]
        keep = (s["slots"] >= 0)[:, None, None]
        k = _values(s["cache"][0][page, :, place], s["cache"][1][page, :, place])
        v = _values(s["cache"][2][page, :, place], s["cache"][3][page, :, place])
        return torch.where(keep, k, torch.zeros_like(k)).to(torch.bfloat16), torch.where(keep, v, torch.zeros_like(v)).to(torch.bfloat16)
    heads, rot = s["heads"], s["rot"]
    x = s["qkv"].float().view(s["tokens"], heads + 2 * kv, d)
    angles = s["table"][s["positions"]].unsqueeze(1)
    cos, sin = angles[..., :rot // 2], angles[..., rot // 2:]
    q = _rotated(_normed(x[:, :heads], s["wq"]), cos, sin, rot, s["interleaved"])
    k = _rotated(_normed(x[:, heads:heads + kv], s["wk"]), cos, sin, rot, s["interleaved"])
    return q.to(torch.bfloat16), _held(k, s["slots"]), _held(x[:, heads + kv:], s["slots"])


def _pairs(case):
    """(query, key) pairs that are seen, and the tokens of the cache that some query sees."""
    pairs = tokens = 0
    for new, old in zip(*_lengths(case)):
        if not case["causal"]:
            pairs += new * old
            tokens += old if new else 0
            continue
        window = case["window"] or old
        first = old
        for p in range(max(0, old - new), old):
            lo = max(0, p - window + 1)
            pairs += p - lo + 1
            first = min(first, lo)
        tokens += old - first
    return pairs, tokens


def work(case):
    d, kv = case["d"], case["kv"]
    held = kv * (d + d // 16)   # bytes of one token's keys and values in the cache
    if case["op"] == "attn":
        pairs, tokens = _pairs(case)
        rows = sum(_lengths(case)[0])
        return {"bytes": max(1, tokens * held + 4 * rows * case["heads"] * d), "flops": 4 * pairs * case["heads"] * d}
    t = case["tokens"]
    back = t * kv * d * 4
    if case["op"] == "read":
        return {"bytes": t * (held + 8) + back, "flops": 2 * t * kv * d}
    o = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "write":
        return {"bytes": t * (2 * kv * d * o + held + 8) + back, "flops": 8 * t * kv * d}
    return {"bytes": t * ((case["heads"] + 2 * kv) * d * o + 4 * case["rot"] + 16 + 2 * case["heads"] * d + held) + back,
            "flops": t * d * (8 * case["heads"] + 16 * kv)}


def _power(n):
    """2^n in 64 bits for whole n, from its bits: exact."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_held(x, slots):
    """The nearest value of the format, by comparisons with the borders between neighbours, in 64 bits."""
    blocks = x.double().unflatten(-1, (-1, 32))
    _, power = torch.frexp(blocks.abs().max(-1, keepdim=True).values)
    unit = _power(power - 3)
    a = blocks.abs() * _power(3 - power)
    value = torch.zeros_like(a)
    # (border, whether the border itself goes up, the step there)
    for border, up, step in ((0.25, False, 0.5), (0.75, True, 0.5), (1.25, False, 0.5), (1.75, True, 0.5), (2.5, False, 1.0), (3.5, True, 1.0), (5.0, False, 2.0)):
        value += step * (a >= border if up else a > border)
    value = torch.copysign(value * unit, blocks).flatten(-2)
    value[slots < 0] = 0.0
    return value


def _exact_values(codes, scales):
    low, high = torch.bitwise_and(codes, 15).long(), torch.bitwise_right_shift(codes, 4).long()
    n = torch.stack([low, high], -1).flatten(-2)
    field, frac = (n % 8) // 2, (n % 2).double()
    mag = torch.where(field == 0, frac * 0.5, (1.0 + 0.5 * frac) * _power(field - 1))
    mag = torch.where(n >= 8, -mag, mag)
    return mag * _power(scales.long().repeat_interleave(32, -1) - 127)


def exact(case, seed):
    """From the definitions, in 64 bits: sequence by sequence, a softmax over the keys that are seen."""
    s = prepare(case, seed)
    kv, d, page = case["kv"], case["d"], case["page"]
    if case["op"] == "write":
        return _exact_held(s["k"], s["slots"]), _exact_held(s["v"], s["slots"])
    if case["op"] == "read":
        both = []
        for c in (0, 2):
            x = _exact_values(s["cache"][c], s["cache"][c + 1]).transpose(1, 2).reshape(-1, kv, d)
            x = x[s["slots"].clamp(min=0)]
            x[s["slots"] < 0] = 0.0
            both.append(x)
        return tuple(both)
    heads = case["heads"]
    if case["op"] == "rope":
        x = s["qkv"].double().view(case["tokens"], -1, d)
        q, k, v = x.split([heads, kv, kv], 1)
        angles = s["table"].double()[s["positions"]]
        half = case["rot"] // 2
        turn = torch.complex(angles[:, :half], angles[:, half:]).unsqueeze(1)
        made = []
        for y, w in ((q, s["wq"]), (k, s["wk"])):
            if w is not None:
                y = y / torch.sqrt(torch.linalg.vector_norm(y, dim=-1, keepdim=True).square() / d + EPS) * w.double()
            y = y.clone()
            first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else (slice(0, half), slice(half, 2 * half))
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            made.append(y)
        return made[0], _exact_held(made[1], s["slots"]), _exact_held(v, s["slots"])
    out = torch.zeros(s["total"], heads, d, dtype=torch.float64, device="cuda")
    at = 0
    for i, (new, old) in enumerate(zip(*_lengths(case))):
        if new == 0 or old == 0:
            at += new
            continue
        pages = s["table"][i, :-(-old // page)].long()
        keys, values = (_exact_values(s["cache"][c][pages], s["cache"][c + 1][pages]).permute(1, 0, 2, 3).reshape(kv, -1, d)[:, :old] for c in (0, 2))
        pos = torch.arange(old - new, old, device="cuda")[:, None]
        j = torch.arange(old, device="cuda")
        hidden = torch.zeros(new, old, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden = j > pos
            if case["window"]:
                hidden |= j <= pos - case["window"]
        for h in range(heads):
            t = s["q"][at:at + new, h].double() @ keys[h // (heads // kv)].t() * s["scale"]
            t[hidden] = -math.inf
            if s["sink"] is not None:
                t = torch.cat([t, s["sink"][h].double().expand(new, 1)], 1)
            t = torch.nan_to_num(torch.softmax(t, 1))[:, :old]
            out[at:at + new, h] = t @ values[h // (heads // kv)]
        at += new
    return out
