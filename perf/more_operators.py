"""Cases of the operators that take new tokens of a prompt, a chunk or a draft through the 4-bit KV cache: rotary positions, the
append with the rotation on its way, and the attention of several new tokens per sequence over the paged cache.

`own` chooses the side: False computes each operator with elementary torch operations (FP32; FP64 for angles and for values next to
a border of the 4-bit grid), True makes the package's calls.
4-bit data is MXFP4 (OCP MX v1.0): E2M1 codes, two per byte with the even element in the low nibble, and one E8M0 scale
(2^(code - 127)) per 32 elements.
"""
import functools
import math
import random

import torch

own = False

FLOATS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
FOUR_BIT = 0.5 + 1 / 32  # bytes an element takes with its share of a scale
PIECE = 1 << 28  # logits that the plain attention holds at a time


def listed():
    return [
        # queries and keys of one token of a decode step, the shortest call
        dict(name="rope_one_token", op="rope", tokens=1, heads=36, dim=128, rot=128, pairs="half", far=5000, magnitude=1.0, x="bf16", pad=4),
        # a draft batch in FP32 whose whole head of 96 rotates, frequencies stretched for a long context with their magnitude
        dict(name="rope_scaled_draft", op="rope", tokens=129, heads=9, dim=96, rot=96, pairs="half", far=130000, magnitude=1.2, x="f32", pad=0),
        # a prompt far into a document: neighbouring elements pair up in the first quarter of each head
        dict(name="rope_prompt_part", op="rope", tokens=7001, heads=20, dim=256, rot=64, pairs="neighbours", far=1000000, magnitude=1.0, x="f16", pad=2),
        # every sequence of a decode batch adds one token
        dict(name="append_step", op="append", seqs=64, new=1, before=8192, heads=4, group=16, dim=128, rot=128, pairs="half", page=16, kv="bf16"),
        # a few drafts far behind their prompts, an odd group of query heads and half of the head rotated
        dict(name="append_drafts", op="append", seqs=5, new=9, before=200000, heads=2, group=7, dim=64, rot=32, pairs="neighbours", page=32, kv="f16"),
        # prompts of different lengths enter the cache, some behind a cached prefix
        dict(name="append_prompts", op="append", seqs=13, new=6000, before=500, heads=8, group=4, dim=128, rot=128, pairs="half", page=64, kv="bf16"),
        # the first words of a few conversations, one of them with nothing new
        dict(name="chunk_short", op="chunk", seqs=3, new=20, before=25, heads=2, group=5, dim=64, page=16, q="f16", window=0, idle=1),
        # drafts of a decode batch, verified in one pass
        dict(name="chunk_drafts", op="chunk", seqs=16, new=5, before=8192, heads=4, group=8, dim=128, page=16, q="bf16", window=0, idle=0),
        # a short question about a long document
        dict(name="chunk_on_document", op="chunk", seqs=1, new=7, before=131000, heads=8, group=5, dim=128, page=64, q="f16", window=0, idle=0),
        # one piece of a long prompt, taken chunk by chunk
        dict(name="chunk_of_prompt", op="chunk", seqs=1, new=2048, before=30011, heads=4, group=7, dim=128, page=64, q="f16", window=0, idle=0),
        # a batch of follow-up prompts in a layer that sees the last 1000 keys, with wide heads
        dict(name="chunk_window", op="chunk", seqs=24, new=1500, before=4000, heads=2, group=6, dim=256, page=128, q="bf16", window=1000, idle=2),
        # a whole prompt from an empty cache
        dict(name="chunk_prompt", op="chunk", seqs=1, new=8192, before=0, heads=4, group=16, dim=128, page=64, q="bf16", window=0, idle=0),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rope", "append", "chunk", "chunk"])
    pairs = rng.choice(["half", "neighbours"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        heads, magnitude = _spread(rng, 1, 80), rng.choice([1.0, 1.0, round(rng.uniform(0.8, 1.5), 3)])
        tokens = _spread(rng, 1, min(8192, 7001 * 20 * 256 // (heads * dim)))
        return dict(op=op, tokens=tokens, heads=heads, dim=dim, rot=16 * rng.randint(1, dim // 16), pairs=pairs, far=_spread(rng, 16, 1000000), magnitude=magnitude, x=rng.choice(["bf16", "f16", "f32"]), pad=rng.choice([0, 0, 1, 2, 8]))
    seqs, heads, dim = _spread(rng, 1, 64 if op == "append" else 32), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    page, group = rng.choice([16, 32, 64, 128, 256]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if op == "append":
        new = rng.choice([1, _spread(rng, 1, 6000)])
        new = max(1, min(new, 78000 * 5 * 128 // (seqs * (group + 1) * dim)))
        return dict(op=op, seqs=seqs, new=new, before=_spread(rng, 1, 200000), heads=heads, group=group, dim=dim, rot=rng.choice([dim, dim, dim // 2, dim // 4]), pairs=pairs, page=page, kv=rng.choice(["bf16", "f16"]))
    new, before = _spread(rng, 1, 8192), rng.choice([0, _spread(rng, 1, 131000), _spread(rng, 1, 131000)])
    before = min(before, 64 * 8192 * 4 * 128 // (seqs * heads * dim))  # the cache that a case holds
    most = 8192 * 4096 * 64 * 128  # rows by keys by elements of the largest
    while new > 1 and seqs * new * (before + new / 2) * heads * group * dim > most:
        new -= -(-new // 16)
    return dict(op=op, seqs=seqs, new=new, before=before, heads=heads, group=group, dim=dim, page=page, q=rng.choice(["bf16", "f16"]), window=rng.choice([0, 0, 1000]), idle=rng.choice([0, 1]) if seqs > 1 else 0)


def _lengths(case):
    """(cached, new) of a case's sequences. One has the most new tokens, and the most before them where these are attended to."""
    r = random.Random("%s %s" % (case["op"], sorted((k, v) for k, v in case.items() if k not in ("name", "op"))))
    before, new = case["before"], case["new"]
    some = []
    for i in range(case["seqs"]):
        n = new if i == 0 else _spread(r, 1, new)
        if case["op"] == "append":
            some.append((r.randint(0, before), n))
        else:
            some.append((before if i == 0 else r.randint(before // 8, before), 0 if i and i <= case["idle"] else n))
    return some


def _pairs_seen(case):
    """(query, key) pairs that attention takes, over the sequences."""
    total = 0
    for before, new in _lengths(case):
        w = case["window"] or before + new
        short = min(new, max(0, w - before))  # queries that see everything before them
        total += short * before + short * (short + 1) // 2 + (new - short) * w
    return total


def _keys_seen(case):
    return sum(0 if not n else n + (min(b, case["window"] - 1) if case["window"] else b) for b, n in _lengths(case))


def work(case):
    if case["op"] == "rope":
        values = case["tokens"] * case["heads"] * case["dim"]
        turned = case["tokens"] * case["heads"] * case["rot"]
        return {"bytes": 2 * values * BYTES[case["x"]] + 4 * case["tokens"], "flops": 3 * turned}
    tokens = sum(n for _, n in _lengths(case))
    rows = tokens * case["heads"] * case["dim"]
    if case["op"] == "append":  # queries in and out; keys and values in, into the cache, and read back
        return {"bytes": 2 * rows * (case["group"] * BYTES[case["kv"]] + 2 * (BYTES[case["kv"]] + FOUR_BIT)), "flops": rows * (3 * case["group"] + 7)}
    ends = 2 * rows * case["group"] * BYTES[case["q"]] + 4 * tokens * case["heads"] * case["group"]
    keys = 2 * _keys_seen(case) * case["heads"] * case["dim"] * FOUR_BIT
    return {"bytes": keys + ends, "flops": 4 * _pairs_seen(case) * case["heads"] * case["group"] * case["dim"]}


def _freqs(rot, stretched):
    """Radians per position of each pair. Stretched: slow ones, with less than a turn in 4096 positions, go 8 times slower, fast
    ones, with more than 32, stay, and those between are mixed."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if stretched:
        keep = ((4096 * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        f = f * (keep + (1 - keep) / 8)
    return f


def _inputs(case, seed):
    """What the case computes from, the same for every side."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "rope":
        t, heads, dim = case["tokens"], case["heads"], case["dim"]
        wide = normal(t, heads + case["pad"], dim).to(FLOATS[case["x"]])
        start = r.randint(0, case["far"])
        if t > 256:  # a prompt
            pos = torch.arange(start, start + t, dtype=torch.int32, device="cuda")
        else:
            pos = torch.randint(0, case["far"] + 1, (t,), generator=g, device="cuda", dtype=torch.int32)
        return {"x": wide[:, :heads], "pos": pos, "freqs": _freqs(case["rot"], case["magnitude"] != 1).cuda()}
    order = list(range(case["seqs"]))
    r.shuffle(order)  # which request has which length
    lengths = [_lengths(case)[i] for i in order]
    heads, group, dim, page = case["heads"], case["group"], case["dim"], case["page"]
    append = case["op"] == "append"
    kind = FLOATS[case["kv" if append else "q"]]
    news, held = [n for _, n in lengths], [b + n for b, n in lengths]
    tokens = sum(news) if append else sum(held)
    loud = 1 + 3 * (torch.rand(1, heads, dim, generator=g, device="cuda") < 0.05)  # keys have channels of their own size
    k, v = normal(tokens, heads, dim) * loud, normal(tokens, heads, dim) * 0.7
    q = normal(sum(news), heads * group, dim)
    if append:  # one projection's output
        qkv = torch.cat([q, k, v], 1).to(kind)
        q, k, v = qkv.split([heads * group, heads, heads], 1)
    else:
        q, k, v = q.to(kind), k.to(kind), v.to(kind)
    per = [-(-t // page) for t in held]
    pages = torch.randperm(sum(per), generator=g, device="cuda").to(torch.int32)  # pages come in any order
    table = torch.zeros(case["seqs"], max(1, max(per)), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(per):
        table[i, :n] = pages[at : at + n]
        at += n
    s = {"q": q, "k": k, "v": v, "table": table, "pages": max(1, sum(per)), "held": held, "news": news}
    s["before"] = torch.tensor([b for b, _ in lengths], dtype=torch.int32, device="cuda")
    s["cu"] = torch.tensor([0] + [sum(news[: i + 1]) for i in range(len(news))], dtype=torch.int32, device="cuda")
    if append:
        s["freqs"] = _freqs(case["rot"], False).cuda()
    return s


@functools.lru_cache
def _tables():
    """The values of the codes and of the scales, exact: powers of two come from here and not from a library's exp2 or pow."""
    return torch.tensor(E2M1 + [-x for x in E2M1], device="cuda"), torch.tensor([2.0 ** (i - 127) for i in range(255)] + [math.nan], device="cuda")


def _quantise(v):
    """(codes, scales) of v [..., n] in MXFP4, in the plain order: codes uint8 [..., n / 2], scales uint8 [..., n / 32]."""
    a = v.unflatten(-1, (-1, 32))
    top = a.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top)[1] - 3).clamp(-127, 127)
    e = torch.where(top > 0, e, torch.full_like(e, -127))
    a = a / _tables()[1].to(a.dtype)[e + 127]
    m = a.abs()
    c = (m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5)
    c = (c + 8 * torch.signbit(a)).to(torch.uint8).flatten(-2)
    return c[..., 0::2] + 16 * c[..., 1::2], (e.squeeze(-1) + 127).to(torch.uint8)


def _values(codes, scales):
    """The FP32 values of plain-order MXFP4."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    code, scale = _tables()
    return (code[c].unflatten(-1, (-1, 32)) * scale[scales.long()].unsqueeze(-1)).flatten(-2)


def _rotate(x, pos, freqs, pairs, magnitude=1.0):
    """x [tokens, heads, dim] in FP32 or FP64 with its pairs turned by their tokens' positions, the angles in FP64."""
    angle = pos.double()[:, None, None] * freqs
    cos, sin = (torch.cos(angle) * magnitude).to(x.dtype), (torch.sin(angle) * magnitude).to(x.dtype)
    rot = 2 * freqs.numel()
    a, b = x[..., :rot].chunk(2, -1) if pairs == "half" else (x[..., :rot:2], x[..., 1:rot:2])
    turned = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat(turned, -1) if pairs == "half" else torch.stack(turned, -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _positions(s):
    """The sequence and the position of each new token."""
    n = torch.tensor(s["news"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(s["news"]), device="cuda"), n)
    return seq, torch.arange(len(seq), device="cuda") - s["cu"].long()[seq] + s["before"].long()[seq]


def _slots(s, seq, pos, page):
    return s["table"].long()[seq, pos // page] * page + pos % page


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from output_centric_expert_gb300 import block_ops as ops
    s["case"] = case
    if "freqs" in s and own:  # a model's rotation, made once
        s["rope"] = ops.Rope(s["freqs"], interleaved=case["pairs"] == "neighbours", magnitude=case.get("magnitude", 1.0))
    if case["op"] == "rope":
        s["out"] = torch.empty(s["x"].shape, dtype=s["x"].dtype, device="cuda")
        return s
    heads, group, dim, page = case["heads"], case["group"], case["dim"], case["page"]
    s["out"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    if case["op"] == "append":
        if own:
            s["cache"] = ops.Kv4Cache(s["pages"], page, heads, dim)
            s["k_out"], s["v_out"] = (torch.empty(s["k"].shape, dtype=s["k"].dtype, device="cuda") for _ in range(2))
        else:
            shape = (s["pages"] * page, heads)
            s["cache"] = [torch.zeros(*shape, n, dtype=torch.uint8, device="cuda") for n in (dim // 2, dim // 32, dim // 2, dim // 32)]
        return s
    if own:  # a cache that holds the sequences, their new tokens among them
        s["cache"] = ops.Kv4Cache(s["pages"], page, heads, dim)
        cu = torch.tensor([0] + [sum(s["held"][: i + 1]) for i in range(len(s["held"]))], dtype=torch.int32, device="cuda")
        ops.wd_kv4_append(s["cache"], s["k"], s["v"], s["table"], torch.zeros_like(s["before"]), cu)
        s["work"] = ops.kv4_chunk_workspace(s["cache"], s["q"].shape[0], heads * group)
        s["lse"] = torch.empty(s["q"].shape[:2], device="cuda")
    else:
        held = torch.tensor(s["held"], device="cuda")
        seq = torch.repeat_interleave(torch.arange(case["seqs"], device="cuda"), held)
        pos = torch.arange(len(seq), device="cuda") - (torch.cumsum(held, 0) - held)[seq]
        at = _slots(s, seq, pos, page)
        s["cache"] = []
        for x in (s["k"], s["v"]):
            for part in _quantise(x.float()):
                kept = torch.zeros(s["pages"] * page, *part.shape[1:], dtype=torch.uint8, device="cuda")
                kept[at] = part
                s["cache"].append(kept)
    del s["k"], s["v"]
    return s


def _run_own(s, case):
    from output_centric_expert_gb300 import block_ops as ops

    if case["op"] == "rope":
        return ops.wd_rope(s["rope"], s["x"], s["pos"], s["out"])
    if case["op"] == "append":  # the cache's values are what the new tokens read back as
        ops.wd_kv4_rope_append(s["cache"], s["rope"], s["q"], s["k"], s["v"], s["table"], s["before"], s["out"], s["cu"])
        ops.wd_kv4_gather(s["cache"], s["table"], s["before"], s["k_out"], s["v_out"], s["cu"])
        return s["out"], s["k_out"], s["v_out"]
    ops.wd_kv4_attend_chunk(s["cache"], s["q"], s["table"], s["before"], s["out"], s["work"], s["cu"], lse=s["lse"], window=case["window"])
    return s["out"], s["lse"]


def _attend(s, case):
    heads, group, dim = case["heads"], case["group"], case["dim"]
    outs, sums, row = [], [], 0
    for i, (held, new) in enumerate(zip(s["held"], s["news"])):
        if not new:
            continue
        at = torch.arange(held, device="cuda")
        slots = _slots(s, torch.full_like(at, i), at, case["page"])
        k, ks, v, vs = (x[slots] for x in s["cache"])
        k, v = _values(k, ks).transpose(0, 1), _values(v, vs).transpose(0, 1)
        step = max(1, PIECE // (heads * group * held))
        for first in range(0, new, step):
            n = min(step, new - first)
            q = s["q"][row + first : row + first + n].float().unflatten(1, (heads, group))
            pos = held - new + first + torch.arange(n, device="cuda")
            logits = torch.einsum("nhgd,htd->hgnt", q, k) * dim ** -0.5
            hidden = at > pos[:, None]
            if case["window"]:
                hidden |= at <= pos[:, None] - case["window"]
            logits.masked_fill_(hidden, -math.inf)
            top = logits.amax(-1, keepdim=True)
            p = torch.exp(logits.sub_(top))
            total = p.sum(-1, keepdim=True)
            out = torch.einsum("hgnt,htd->nhgd", p, v) / total.permute(2, 0, 1, 3)
            outs.append(out.flatten(1, 2).to(s["q"].dtype))
            sums.append((top + torch.log(total)).squeeze(-1).permute(2, 0, 1).flatten(1, 2))
        row += new
    return torch.cat(outs), torch.cat(sums)


def run(state):
    s, case = state, state["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "rope":
        return _rotate(s["x"].float(), s["pos"], s["freqs"], case["pairs"], case["magnitude"]).to(s["x"].dtype)
    if case["op"] == "chunk":
        return _attend(s, case)
    seq, pos = _positions(s)
    slots = _slots(s, seq, pos, case["page"])
    back = [_rotate(s["q"].float(), pos, s["freqs"], case["pairs"]).to(s["q"].dtype)]
    k = _rotate(s["k"].double(), pos, s["freqs"], case["pairs"])  # FP32 would put some on the other side of a border
    for i, x in enumerate((k, s["v"].float())):
        cache = s["cache"][2 * i : 2 * i + 2]
        for held, part in zip(cache, _quantise(x)):
            held[slots] = part
        back.append(_values(*(held[slots] for held in cache)).to(s["k"].dtype))
    return tuple(back)


def _nearest(v):
    """v [..., n] rounded to MXFP4, in 64 bits: the step of a value is half, one or two units of its block's scale."""
    a = v.double().reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    top = a.abs().max(-1, keepdim=True).values
    power = torch.clamp((top.view(torch.int64) >> 52) - 1025, -127, 127)  # the exponent field, less E2M1's own two
    unit = ((power + 1023) << 52).view(torch.float64)
    a = a / torch.where(top > 0, unit, torch.ones_like(unit))
    m = a.abs()
    step = 0.5 * (1 + (m >= 2).double() + 2 * (m >= 4).double())
    return (torch.sign(a) * torch.clamp(torch.round(m / step) * step, max=6.0) * torch.where(top > 0, unit, torch.zeros_like(unit))).reshape(v.shape)


def _turned(x, pos, freqs, pairs, magnitude=1.0):
    """x with its pairs as complex numbers times e^(i angle)."""
    x, rot = x.double(), 2 * freqs.numel()
    if pairs == "half":
        z = torch.complex(x[..., : rot // 2], x[..., rot // 2 : rot])
    else:
        z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous())
    angle = torch.outer(pos.double(), freqs)
    z = z * torch.polar(torch.full_like(angle, magnitude), angle).unsqueeze(1)
    y = x.clone()
    if pairs == "half":
        y[..., : rot // 2], y[..., rot // 2 : rot] = z.real, z.imag
    else:
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    return y


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rope":
        return _turned(s["x"], s["pos"], s["freqs"], case["pairs"], case["magnitude"])
    if case["op"] == "append":
        pos = torch.cat([torch.arange(h - n, h, device="cuda") for h, n in zip(s["held"], s["news"])])
        q, k = (_turned(s[x], pos, s["freqs"], case["pairs"]) for x in "qk")
        return q, _nearest(k), _nearest(s["v"])
    heads, group = case["heads"], case["group"]
    outs, sums, key, row = [], [], 0, 0
    for held, new in zip(s["held"], s["news"]):
        k, v = (_nearest(s[x][key : key + held]) for x in "kv")
        key += held
        step = max(1, (1 << 27) // (heads * group * max(1, held)))
        for first in range(0, new, step):
            n = min(step, new - first)
            pos = torch.arange(held - new + first, held - new + first + n, device="cuda")
            end = held - new + first + n
            start = max(0, end - n - case["window"] + 1) if case["window"] else 0
            at = torch.arange(start, end, device="cuda")
            q = s["q"][row + first : row + first + n].double().reshape(n, heads, group, -1).permute(1, 2, 0, 3).flatten(1, 2)
            z = torch.matmul(q, k[start:end].permute(1, 2, 0)).unflatten(1, (group, n)) / math.sqrt(case["dim"])
            gone = pos[:, None] - at
            z = torch.where((gone >= 0) & (gone < (case["window"] or held)), z, -math.inf)
            total = torch.logsumexp(z, -1)
            o = torch.matmul(torch.exp(z - total[..., None]).flatten(1, 2), v[start:end].permute(1, 0, 2))
            outs.append(o.unflatten(1, (group, n)).permute(2, 0, 1, 3).flatten(1, 2))
            sums.append(total.permute(2, 0, 1).flatten(1, 2))
        row += new
    return torch.cat(outs), torch.cat(sums)
