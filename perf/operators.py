"""The serving and position operators beside the attention layer, as they are measured.

A case names one operator and its sizes; ``run`` computes it in plain torch
operations, or, where ``own`` is true, through the package's entry points:

  rope_fwd, rope_bwd  rotary positions with one to four axes on Q and K
  cache_write         K and V of new tokens into a paged cache (as they are, or e4m3 with a scale per row)
  cache_read          the tokens of each sequence gathered back from their pages
  attn_decode         attention of one new token per sequence over the paged cache
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
_BYTES = {"bf16": 2, "fp32": 4, "e4m3": 1}
E4M3_MAX = 448.0
MIN_AMAX = 2.0 ** -100


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # rotary: a decode step of 16 sequences far into their contexts
        dict(name="rope_step", op="rope_fwd", tokens=16, hq=32, hkv=8, d=128, rot=128, axes=1, span=131072,
             dtype="bf16", out="bf16", layout="head", pairs="half"),
        # a video of 19 frames of 30 x 30 patches, three axes
        dict(name="rope_video", op="rope_fwd", tokens=17100, hq=32, hkv=8, d=128, rot=128, axes=3, span=4096,
             dtype="bf16", out="bf16", layout="seq", pairs="half"),
        # the gradients of the 64K layer (fp32, sequence layout), on their way to the projection's backward
        dict(name="rope_grad_64k", op="rope_bwd", tokens=65536, hq=32, hkv=8, d=128, rot=128, axes=1, span=65536,
             dtype="fp32", out="bf16", layout="seq", pairs="half"),
        # one new token each of 64 sequences
        dict(name="write_step_e4m3", op="cache_write", seqs=64, tokens=64, hkv=8, d=128, page=16, dtype="bf16",
             cache="e4m3", layout="head"),
        # the prompts of the packed workload
        dict(name="write_packed_e4m3", op="cache_write", seqs=12, tokens=131072, hkv=8, d=128, page=64, dtype="bf16",
             cache="e4m3", layout="head"),
        # a chunk of one prompt, kept as it is
        dict(name="write_chunk_bf16", op="cache_write", seqs=1, tokens=8191, hkv=8, d=64, page=16, dtype="bf16",
             cache="bf16", layout="seq"),
        # a few short prefixes
        dict(name="read_few_bf16", op="cache_read", seqs=5, tokens=2047, hkv=8, d=128, page=16, dtype="bf16",
             cache="bf16", layout="seq"),
        # a long context brought back for another prompt chunk
        dict(name="read_64k_e4m3", op="cache_read", seqs=1, tokens=65536, hkv=8, d=128, page=64, dtype="bf16",
             cache="e4m3", layout="head"),
        # the first tokens of one answer: latency
        dict(name="decode_one_short", op="attn_decode", seqs=1, longest=777, ragged=False, hq=32, hkv=8, d=128, page=16,
             dtype="bf16", cache="bf16", layout="head"),
        # a served batch, lengths as the packed documents'
        dict(name="decode_batch_bf16", op="attn_decode", seqs=64, longest=32768, ragged=True, hq=32, hkv=8, d=128,
             page=16, dtype="bf16", cache="bf16", layout="head"),
        # one sequence of a million tokens, 8-bit cache
        dict(name="decode_million_e4m3", op="attn_decode", seqs=1, longest=1048576, ragged=False, hq=32, hkv=8, d=128,
             page=64, dtype="bf16", cache="e4m3", layout="head"),
        # full-precision heads of their own
        dict(name="decode_mha_fp32", op="attn_decode", seqs=24, longest=4096, ragged=True, hq=8, hkv=8, d=64, page=32,
             dtype="fp32", cache="fp32", layout="seq"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_fwd", "rope_bwd", "cache_write", "cache_read", "attn_decode", "attn_decode"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 4, 6, 8, 16])
    layout = rng.choice(["seq", "head"])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if op in ("rope_fwd", "rope_bwd"):
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        out = "bf16" if dtype == "bf16" else rng.choice(["bf16", "fp32"]) if op == "rope_bwd" else "fp32"
        rot = rng.choice([d, d, d // 2, 48])
        return dict(op=op, tokens=min(_log(rng, 1, 65536), (1 << 28) // (hkv * (group + 1) * d)), hq=hkv * group, hkv=hkv,
                    d=d, rot=rot, axes=rng.choice([1, 1, 2, 3, 4]), span=_log(rng, 16, 1 << 20), dtype=dtype, out=out,
                    layout=layout, pairs=rng.choice(["half", "half", "adjacent"]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    cache = rng.choice([dtype, "e4m3"])
    if op in ("cache_write", "cache_read"):
        tokens = _log(rng, 1, 100000)
        return dict(op=op, seqs=min(tokens, _log(rng, 1, 100)), tokens=tokens, hkv=hkv, d=d, page=page, dtype=dtype,
                    cache=cache, layout=layout)
    if dtype == "fp32":
        cache = "fp32"
    longest = _log(rng, 1, 131072)
    seqs = _log(rng, 1, min(128, max(1, (1 << 30) // (longest * hkv * d * _BYTES[cache]))))
    return dict(op=op, seqs=seqs, longest=longest, ragged=rng.random() < 0.7, hq=hkv * group, hkv=hkv, d=d, page=page,
                dtype=dtype, cache=cache, layout=layout)


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, spread evenly over their logarithm, in a mixed order."""
    return [int(round(lo * (hi / lo) ** ((i * 0.6180339887498949 + 0.5) % 1.0))) for i in range(n)]


def _lengths(c):
    """The cached length of every sequence of an attention case: the first is the longest, and a ragged batch
    of four or more has an empty place."""
    n, top = c["seqs"], c["longest"]
    if not c["ragged"]:
        return [top] * n
    got = [top] + _spread(n - 1, max(1, top // 64), top)
    if n >= 4:
        got[n // 2] = 0
    return got


def _new(c):
    """(new tokens, tokens that were there before) of every sequence of a cache case."""
    n, t = c["seqs"], c["tokens"]
    if n == t:
        return [1] * n, [37 * i % 211 + 5 for i in range(n)]
    w = _spread(n, 1, 64)
    new = [max(1, (t - n) * x // sum(w)) for x in w] if t > n else [1] * n
    new[0] += t - sum(new)
    return new, [37 * i % 211 for i in range(n)]


def work(c):
    if c["op"] in ("rope_fwd", "rope_bwd"):
        n = c["tokens"] * (c["hq"] + c["hkv"]) * c["d"]
        return {"bytes": n * (_BYTES[c["dtype"]] + _BYTES[c["out"]]) + 4 * c["axes"] * c["tokens"], "flops": 3 * n * c["rot"] // c["d"]}
    if c["op"] in ("cache_write", "cache_read"):
        n = 2 * c["tokens"] * c["hkv"]
        return {"bytes": n * c["d"] * (_BYTES[c["dtype"]] + _BYTES[c["cache"]]) + (4 * n if c["cache"] == "e4m3" else 0),
                "flops": 2 * n * c["d"] if c["cache"] == "e4m3" else 0}
    total = sum(_lengths(c))
    rows = 2 * total * c["hkv"]
    return {"bytes": rows * c["d"] * _BYTES[c["cache"]] + (4 * rows if c["cache"] == "e4m3" else 0)
            + c["seqs"] * c["hq"] * (2 * c["d"] * _BYTES[c["dtype"]] + 4), "flops": 4 * total * c["hq"] * c["d"]}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _heads(g, tokens, h, d, dtype, layout, gain=1.0):
    """N(0, gain^2), [tokens, h, d] or, in head layout, [h, tokens, d]."""
    shape = (h, tokens, d) if layout == "head" else (tokens, h, d)
    return (torch.randn(shape, generator=g, device="cuda") * gain).to(_DT[dtype])


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(g, pages, extra=1):
    """A page table with the pages of every sequence in a mixed order; entries of no page are -1."""
    total = sum(pages)
    order = torch.randperm(total + 3, generator=g, device="cuda")[:total].to(torch.int32)
    width = max(pages) + extra
    at = torch.zeros(len(pages), dtype=torch.int64)
    at[1:] = torch.cumsum(torch.tensor(pages, dtype=torch.int64), 0)[:-1]
    col = torch.arange(width, device="cuda")
    used = col[None] < _ints(pages)[:, None]
    where = (at.cuda()[:, None] + col[None]).clamp_(max=max(total - 1, 0))
    return torch.where(used, order[where] if total else torch.zeros_like(where, dtype=torch.int32), -1).to(torch.int32).contiguous(), total + 3


def _filled(g, c, pages):
    """The two caches (and scales) with rows in every slot."""
    got = []
    for _ in range(2):
        shape = (pages, c["hkv"], c["page"], c["d"])
        codes = torch.empty(shape, dtype=_DT[c["cache"]], device="cuda")
        scale = torch.empty(shape[:3], device="cuda") if c["cache"] == "e4m3" else None
        step = max(1, (1 << 27) // (c["hkv"] * c["page"] * c["d"]))
        for i in range(0, pages, step):
            x = torch.randn((min(step, pages - i),) + shape[1:], generator=g, device="cuda")
            if scale is None:
                codes[i:i + step] = x.to(codes.dtype)
            else:
                amax = x.abs().amax(-1)
                codes[i:i + step] = (x * (E4M3_MAX / amax)[..., None]).to(codes.dtype)
                scale[i:i + step] = amax / E4M3_MAX
        got.append((codes, scale))
    return got


def prepare(c, seed):
    g = _gen(seed)
    if c["op"] in ("rope_fwd", "rope_bwd"):
        half = c["rot"] // 2
        return {"c": c,
                "q": _heads(g, c["tokens"], c["hq"], c["d"], c["dtype"], c["layout"]),
                "k": _heads(g, c["tokens"], c["hkv"], c["d"], c["dtype"], c["layout"]),
                "pos": torch.randint(0, c["span"], (c["axes"], c["tokens"]), generator=g, device="cuda", dtype=torch.int32),
                "freq": torch.tensor([1e6 ** (-i / half) for i in range(half)], dtype=torch.float64),
                "axis": torch.tensor([i * c["axes"] // half for i in range(half)], dtype=torch.int32)}
    if c["op"] in ("cache_write", "cache_read"):
        new, before = _new(c)
        first = before if c["op"] == "cache_read" else [0] * len(new)
        pages = [-(-(a + b) // c["page"]) for a, b in zip(new, before)]
        table, n = _table(g, pages)
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        s = {"c": c, "table": table, "cu": _ints(cu), "first": _ints(first), "lens": _ints([a + b for a, b in zip(new, before)])}
        if c["op"] == "cache_read":
            (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _filled(g, c, n)
            return s
        for x in ("k", "v"):
            s[x] = _heads(g, c["tokens"], c["hkv"], c["d"], c["dtype"], c["layout"])
            s[x + "c"] = torch.zeros((n, c["hkv"], c["page"], c["d"]), dtype=_DT[c["cache"]], device="cuda")
            s[x + "s"] = torch.zeros((n, c["hkv"], c["page"]), device="cuda") if c["cache"] == "e4m3" else None
        return s
    lens = _lengths(c)
    table, n = _table(g, [-(-x // c["page"]) for x in lens])
    s = {"c": c, "table": table, "lens": _ints(lens), "longest": max(lens)}
    (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _filled(g, c, n)
    # scores of a spread of about 2, as trained heads have
    s["q"] = _heads(g, c["seqs"], c["hq"], c["d"], c["dtype"], c["layout"], 2.0)
    return s


# ------------------------------------------------------------------ the plain forms

def _tokens_first(x, c):
    return x.transpose(0, 1) if c["layout"] == "head" else x


def _rope(s):
    c, half = s["c"], s["c"]["rot"] // 2
    # angles in 64 bits: those of far positions lose everything in 32
    ang = s["pos"].double()[s["axis"].long().cuda()] * s["freq"].cuda()[:, None]
    if c["op"] == "rope_bwd":
        ang = -ang
    cos, sin = ang.cos().float().T[:, None], ang.sin().float().T[:, None]
    out = []
    for x in (s["q"], s["k"]):
        x = _tokens_first(x, c).float()
        if c["pairs"] == "half":
            a, b = x[..., :half], x[..., half:2 * half]
        else:
            a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = (a * cos - b * sin, a * sin + b * cos)
        y = torch.cat(y, -1) if c["pairs"] == "half" else torch.stack(y, -1).flatten(-2)
        y = torch.cat((y, x[..., c["rot"]:]), -1).to(_DT[c["out"]])
        out.append(_tokens_first(y, c).contiguous())
    return out


def _slots(s, first):
    """(page, slot in the page) of every token of the packed sequences."""
    c = s["c"]
    t = torch.arange(c["tokens"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    p = first.long()[b] + t - s["cu"].long()[b]
    return s["table"].long()[b, p // c["page"]], p % c["page"]


def _write(s):
    c = s["c"]
    page, slot = _slots(s, s["lens"] - (s["cu"][1:] - s["cu"][:-1]))
    out = []
    for x in ("k", "v"):
        rows = _tokens_first(s[x], c)
        if c["cache"] == "e4m3":
            y = rows.float()
            amax = y.abs().amax(-1).clamp(min=MIN_AMAX)
            most = torch.full_like(amax, E4M3_MAX)
            s[x + "s"][page, :, slot] = amax / most
            rows = (y * (most / amax)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            s[x + "c"].view(torch.uint8)[page, :, slot] = rows
            out += [s[x + "c"], s[x + "s"]]
        else:
            s[x + "c"][page, :, slot] = rows
            out.append(s[x + "c"])
    return out


def _read(s):
    c = s["c"]
    page, slot = _slots(s, s["first"])
    out = []
    for x in ("k", "v"):
        y = s[x + "c"].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn) if c["cache"] == "e4m3" else s[x + "c"][page, :, slot]
        if c["cache"] == "e4m3":
            y = y.float() * s[x + "s"][page, :, slot][..., None]
        out.append(_tokens_first(y.to(_DT[c["dtype"]]), c).contiguous())
    return out


def _decode(s):
    c, n = s["c"], s["longest"]
    b, g = c["seqs"], c["hq"] // c["hkv"]
    cols = -(-n // c["page"])
    pages = s["table"][:, :cols].long().clamp(min=0)
    seen = torch.arange(cols * c["page"], device="cuda") < s["lens"][:, None]
    kv = []
    for x in ("k", "v"):
        rows = s[x + "c"].view(torch.uint8)[pages].view(torch.float8_e4m3fn) if c["cache"] == "e4m3" else s[x + "c"][pages]
        rows = rows.float()
        if c["cache"] == "e4m3":
            rows = rows * s[x + "s"][pages][..., None]
        rows = rows.permute(0, 2, 1, 3, 4).reshape(b, c["hkv"], cols * c["page"], c["d"])
        kv.append(rows.masked_fill(~seen[:, None, :, None], 0.0))
    q = _tokens_first(s["q"], c).float().reshape(b, c["hkv"], g, c["d"])
    score = (q @ kv[0].transpose(-1, -2)) / math.sqrt(c["d"])
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p @ kv[1]) / total.clamp(min=1e-30)
    lse = (top + total.log()).squeeze(-1)
    o = o.reshape(b, c["hq"], c["d"]).to(_DT[c["dtype"]])
    return [_tokens_first(o, c).contiguous(), lse.reshape(b, c["hq"])]


# ------------------------------------------------------------------ the calls

def _own_run(s):
    from long_context_sequence_seq_gb300 import ulysses as U
    c = s["c"]
    if c["op"] in ("rope_fwd", "rope_bwd"):
        if c["op"] == "rope_fwd":
            return U.rope_fwd(s["q"], s["k"], s["pos"], s["freq"], s["axis"], layout=c["layout"], pairs=c["pairs"])
        return U.rope_bwd(s["q"], s["k"], s["pos"], s["freq"], s["axis"], layout=c["layout"], pairs=c["pairs"],
                          dtype=_DT[c["out"]])
    if c["op"] == "cache_write":
        U.cache_write(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"],
                      cu_new=None if c["seqs"] == c["tokens"] else s["cu"], k_scale=s["ks"], v_scale=s["vs"],
                      layout=c["layout"])
        return [x for x in (s["kc"], s["ks"], s["vc"], s["vs"]) if x is not None]
    if c["op"] == "cache_read":
        return U.cache_read(s["kc"], s["vc"], s["table"], s["cu"], c["tokens"], first=s["first"], k_scale=s["ks"],
                            v_scale=s["vs"], dtype=_DT[c["dtype"]], layout=c["layout"])
    return U.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], k_scale=s["ks"], v_scale=s["vs"],
                         layout=c["layout"])


def run(s):
    if own:
        return _own_run(s)
    op = s["c"]["op"]
    return _rope(s) if op in ("rope_fwd", "rope_bwd") else _write(s) if op == "cache_write" else _read(s) if op == "cache_read" else _decode(s)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rope(c, s):
    sign = -1.0 if c["op"] == "rope_bwd" else 1.0
    turn = torch.empty((c["tokens"], c["rot"] // 2), dtype=torch.complex128, device="cuda")
    for i in range(c["rot"] // 2):
        a = sign * float(s["freq"][i]) * s["pos"][int(s["axis"][i])].to(torch.float64)
        turn[:, i] = torch.complex(a.cos(), a.sin())
    out = []
    for x in (s["q"], s["k"]):
        y = x.double()
        w = turn[None] if c["layout"] == "head" else turn[:, None]
        h = c["rot"] // 2
        ia = torch.arange(h, device="cuda") * (1 if c["pairs"] == "half" else 2)
        ib = ia + (h if c["pairs"] == "half" else 1)
        z = torch.complex(y[..., ia], y[..., ib]) * w
        y[..., ia], y[..., ib] = z.real, z.imag
        out.append(y)
    return out


def _each_token(c, s, first):
    """(sequence's rows in the packed tensor, their pages, their slots), a sequence at a time."""
    cu, table = s["cu"].tolist(), s["table"].long()
    for b in range(c["seqs"]):
        p = torch.arange(cu[b + 1] - cu[b], device="cuda") + first[b]
        yield slice(cu[b], cu[b + 1]), table[b][p // c["page"]], p % c["page"]


def _exact_write(c, s):
    new = [y - x for x, y in zip(s["cu"].tolist(), s["cu"].tolist()[1:])]
    first = [a - b for a, b in zip(s["lens"].tolist(), new)]
    out = []
    for x in ("k", "v"):
        rows, codes = s[x].double(), torch.zeros(s[x + "c"].shape, dtype=torch.float64, device="cuda")
        scale = None if s[x + "s"] is None else torch.zeros(s[x + "s"].shape, dtype=torch.float64, device="cuda")
        for at, page, slot in _each_token(c, s, first):
            y = rows[:, at].transpose(0, 1) if c["layout"] == "head" else rows[at]
            if scale is not None:
                f = y.abs().max(-1).values.clamp(min=MIN_AMAX) / E4M3_MAX
                scale[page, :, slot] = f
                y = y / f[..., None]
            codes[page, :, slot] = y
        out += [codes] if scale is None else [codes, scale]
    return out


def _exact_read(c, s):
    first, out = s["first"].tolist(), []
    for x in ("k", "v"):
        got = torch.empty((c["tokens"], c["hkv"], c["d"]), dtype=torch.float64, device="cuda")
        cache = s[x + "c"].float()
        for at, page, slot in _each_token(c, s, first):
            y = cache[page, :, slot].double()
            got[at] = y if s[x + "s"] is None else y * s[x + "s"][page, :, slot].double()[..., None]
        out.append(got.transpose(0, 1).contiguous() if c["layout"] == "head" else got)
    return out


def _exact_decode(c, s):
    q = (s["q"].transpose(0, 1) if c["layout"] == "head" else s["q"]).double()
    group = c["hq"] // c["hkv"]
    o = torch.zeros((c["seqs"], c["hq"], c["d"]), dtype=torch.float64, device="cuda")
    lse = torch.full((c["seqs"], c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if not n:
            continue
        pages = s["table"][b, :-(-n // c["page"])].long()
        for h in range(c["hkv"]):
            k, v = (s[x + "c"][:, h].view(torch.uint8)[pages].view(torch.float8_e4m3fn) if c["cache"] == "e4m3" else s[x + "c"][pages, h]
                    for x in ("k", "v"))
            k, v = (x.float().double().reshape(-1, c["d"])[:n] for x in (k, v))
            if c["cache"] == "e4m3":
                k, v = (x * s[w][pages, h].reshape(-1)[:n, None].double() for x, w in ((k, "ks"), (v, "vs")))
            z = k @ q[b, h * group:(h + 1) * group].T * c["d"] ** -0.5
            lse[b, h * group:(h + 1) * group] = torch.logsumexp(z, 0)
            o[b, h * group:(h + 1) * group] = torch.softmax(z, 0).T @ v
    return [o.transpose(0, 1).contiguous() if c["layout"] == "head" else o, lse]


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("rope_fwd", "rope_bwd"):
        return _exact_rope(c, s)
    return {"cache_write": _exact_write, "cache_read": _exact_read, "attn_decode": _exact_decode}[c["op"]](c, s)
