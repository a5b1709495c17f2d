"""Long contexts in less memory: the cache held in 4 bits, the attention weight its tokens gather, and their eviction.

A case names one operator and its sizes; ``run`` computes it in plain torch
operations, or, where ``own`` is true, through the package's entry points:

  write_4bit    K and V of new tokens into a 4-bit paged cache, and those tokens read back as later chunks see them
  read_4bit     the tokens of each sequence gathered back from a 4-bit cache
  decode_4bit   attention of one new token per sequence over a 4-bit cache
  decode_seen   the same over any cache, adding each cached token's attention weight to what it has gathered
  evict         the tokens with the least weight taken out of each sequence and head, the others closed up in order

Four bits: codes of e2m1 (0, 1/2, 1, 3/2, 2, 3, 4, 6 and their negatives), an
e4m3 scale for every 16 of them and a power of two (in fp32) for the row.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn, "e2m1": torch.uint8}
_BYTES = {"bf16": 2, "fp32": 4, "e4m3": 1, "e2m1": 0.5625}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E4M3_MAX = 448.0
MOST = 6.0 * E4M3_MAX          # the largest code under the largest block scale
MIN_AMAX = 2.0 ** -100


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a chunk of one prompt on its way into the cache
        dict(name="write_chunk", op="write_4bit", seqs=1, tokens=8191, hkv=8, d=128, page=64, dtype="bf16", layout="head"),
        # the prompts of the packed workload
        dict(name="write_packed", op="write_4bit", seqs=12, tokens=131072, hkv=8, d=128, page=64, dtype="bf16", layout="head"),
        # a few short prefixes
        dict(name="read_few", op="read_4bit", seqs=5, tokens=2047, hkv=8, d=64, page=16, dtype="bf16", layout="seq"),
        # a long context brought back for another prompt chunk
        dict(name="read_64k", op="read_4bit", seqs=1, tokens=65536, hkv=8, d=128, page=64, dtype="bf16", layout="head"),
        # the first tokens of one answer: latency
        dict(name="decode_one_short", op="decode_4bit", seqs=1, longest=777, ragged=False, hq=32, hkv=8, d=128, page=16,
             dtype="bf16", cache="e2m1", layout="head"),
        # a served batch, lengths as the packed documents'
        dict(name="decode_batch", op="decode_4bit", seqs=64, longest=32768, ragged=True, hq=32, hkv=8, d=128, page=64,
             dtype="bf16", cache="e2m1", layout="head"),
        # one sequence of a million tokens
        dict(name="decode_million", op="decode_4bit", seqs=1, longest=1048576, ragged=False, hq=32, hkv=8, d=128, page=64,
             dtype="bf16", cache="e2m1", layout="head"),
        # a step of an answer whose cached tokens are being weighed
        dict(name="seen_one_short", op="decode_seen", seqs=1, longest=4099, ragged=False, hq=32, hkv=8, d=128, page=16,
             dtype="bf16", cache="bf16", layout="head"),
        # the served batch, weighed
        dict(name="seen_batch", op="decode_seen", seqs=64, longest=16384, ragged=True, hq=32, hkv=8, d=128, page=16,
             dtype="bf16", cache="bf16", layout="head"),
        # a page's worth of tokens over the budget of 4096, 16 sequences
        dict(name="evict_page", op="evict", seqs=16, longest=4160, ragged=False, keep=4096, recent=512, hkv=8, d=128, page=64,
             dtype="bf16", cache="bf16"),
        # a long prompt cut to what its answer needs
        dict(name="evict_prompt", op="evict", seqs=1, longest=131072, ragged=False, keep=8192, recent=1024, hkv=8, d=128,
             page=64, dtype="bf16", cache="e4m3"),
        # half of a served batch's longest sequences, 4-bit cache
        dict(name="evict_batch", op="evict", seqs=64, longest=16384, ragged=True, keep=4096, recent=256, hkv=8, d=128, page=64,
             dtype="bf16", cache="e2m1"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write_4bit", "read_4bit", "decode_4bit", "decode_4bit", "decode_seen", "decode_seen", "evict", "evict"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 4, 6, 8, 16])
    layout = rng.choice(["seq", "head"])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("write_4bit", "read_4bit"):
        tokens = _log(rng, 1, 100000)
        return dict(op=op, seqs=min(tokens, _log(rng, 1, 100)), tokens=tokens, hkv=hkv, d=d, page=page, dtype=dtype, layout=layout)
    cache = "e2m1" if op == "decode_4bit" else rng.choice([dtype, "e4m3", "e2m1"])
    longest = _log(rng, 1, 131072 if op != "evict" else 65536)
    seqs = _log(rng, 1, min(128, max(1, (1 << 29) // (longest * hkv * d))))
    if op != "evict":
        return dict(op=op, seqs=seqs, longest=longest, ragged=rng.random() < 0.7, hq=hkv * group, hkv=hkv, d=d, page=page,
                    dtype=dtype, cache=cache, layout=layout)
    keep = _log(rng, 1, longest)
    return dict(op=op, seqs=seqs, longest=longest, ragged=rng.random() < 0.7, keep=keep, recent=rng.choice([0, keep // 8, keep // 2]),
                hkv=hkv, d=d, page=page, dtype=dtype, cache=cache)


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, spread evenly over their logarithm, in a mixed order."""
    return [int(round(lo * (hi / lo) ** ((i * 0.6180339887498949 + 0.5) % 1.0))) for i in range(n)]


def _lengths(c):
    """The cached length of every sequence: the first is the longest, and a ragged batch of four or more has an
    empty place."""
    n, top = c["seqs"], c["longest"]
    if not c["ragged"]:
        return [top] * n
    got = [top] + _spread(n - 1, max(1, top // 64), top)
    if n >= 4:
        got[n // 2] = 0
    return got


def _new(c):
    """(new tokens, tokens that were there before) of every sequence of a write or read."""
    n, t = c["seqs"], c["tokens"]
    if n == t:
        return [1] * n, [37 * i % 211 + 5 for i in range(n)]
    w = _spread(n, 1, 64)
    new = [max(1, (t - n) * x // sum(w)) for x in w]
    new[0] += t - sum(new)
    return new, [37 * i % 211 for i in range(n)]


def work(c):
    row = c["d"] * _BYTES[c.get("cache", "e2m1")] + (4 if c.get("cache", "e2m1") in ("e4m3", "e2m1") else 0)
    if c["op"] in ("write_4bit", "read_4bit"):
        n = 2 * c["tokens"] * c["hkv"]
        if c["op"] == "read_4bit":
            return {"bytes": int(n * (row + c["d"] * _BYTES[c["dtype"]])), "flops": 2 * n * c["d"]}
        # the rows in, their codes out and the weights' zeros; the codes in again, bf16 rows out
        return {"bytes": int(n * (c["d"] * _BYTES[c["dtype"]] + 2 * row + 2 * c["d"] + 2)), "flops": 5 * n * c["d"]}
    lens = _lengths(c)
    if c["op"] == "evict":
        kept = sum(min(n, c["keep"]) for n in lens)
        # every weight once; the kept rows out of their places and into their new ones, K, V and weight
        b = 4 * sum(lens) * c["hkv"] + 2 * kept * c["hkv"] * (2 * row + 4)
        if c["cache"] == "e2m1":   # and read back
            b += 2 * kept * c["hkv"] * (row + 2 * c["d"])
        return {"bytes": int(b), "flops": sum(lens) * c["hkv"]}
    total = sum(lens)
    return {"bytes": int(2 * total * c["hkv"] * row + c["seqs"] * c["hq"] * (2 * c["d"] * _BYTES[c["dtype"]] + 4)
                         + (8 * total * c["hkv"] if c["op"] == "decode_seen" else 0)), "flops": 4 * total * c["hq"] * c["d"]}


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


def _empty_cache(c, pages):
    width = c["d"] * 9 // 16 if c["cache"] == "e2m1" else c["d"]
    codes = torch.zeros((pages, c["hkv"], c["page"], width), dtype=_DT[c["cache"]], device="cuda")
    return codes, torch.zeros(codes.shape[:3], device="cuda") if c["cache"] in ("e4m3", "e2m1") else None


def _filled(g, c, pages):
    """The two caches (and scales) with rows in every slot."""
    got = []
    for _ in range(2):
        codes, scale = _empty_cache(c, pages)
        step = max(1, (1 << 25) // (c["hkv"] * c["page"] * c["d"]))
        for i in range(0, pages, step):
            x = torch.randn((min(step, pages - i), c["hkv"], c["page"], c["d"]), generator=g, device="cuda")
            if c["cache"] == "e2m1":
                part, blocks = _parts(codes[i:i + step], c)
                part[:], blocks[:], scale[i:i + step] = _quantised(x)
            elif c["cache"] == "e4m3":
                amax = x.abs().amax(-1)
                codes[i:i + step] = (x * (E4M3_MAX / amax)[..., None]).to(codes.dtype)
                scale[i:i + step] = amax / E4M3_MAX
            else:
                codes[i:i + step] = x.to(codes.dtype)
        got.append((codes, scale))
    return got


def prepare(c, seed):
    g = _gen(seed)
    if c["op"] in ("write_4bit", "read_4bit"):
        c = dict(c, cache="e2m1")
        new, before = _new(c)
        pages = [-(-(a + b) // c["page"]) for a, b in zip(new, before)]
        table, n = _table(g, pages)
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        s = {"c": c, "table": table, "cu": _ints(cu), "first": _ints(before), "lens": _ints([a + b for a, b in zip(new, before)])}
        if c["op"] == "read_4bit":
            (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _filled(g, c, n)
            return s
        for x in ("k", "v"):
            # channels of different sizes, as K's have
            gain = torch.exp(0.7 * torch.randn((c["d"],), generator=g, device="cuda"))
            s[x] = (_heads(g, c["tokens"], c["hkv"], c["d"], "fp32", c["layout"]) * gain).to(_DT[c["dtype"]])
            s[x + "c"], s[x + "s"] = _empty_cache(c, n)
        s["seen"] = torch.rand((n, c["hkv"], c["page"]), generator=g, device="cuda")
        return s
    lens = _lengths(c)
    table, n = _table(g, [-(-x // c["page"]) for x in lens])
    s = {"c": c, "table": table, "lens": _ints(lens), "longest": max(lens)}
    (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _filled(g, c, n)
    if c["op"] == "evict":
        # what tokens have gathered: most of them little, some equal
        s["seen"] = torch.floor(torch.exp(1.5 * torch.randn((n, c["hkv"], c["page"]), generator=g, device="cuda")) * 64) / 64
        s["keep"] = _ints([c["keep"]] * c["seqs"])
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + min(x, c["keep"]))
        s["cu"], s["kept"] = _ints(cu), cu[-1]
        return s
    s["seen"] = torch.rand((n, c["hkv"], c["page"]), generator=g, device="cuda")
    # scores of a spread of about 2, as trained heads have
    s["q"] = _heads(g, c["seqs"], c["hq"], c["d"], c["dtype"], c["layout"], 2.0)
    return s


# ------------------------------------------------------------------ the plain forms

def _parts(cache, c):
    """Codes and block scales of a 4-bit cache: each page and head holds the codes of its tokens, then their scales."""
    flat, at = cache.view(*cache.shape[:2], -1), c["page"] * c["d"] // 2
    return (flat[..., :at].unflatten(-1, (c["page"], c["d"] // 2)),
            flat[..., at:].unflatten(-1, (c["page"], c["d"] // 16)))


def _quantised(x):
    """Codes (two a byte, the first in the low half), block scales (as bytes) and row scale of rows x."""
    x = x.float()
    amax = x.abs().amax(-1).clamp(min=MIN_AMAX)
    part, e = torch.frexp(amax / torch.full_like(amax, MOST))
    scale = ((e - (part == 0.5).int() + 127) << 23).view(torch.float32)          # the least power of two with amax <= MOST * scale
    y = (x / scale[..., None]).unflatten(-1, (-1, 16))
    block = y.abs().amax(-1)
    block = (block / torch.full_like(block, 6.0)).to(torch.float8_e4m3fn)
    b = block.float()[..., None]
    z = torch.where(b > 0, y / torch.where(b > 0, b, torch.ones_like(b)), torch.zeros_like(y))
    a = z.abs()
    # half way goes to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8) + (a >= 1.75).to(torch.uint8)
            + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8) + (a > 5.0).to(torch.uint8) + 8 * z.signbit().to(torch.uint8))
    code = code.flatten(-2)
    return code[..., ::2] + 16 * code[..., 1::2], block.view(torch.uint8), scale


def _values(codes, blocks, scale):
    """Rows in fp32 from codes, block scales and row scales."""
    pairs = torch.tensor([[(-1.0 if n & 8 else 1.0) * E2M1[n & 7] for n in (i & 15, i >> 4)] for i in range(256)], device="cuda")
    x = pairs.index_select(0, codes.reshape(-1).int()).view(*codes.shape[:-1], -1, 16)
    x = x * blocks.contiguous().view(torch.float8_e4m3fn).float()[..., None]
    return x.flatten(-2) * scale[..., None]


def _tokens_first(x, c):
    return x.transpose(0, 1) if c["layout"] == "head" else x


def _slots(s, first):
    """(page, slot in the page) of every token of the packed sequences."""
    c = s["c"]
    t = torch.arange(c["tokens"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    p = first.long()[b] + t - s["cu"].long()[b]
    return s["table"].long()[b, p // c["page"]], p % c["page"]


def _read_at(s, page, slot, dtype):
    """K and V rows [tokens, heads, d] of places in the cache."""
    out = []
    for x in ("k", "v"):
        codes, blocks = _parts(s[x + "c"], s["c"])
        out.append(_values(codes[page, :, slot], blocks[page, :, slot], s[x + "s"][page, :, slot]).to(dtype))
    return out


def _write(s):
    c = s["c"]
    page, slot = _slots(s, s["first"])
    for x in ("k", "v"):
        codes, blocks = _parts(s[x + "c"], c)
        codes[page, :, slot], blocks[page, :, slot], s[x + "s"][page, :, slot] = _quantised(_tokens_first(s[x], c))
    s["seen"][page, :, slot] = 0.0
    return [_tokens_first(x, c).contiguous() for x in _read_at(s, page, slot, torch.bfloat16)] + [s["seen"]]


def _read(s):
    page, slot = _slots(s, s["first"])
    return [_tokens_first(x, s["c"]).contiguous() for x in _read_at(s, page, slot, _DT[s["c"]["dtype"]])]


def _decode(s):
    c = s["c"]
    b, g = c["seqs"], c["hq"] // c["hkv"]
    cols = -(-s["longest"] // c["page"])
    pages = s["table"][:, :cols].long().clamp(min=0)
    seen = torch.arange(cols * c["page"], device="cuda") < s["lens"][:, None]
    kv = []
    for x in ("k", "v"):
        if c["cache"] == "e2m1":
            codes, blocks = _parts(s[x + "c"], c)
            rows = _values(codes[pages], blocks[pages], s[x + "s"][pages])
        elif c["cache"] == "e4m3":
            rows = s[x + "c"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() * s[x + "s"][pages][..., None]
        else:
            rows = s[x + "c"][pages].float()
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
    out = [_tokens_first(o, c).contiguous(), lse.reshape(b, c["hq"])]
    if c["op"] == "decode_seen":
        # a slot gets one weight; the places behind a sequence's end add nothing to some page's
        w = (p / total.clamp(min=1e-30)).sum(2).reshape(b, c["hkv"], cols, c["page"]).transpose(1, 2)
        s["seen"].index_add_(0, pages.reshape(-1), w.reshape(b * cols, c["hkv"], c["page"]))
        out.append(s["seen"])
    return out


def _evict(s):
    c = s["c"]
    h, n = c["hkv"], s["longest"]
    top = min(n, c["keep"])
    pos = torch.arange(n, device="cuda")
    pages = s["table"].long().clamp(min=0)[:, pos // c["page"]]                                    # [b, n]
    lens, keep = s["lens"].long()[:, None, None], s["keep"].long()[:, None, None]
    w = s["seen"][pages, :, (pos % c["page"])[None]].transpose(1, 2)                               # [b, h, n]
    left = torch.minimum(lens, keep)                                                               # tokens that stay
    last = torch.minimum(left, torch.full_like(left, c["recent"]))
    old = pos < lens - last
    # the heaviest of the old ones, the lower place first among equals
    order = torch.where(old, w, torch.full_like(w, -math.inf)).sort(dim=-1, descending=True, stable=True).indices
    stays = torch.zeros_like(old.expand_as(w)).scatter(-1, order, (pos < left - last).expand_as(order))
    stays = stays | ((pos >= lens - last) & (pos < lens))
    src = (~stays).to(torch.uint8).sort(dim=-1, stable=True).indices[..., :top]                        # [b, h, top]
    # rows of no token repeat the move of the first sequence's first: the same value in the same place
    none = torch.arange(top, device="cuda") >= left
    b = torch.where(none, 0, torch.arange(c["seqs"], device="cuda")[:, None, None])
    r = torch.where(none, 0, torch.arange(top, device="cuda"))
    src = src[b, torch.arange(h, device="cuda")[:, None], r]
    heads = torch.arange(h, device="cuda")[:, None].expand_as(src)
    at, to = (pages[b, src], heads, src % c["page"]), (pages[b, r], heads, r % c["page"])
    for x in ("kc", "vc", "ks", "vs", "seen"):
        if s[x] is None:
            continue
        for t in _parts(s[x], c) if x[1] == "c" and c["cache"] == "e2m1" else [s[x].view(torch.uint8) if c["cache"] == "e4m3" and x[1] == "c" else s[x]]:
            t[to] = t[at]
    return _evicted(s, left[:, 0, 0].to(torch.int32))


def _evicted(s, left):
    """What an eviction leaves: the new lengths, the weights and the cache, a 4-bit one as the values of its tokens."""
    c = s["c"]
    if c["cache"] != "e2m1":
        return [x for x in (left, s["seen"], s["kc"], s["ks"], s["vc"], s["vs"]) if x is not None]
    if own:
        from long_context_sequence_seq_gb300 import ulysses as U
        return [left, s["seen"], s["ks"], s["vs"], *U.cache_read(s["kc"], s["vc"], s["table"], s["cu"], s["kept"], k_scale=s["ks"],
                                                                  v_scale=s["vs"], dtype=torch.bfloat16)]
    t = torch.arange(s["kept"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    p = t - s["cu"].long()[b]
    return [left, s["seen"], s["ks"], s["vs"], *(x.contiguous() for x in _read_at(s, s["table"].long()[b, p // c["page"]], p % c["page"],
                                                                                   torch.bfloat16))]


# ------------------------------------------------------------------ the calls

def _own_run(s):
    from long_context_sequence_seq_gb300 import ulysses as U
    c = s["c"]
    scales = dict(k_scale=s["ks"], v_scale=s["vs"])
    if c["op"] == "write_4bit":
        U.cache_write(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"], cu_new=None if c["seqs"] == c["tokens"] else s["cu"],
                      layout=c["layout"], weights=s["seen"], **scales)
        return [*U.cache_read(s["kc"], s["vc"], s["table"], s["cu"], c["tokens"], first=s["first"], dtype=torch.bfloat16,
                              layout=c["layout"], **scales), s["seen"]]
    if c["op"] == "read_4bit":
        return U.cache_read(s["kc"], s["vc"], s["table"], s["cu"], c["tokens"], first=s["first"], dtype=_DT[c["dtype"]],
                            layout=c["layout"], **scales)
    if c["op"] == "evict":
        return _evicted(s, U.cache_evict(s["kc"], s["vc"], s["seen"], s["table"], s["lens"], s["keep"], recent=c["recent"], **scales))
    if c["op"] == "decode_4bit":
        return U.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], layout=c["layout"], **scales)
    return [*U.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], layout=c["layout"], weights=s["seen"], **scales), s["seen"]]


def run(s):
    if own:
        return _own_run(s)
    op = s["c"]["op"]
    return _write(s) if op == "write_4bit" else _read(s) if op == "read_4bit" else _evict(s) if op == "evict" else _decode(s)


# ------------------------------------------------------------------ the definitions in 64 bits

def _nearest(a, bits, low, most):
    """a >= 0 to `bits` fraction bits (2^low the smallest binade), half way to even, at most `most`."""
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -60))).clamp(min=low)
    step = torch.exp2(e - bits)
    return (torch.round(a / step) * step).clamp(max=most)


def _exact_rounded(x):
    """Rows as a 4-bit cache holds them."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for i in range(0, len(x), 4096):
        y = x[i:i + 4096].double()
        f = torch.exp2(torch.ceil(torch.log2(y.abs().amax(-1, keepdim=True).clamp(min=MIN_AMAX) / MOST)))
        y = (y / f).unflatten(-1, (-1, 16))
        b = _nearest(y.abs().amax(-1, keepdim=True) / 6.0, 3, -6, E4M3_MAX)
        z = torch.where(b > 0, _nearest(y.abs() / b.clamp(min=1e-9), 1, 0, 6.0) * y.sign(), torch.zeros_like(y))
        out[i:i + 4096] = (z * b).flatten(-2) * f
    return out


def _exact_rows(c, s, x, page, slot=None, h=None):
    """Rows of cache x (k or v) in 64 bits: pages `page` whole, of head h, or places (page, slot) of all heads."""
    def pick(t):
        return t[page, h] if slot is None else t[page, :, slot]
    if c["cache"] == "e2m1":
        at = c["page"] * c["d"] // 2
        flat = s[x + "c"].flatten(2)
        codes = pick(flat[..., :at].unflatten(2, (c["page"], -1)))
        blocks = pick(flat[..., at:].unflatten(2, (c["page"], -1))).contiguous().view(torch.float8_e4m3fn).double()
        table = torch.tensor([*E2M1, *(-v for v in E2M1)], dtype=torch.float64, device="cuda")
        two = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1).flatten(-2)
        return two * blocks.repeat_interleave(16, -1) * pick(s[x + "s"]).double()[..., None]
    rows = (pick(s[x + "c"].view(torch.uint8)).contiguous().view(torch.float8_e4m3fn).float() if c["cache"] == "e4m3" else pick(s[x + "c"])).double()
    return rows * pick(s[x + "s"]).double()[..., None] if c["cache"] == "e4m3" else rows


def _each_token(c, s):
    """(sequence's rows in the packed tensor, their pages, their slots), a sequence at a time."""
    cu, first, table = s["cu"].tolist(), s["first"].tolist(), s["table"].long()
    for b in range(c["seqs"]):
        p = torch.arange(cu[b + 1] - cu[b], device="cuda") + first[b]
        yield slice(cu[b], cu[b + 1]), table[b][p // c["page"]], p % c["page"]


def _exact_write(c, s):
    out = [_exact_rounded(s[x]) for x in ("k", "v")]
    seen = s["seen"].double()
    for _, page, slot in _each_token(c, s):
        seen[page, :, slot] = 0.0
    return out + [seen]


def _exact_read(c, s):
    out = []
    for x in ("k", "v"):
        got = torch.empty((c["tokens"], c["hkv"], c["d"]), dtype=torch.float64, device="cuda")
        for at, page, slot in _each_token(c, s):
            got[at] = _exact_rows(c, s, x, page, slot)
        out.append(got.transpose(0, 1).contiguous() if c["layout"] == "head" else got)
    return out


def _exact_decode(c, s):
    q = (s["q"].transpose(0, 1) if c["layout"] == "head" else s["q"]).double()
    group = c["hq"] // c["hkv"]
    o = torch.zeros((c["seqs"], c["hq"], c["d"]), dtype=torch.float64, device="cuda")
    lse = torch.full((c["seqs"], c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    seen = s["seen"].double()
    for b, n in enumerate(s["lens"].tolist()):
        if not n:
            continue
        pages = s["table"][b, :-(-n // c["page"])].long()
        at = torch.arange(n, device="cuda")
        for h in range(c["hkv"]):
            k, v = (_exact_rows(c, s, x, pages, h=h).flatten(0, 1)[:n] for x in ("k", "v"))
            z = k @ q[b, h * group:(h + 1) * group].T * c["d"] ** -0.5
            lse[b, h * group:(h + 1) * group] = torch.logsumexp(z, 0)
            p = torch.softmax(z, 0)
            o[b, h * group:(h + 1) * group] = p.T @ v
            seen[pages[at // c["page"]], h, at % c["page"]] += p.sum(1)
    out = [o.transpose(0, 1).contiguous() if c["layout"] == "head" else o, lse]
    return out + [seen] if c["op"] == "decode_seen" else out


def _exact_evict(c, s):
    whole = [s["seen"].double()]
    for x in ("k", "v"):
        if c["cache"] == "e2m1":
            whole.append(_exact_rows(c, s, x, torch.arange(len(s["kc"]), device="cuda"), h=slice(None)))
        else:
            whole.append(s[x + "c"].float().double())
        whole.append(None if s[x + "s"] is None else s[x + "s"].double())
    left, rows = [], [[], []]
    for b, n in enumerate(s["lens"].tolist()):
        m = min(n, c["keep"])
        left.append(m)
        last = min(m, c["recent"])
        p = torch.arange(n, device="cuda")
        page, slot = s["table"][b].long()[p // c["page"]], p % c["page"]
        for h in range(c["hkv"]):
            # places by falling weight, then by rising place: the first m - last of the old ones stay
            w = s["seen"][page, h, slot][:n - last].double()
            best = torch.sort(-w, stable=True).indices[:m - last]
            src = torch.cat((torch.sort(best).values, p[n - last:]))
            for t in whole:
                if t is not None:
                    t[page[:m], h, slot[:m]] = t[page[src], h, slot[src]]
        for i in range(2):
            rows[i].append(whole[1 + 2 * i][page[:m], :, slot[:m]])
    left = torch.tensor(left, dtype=torch.int32, device="cuda")
    if c["cache"] != "e2m1":
        return [left, *(t for t in whole if t is not None)]
    return [left, whole[0], whole[2], whole[4], torch.cat(rows[0]), torch.cat(rows[1])]


def exact(c, seed):
    s = prepare(c, seed)
    c = s["c"]
    return {"write_4bit": _exact_write, "read_4bit": _exact_read, "evict": _exact_evict}.get(c["op"], _exact_decode)(c, s)
