"""Measured cases of the rotation of queries and keys, the append to the 8-bit
key/value cache and the attention of chunks over it.

Three operators of the serving path between the coded q/k/v products and the
o product:

* ``rope``    rotary positions, on one axis (text) or three (time, height and
  width of image and video patches), of packed queries and keys;
* ``append``  new keys and values as the products leave them (float32, or 16
  bits) into the paged 8-bit cache, keys rotated on the way and the queries
  beside them, and the touched pages read back, which is the state the call
  updated;
* ``chunk``   attention of a chunk of new tokens per sequence over the cache,
  in which the chunk's own keys and values are already: pieces of prompts,
  drafted tokens, and batches of both with single tokens.

``run`` computes each in its plain form (elementary torch operations in 32
bits, angles in 64) or, where ``own`` is true, with the framework's kernels.
``exact`` is the definition in 64 bits.

Cache layout: ``k_codes`` int8 [pages][kv heads][page tokens][dim], ``v_codes``
int8 [pages][kv heads][dim][page tokens], ``k_scales`` / ``v_scales`` float32
[pages][kv heads]; value = code * scale.  Sequence b's token p is in page
``table[b][p // page]`` at row ``p % page``.

Rotation: pair i of a head's first 2 P elements is (i, i + P), or (2 i, 2 i + 1)
where adjacent; it turns by position * freqs[i], the position being that of the
pair's axis.
"""
import math
import random

import torch

own = False

# Head layouts (query heads, key/value heads, head dimension) of the three
# weight stacks that the framework's workloads are shaped after, as their
# projection sizes give them, and two generic grouped layouts.
HEADS = {
    "h32x64": (32, 32, 64),     # 2048-wide projections
    "h32x96": (32, 32, 96),     # joint qkv projection of 3 x 32 x 96
    "g4x128": (32, 8, 128),     # 4096-wide q, 1024-wide k and v
    "g8x128": (64, 8, 128),
    "g7x64": (14, 2, 64),       # a group that is no power of two
}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
PAGES = (16, 32, 64, 128)


def listed():
    return [
        # the new token of each of a few users, from the products: all latency
        {"name": "rope_step", "op": "rope", "heads": "g4x128", "dtype": "f32", "out": "bf16", "seqs": 5, "longest": 1, "prefix": 900,
         "axes": 1, "share": 1.0, "adjacent": False},
        # an image's patches behind some text, positions on three axes
        {"name": "rope_image", "op": "rope", "heads": "g7x64", "dtype": "bf16", "out": "bf16", "seqs": 3, "longest": 2741, "prefix": 0,
         "axes": 3, "share": 1.0, "adjacent": False},
        # one long document, half of each head rotated
        {"name": "rope_long", "op": "rope", "heads": "h32x96", "dtype": "f16", "out": "f16", "seqs": 1, "longest": 32768, "prefix": 100000,
         "axes": 1, "share": 0.5, "adjacent": True},
        # the new token of every sequence of a decode batch, from the products
        {"name": "append_step", "op": "append", "heads": "g4x128", "dtype": "f32", "out": "bf16", "seqs": 16, "longest": 1, "prefix": 2000,
         "axes": 1, "share": 1.0, "adjacent": False, "page": 64},
        # pieces of images and text that begin inside partly filled pages
        {"name": "append_ragged", "op": "append", "heads": "h32x96", "dtype": "f16", "out": "f16", "seqs": 12, "longest": 1001, "prefix": 500,
         "axes": 3, "share": 0.5, "adjacent": False, "page": 32},
        # one long document's queries, keys and values
        {"name": "append_long", "op": "append", "heads": "g4x128", "dtype": "bf16", "out": "bf16", "seqs": 1, "longest": 32768, "prefix": 0,
         "axes": 1, "share": 1.0, "adjacent": False, "page": 64},
        # a few drafted tokens of one user's first answer: all latency
        {"name": "chunk_short", "op": "chunk", "heads": "h32x64", "dtype": "bf16", "seqs": 1, "longest": 5, "prefix": 85, "page": 16},
        # drafted tokens of a batch, to be verified over ragged contexts
        {"name": "chunk_drafts", "op": "chunk", "heads": "g4x128", "dtype": "bf16", "seqs": 24, "longest": 7, "prefix": 12000, "page": 64},
        # a turn of one conversation behind a long context
        {"name": "chunk_turn", "op": "chunk", "heads": "g8x128", "dtype": "f16", "seqs": 1, "longest": 61, "prefix": 40003, "page": 128},
        # a batch that mixes pieces of prompts with short and single tokens
        {"name": "chunk_mixed", "op": "chunk", "heads": "h32x96", "dtype": "f16", "seqs": 18, "longest": 500, "prefix": 5001, "page": 32},
        # the first piece of a prompt, nothing in front
        {"name": "chunk_first", "op": "chunk", "heads": "g7x64", "dtype": "bf16", "seqs": 2, "longest": 4099, "prefix": 0, "page": 16},
        # a piece of one long document
        {"name": "chunk_long", "op": "chunk", "heads": "g4x128", "dtype": "bf16", "seqs": 1, "longest": 2048, "prefix": 30720, "page": 64},
    ]


# draw(): the longest sequence, the largest batch and the longest prefix of each
# operator, and the most elements that the plain form's largest intermediate
# may have (those of the listed chunk_long, append_long and rope_long)
_TOP = {
    "rope": (32768, 64, 1 << 20, 32768 * 64 * 96),
    "append": (32768, 64, 32768, 32768 * 8 * 128),
    "chunk": (4096, 64, 131072, 32 * 2048 * 32768),
}


def _spread(rng, top):
    return round(math.exp(rng.uniform(0.0, math.log(top))))


def draw(rng):
    op = rng.choice(sorted(_TOP))
    longest, seqs, prefix, most = _TOP[op]
    while True:
        case = {"op": op, "heads": rng.choice(sorted(HEADS)), "seqs": _spread(rng, seqs), "longest": _spread(rng, longest),
                "prefix": _spread(rng, prefix) if rng.random() < 0.75 else 0}
        case["dtype"] = rng.choice(("bf16", "f16"))
        if op != "chunk":
            case["out"] = case["dtype"]
            if rng.random() < 0.4:
                case["dtype"] = "f32"
            case["axes"] = rng.choice((1, 1, 3))
            case["share"] = rng.choice((1.0, 1.0, 0.5))
            case["adjacent"] = rng.random() < 0.3
        if op != "rope":
            case["page"] = rng.choice(PAGES)
        h, kv, d = HEADS[case["heads"]]
        n, both = case["seqs"], case["longest"] + case["prefix"]
        if op == "rope":
            size = n * case["longest"] * (h + kv) * d
        elif op == "append":
            size = n * kv * d * both
        else:
            size = max(n * h * case["longest"] * both, 2 * n * kv * d * both)
        if size <= most:
            return case


def _lengths(case):
    """(new tokens, earlier tokens) of each sequence: the first is the longest,
    the others spread over the logarithm from a 32nd of it on, and a batch of
    four or more has an empty sequence (a slot that waits) and one of a single
    token."""
    rng = random.Random("%(op)s %(seqs)d %(longest)d %(prefix)d" % case)
    n = case["seqs"]
    spread = lambda top: round(top * math.exp(rng.uniform(-math.log(32.0), 0.0)))  # noqa: E731
    new = [case["longest"]] + [max(1, spread(case["longest"])) for _ in range(n - 1)]
    held = [case["prefix"]] + [spread(case["prefix"]) for _ in range(n - 1)]
    if n >= 4:
        new[-1], new[-2] = 0, 1
    return new, held


def _running(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


def work(case):
    h, kv, d = HEADS[case["heads"]]
    new, held = _lengths(case)
    total, size = sum(new), 4 if case["dtype"] == "f32" else 2
    if case["op"] == "chunk":
        pairs = sum(a * (a + b) - a * (a - 1) // 2 for a, b in zip(new, held))
        read = sum(a + b for a, b in zip(new, held) if a)
        return {"bytes": 2 * kv * d * read + 4 * h * d * total, "flops": 4 * d * h * pairs}
    if case["op"] == "rope":
        return {"bytes": (size + 2) * (h + kv) * d * total + 4 * case["axes"] * total, "flops": 3 * (h + kv) * d * total}
    page = case["page"]
    back = sum(b + a - b // page * page for a, b in zip(new, held) if a)
    # queries in and out, keys and values in and their codes out, then the codes in and 16-bit values out
    moved = (size + 2) * h * d * total + 2 * kv * d * ((size + 1) * total + 3 * back)
    return {"bytes": moved, "flops": 3 * (h + kv) * d * total + 2 * kv * d * (total + back)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _keys(g, n, kv, d):
    """Keys: unit noise over a fixed offset per channel, a few channels large."""
    off = 0.5 * torch.randn(kv, d, device="cuda", generator=g)
    gain = 1.0 + 3.0 * (torch.rand(kv, d, device="cuda", generator=g) < 0.03)
    return (torch.randn(n, kv, d, device="cuda", generator=g) + off) * gain


def _quantize(x):
    """[pages][kv][tokens][dim] to codes and scales: a full page at once."""
    scale = x.abs().amax((2, 3)) * (1.0 / 127.0)
    return torch.round(x * torch.reciprocal(scale)[:, :, None, None]).to(torch.int8), scale


def _positions(case, new, held):
    """[axes][rows]: a sequence's places; on three axes a quarter of it is text
    and the rest patches of one image behind it, row by row of a square."""
    at = []
    for n, p in zip(new, held):
        i = torch.arange(n, device="cuda")
        if case["axes"] == 1:
            at.append((p + i)[None])
            continue
        text = n // 4
        wide = math.isqrt(max(n - text, 1))
        j = (i - text).clamp(min=0)
        flat = torch.minimum(i, torch.full_like(i, text))
        at.append(p + torch.stack([flat, flat + j // wide, flat + j % wide]))
    return torch.cat(at, 1).to(torch.int32)


def _axes_of(case, pairs):
    """The axis of each pair: a quarter time, the rest height and width."""
    if case["axes"] == 1:
        return [0] * pairs
    t = pairs // 4
    u = (pairs - t) // 2
    return [0] * t + [1] * u + [2] * (pairs - t - u)


def _rotary(s, case, d):
    s["pairs"] = int(d * case["share"]) // 2
    i = torch.arange(s["pairs"], dtype=torch.float64)
    s["freqs"] = (500000.0 ** (-i / s["pairs"])).float().cuda()
    s["axes"] = _axes_of(case, s["pairs"])
    s["axis"] = torch.tensor(s["axes"], device="cuda")
    s["rotary"] = None     # the framework's handle, made in the first pass as a program makes it once


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    h, kv, d = HEADS[case["heads"]]
    dtype = DTYPES[case["dtype"]]
    new, held = _lengths(case)
    n, total = len(new), sum(new)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": case, "status": torch.zeros(n, dtype=torch.int32, device="cuda"), "scale": 1.0 / math.sqrt(d)}
    s["q"] = (1.5 * torch.randn(total, h, d, device="cuda", generator=g)).to(dtype)
    if case["op"] != "chunk":
        _rotary(s, case, d)
        s["positions"] = _positions(case, new, held)
    if case["op"] == "rope":
        s["k"] = _keys(g, total, kv, d).to(dtype)
        return s
    page = case["page"]
    count = [-(-(a + b) // page) for a, b in zip(new, held)]
    pages = sum(count) + 3
    where = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    at = _running(count)
    table = torch.full((n, max(count + [1])), -1, dtype=torch.int32, device="cuda")
    for b in range(n):
        table[b, : count[b]] = where[at[b]: at[b + 1]]
    s["table"] = table
    s["k_codes"], s["k_scales"] = _quantize(_keys(g, pages * page, kv, d).view(pages, page, kv, d).transpose(1, 2))
    v, s["v_scales"] = _quantize(torch.randn(pages, kv, page, d, device="cuda", generator=g))
    s["k_codes"], s["v_codes"] = s["k_codes"].contiguous(), v.transpose(2, 3).contiguous()
    s["cu"] = ints(_running(new))
    if case["op"] == "chunk":
        s["lens"], s["most"] = ints([a + b for a, b in zip(new, held)]), max(new)
        return s
    s["k"] = (1.2 * _keys(g, total, kv, d)).to(dtype)
    s["v"] = (1.2 * torch.randn(total, kv, d, device="cuda", generator=g)).to(dtype)
    s["held"] = ints(held)
    first = [b // page * page for b in held]
    back = [a + b - f if a else 0 for a, b, f in zip(new, held, first)]
    s["first"], s["cu_out"], s["n_out"] = ints(first), ints(_running(back)), sum(back)
    s["n_pages"] = sum(-(-(a + b) // page) - b // page if a else 0 for a, b in zip(new, held))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _handles(ent, s):
    """What a program makes once: the rotation's plan and the cache."""
    if s.get("rotary") is None and "freqs" in s:
        s["rotary"] = ent.Rotary(s["freqs"], axes=s["axes"], interleaved=s["case"]["adjacent"])
    if s.get("cache") is None and "k_codes" in s:
        s["cache"] = ent.KVCache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])


def _own_rope(s):
    import entropy_coded_weight_canonical_amd as ent

    _handles(ent, s)
    return list(ent.rope(s["rotary"], s["q"], s["k"], s["positions"], dtype=DTYPES[s["case"]["out"]]))


def _own_append(s):
    import entropy_coded_weight_canonical_amd as ent

    _handles(ent, s)
    # (text needs no positions: a token's place in its sequence is its position)
    q = ent.kv_append(s["cache"], s["rotary"], s["k"], s["v"], s["table"], s["held"], s["cu"], s["status"], q=s["q"],
                      positions=s["positions"] if s["case"]["axes"] > 1 else None, dtype=DTYPES[s["case"]["out"]])
    k, v = ent.kv_load(s["cache"], s["table"], s["first"], s["cu_out"], s["n_out"], s["status"], dtype=DTYPES[s["case"]["out"]])
    return [q, k, v, s["k_scales"], s["v_scales"]]


def _own_chunk(s):
    import entropy_coded_weight_canonical_amd as ent

    _handles(ent, s)
    return ent.attn_chunk(s["q"], s["cache"], s["table"], s["lens"], s["cu"], s["status"], scale=s["scale"])


_OWN = {"rope": _own_rope, "append": _own_append, "chunk": _own_chunk}


def _turned(s, x):
    """x [rows][heads][dim] rotated, in 32 bits; angles in 64."""
    p = s["pairs"]
    angle = s["positions"][s["axis"]].double().t() * s["freqs"].double()        # [rows][pairs]
    c, n = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = x.float()
    a, b = (x[..., 0: 2 * p: 2], x[..., 1: 2 * p: 2]) if s["case"]["adjacent"] else (x[..., :p], x[..., p: 2 * p])
    a, b = a * c - b * n, b * c + a * n
    both = torch.stack([a, b], -1).flatten(-2) if s["case"]["adjacent"] else torch.cat([a, b], -1)
    return torch.cat([both, x[..., 2 * p:]], -1)


def _plain_rope(s):
    dtype = DTYPES[s["case"]["out"]]
    return [_turned(s, s["q"]).to(dtype), _turned(s, s["k"]).to(dtype)]


def _grown(codes, old, x, is_new, is_held):
    """A page's codes and scales after the new rows `x` ([items][rows][kv][dim];
    `codes` [items][kv][rows][dim]): the scale grows to cover them, what the
    page held is requantized to it."""
    x = x.permute(0, 2, 1, 3)
    is_new, is_held = is_new[:, None, :, None], is_held[:, None, :, None]
    top = x.abs().mul_(is_new).amax((2, 3))
    before = old * is_held.any(2)[:, :, 0]
    scale = torch.maximum(before, top * (1.0 / 127.0))
    again = torch.round(codes.float() * (before / scale)[:, :, None, None])
    fresh = torch.round(x * torch.reciprocal(scale)[:, :, None, None])
    out = torch.where(is_new, fresh, torch.where(is_held, again, codes.float()))
    return out.to(torch.int8), scale


def _plain_append(s):
    page, dtype = s["case"]["page"], DTYPES[s["case"]["out"]]
    held, cu, table = s["held"].long(), s["cu"].long(), s["table"].long()
    q, k, v = _turned(s, s["q"]).to(dtype), _turned(s, s["k"]), s["v"].float()
    new = cu[1:] - cu[:-1]
    dev = table.device
    # the pages that get new rows, one after another
    first = held // page
    count = torch.where(new > 0, (held + new + page - 1) // page - first, 0)
    seq = torch.repeat_interleave(torch.arange(held.numel(), device=dev), count, output_size=s["n_pages"])
    begin = torch.cumsum(count, 0) - count
    local = first[seq] + torch.arange(s["n_pages"], device=dev) - begin[seq]
    ids = table[seq, local]
    pos = local[:, None] * page + torch.arange(page, device=dev)
    is_held = pos < held[seq][:, None]
    is_new = ~is_held & (pos < (held + new)[seq][:, None])
    row = (cu[seq][:, None] + pos - held[seq][:, None]).clamp_(0, max(k.shape[0] - 1, 0))
    codes, s["k_scales"][ids] = _grown(s["k_codes"][ids], s["k_scales"][ids], k[row], is_new, is_held)
    s["k_codes"][ids] = codes
    codes, s["v_scales"][ids] = _grown(s["v_codes"][ids].transpose(2, 3), s["v_scales"][ids], v[row], is_new, is_held)
    s["v_codes"][ids] = codes.transpose(2, 3)
    # the touched pages, back in 16 bits
    cu = s["cu_out"].long()
    seq = torch.repeat_interleave(torch.arange(cu.numel() - 1, device=dev), cu[1:] - cu[:-1], output_size=s["n_out"])
    pos = s["first"].long()[seq] + torch.arange(s["n_out"], device=dev) - cu[seq]
    ids, row = table[seq, pos // page], pos % page
    k = s["k_codes"][ids, :, row].float().mul_(s["k_scales"][ids][:, :, None])
    v = s["v_codes"][ids, :, :, row].float().mul_(s["v_scales"][ids][:, :, None])
    return [q, k.to(dtype), v.to(dtype), s["k_scales"], s["v_scales"]]


def _plain_chunk(s):
    q, lens, cu = s["q"], s["lens"].long(), s["cu"].long()
    h, kv, d = HEADS[s["case"]["heads"]]
    table = s["table"].long().clamp(min=0)
    n, wide = table.shape
    nq, tokens = s["most"], wide * s["case"]["page"]
    # [n][pages][kv][...] to one key matrix and one value matrix per sequence and head
    k = s["k_codes"][table].float().mul_(s["k_scales"][table][..., None, None])
    k = k.permute(0, 2, 4, 1, 3).reshape(n * kv, d, tokens)
    v = s["v_codes"][table].float().mul_(s["v_scales"][table][..., None, None])
    v = v.permute(0, 2, 1, 4, 3).reshape(n * kv, tokens, d)
    # the packed rows as padded batches
    new = cu[1:] - cu[:-1]
    i = torch.arange(nq, device=q.device)
    at = (cu[:-1, None] + torch.minimum(i[None], new[:, None] - 1)).clamp_(0, q.shape[0] - 1)
    qq = q[at].float().view(n, nq, kv, h // kv, d).permute(0, 2, 3, 1, 4).reshape(n * kv, h // kv * nq, d)
    last = (lens - new)[:, None] + i                                               # [n][nq]
    hidden = torch.arange(tokens, device=q.device) > torch.minimum(last, lens[:, None] - 1)[..., None]
    scores = torch.matmul(qq, k).mul_(s["scale"]).view(n, kv, h // kv, nq, tokens)
    # softmax without the hidden places, in place; a row that has none left is zero
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    scores.sub_(scores.amax(-1, keepdim=True).clamp_(min=-3e38)).exp_()
    scores.div_(scores.sum(-1, keepdim=True).clamp_(min=1e-38))
    o = torch.matmul(scores.view(n * kv, h // kv * nq, tokens), v)
    o = o.view(n, kv, h // kv, nq, d).permute(0, 3, 1, 2, 4).reshape(n * nq, h, d).to(q.dtype)
    # back to the packed rows
    seq = torch.repeat_interleave(torch.arange(n, device=q.device), new, output_size=q.shape[0])
    return o[seq * nq + torch.arange(q.shape[0], device=q.device) - cu[seq]]


_PLAIN = {"rope": _plain_rope, "append": _plain_append, "chunk": _plain_chunk}


# ---------------------------------------------------------------------------
# the definition in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "chunk": _exact_chunk}[case["op"]](s)


def _exact_turned(s, x):
    """A pair as a complex number, times exp(i angle)."""
    x = x.double()
    p = s["pairs"]
    place = s["positions"].double()
    angle = torch.stack([place[a] * s["freqs"][i].double() for i, a in enumerate(s["axes"])], 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    out = x.clone()
    if s["case"]["adjacent"]:
        z = torch.complex(x[..., 0: 2 * p: 2], x[..., 1: 2 * p: 2]) * turn
        out[..., 0: 2 * p: 2], out[..., 1: 2 * p: 2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :p].contiguous(), x[..., p: 2 * p].contiguous()) * turn
        out[..., :p], out[..., p: 2 * p] = z.real, z.imag
    return out


def _exact_rope(s):
    return [_exact_turned(s, s["q"]), _exact_turned(s, s["k"])]


def _exact_append(s):
    page = s["case"]["page"]
    held, cu, first, table = s["held"].tolist(), s["cu"].tolist(), s["first"].tolist(), s["table"].tolist()
    new = {"k": _exact_turned(s, s["k"]), "v": s["v"].double()}
    scales = {"k": s["k_scales"].double(), "v": s["v_scales"].double()}
    rows = {"k": [], "v": []}
    for b in range(len(held)):
        end = held[b] + cu[b + 1] - cu[b]
        for lead in range(first[b], end if end > held[b] else first[b], page):
            at = table[b][lead // page]
            keep = min(max(held[b] - lead, 0), page)
            take = min(end - lead, page) - keep
            for name, codes in (("k", s["k_codes"][at]), ("v", s["v_codes"][at].transpose(1, 2))):
                was = scales[name][at].clone()
                x = new[name][cu[b] + lead + keep - held[b]:][:take].transpose(0, 1)          # [kv][take][d]
                now = x.abs().amax((1, 2)) / 127
                if keep:
                    now = torch.maximum(now, was)
                scales[name][at] = now
                now = now[:, None, None]
                old = torch.round(codes[:, :keep].double() * (was[:, None, None] / now)) * now
                rows[name].append(torch.cat([old, torch.round(x / now) * now], 1).transpose(0, 1))
    return [_exact_turned(s, s["q"]), torch.cat(rows["k"]), torch.cat(rows["v"]), scales["k"], scales["v"]]


def _exact_head(q, k, v, scale, behind):
    """One head: row i of q sees the keys up to i + behind."""
    logits = (q @ k.t()) * scale
    i = torch.arange(q.shape[0], device=q.device)[:, None] + behind
    seen = torch.arange(k.shape[0], device=q.device)[None, :] <= i
    logits = logits.masked_fill(~seen, -math.inf)
    w = torch.exp(logits - logits.max(1, keepdim=True).values)
    return (w @ v) / w.sum(1, keepdim=True)


def _exact_chunk(s):
    h, kv, d = HEADS[s["case"]["heads"]]
    page, cu, lens = s["case"]["page"], s["cu"].tolist(), s["lens"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, tokens in enumerate(lens):
        i0, i1 = cu[b], cu[b + 1]
        if i1 == i0:
            continue
        ids = s["table"][b, : -(-tokens // page)].long()
        for g in range(kv):
            k = (s["k_codes"][ids, g].double() * s["k_scales"][ids, g].double()[:, None, None]).reshape(-1, d)[:tokens]
            v = s["v_codes"][ids, g].double() * s["v_scales"][ids, g].double()[:, None, None]
            v = v.transpose(1, 2).reshape(-1, d)[:tokens]
            for head in range(g * (h // kv), (g + 1) * (h // kv)):
                out[i0:i1, head] = _exact_head(s["q"][i0:i1, head].double(), k, v, s["scale"], tokens - (i1 - i0))
    return out
