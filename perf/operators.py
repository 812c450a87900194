"""Measured cases of the attention operators and the 8-bit key/value cache.

Four operators of the serving path around the coded weight products:

* ``prompt``  causal attention of packed prompts of different lengths with
  grouped heads, optionally behind earlier tokens (keys and values longer than
  the queries);
* ``store``   new keys and values written into the paged 8-bit cache (one scale
  per page and head, requantized when a page's range grows), and the touched
  pages read back, which is the state the call updated;
* ``load``    a cached prefix read back as 16-bit keys and values;
* ``step``    attention of one new token per sequence over the 8-bit cache.

``run`` computes each in its plain form (elementary torch operations in 32
bits) or, where ``own`` is true, with the framework's kernels.  ``exact`` is
the definition in 64 bits.

Cache layout: ``k_codes`` int8 [pages][kv heads][page tokens][dim], ``v_codes``
int8 [pages][kv heads][dim][page tokens], ``k_scales`` / ``v_scales`` float32
[pages][kv heads]; value = code * scale.  Sequence b's token p is in page
``table[b][p // page]`` at row ``p % page``.
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
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
PAGES = (16, 32, 64, 128)


def listed():
    return [
        # a short question to one user: all latency
        {"name": "prompt_short", "op": "prompt", "heads": "h32x64", "dtype": "bf16", "seqs": 1, "longest": 37, "prefix": 0},
        # a batch of mixed prompts, some behind an already processed prefix
        {"name": "prompt_packed", "op": "prompt", "heads": "h32x96", "dtype": "f16", "seqs": 12, "longest": 1531, "prefix": 2000},
        # one long document
        {"name": "prompt_long", "op": "prompt", "heads": "g4x128", "dtype": "bf16", "seqs": 1, "longest": 16384, "prefix": 0},
        # the new token of every sequence of a small decode batch
        {"name": "store_step", "op": "store", "heads": "g4x128", "dtype": "bf16", "seqs": 16, "longest": 1, "prefix": 2000, "page": 64},
        # ragged prompt pieces that begin inside partly filled pages
        {"name": "store_ragged", "op": "store", "heads": "h32x96", "dtype": "f16", "seqs": 12, "longest": 1001, "prefix": 500, "page": 32},
        # one long document's keys and values
        {"name": "store_long", "op": "store", "heads": "g4x128", "dtype": "bf16", "seqs": 1, "longest": 32768, "prefix": 0, "page": 64},
        # a conversation's prefix, back for its next turn
        {"name": "load_prefix", "op": "load", "heads": "h32x64", "dtype": "bf16", "seqs": 1, "longest": 700, "prefix": 0, "page": 16},
        # the prefixes of a batch
        {"name": "load_ragged", "op": "load", "heads": "g4x128", "dtype": "f16", "seqs": 24, "longest": 8190, "prefix": 0, "page": 64},
        # the first tokens of one user's answer: all latency
        {"name": "step_short", "op": "step", "heads": "h32x64", "dtype": "bf16", "seqs": 1, "longest": 90, "prefix": 0, "page": 16},
        # a small batch, one key head per query head
        {"name": "step_batch8", "op": "step", "heads": "h32x96", "dtype": "f16", "seqs": 8, "longest": 4099, "prefix": 0, "page": 32},
        # one user with a very long context: the work has to be split along it
        {"name": "step_one_long", "op": "step", "heads": "g4x128", "dtype": "bf16", "seqs": 1, "longest": 131072, "prefix": 0, "page": 64},
        # a full decode batch of ragged contexts
        {"name": "step_batch64", "op": "step", "heads": "g4x128", "dtype": "bf16", "seqs": 64, "longest": 16384, "prefix": 0, "page": 64},
    ]


# draw(): the longest sequence and the largest batch of each operator, and the
# elements that the plain form's largest intermediate may have (those of the
# listed prompt_long, store_long and step_batch64)
_TOP = {
    "prompt": (16384, 16, 32 * 16384 * 16384),
    "store": (32768, 64, 32768 * 8 * 128),
    "load": (32768, 64, 64 * 16384 * 8 * 128 // 4),
    "step": (131072, 64, 64 * 16384 * 8 * 128),
}


def draw(rng):
    op = rng.choice(sorted(_TOP))
    longest_top, seqs_top, most = _TOP[op]
    while True:
        case = {
            "op": op,
            "heads": rng.choice(sorted(HEADS)),
            "dtype": rng.choice(sorted(DTYPES)),
            "seqs": round(math.exp(rng.uniform(0.0, math.log(seqs_top)))),
            "longest": round(math.exp(rng.uniform(0.0, math.log(longest_top)))),
            "prefix": 0,
        }
        if op in ("prompt", "store") and rng.random() < 0.5:
            case["prefix"] = round(math.exp(rng.uniform(0.0, math.log(4096))))
        if op != "prompt":
            case["page"] = rng.choice(PAGES)
        h, kv, d = HEADS[case["heads"]]
        both = case["longest"] + case["prefix"]
        size = case["seqs"] * (h * case["longest"] * both if op == "prompt" else kv * d * both)
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
    total, both = sum(new), sum(new) + sum(held)
    if case["op"] == "prompt":
        pairs = sum(a * (a + b) - a * (a - 1) // 2 for a, b in zip(new, held))
        return {"bytes": 2 * d * (2 * h * total + 2 * kv * both), "flops": 4 * d * h * pairs}
    if case["op"] == "store":
        page = case["page"]
        back = sum(b + a - b // page * page for a, b in zip(new, held))
        # keys and values in and their codes out, then the codes in and 16-bit values out
        return {"bytes": 2 * kv * d * (3 * total + 3 * back), "flops": 2 * kv * d * (2 * total + back)}
    if case["op"] == "load":
        return {"bytes": 2 * kv * d * 3 * total, "flops": 2 * kv * d * total}
    return {"bytes": 2 * kv * d * total + 4 * h * d * case["seqs"], "flops": 4 * d * h * total}


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


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    h, kv, d = HEADS[case["heads"]]
    dtype = DTYPES[case["dtype"]]
    new, held = _lengths(case)
    n, total = len(new), sum(new)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": case, "status": torch.zeros(n, dtype=torch.int32, device="cuda"), "scale": 1.0 / math.sqrt(d)}
    if case["op"] == "prompt":
        both = [a + b for a, b in zip(new, held)]
        s["q"] = (1.5 * torch.randn(total, h, d, device="cuda", generator=g)).to(dtype)
        s["k"] = _keys(g, sum(both), kv, d).to(dtype)
        s["v"] = torch.randn(sum(both), kv, d, device="cuda", generator=g).to(dtype)
        s["cu_q"], s["cu_k"] = ints(_running(new)), ints(_running(both))
        s["most_q"], s["most_k"] = max(new), max(both)
        return s
    page = case["page"]
    count = [-(-(a + b) // page) for a, b in zip(new, held)]
    pages = sum(count) + 3
    where = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    wide = max(count + [1])
    at = _running(count)
    s["table"] = torch.full((n, wide), -1, dtype=torch.int32, device="cuda")
    for b in range(n):
        s["table"][b, : count[b]] = where[at[b]: at[b + 1]]
    s["k_codes"], s["k_scales"] = _quantize(_keys(g, pages * page, kv, d).view(pages, page, kv, d).transpose(1, 2))
    v, s["v_scales"] = _quantize(torch.randn(pages, kv, page, d, device="cuda", generator=g))
    s["k_codes"], s["v_codes"] = s["k_codes"].contiguous(), v.transpose(2, 3).contiguous()
    if case["op"] == "step":
        s["lens"] = ints(new)
        s["q"] = (1.5 * torch.randn(n, h, d, device="cuda", generator=g)).to(dtype)
        return s
    if case["op"] == "store":
        s["k"] = (1.2 * _keys(g, total, kv, d)).to(dtype)
        s["v"] = (1.2 * torch.randn(total, kv, d, device="cuda", generator=g)).to(dtype)
        s["held"], s["cu_new"] = ints(held), ints(_running(new))
        first = [b // page * page for b in held]
    else:
        first = [0] * n
    back = [a + b - f for a, b, f in zip(new, held, first)]
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


def _cache(ent, s):
    return ent.KVCache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])


def _own_prompt(s):
    import entropy_coded_weight_canonical_amd as ent

    return ent.attn_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["status"], scale=s["scale"])


def _own_store(s):
    import entropy_coded_weight_canonical_amd as ent

    ent.kv_store(_cache(ent, s), s["k"], s["v"], s["table"], s["held"], s["cu_new"], s["status"])
    return [*_own_load(s), s["k_scales"], s["v_scales"]]


def _own_load(s):
    import entropy_coded_weight_canonical_amd as ent

    return ent.kv_load(_cache(ent, s), s["table"], s["first"], s["cu_out"], s["n_out"], s["status"],
                       dtype=DTYPES[s["case"]["dtype"]])


def _own_step(s):
    import entropy_coded_weight_canonical_amd as ent

    return ent.attn_cache(s["q"], _cache(ent, s), s["table"], s["lens"], s["status"], scale=s["scale"])


_OWN = {"prompt": _own_prompt, "store": _own_store, "load": _own_load, "step": _own_step}


def _softmax_rows(scores, hidden):
    """Softmax over the last axis without the hidden places; a row that has
    none left is zero.  Works in place of its argument."""
    scores.masked_fill_(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_(min=-3e38)
    scores.sub_(top).exp_()
    scores.div_(scores.sum(-1, keepdim=True).clamp_(min=1e-38))
    return scores


def _plain_prompt(s):
    q, k, v, cu_q, cu_k = s["q"], s["k"], s["v"], s["cu_q"].long(), s["cu_k"].long()
    h, kv, d = HEADS[s["case"]["heads"]]
    n, nq, nk = cu_q.numel() - 1, s["most_q"], s["most_k"]
    lq, lk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    # the packed rows as padded batches
    rq = torch.arange(nq, device=q.device)
    rk = torch.arange(nk, device=q.device)
    at_q = (cu_q[:-1, None] + torch.minimum(rq[None], lq[:, None] - 1)).clamp_(0, q.shape[0] - 1)
    at_k = (cu_k[:-1, None] + torch.minimum(rk[None], lk[:, None] - 1)).clamp_(0, k.shape[0] - 1)
    qq = q[at_q].float().view(n, nq, kv, h // kv, d).permute(0, 2, 3, 1, 4).reshape(n * kv, h // kv * nq, d)
    kk = k[at_k].float().permute(0, 2, 3, 1).reshape(n * kv, d, nk).contiguous()
    vv = v[at_k].float().permute(0, 2, 1, 3).reshape(n * kv, nk, d).contiguous()
    hidden = rk[None, None] > (rq[None, :, None] + (lk - lq)[:, None, None])      # [n][nq][nk]
    hidden = hidden | (rk[None, None] >= lk[:, None, None])
    scores = torch.matmul(qq, kk).mul_(s["scale"]).view(n, kv, h // kv, nq, nk)
    p = _softmax_rows(scores, hidden[:, None, None])
    o = torch.matmul(p.view(n * kv, h // kv * nq, nk), vv)
    o = o.view(n, kv, h // kv, nq, d).permute(0, 3, 1, 2, 4).reshape(n * nq, h, d).to(q.dtype)
    # back to the packed rows
    seq = torch.repeat_interleave(torch.arange(n, device=q.device), lq, output_size=q.shape[0])
    return o[seq * nq + torch.arange(q.shape[0], device=q.device) - cu_q[seq]]


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


def _plain_store(s):
    page = s["case"]["page"]
    held, cu, table = s["held"].long(), s["cu_new"].long(), s["table"].long()
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
    row = (cu[seq][:, None] + pos - held[seq][:, None]).clamp_(0, max(s["k"].shape[0] - 1, 0))
    codes, s["k_scales"][ids] = _grown(s["k_codes"][ids], s["k_scales"][ids], s["k"][row].float(), is_new, is_held)
    s["k_codes"][ids] = codes
    codes, s["v_scales"][ids] = _grown(s["v_codes"][ids].transpose(2, 3), s["v_scales"][ids], s["v"][row].float(), is_new,
                                       is_held)
    s["v_codes"][ids] = codes.transpose(2, 3)
    return [*_plain_load(s), s["k_scales"], s["v_scales"]]


def _plain_load(s):
    page, dtype = s["case"]["page"], DTYPES[s["case"]["dtype"]]
    cu, table = s["cu_out"].long(), s["table"].long()
    dev = table.device
    seq = torch.repeat_interleave(torch.arange(cu.numel() - 1, device=dev), cu[1:] - cu[:-1], output_size=s["n_out"])
    pos = s["first"].long()[seq] + torch.arange(s["n_out"], device=dev) - cu[seq]
    ids, row = table[seq, pos // page], pos % page
    k = s["k_codes"][ids, :, row].float().mul_(s["k_scales"][ids][:, :, None])
    v = s["v_codes"][ids, :, :, row].float().mul_(s["v_scales"][ids][:, :, None])
    return [k.to(dtype), v.to(dtype)]


def _plain_step(s):
    q, lens = s["q"], s["lens"].long()
    h, kv, d = HEADS[s["case"]["heads"]]
    table = s["table"].long().clamp_(min=0)
    n, wide = table.shape
    tokens = wide * s["case"]["page"]
    # [n][pages][kv][...] to one key matrix and one value matrix per sequence and head
    k = s["k_codes"][table].float().mul_(s["k_scales"][table][..., None, None])
    k = k.permute(0, 2, 4, 1, 3).reshape(n * kv, d, tokens)
    v = s["v_codes"][table].float().mul_(s["v_scales"][table][..., None, None])
    v = v.permute(0, 2, 1, 4, 3).reshape(n * kv, tokens, d)
    scores = torch.matmul(q.float().view(n * kv, h // kv, d), k).mul_(s["scale"]).view(n, h, tokens)
    p = _softmax_rows(scores, (torch.arange(tokens, device=q.device)[None] >= lens[:, None])[:, None])
    return torch.matmul(p.view(n * kv, h // kv, tokens), v).view(n, h, d).to(q.dtype)


_PLAIN = {"prompt": _plain_prompt, "store": _plain_store, "load": _plain_load, "step": _plain_step}


# ---------------------------------------------------------------------------
# the definition in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "store": _exact_store, "load": _exact_load, "step": _exact_step}[case["op"]](s)


def _exact_head(q, k, v, scale, behind):
    """One head: row i of q sees the keys up to i + behind."""
    logits = (q @ k.t()) * scale
    i = torch.arange(q.shape[0], device=q.device)[:, None] + behind
    j = torch.arange(k.shape[0], device=q.device)[None, :]
    w = torch.exp(torch.where(j <= i, logits - logits.masked_fill(j > i, -math.inf).max(1, keepdim=True).values, -math.inf))
    return (w @ v) / w.sum(1, keepdim=True)


def _exact_prompt(s):
    h, kv, d = HEADS[s["case"]["heads"]]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(len(cu_q) - 1):
        (i0, i1), (j0, j1) = cu_q[b: b + 2], cu_k[b: b + 2]
        if i1 == i0:
            continue
        for head in range(h):
            g = head // (h // kv)
            out[i0:i1, head] = _exact_head(s["q"][i0:i1, head].double(), s["k"][j0:j1, g].double(), s["v"][j0:j1, g].double(),
                                           s["scale"], (j1 - j0) - (i1 - i0))
    return out


def _exact_rows(s, b, lo, hi):
    """Keys and values of sequence b's tokens lo .. hi-1 in the cache."""
    page = s["case"]["page"]
    ids = [int(i) for i in s["table"][b, lo // page: -(-hi // page)].tolist()]
    k = torch.cat([s["k_codes"][i].double() * s["k_scales"][i].double()[:, None, None] for i in ids], 1)
    v = torch.cat([s["v_codes"][i].double() * s["v_scales"][i].double()[:, None, None] for i in ids], 2)
    lead = lo // page * page
    return k[:, lo - lead: hi - lead].transpose(0, 1), v[:, :, lo - lead: hi - lead].permute(2, 0, 1)


def _exact_load(s):
    cu, first = s["cu_out"].tolist(), s["first"].tolist()
    got = [_exact_rows(s, b, first[b], first[b] + cu[b + 1] - cu[b]) for b in range(len(first)) if cu[b + 1] > cu[b]]
    return [torch.cat([x[0] for x in got]), torch.cat([x[1] for x in got])]


def _exact_store(s):
    page = s["case"]["page"]
    held, cu, first, table = s["held"].tolist(), s["cu_new"].tolist(), s["first"].tolist(), s["table"].tolist()
    scales = {"k": s["k_scales"].double(), "v": s["v_scales"].double()}
    rows = {"k": [], "v": []}
    for b in range(len(held)):
        end = held[b] + cu[b + 1] - cu[b]
        for lead in range(first[b], end, page):
            at = table[b][lead // page]
            keep = min(max(held[b] - lead, 0), page)
            take = min(end - lead, page) - keep
            for name, codes in (("k", s["k_codes"][at]), ("v", s["v_codes"][at].transpose(1, 2))):
                was = scales[name][at].clone()
                x = s[name][cu[b] + lead + keep - held[b]:][:take].double().transpose(0, 1)          # [kv][take][d]
                now = x.abs().amax((1, 2)) / 127 if take else torch.zeros_like(was)
                if keep:
                    now = torch.maximum(now, was)
                scales[name][at] = now
                now = now[:, None, None]
                old = torch.round(codes[:, :keep].double() * (was[:, None, None] / now)) * now
                rows[name].append(torch.cat([old, torch.round(x / now) * now], 1).transpose(0, 1))
    return [torch.cat(rows["k"]), torch.cat(rows["v"]), scales["k"], scales["v"]]


def _exact_step(s):
    h, kv, d = HEADS[s["case"]["heads"]]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n:
            k, v = _exact_rows(s, b, 0, n)
            for head in range(h):
                out[b, head] = _exact_head(s["q"][b, head: head + 1].double(), k[:, head // (h // kv)], v[:, head // (h // kv)],
                                           s["scale"], n - 1)[0]
    return out
