"""The latent-attention operators, as they are measured: cases, inputs, plain forms, 64-bit values.

Latent attention keeps one vector a token for all heads: a latent c of 512 channels and, where the model
rotates positions, a key part r of 64 channels.  Four operators serve it:

  append   writes new tokens' [c | r] rows into a paged cache, r (and the queries' r part) rotated on the way
  gather   reads cached rows back, packed, for the up-projection of a cached prefix
  decode   the absorbed form: queries already in latent space attend over the paged cache
  prefill  the expanded form: per-head keys and values of a prompt, the r part shared by the heads

Where ``own`` is false, ``run`` computes them with elementary torch operations in 32 bits (angles in 64).
"""
import math
import random

import torch

own = False

LATENT = 512   # channels of the latent
NOPE = 128     # per-head key / value / query channels of the expanded form (the library's head width)
DEV = "cuda"


def listed():
    return [
        # one new token for each of 64 running sequences: a serving step, 32 heads of queries rotated with it
        {"name": "append step 64", "op": "append", "n": 64, "new": 1, "ctx": 8192, "heads": 32, "page": 64,
         "interleaved": False},
        # eight ragged prompts of up to 2048 tokens written at once, small pages
        {"name": "append prompts 8x2048", "op": "append", "n": 8, "new": 2048, "ctx": 2048, "heads": 32,
         "page": 16, "interleaved": True},
        # one short cached prefix read back
        {"name": "gather 1x1000", "op": "gather", "n": 1, "ctx": 1000, "page": 16, "rope": 64},
        # sixteen cached prefixes of up to 16384 tokens
        {"name": "gather 16x16384", "op": "gather", "n": 16, "ctx": 16384, "page": 64, "rope": 64},
        # one user, one token, a short context: latency alone counts
        {"name": "decode 1x1024", "op": "decode", "n": 1, "tokens": 1, "ctx": 1024, "heads": 32, "page": 64,
         "rope": 64},
        # 64 users with ragged contexts
        {"name": "decode 64x8192", "op": "decode", "n": 64, "tokens": 1, "ctx": 8192, "heads": 32, "page": 64,
         "rope": 64},
        # the KDA decode benchmark's 256 sequences x 32 heads; no rotated part (position-free layers)
        {"name": "decode 256x8192 no rope", "op": "decode", "n": 256, "tokens": 1, "ctx": 8192, "heads": 32,
         "page": 64, "rope": 0},
        # a step of four tokens (drafted tokens being checked) of a 16-head shard, small pages
        {"name": "decode 32x4096 t4", "op": "decode", "n": 32, "tokens": 4, "ctx": 4096, "heads": 16, "page": 16,
         "rope": 64},
        # one very long context: the work of a single sequence over the whole card
        {"name": "decode 1x131072", "op": "decode", "n": 1, "tokens": 1, "ctx": 131072, "heads": 32, "page": 128,
         "rope": 64},
        # three short ragged prompts
        {"name": "prefill 3x100", "op": "prefill", "n": 3, "new": 100, "past": 0, "heads": 32, "rope": 64,
         "ragged": True},
        # two sequences' chunks of 1024 tokens over 16384 tokens already cached; no rotated part
        {"name": "prefill 2x1024+16384", "op": "prefill", "n": 2, "new": 1024, "past": 16384, "heads": 32,
         "rope": 0, "ragged": False},
        # the KDA prefill benchmark's 4 x 8192 tokens x 32 heads
        {"name": "prefill 4x8192", "op": "prefill", "n": 4, "new": 8192, "past": 0, "heads": 32, "rope": 64,
         "ragged": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "gather", "decode", "decode", "prefill"])
    page = rng.choice([16, 32, 64, 128, 256])
    rope = rng.choice([0, 64, 64])
    heads = rng.choice([1, 4, 8, 12, 16, 20, 32, 40, 64])
    if op == "append":
        n = _log(rng, 1, 256)
        new = 1 if rng.random() < 0.5 else _log(rng, 1, max(1, 16384 // n))
        return {"op": op, "n": n, "new": new, "ctx": new + _log(rng, 1, 8192), "heads": min(heads, 32), "page": page,
                "interleaved": rng.random() < 0.5}
    if op == "gather":
        n = _log(rng, 1, 64)
        return {"op": op, "n": n, "ctx": _log(rng, 1, 262144 // n), "page": page, "rope": rope}
    if op == "decode":
        tokens = rng.choice([1, 1, 1, 2, 3, 5, 8, 16])
        n = _log(rng, 1, 256)
        ctx = _log(rng, 16, min(131072, 2097152 // n * 32 // max(32, heads * tokens)))
        return {"op": op, "n": n, "tokens": tokens, "ctx": max(tokens, ctx), "heads": heads, "page": page, "rope": rope}
    n = _log(rng, 1, 8)
    heads = min(heads, 32)
    new = _log(rng, 1, 4096)
    past = 0 if rng.random() < 0.5 else _log(rng, 1, 8192)
    while n * heads * new * (new + past) > 4 * 32 * 8192 * 4096:
        new, past = new * 2 // 3 + 1, past * 2 // 3
    return {"op": op, "n": n, "new": new, "past": past, "heads": heads, "rope": rope, "ragged": rng.random() < 0.7}


def _scale(rope):
    return (NOPE + rope) ** -0.5


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _lengths(case):
    """A case's sequence lengths: (new tokens, tokens in all), a list each.  They belong to the case, so that
    its outputs have one shape; the longest sequence comes first, the others are uniform below it."""
    r, n, op = random.Random(case["n"]), case["n"], case["op"]
    if op == "append":
        new = [case["new"]] + [r.randint(1, case["new"]) for _ in range(n - 1)]
        return new, [k + r.randint(0, case["ctx"] - case["new"]) for k in new]
    if op == "prefill":
        new, past = case["new"], case["past"]
        if not case["ragged"]:
            return [new] * n, [new + past] * n
        nq = [new] + [r.randint((new + 1) // 2, new) for _ in range(n - 1)]
        return nq, [k + r.randint(0, past) for k in nq]
    least = max(case.get("tokens", 1), (case["ctx"] + 3) // 4)
    return None, [case["ctx"]] + [r.randint(least, case["ctx"]) for _ in range(n - 1)]


def _paged(lens, top, page, rope, g):
    """A cache that holds `lens` tokens a sequence on pages in random order, and its block table."""
    per = -(-top // page)
    used = (lens + page - 1) // page
    total = int(used.sum())
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    at = torch.arange(per, device=DEV)[None, :] < used[:, None]
    table = torch.full((lens.numel(), per), -1, dtype=torch.int32, device=DEV)
    table[at] = order
    return _randn((total, page, LATENT + rope), g), table


def _offsets(counts):
    return torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), counts.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    new, lens = (x and torch.tensor(x, device=DEV) for x in _lengths(case))
    if case["op"] == "append":
        cache, table = _paged(lens, case["ctx"], case["page"], 64, g)
        total = int(new.sum())
        s.update(cache=cache, table=table, lens=lens.to(torch.int32), cu=_offsets(new),
                 latent=_randn((total, LATENT), g), rope_k=_randn((total, 64), g),
                 # the queries' rotated part is the end of each head's query row
                 q=_randn((total, case["heads"], NOPE + 64), g),
                 freq=(10000.0 ** (-torch.arange(32, device=DEV, dtype=torch.float64) / 32)).float())
    elif case["op"] == "gather":
        cache, table = _paged(lens, case["ctx"], case["page"], case["rope"], g)
        s.update(cache=cache, table=table, cu=_offsets(lens), total=int(lens.sum()))
    elif case["op"] == "decode":
        cache, table = _paged(lens, case["ctx"], case["page"], case["rope"], g)
        rows = case["n"] * case["tokens"]
        s.update(cache=cache, table=table, lens=lens.to(torch.int32),
                 q_latent=_randn((rows, case["heads"], LATENT), g),
                 q_rope=_randn((rows, case["heads"], case["rope"]), g) if case["rope"] else None)
        if own:
            import linear_attention_06_gb300 as kda
            size = kda.kda_latent_decode_workspace_size(case["n"], rows, case["heads"], case["rope"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    else:
        t, u = int(new.sum()), int(lens.sum())
        # the up-projection gives each token and head its key and value side by side
        kv = _randn((u, case["heads"], 2 * NOPE), g)
        s.update(q=_randn((t, case["heads"], NOPE + case["rope"]), g), k=kv[..., :NOPE], v=kv[..., NOPE:],
                 rope_k=_randn((u, case["rope"]), g) if case["rope"] else None, cu_q=_offsets(new),
                 cu_k=_offsets(lens), most_q=int(new.max()), most_k=int(lens.max()))
    return s


def run(s):
    return _own(s) if own else PLAIN[s["op"]](s)


# ---------------------------------------------------------------- the framework's operators

def _own(s):
    import linear_attention_06_gb300 as kda
    if s["op"] == "append":
        q = kda.kda_latent_append(s["latent"], s["rope_k"], s["cache"], s["table"], s["lens"], inv_freq=s["freq"],
                                  interleaved=s["interleaved"], q_rope=s["q"][..., NOPE:], cu_seqlens=s["cu"])
        return s["cache"], q
    if s["op"] == "gather":
        return kda.kda_latent_gather(s["cache"], s["table"], s["cu"], s["total"])
    if s["op"] == "decode":
        return kda.kda_latent_decode(s["q_latent"], s["q_rope"], s["cache"], s["table"], s["lens"],
                                     _scale(s["rope"]), lse=True, workspace=s["workspace"])
    return kda.kda_latent_prefill(s["q"], s["k"], s["v"], s["rope_k"], _scale(s["rope"]), cu_seqlens=s["cu_q"],
                                  cu_seqlens_k=s["cu_k"], lse=True)


# ---------------------------------------------------------------- plain forms

def _plain_append(s):
    cu, cache, page = s["cu"].long(), s["cache"], s["page"]
    row = torch.arange(s["latent"].shape[0], device=DEV)
    seq = torch.searchsorted(cu, row, right=True) - 1
    pos = s["lens"].long()[seq] - cu[seq + 1] + row
    angle = pos.double()[:, None] * s["freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()

    def rotate(x, c, d):
        x = x.float()
        a, b = (x[..., 0::2], x[..., 1::2]) if s["interleaved"] else (x[..., :32], x[..., 32:])
        y = (a * c - b * d, a * d + b * c)
        y = torch.stack(y, -1).flatten(-2) if s["interleaved"] else torch.cat(y, -1)
        return y.to(torch.bfloat16)

    where = s["table"].long()[seq, pos // page] * page + pos % page
    cache.view(-1, LATENT + 64)[where] = torch.cat([s["latent"], rotate(s["rope_k"], cos, sin)], 1)
    return cache, rotate(s["q"][..., NOPE:], cos[:, None], sin[:, None])


def _plain_gather(s):
    cu, page = s["cu"].long(), s["page"]
    row = torch.arange(s["total"], device=DEV)
    seq = torch.searchsorted(cu, row, right=True) - 1
    pos = row - cu[seq]
    x = s["cache"].view(-1, LATENT + s["rope"])[s["table"].long()[seq, pos // page] * page + pos % page]
    return (x[:, :LATENT].contiguous(), x[:, LATENT:].contiguous()) if s["rope"] else (x, None)


def _softmax_rows(x):
    """exp(x - max) in place, its sums and the log-sum-exp; a row of -inf gives zeros."""
    m = x.amax(-1, keepdim=True)
    z = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x.sub_(z).exp_()
    total = x.sum(-1, keepdim=True)
    return total, (z + total.log()).squeeze(-1)


def _plain_decode(s):
    n, page, tokens, heads = s["n"], s["page"], s["tokens"], s["heads"]
    width = LATENT + s["rope"]
    at = s["table"].long().clamp_min(0)[:, :, None] * page + torch.arange(page, device=DEV)
    c = s["cache"].view(-1, width)[at.view(n, -1)].float()
    q = s["q_latent"] if s["q_rope"] is None else torch.cat([s["q_latent"], s["q_rope"]], -1)
    x = torch.bmm(q.float().view(n, tokens * heads, width), c.transpose(1, 2)).mul_(_scale(s["rope"]))
    limit = (s["lens"].long()[:, None] - tokens + 1 + torch.arange(tokens, device=DEV)).repeat_interleave(heads, 1)
    x.masked_fill_(torch.arange(c.shape[1], device=DEV) >= limit[:, :, None], -math.inf)
    total, lse = _softmax_rows(x)
    o = torch.bmm(x, c[..., :LATENT]) / total.clamp_min(1e-38)
    return o.to(torch.bfloat16).view(n * tokens, heads, LATENT), lse.view(n * tokens, heads)


def _plain_prefill(s):
    n, heads, mq, mk = s["n"], s["heads"], s["most_q"], s["most_k"]
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    nq, nk = cq[1:] - cq[:-1], ck[1:] - ck[:-1]
    iq, ik = torch.arange(mq, device=DEV), torch.arange(mk, device=DEV)
    k = s["k"] if s["rope_k"] is None else torch.cat(
        [s["k"], s["rope_k"][:, None].expand(-1, heads, -1)], -1)

    def padded(x, cu, i):
        at = (cu[:-1, None] + i).clamp_max(x.shape[0] - 1)
        return x[at].transpose(1, 2).float()          # [n, heads, longest, channels]

    x = (padded(s["q"], cq, iq) @ padded(k, ck, ik).transpose(2, 3)).mul_(_scale(s["rope"]))
    limit = (nk - nq)[:, None] + iq                   # the last key that query i sees
    hidden = ik > limit[:, :, None]
    x.masked_fill_(hidden[:, None], -math.inf)
    total, lse = _softmax_rows(x)
    o = (x @ padded(s["v"], ck, ik)).div_(total)
    live = iq < nq[:, None]
    return o.transpose(1, 2)[live].to(torch.bfloat16), lse.transpose(1, 2)[live]


PLAIN = {"append": _plain_append, "gather": _plain_gather, "decode": _plain_decode, "prefill": _plain_prefill}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    new, lens = _lengths(case)
    width, total = LATENT + case.get("rope", 64), sum(lens)
    if case["op"] == "append":
        return {"bytes": sum(new) * (4 * width + 4 * 64 * case["heads"]), "flops": sum(new) * 64 * 3 * (1 + case["heads"])}
    if case["op"] == "gather":
        return {"bytes": total * 4 * width, "flops": 0}
    if case["op"] == "decode":
        rows = case["tokens"] * case["heads"]
        return {"bytes": total * 2 * width + case["n"] * rows * (2 * width + 2 * LATENT + 4),
                "flops": 2 * rows * total * (width + LATENT)}
    h, wide = case["heads"], NOPE + case["rope"]
    pairs = sum(q * (k - q) + q * (q + 1) / 2 for q, k in zip(new, lens))
    return {"bytes": h * (sum(new) * (2 * (wide + NOPE) + 4) + total * 4 * NOPE) + total * 2 * case["rope"],
            "flops": 2 * h * pairs * (wide + NOPE)}


# ---------------------------------------------------------------- the values, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s)


def _exact_append(s):
    cu, lens, table, page = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist(), s["page"]
    cache = s["cache"].double()
    flat = cache.view(-1, LATENT + 64)
    queries = s["q"][..., NOPE:].double()
    turned = torch.empty_like(queries)

    def turn(x, unit):                                # pairs as complex numbers times e^(i angle)
        if s["interleaved"]:
            return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:-1], 32, 2)) * unit).flatten(-2)
        z = torch.complex(x[..., :32], x[..., 32:]) * unit
        return torch.cat([z.real, z.imag], -1)

    for n in range(s["n"]):
        a, b = cu[n], cu[n + 1]
        pos = torch.arange(lens[n] - (b - a), lens[n], device=DEV)
        angle = torch.outer(pos.double(), s["freq"].double())
        unit = torch.polar(torch.ones_like(angle), angle)
        pages = torch.tensor(table[n], device=DEV)[torch.div(pos, page, rounding_mode="floor")]
        slot = pages * page + pos % page
        flat[slot, :LATENT] = s["latent"][a:b].double()
        flat[slot, LATENT:] = turn(s["rope_k"][a:b].double(), unit)
        turned[a:b] = turn(queries[a:b], unit[:, None])
    return cache, turned


def _rows(s, n, count):
    """The first `count` cached rows of sequence n, in 64 bits."""
    pages = s["table"][n, : -(-count // s["page"])].long()
    return s["cache"][pages].reshape(-1, LATENT + s["rope"])[:count].double()


def _exact_gather(s):
    cu = s["cu"].tolist()
    x = torch.cat([_rows(s, n, cu[n + 1] - cu[n]) for n in range(s["n"])])
    return (x[:, :LATENT], x[:, LATENT:]) if s["rope"] else (x, None)


def _exact_decode(s):
    t, outs, sums = s["tokens"], [], []
    for n, length in enumerate(s["lens"].tolist()):
        c = _rows(s, n, length)
        q = s["q_latent"][n * t:(n + 1) * t].double()
        if s["q_rope"] is not None:
            q = torch.cat([q, s["q_rope"][n * t:(n + 1) * t].double()], -1)
        for j in range(t):
            seen = c[: length - t + 1 + j]
            x = q[j] @ seen.T * _scale(s["rope"])
            sums.append(torch.logsumexp(x, -1))
            outs.append(torch.softmax(x, -1) @ seen[:, :LATENT])
    return torch.stack(outs), torch.stack(sums)


def _exact_prefill(s):
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    out = torch.empty((*s["q"].shape[:2], NOPE), dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    for n in range(s["n"]):
        a, b, c, d = cq[n], cq[n + 1], ck[n], ck[n + 1]
        for h in range(s["heads"]):
            k = s["k"][c:d, h].double()
            if s["rope_k"] is not None:
                k = torch.cat([k, s["rope_k"][c:d].double()], -1)
            x = s["q"][a:b, h].double() @ k.T * _scale(s["rope"])
            x += torch.full_like(x, -math.inf).triu_(d - c - (b - a) + 1)
            lse[a:b, h] = torch.logsumexp(x, -1)
            out[a:b, h] = torch.softmax(x, -1) @ s["v"][c:d, h].double()
    return out, lse
