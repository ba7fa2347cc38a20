"""The operators of the 8-bit latent cache, as they are measured: cases, inputs, plain forms, 64-bit values.

The paged latent cache keeps one row a token for all heads: a latent of 512 channels and, where the model
rotates positions, a key part of 64 channels.  Held in 8 bits, a row is e4m3 numbers with one power of two
2^e for the row, the smallest with max |row| <= 448 * 2^e (e from -64 to 120; a row of zeros has -64).  Three
operators serve it:

  write    new tokens' rows quantised into the cache (key part and queries rotated on the way), then read back
  gather   cached rows read back, packed, as bf16 for the up-projection of a cached prefix
  decode   the absorbed form: queries already in latent space attend over the 8-bit cache

Where ``own`` is false, ``run`` computes them with elementary torch operations in 32 bits (angles in 64).
"""
import math
import random

import torch

own = False

LATENT = 512   # channels of the latent
NOPE = 128     # per-head key channels of the expanded form (the library's head width)
E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu
DEV = "cuda"


def listed():
    return [
        # one new token for each of 64 running sequences: a serving step, 32 heads of queries rotated with it
        {"name": "write step 64", "op": "write", "n": 64, "new": 1, "ctx": 8192, "heads": 32, "page": 64, "rope": 64,
         "interleaved": False},
        # one ragged prompt of 777 tokens in a model that does not rotate positions
        {"name": "write prompt 1x777 no rope", "op": "write", "n": 1, "new": 777, "ctx": 777, "heads": 32, "page": 128,
         "rope": 0, "interleaved": False},
        # eight ragged prompts of up to 2048 tokens written at once, small pages
        {"name": "write prompts 8x2048", "op": "write", "n": 8, "new": 2048, "ctx": 2048, "heads": 32, "page": 16,
         "rope": 64, "interleaved": True},
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
        # the same with 64 heads: twice the arithmetic a cached byte
        {"name": "decode 64x8192 h64", "op": "decode", "n": 64, "tokens": 1, "ctx": 8192, "heads": 64, "page": 64,
         "rope": 64},
        # the KDA decode benchmark's 256 sequences x 32 heads; no rotated part (position-free layers)
        {"name": "decode 256x8192 no rope", "op": "decode", "n": 256, "tokens": 1, "ctx": 8192, "heads": 32,
         "page": 64, "rope": 0},
        # a step of four tokens (drafted tokens being checked) of a 16-head shard, small pages
        {"name": "decode 32x4096 t4", "op": "decode", "n": 32, "tokens": 4, "ctx": 4096, "heads": 16, "page": 16,
         "rope": 64},
        # 100 short odd contexts of a 12-head shard
        {"name": "decode 100x401 h12", "op": "decode", "n": 100, "tokens": 1, "ctx": 401, "heads": 12, "page": 32,
         "rope": 64},
        # one very long context: the work of a single sequence over the whole card
        {"name": "decode 1x131072", "op": "decode", "n": 1, "tokens": 1, "ctx": 131072, "heads": 32, "page": 128,
         "rope": 64},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "gather", "decode", "decode", "decode"])
    page = rng.choice([16, 32, 64, 128, 256])
    rope = rng.choice([0, 64, 64])
    heads = rng.choice([1, 4, 8, 12, 16, 20, 32, 40, 64])
    if op == "write":
        n = _log(rng, 1, 256)
        new = 1 if rng.random() < 0.5 else _log(rng, 1, max(1, 16384 // n))
        return {"op": op, "n": n, "new": new, "ctx": new + _log(rng, 1, 8192), "heads": min(heads, 32), "page": page,
                "rope": rope, "interleaved": rng.random() < 0.5}
    if op == "gather":
        n = _log(rng, 1, 64)
        return {"op": op, "n": n, "ctx": _log(rng, 1, 262144 // n), "page": page, "rope": rope}
    tokens = rng.choice([1, 1, 1, 2, 3, 5, 8, 16])
    n = _log(rng, 1, 256)
    ctx = _log(rng, 16, min(131072, 2097152 // n * 32 // max(32, heads * tokens)))
    return {"op": op, "n": n, "tokens": tokens, "ctx": max(tokens, ctx), "heads": heads, "page": page, "rope": rope}


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
    if op == "write":
        new = [case["new"]] + [r.randint(1, case["new"]) for _ in range(n - 1)]
        return new, [k + r.randint(0, case["ctx"] - case["new"]) for k in new]
    least = max(case.get("tokens", 1), (case["ctx"] + 3) // 4)
    return None, [case["ctx"]] + [r.randint(least, case["ctx"]) for _ in range(n - 1)]


def _paged(lens, top, page, rope, g):
    """An 8-bit cache that holds `lens` tokens a sequence on pages in random order, its rows' powers of two and
    its block table.  Rows are about N(0, 1) times 1/2, 1 or 2, as e4m3 numbers of up to 448."""
    per = -(-top // page)
    used = (lens + page - 1) // page
    total = int(used.sum())
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    at = torch.arange(per, device=DEV)[None, :] < used[:, None]
    table = torch.full((lens.numel(), per), -1, dtype=torch.int32, device=DEV)
    table[at] = order
    rows = torch.randn((total, page, LATENT + rope), generator=g, device=DEV).mul_(100).clamp_(-448, 448).to(E4M3)
    powers = torch.randint(119, 122, (total, page), generator=g, device=DEV).to(torch.uint8)
    return rows, powers.view(E8M0), table


def _offsets(counts):
    return torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), counts.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    new, lens = (x and torch.tensor(x, device=DEV) for x in _lengths(case))
    cache, powers, table = _paged(lens, case["ctx"], case["page"], case["rope"], g)
    s.update(cache=cache, powers=powers, table=table, lens=lens.to(torch.int32))
    if case["op"] == "write":
        total, rope = int(new.sum()), case["rope"]
        # rows of different sizes, as different layers' and tokens' are
        size = torch.exp2(torch.randint(-3, 4, (total, 1), generator=g, device=DEV).float()).to(torch.bfloat16)
        s.update(cu=_offsets(new), total=total, starts=(lens - new).to(torch.int32), latent=_randn((total, LATENT), g) * size,
                 rope_k=_randn((total, 64), g) * size if rope else None,
                 # the queries' rotated part is the end of each head's query row
                 q=_randn((total, case["heads"], NOPE + 64), g) if rope else None,
                 freq=(10000.0 ** (-torch.arange(32, device=DEV, dtype=torch.float64) / 32)).float())
    elif case["op"] == "gather":
        s.update(cu=_offsets(lens), total=int(lens.sum()))
    else:
        rows = case["n"] * case["tokens"]
        s.update(q_latent=_randn((rows, case["heads"], LATENT), g),
                 q_rope=_randn((rows, case["heads"], case["rope"]), g) if case["rope"] else None)
        if own:
            import linear_attention_06_gb300 as kda
            size = kda.kda_latent_decode_q8_workspace_size(case["n"], rows, case["heads"], case["rope"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return s


def run(s):
    return _own(s) if own else PLAIN[s["op"]](s)


# ---------------------------------------------------------------- the framework's operators

def _own(s):
    import linear_attention_06_gb300 as kda
    if s["op"] == "write":
        q = kda.kda_latent_append_q8(s["latent"], s["rope_k"], s["cache"], s["powers"], s["table"], s["lens"],
                                     inv_freq=s["freq"] if s["rope"] else None, interleaved=s["interleaved"],
                                     q_rope=s["q"][..., NOPE:] if s["rope"] else None, cu_seqlens=s["cu"])
        return (*kda.kda_latent_gather_q8(s["cache"], s["powers"], s["table"], s["cu"], s["total"], s["starts"]), q)
    if s["op"] == "gather":
        return kda.kda_latent_gather_q8(s["cache"], s["powers"], s["table"], s["cu"], s["total"])
    return kda.kda_latent_decode_q8(s["q_latent"], s["q_rope"], s["cache"], s["powers"], s["table"], s["lens"],
                                    _scale(s["rope"]), lse=True, workspace=s["workspace"])


# ---------------------------------------------------------------- plain forms

def _read(s, seq, pos):
    """The values that cached rows stand for, in 32 bits."""
    page, width = s["page"], LATENT + s["rope"]
    at = s["table"].long()[seq, pos // page] * page + pos % page
    x = s["cache"].view(torch.uint8).view(-1, width)[at].view(E4M3).float()
    return x * torch.exp2(s["powers"].view(torch.uint8).view(-1)[at].float() - 127)[:, None]


def _split(s, x):
    x = x.to(torch.bfloat16)
    return (x[:, :LATENT].contiguous(), x[:, LATENT:].contiguous()) if s["rope"] else (x, None)


def _plain_write(s):
    cu, page, width = s["cu"].long(), s["page"], LATENT + s["rope"]
    row = torch.arange(s["total"], device=DEV)
    seq = torch.searchsorted(cu, row, right=True) - 1
    pos = s["lens"].long()[seq] - cu[seq + 1] + row
    x, q = s["latent"].float(), None
    if s["rope"]:
        angle = pos.double()[:, None] * s["freq"].double()
        cos, sin = angle.cos().float(), angle.sin().float()

        def rotate(x, c, d):
            x = x.float()
            a, b = (x[..., 0::2], x[..., 1::2]) if s["interleaved"] else (x[..., :32], x[..., 32:])
            y = (a * c - b * d, a * d + b * c)
            return torch.stack(y, -1).flatten(-2) if s["interleaved"] else torch.cat(y, -1)

        x = torch.cat([x, rotate(s["rope_k"], cos, sin)], 1)
        q = rotate(s["q"][..., NOPE:], cos[:, None], sin[:, None]).to(torch.bfloat16)
    most = x.abs().amax(1)
    part, e = torch.frexp(most)                       # most = part * 2^e, part in [1/2, 1); 448 = 7/8 * 2^9
    e = torch.where(most > 0, e - 9 + (part > 0.875), -64).clamp(-64, 120)
    x = (x * torch.exp2(-e.float())[:, None]).to(E4M3)
    at = s["table"].long()[seq, pos // page] * page + pos % page
    s["cache"].view(torch.uint8).view(-1, width)[at] = x.view(torch.uint8)
    s["powers"].view(torch.uint8).view(-1)[at] = (e + 127).to(torch.uint8)
    return (*_split(s, _read(s, seq, pos)), q)


def _plain_gather(s):
    cu = s["cu"].long()
    row = torch.arange(s["total"], device=DEV)
    seq = torch.searchsorted(cu, row, right=True) - 1
    return _split(s, _read(s, seq, row - cu[seq]))


def _plain_decode(s):
    n, page, tokens, heads = s["n"], s["page"], s["tokens"], s["heads"]
    width = LATENT + s["rope"]
    at = (s["table"].long().clamp_min(0)[:, :, None] * page + torch.arange(page, device=DEV)).view(n, -1)
    c = s["cache"].view(torch.uint8).view(-1, width)[at].view(E4M3).float()
    c.mul_(torch.exp2(s["powers"].view(torch.uint8).view(-1)[at].float() - 127)[..., None])
    q = s["q_latent"] if s["q_rope"] is None else torch.cat([s["q_latent"], s["q_rope"]], -1)
    x = torch.bmm(q.float().view(n, tokens * heads, width), c.transpose(1, 2)).mul_(_scale(s["rope"]))
    limit = (s["lens"].long()[:, None] - tokens + 1 + torch.arange(tokens, device=DEV)).repeat_interleave(heads, 1)
    x.masked_fill_(torch.arange(c.shape[1], device=DEV) >= limit[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.bmm(x, c[..., :LATENT]) / total.clamp_min(1e-38)
    lse = (m + total.log()).squeeze(-1)
    return o.to(torch.bfloat16).view(n * tokens, heads, LATENT), lse.view(n * tokens, heads)


PLAIN = {"write": _plain_write, "gather": _plain_gather, "decode": _plain_decode}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    new, lens = _lengths(case)
    width, total = LATENT + case["rope"], sum(lens)
    held = width + 1                                  # a cached row with its power of two
    if case["op"] == "write":                         # rows in, cached and read back; queries in and out
        return {"bytes": sum(new) * (2 * width + held + 2 * width + (4 * 64 * case["heads"] if case["rope"] else 0)),
                "flops": sum(new) * (3 * 64 * (1 + case["heads"]) if case["rope"] else 0)}
    if case["op"] == "gather":
        return {"bytes": total * (held + 2 * width), "flops": 0}
    rows = case["tokens"] * case["heads"]
    return {"bytes": total * held + case["n"] * rows * (2 * width + 2 * LATENT + 4),
            "flops": 2 * rows * total * (width + LATENT)}


# ---------------------------------------------------------------- the values, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s)


def _held(s, n, first, last):
    """Cached rows first .. last - 1 of sequence n, in 64 bits."""
    pages = s["table"][n, : -(-last // s["page"])].long()
    x = s["cache"].view(torch.uint8)[pages].view(E4M3).double()
    x = x * _two(s["powers"].view(torch.uint8)[pages].double() - 127)[..., None]
    return x.reshape(-1, LATENT + s["rope"])[first:last]


def _halves(s, x):
    return (x[:, :LATENT], x[:, LATENT:]) if s["rope"] else (x, None)


def _to_e4m3(x):
    """The nearest e4m3 number (ties to even) to each x of up to 448, from the definition: steps of 2^-3 of the
    number's power of two, and of 2^-9 below 2^-6."""
    size = x.abs().clamp_min(2.0 ** -6)
    k = torch.floor(torch.log2(size))
    k = k + (_two(k + 1) <= size).double() - (_two(k) > size).double()        # a logarithm may miss its whole number
    return torch.round(x * _two(3 - k)) * _two(k - 3)


def _two(k):
    """2^k exactly, for whole k from -1022 to 1023: the number of 64 bits with this exponent."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _exact_write(s):
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    rows = s["latent"].double()
    turned = None
    if s["rope"]:
        def turn(x, unit):                            # pairs as complex numbers times e^(i angle)
            if s["interleaved"]:
                pairs = torch.view_as_complex(x.reshape(*x.shape[:-1], 32, 2)) * unit
                return torch.view_as_real(pairs).flatten(-2)
            z = torch.complex(x[..., :32], x[..., 32:]) * unit
            return torch.cat([z.real, z.imag], -1)

        pos = torch.cat([torch.arange(n - (b - a), n, device=DEV) for a, b, n in zip(cu[:-1], cu[1:], lens)])
        angle = torch.outer(pos.double(), s["freq"].double())
        unit = torch.polar(torch.ones_like(angle), angle)
        rows = torch.cat([rows, turn(s["rope_k"].double(), unit)], 1)
        turned = turn(s["q"][..., NOPE:].double(), unit[:, None])
    most = rows.abs().amax(1, keepdim=True)
    power = torch.ceil(torch.log2(most.clamp_min(2.0 ** -200) / 448))
    power = power + (448 * _two(power) < most).double() - (448 * _two(power - 1) >= most).double()
    power = power.clamp(-64, 120)
    return (*_halves(s, _to_e4m3(rows * _two(-power)) * _two(power)), turned)


def _exact_gather(s):
    cu = s["cu"].tolist()
    return _halves(s, torch.cat([_held(s, n, 0, cu[n + 1] - cu[n]) for n in range(s["n"])]))


def _exact_decode(s):
    t, outs, sums = s["tokens"], [], []
    for n, length in enumerate(s["lens"].tolist()):
        c = _held(s, n, 0, length)
        q = s["q_latent"][n * t:(n + 1) * t].double()
        if s["q_rope"] is not None:
            q = torch.cat([q, s["q_rope"][n * t:(n + 1) * t].double()], -1)
        for j in range(t):
            seen = c[: length - t + 1 + j]
            x = q[j] @ seen.T * _scale(s["rope"])
            sums.append(torch.logsumexp(x, -1))
            outs.append(torch.softmax(x, -1) @ seen[:, :LATENT])
    return torch.stack(outs), torch.stack(sums)
