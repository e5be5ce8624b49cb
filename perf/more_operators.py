"""Measured cases of attention and the paged key-value cache that it reads.

Three operators, each with a plain form in elementary torch operations (32-bit
arithmetic, one rounding at the end) and the library's calls:

  cache    new tokens' keys and values written into a paged cache, as they are
           or quantized in blocks of 32 channels (e4m3 or e2m1 values with a
           power of two as the block's scale), and the same rows read back
  paged    o = softmax(scale q K^T) V for one new token of each sequence, whose
           keys and values lie in pages of such a cache
  prompt   the same for whole prompts: packed sequences of different lengths or
           a batch, causal or not, query heads that share key heads
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 32                                   # channels that share a scale
TOP = {"fp8": (8, 3, -6, 448.0), "fp4": (2, 1, 0, 6.0)}     # largest exponent, mantissa bits, smallest exponent, largest value


def listed():
    return [
        # one new token of four sequences, fp4 cache: latency
        {"name": "cache_token", "op": "cache", "tokens": 4, "heads": 8, "dim": 128, "page": 16, "pages": 64,
         "kind": "fp4", "dtype": "bf16", "padding": 0},
        # a padded batch of ragged prompts, an odd number of heads, half precision
        {"name": "cache_odd", "op": "cache", "tokens": 1999, "heads": 3, "dim": 96, "page": 32, "pages": 80,
         "kind": "fp8", "dtype": "f16", "padding": 357},
        # the prompts of a busy server, fp4 cache
        {"name": "cache_prompts", "op": "cache", "tokens": 32768, "heads": 8, "dim": 128, "page": 64, "pages": 600,
         "kind": "fp4", "dtype": "bf16", "padding": 0},
        # one short sequence, grouped heads, cache in bf16: latency
        {"name": "paged_token", "op": "paged", "lengths": "301", "q_heads": 32, "k_heads": 8, "dim": 128, "page": 16,
         "kind": "same", "dtype": "bf16"},
        # ragged requests, one of them just admitted and one empty, three heads a key head, fp8 cache
        {"name": "paged_odd", "op": "paged", "lengths": "1,0,77,1500,333,4099", "q_heads": 9, "k_heads": 3, "dim": 96,
         "page": 8, "kind": "fp8", "dtype": "f16"},
        # sixteen requests of a chat server, cache in bf16
        {"name": "paged_batch", "op": "paged",
         "lengths": "4000,310,2048,95,1200,7777,640,3300,150,5120,2900,1,8191,450,1750,980",
         "q_heads": 32, "k_heads": 8, "dim": 128, "page": 64, "kind": "same", "dtype": "bf16"},
        # eight long documents, fp4 cache
        {"name": "paged_long", "op": "paged", "lengths": "32768,30001,32768,32000,28123,32767,32768,31000", "q_heads": 32,
         "k_heads": 8, "dim": 128, "page": 64, "kind": "fp4", "dtype": "bf16"},
        # one short prompt: latency
        {"name": "prompt_short", "op": "prompt", "q_lens": "128", "k_lens": "128", "q_heads": 16, "k_heads": 4,
         "dim": 64, "causal": True, "packed": False, "dtype": "bf16"},
        # one picture's 1024 image and 512 text tokens, every token sees every other, heads out of the packed projection
        {"name": "prompt_image", "op": "prompt", "q_lens": "1536", "k_lens": "1536", "q_heads": 24, "k_heads": 24,
         "dim": 128, "causal": False, "packed": True, "dtype": "bf16"},
        # ragged prompts packed one behind the other, one of a single token and one empty
        {"name": "prompt_ragged", "op": "prompt", "q_lens": "1,999,0,2501,63,1777,3001,130",
         "k_lens": "1,999,0,2501,63,1777,3001,130", "q_heads": 32, "k_heads": 8, "dim": 128, "causal": True,
         "packed": True, "dtype": "bf16"},
        # the next pieces of two long prompts against everything before them, an odd head size
        {"name": "prompt_chunk", "op": "prompt", "q_lens": "200,33", "k_lens": "9001,4242", "q_heads": 9, "k_heads": 3,
         "dim": 72, "causal": True, "packed": False, "dtype": "f16"},
        # one long prompt
        {"name": "prompt_long", "op": "prompt", "q_lens": "16384", "k_lens": "16384", "q_heads": 32, "k_heads": 8,
         "dim": 128, "causal": True, "packed": False, "dtype": "bf16"},
    ]


def _lens(text):
    return [int(n) for n in text.split(",")]


def _width(case):
    """Bytes of one row of a cache, scales included, as a number of bits a value."""
    return {"same": 16.0, "fp8": 8.25, "fp4": 4.25}[case["kind"]]


# The largest work of a drawn case: that of the largest listed ones.
MOST_CACHE = 32768 * 8 * 128
MOST_PAGED = sum(_lens("32768,30001,32768,32000,28123,32767,32768,31000")) * 8 * 128 * 4.25   # bits of the keys
MOST_PROMPT = 16384 * 16384 // 2 * 32 * 128


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(("cache", "paged", "prompt"))
    if op == "cache":
        kind = rng.choice(("same", "fp8", "fp4", "fp4"))
        dim = rng.choice((32, 64, 96, 128, 128, 192, 256) if kind != "same" else (64, 72, 80, 128, 256))
        heads, page = rng.choice((1, 2, 3, 4, 5, 8, 8, 16)), rng.choice((8, 16, 32, 64, 128, 256))
        tokens = _log(rng, 1, MOST_CACHE // (dim * heads))
        tokens = min(tokens, 65536)
        return {"op": op, "tokens": tokens, "heads": heads, "dim": dim, "page": page,
                "pages": -(-tokens // page) + rng.randint(1, 40), "kind": kind, "dtype": rng.choice(("bf16", "bf16", "f16")),
                "padding": rng.choice((0, 0, tokens // 5))}
    ks = rng.choice((1, 1, 2, 3, 4, 8))
    qs = ks * rng.choice((1, 2, 3, 4, 4, 8, 16))
    if op == "paged":
        kind = rng.choice(("same", "fp8", "fp4"))
        dim = rng.choice((64, 96, 128, 128, 192, 256) if kind != "same" else (64, 72, 80, 128, 256))
        case = {"op": op, "lengths": "", "q_heads": qs, "k_heads": ks, "dim": dim, "page": rng.choice((8, 16, 32, 64, 128, 256)),
                "kind": kind, "dtype": rng.choice(("bf16", "bf16", "f16"))}
        batch = _log(rng, 1, 48)
        each = max(1, int(MOST_PAGED / (_width(case) * ks * dim * batch * max(1, qs // ks / 4))))
        top = _log(rng, 16, min(131072, max(16, each)))
        lengths = [_log(rng, 1, top) if rng.random() < 0.5 else rng.randint(0, top) for _ in range(batch)]
        lengths[rng.randrange(batch)] = top
        case["lengths"] = ",".join(map(str, lengths))
        return case
    dim = rng.choice((64, 72, 80, 96, 128, 128, 128, 192, 256))
    count = _log(rng, 1, 8)
    top = _log(rng, 16, min(16384, max(16, int(math.sqrt(MOST_PROMPT / (qs * dim * count))))))
    q_lens = [_log(rng, 1, top) if rng.random() < 0.5 else rng.randint(0, top) for _ in range(count)]
    q_lens[rng.randrange(count)] = top
    how = rng.choice(("self", "self", "after", "other"))
    k_lens = list(q_lens)
    if how == "after":      # pieces of longer prompts
        q_lens = [min(n, rng.choice((1, 16, 100, 512))) for n in q_lens]
    elif how == "other":    # keys of another text
        k_lens = [rng.randint(0, top) for _ in q_lens]
    return {"op": op, "q_lens": ",".join(map(str, q_lens)), "k_lens": ",".join(map(str, k_lens)), "q_heads": qs,
            "k_heads": ks, "dim": dim, "causal": rng.random() < 0.6, "packed": how == "self" and rng.random() < 0.6,
            "dtype": rng.choice(("bf16", "bf16", "f16"))}


# ---- inputs -----------------------------------------------------------------


def _normal(g, shape, dtype=torch.float32):
    """Heads as projections make them: a few channels are larger than the others."""
    x = torch.randn(shape, generator=g, device="cuda")
    x[..., torch.randint(0, shape[-1], (max(1, shape[-1] // 32),), generator=g, device="cuda")] *= 4.0
    return x.to(dtype)


def _pow2(n):
    """2^n of whole n, exact (a power function may be off in its last place)."""
    return ((n.clamp(-126, 127).int() + 127) << 23).view(torch.float32)


def _codes(x, kind):
    """Rows [..., dim] as the bytes of a cache and the exponents (plus 127) of its blocks."""
    top, bits, least, most = TOP[kind]
    x = x.float().unflatten(-1, (-1, BLOCK))
    power = torch.frexp(x.abs().amax(-1))[1] - 1 - top
    x = (x * _pow2(-power.unsqueeze(-1))).clamp(-most, most).flatten(-2)
    scales = (power + 127).clamp(0, 254).to(torch.uint8)
    if kind == "fp8":
        return x.to(torch.float8_e4m3fn), scales
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = torch.bucketize(x.abs(), edges).to(torch.uint8) + 8 * (x < 0).to(torch.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, scales


def _stored(g, case, pages):
    """A filled cache: keys, values and their scales, [pages, heads, page, ...]."""
    shape, out = (pages, case["k_heads"], case["page"], case["dim"]), []
    for _ in range(2):
        x = _normal(g, shape, DT[case["dtype"]])
        out.append((x, None) if case["kind"] == "same" else _codes(x, case["kind"]))
    return {"k": out[0][0], "v": out[1][0], "k_scales": out[0][1], "v_scales": out[1][1]}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, dim = DT[case["dtype"]], case["dim"]
    if case["op"] == "cache":
        tokens, heads, rows = case["tokens"], case["heads"], case["pages"] * case["page"]
        qkv = _normal(g, (tokens, 3, heads, dim), dt)
        slots = torch.randperm(case["pages"], generator=g, device="cuda")[:-(-tokens // case["page"])]
        slots = (slots[:, None] * case["page"] + torch.arange(case["page"], device="cuda")).flatten()[:tokens]
        if case["padding"]:     # places of the padded batch that hold no token
            slots[torch.randperm(tokens, generator=g, device="cuda")[:case["padding"]]] = -1
        shape = (case["pages"], heads, case["page"])
        last, kept = {"same": (dim, dt), "fp8": (dim, torch.float8_e4m3fn), "fp4": (dim // 2, torch.uint8)}[case["kind"]]
        s = {"new_k": qkv[:, 1], "new_v": qkv[:, 2], "slots": slots,
             "values": torch.zeros((2, rows + 1, heads, dim), dtype=dt, device="cuda")}
        for name in ("k", "v"):
            s[name] = torch.zeros((*shape, last), dtype=torch.float32, device="cuda").to(kept)
            s[name + "_scales"] = None if case["kind"] == "same" else torch.zeros((*shape, dim // BLOCK), dtype=torch.uint8, device="cuda")
    elif case["op"] == "paged":
        lengths, page = _lens(case["lengths"]), case["page"]
        need = [-(-n // page) for n in lengths]
        pages = sum(need) + 3
        s = _stored(g, case, pages)
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((len(lengths), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        s.update(q=_normal(g, (len(lengths), case["q_heads"], dim), dt), table=table,
                 lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    else:
        q_lens, k_lens, hq, hk = _lens(case["q_lens"]), _lens(case["k_lens"]), case["q_heads"], case["k_heads"]
        if case["packed"]:      # slices of one projection
            qkv = _normal(g, (sum(q_lens), hq + 2 * hk, dim), dt)
            s = {"q": qkv[:, :hq], "k": qkv[:, hq:hq + hk], "v": qkv[:, hq + hk:]}
        else:
            s = {"q": _normal(g, (sum(q_lens), hq, dim), dt), "k": _normal(g, (sum(k_lens), hk, dim), dt),
                 "v": _normal(g, (sum(k_lens), hk, dim), dt)}
        for name, lens in (("q_starts", q_lens), ("k_starts", k_lens)):
            s[name] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    s["case"] = case
    return s


# ---- one pass -----------------------------------------------------------------


def run(state):
    return {"cache": _run_cache, "paged": _run_paged, "prompt": _run_prompt}[state["case"]["op"]](state)


def _rounded(x, kind):
    """What a block-quantized cache keeps of rows [..., dim], in 32 bits."""
    top, bits, least, most = TOP[kind]
    x = x.float().unflatten(-1, (-1, BLOCK))
    power = (torch.frexp(x.abs().amax(-1, keepdim=True))[1] - 1 - top).clamp(-126, 126)
    x = x * _pow2(-power)
    step = (torch.frexp(x)[1] - 1).clamp(min=least) - bits
    x = (torch.round(x * _pow2(-step)) * _pow2(step)).clamp(-most, most)
    return (x * _pow2(power)).flatten(-2)


def _values(codes, scales, kind):
    """The values that the bytes of a cache stand for, in 32 bits."""
    if kind == "same":
        return codes.float()
    if kind == "fp8":
        x = codes.float()
    else:
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
        table = torch.cat([table, -table])
        x = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    return (x.unflatten(-1, (-1, BLOCK)) * _pow2(scales.int().unsqueeze(-1) - 127)).flatten(-2)


def _handle(s):
    from w4a4_rotated_bit_amd import binding
    return binding, binding.KVCache(s["k"], s["v"], s["k_scales"], s["v_scales"])


def _run_cache(s):
    case = s["case"]
    if own:
        binding, cache = _handle(s)
        binding.convrot_cache_write(s["new_k"], s["new_v"], s["slots"], cache)
        return binding.convrot_cache_read(cache, s["slots"], dtype=s["new_k"].dtype)
    out, rows = [], s["values"].shape[1] - 1
    at = torch.where(s["slots"] < 0, rows, s["slots"])      # padding goes to a row of its own
    for x, kept in zip((s["new_k"], s["new_v"]), s["values"]):
        kept[at] = x if case["kind"] == "same" else _rounded(x, case["kind"]).to(x.dtype)
        out.append(kept[at] * (s["slots"] >= 0)[:, None, None])
    return out


def _run_paged(s):
    case, q = s["case"], s["q"]
    scale = case["dim"] ** -0.5
    if own:
        binding, cache = _handle(s)
        return binding.convrot_attention_paged(q, cache, s["table"], s["lengths"], scale=scale)
    lengths, out = _lens(case["lengths"]), []
    group = case["q_heads"] // case["k_heads"]
    for i, n in enumerate(lengths):     # the host of such a server knows its requests' lengths
        if n == 0:
            out.append(torch.zeros_like(q[i]))
            continue
        pages = s["table"][i, :-(-n // case["page"])].long()
        k, v = (_values(s[x][pages], None if s[x + "_scales"] is None else s[x + "_scales"][pages], case["kind"])
                .transpose(0, 1).flatten(1, 2)[:, :n].contiguous() for x in ("k", "v"))
        x = torch.bmm(q[i].float().unflatten(0, (-1, group)), k.transpose(1, 2).contiguous()) * scale
        x = torch.exp(x - x.amax(-1, keepdim=True))
        out.append((torch.bmm(x, v) / x.sum(-1, keepdim=True)).flatten(0, 1).to(q.dtype))
    return torch.stack(out)


def _run_prompt(s):
    case, q = s["case"], s["q"]
    scale = case["dim"] ** -0.5
    if own:
        from w4a4_rotated_bit_amd import binding
        return binding.convrot_attention(q, s["k"], s["v"], q_starts=s["q_starts"], k_starts=s["k_starts"],
                                         causal=case["causal"], scale=scale)
    group, out = case["q_heads"] // case["k_heads"], torch.zeros(q.shape, dtype=q.dtype, device="cuda")
    at_q = at_k = 0
    for nq, nk in zip(_lens(case["q_lens"]), _lens(case["k_lens"])):
        k = s["k"][at_k:at_k + nk].float().permute(1, 2, 0).repeat_interleave(group, 0).contiguous()
        v = s["v"][at_k:at_k + nk].float().transpose(0, 1).repeat_interleave(group, 0).contiguous()
        for first in range(0, nq if nk else 0, 1024):       # a piece of the rows at a time: the scores of all do not fit
            last = min(nq, first + 1024)
            x = torch.bmm(q[at_q + first:at_q + last].float().transpose(0, 1).contiguous(), k) * scale
            if case["causal"]:      # the last query sees every key
                seen = torch.arange(nk, device="cuda") <= torch.arange(first, last, device="cuda")[:, None] + (nk - nq)
                x = torch.where(seen, x, -math.inf)
                top = x.amax(-1, keepdim=True)
                x = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
            else:
                x = torch.exp(x - x.amax(-1, keepdim=True))
            total = x.sum(-1, keepdim=True)
            y = torch.bmm(x, v) / torch.where(total > 0, total, 1.0)
            out[at_q + first:at_q + last] = y.transpose(0, 1).to(q.dtype)
        at_q, at_k = at_q + nq, at_k + nk
    return out


# ---- what a pass cannot do without ----------------------------------------------


def work(case):
    if case["op"] == "cache":
        values = 2 * (case["tokens"] - case["padding"]) * case["heads"] * case["dim"]
        # read once in 16 bits, kept, read from there, written in 16 bits
        return {"bytes": values * 4 + int(values * _width(case) / 4) + case["tokens"] * 8 * 2, "flops": 2 * values}
    if case["op"] == "paged":
        lengths = _lens(case["lengths"])
        held = sum(lengths) * case["k_heads"] * case["dim"]
        heads = len(lengths) * case["q_heads"] * case["dim"]
        pages = sum(-(-n // case["page"]) for n in lengths)
        return {"bytes": int(2 * held * _width(case) / 8) + 4 * heads + 4 * pages + 4 * len(lengths),
                "flops": 4 * sum(lengths) * case["q_heads"] * case["dim"]}
    q_lens, k_lens = _lens(case["q_lens"]), _lens(case["k_lens"])
    pairs = 0
    for nq, nk in zip(q_lens, k_lens):
        if not case["causal"]:
            pairs += nq * nk
        else:       # row i of nq sees the first max(0, i + 1 + nk - nq) keys
            rows = min(nq, nk)
            pairs += rows * nk - rows * (rows - 1) // 2
    d = case["dim"]
    return {"bytes": 2 * d * (2 * sum(q_lens) * case["q_heads"] + 2 * sum(k_lens) * case["k_heads"]),
            "flops": 4 * pairs * case["q_heads"] * d}


# ---- the definitions in 64 bits ---------------------------------------------------


def _grid(kind):
    """Every value of a format that is not negative, in order."""
    top, bits, least, most = TOP[kind]
    points = [m * 2.0 ** (least - bits) for m in range(1 << bits)]
    points += [(1 + m / (1 << bits)) * 2.0 ** e for e in range(least, top + 1) for m in range(1 << bits)]
    return torch.tensor([p for p in points if p <= most], dtype=torch.float64, device="cuda")


def _power(n):
    """2^n in 64 bits, from a table of exact ones."""
    return torch.tensor([2.0 ** i for i in range(-400, 401)], dtype=torch.float64, device="cuda")[n.long() + 400]


def _nearest(x, kind):
    """x [..., dim] in 64 bits to the nearest value of its block's grid, ties to an even place in it."""
    grid = _grid(kind)
    x = x.reshape(*x.shape[:-1], -1, BLOCK)
    most = x.abs().max(-1, keepdim=True).values.clamp(min=2.0 ** -119)
    unit = _power(torch.floor(torch.log2(most)) - TOP[kind][0])     # 64 bits tell 11-bit values from the power above them
    a = (x / unit).abs().contiguous()
    hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    at = torch.where((up < down) | ((up == down) & (hi % 2 == 0)) | (a >= grid[-1]), hi, lo)
    return (torch.sign(x) * grid[at] * unit).reshape(*x.shape[:-2], -1)


def _wide(s, name, pages, case):
    """Cached rows of some pages as [heads, tokens, dim] in 64 bits."""
    x, kind = s[name][pages], case["kind"]
    if kind == "fp4":
        grid = _grid(kind)
        x = torch.stack([x % 16, x // 16], -1).flatten(-2).long()
        x = grid[x % 8] * (1 - 2 * (x // 8))
    elif kind == "fp8":
        x = x.to(torch.float64)
    else:
        x = x.double()
    if kind != "same":
        x = x * _power(s[name + "_scales"][pages].int() - 127).repeat_interleave(BLOCK, -1)
    return x.permute(1, 0, 2, 3).reshape(case["k_heads"], -1, case["dim"])


def _attended(q, k, v, scale, offset):
    """q [heads, rows, dim], k, v [heads, keys, dim] in 64 bits; row i sees keys up to i + offset (None: all)."""
    x = (q @ k.transpose(1, 2)) * scale
    if offset is not None:
        hidden = torch.ones(x.shape[1:], dtype=torch.bool, device="cuda").triu(offset + 1)
        x = x.masked_fill(hidden, -math.inf)
    x = torch.softmax(x, -1).nan_to_num(0.0) if offset is not None else torch.softmax(x, -1)
    return x @ v


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "cache":
        keep = (s["slots"] >= 0)[:, None, None]
        return [(x.double() if case["kind"] == "same" else _nearest(x.double(), case["kind"])) * keep
                for x in (s["new_k"], s["new_v"])]
    q, scale = s["q"].double(), case["dim"] ** -0.5
    share = case["q_heads"] // case["k_heads"]
    y = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    if case["op"] == "paged":
        for i, n in enumerate(_lens(case["lengths"])):
            if n:
                pages = s["table"][i, :-(-n // case["page"])].long()
                k, v = (_wide(s, name, pages, case)[:, :n] for name in ("k", "v"))
                y[i] = _attended(q[i].reshape(-1, share, case["dim"]), k, v, scale, None).reshape(-1, case["dim"])
        return y
    ends_q, ends_k = s["q_starts"].tolist(), s["k_starts"].tolist()
    for i in range(len(ends_q) - 1):
        (a, b), (c, d) = ends_q[i:i + 2], ends_k[i:i + 2]
        for h in range(case["q_heads"] if d > c else 0):
            k, v = (s[name][c:d, h // share].double()[None] for name in ("k", "v"))
            for first in range(a, b, 8192):
                last = min(b, first + 8192)
                offset = (d - c) - (b - a) + first - a if case["causal"] else None
                y[first:last, h] = _attended(q[None, first:last, h], k, v, scale, offset)[0]
    return y
