"""Measured cases of the operators around a rotated linear in a transformer block.

Three operators, each with a plain form in elementary torch operations (32-bit
arithmetic, angles in 64 bits, one rounding at the end) and the library's call:

  norm     r = a x + gate * P(y);  h = N(r) * weight * (1 + scale) + shift
           (the residual update that ends one sub-block and the modulated norm
           that begins the next; P is y itself or a norm of y)
  rope     rotary positions over several axes for the query and key heads, with
           the per-head RMS norm in front of it where the model has one
  grouped  y = x W^T + bias with 4-bit weights, one scale (and zero point) for
           every 32, 64 or 128 input channels of a row
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
THETA = 10000.0

# The largest work that a drawn case may have: bytes of one matrix for norm and
# of the heads for rope, weights for grouped (those of the largest listed cases).
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
MOST_NORM = 32768 * 4096 * 2
MOST_ROPE = 32768 * 32 * 128 * 2
MOST_GROUPED = 16384 * 16384


def listed():
    return [
        # one token of a decoder layer: residual add and RMS norm with its weight
        {"name": "norm_token", "op": "norm", "rows": 1, "width": 4096, "vectors": 0, "dtype": "bf16", "vec": "bf16",
         "norm": "rms", "post": "none", "gate": False, "modulate": False, "weight": True, "a": 1.0},
        # 1024 image and 512 text tokens of one picture, between the two halves of a diffusion transformer block
        {"name": "norm_image", "op": "norm", "rows": 1536, "width": 4096, "vectors": 1, "dtype": "bf16", "vec": "bf16",
         "norm": "layer", "post": "none", "gate": True, "modulate": True, "weight": False, "a": 1.0},
        # three ragged requests, a width that no vector load divides, a scaled residual
        {"name": "norm_odd", "op": "norm", "rows": 999, "width": 1035, "vectors": 3, "dtype": "f16", "vec": "f32",
         "norm": "layer", "post": "layer", "gate": True, "modulate": True, "weight": True, "a": 0.5},
        # two clips of 16384 video tokens, norms before and after the sub-block
        {"name": "norm_video", "op": "norm", "rows": 32768, "width": 4096, "vectors": 2, "dtype": "bf16",
         "vec": "bf16", "norm": "rms", "post": "rms", "gate": True, "modulate": True, "weight": True, "a": 1.0},
        # four sequences, one new token each, grouped key heads, three axes that share one spectrum, far positions
        {"name": "rope_token", "op": "rope", "batch": 4, "tokens": 1, "q_heads": 32, "k_heads": 8, "dim": 128,
         "axes": "16,24,24", "spectrum": "shared", "layout": "halves", "where": "far", "qk_norm": False,
         "dtype": "bf16", "packed": False, "head_major": False},
        # one picture: queries and keys out of the packed projection, per-head norm, (index, row, column) axes
        {"name": "rope_image", "op": "rope", "batch": 1, "tokens": 1536, "q_heads": 16, "k_heads": 16, "dim": 128,
         "axes": "16,56,56", "spectrum": "own", "layout": "interleaved", "where": "grid", "qk_norm": True,
         "dtype": "bf16", "packed": True, "head_major": False},
        # an odd head size, rotated in part, ragged lengths
        {"name": "rope_odd", "op": "rope", "batch": 3, "tokens": 333, "q_heads": 9, "k_heads": 3, "dim": 72,
         "axes": "22,22,22", "spectrum": "own", "layout": "halves", "where": "far", "qk_norm": True,
         "dtype": "f16", "packed": True, "head_major": False},
        # a long clip: (time, row, column), heads first for the attention that follows
        {"name": "rope_video", "op": "rope", "batch": 1, "tokens": 32768, "q_heads": 16, "k_heads": 16, "dim": 128,
         "axes": "44,42,42", "spectrum": "own", "layout": "interleaved", "where": "video", "qk_norm": True,
         "dtype": "bf16", "packed": True, "head_major": True},
        # the smallest linear, one token: latency
        {"name": "grouped_small", "op": "grouped", "m": 1, "n": 1024, "k": 1024, "group": 64, "zeros": False,
         "bias": True, "dtype": "bf16"},
        # the modulation linear of one picture (six vectors of 2048 from the conditioning vector)
        {"name": "grouped_token", "op": "grouped", "m": 1, "n": 12288, "k": 4096, "group": 128, "zeros": False,
         "bias": True, "dtype": "bf16"},
        # sixteen tokens, zero points, short groups, half precision, an odd number of outputs
        {"name": "grouped_batch", "op": "grouped", "m": 16, "n": 9001, "k": 4128, "group": 32, "zeros": True,
         "bias": False, "dtype": "f16"},
        # the largest weight, a full tile of tokens
        {"name": "grouped_large", "op": "grouped", "m": 32, "n": 16384, "k": 16384, "group": 128, "zeros": True,
         "bias": True, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "rope", "grouped"))
    if op == "norm":
        width = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            width = max(64, width // 64 * 64)
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        rows = _log(rng, 1, max(1, min(32768, MOST_NORM // (width * SIZE[dtype]))))
        vectors = rng.choice((0, 1, rng.randint(2, 4)))
        if vectors:
            rows = max(1, rows // vectors) * vectors
        vec = rng.choice((dtype, "f32"))
        gate = bool(vectors) and rng.random() < 0.7
        modulate = bool(vectors) and (not gate or rng.random() < 0.7)
        return {"op": op, "rows": rows, "width": width, "vectors": vectors, "dtype": dtype, "vec": vec,
                "norm": rng.choice(("layer", "rms")), "post": rng.choice(("none", "none", "rms", "layer")),
                "gate": gate, "modulate": modulate, "weight": rng.random() < 0.5,
                "a": rng.choice((1.0, 1.0, 0.5, 2.0))}
    if op == "rope":
        dim = rng.choice((32, 64, 72, 80, 96, 128, 128, 256))
        q = rng.randint(1, 32)
        k = rng.choice([h for h in range(1, q + 1) if q % h == 0])
        batch = rng.choice((1, 1, 2, 3))
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        tokens = _log(rng, 1, max(1, min(32768, MOST_ROPE // (dim * (q + k) * batch * SIZE[dtype]))))
        axes = rng.choice((1, 2, 3, 3))
        pairs = dim // 2 if rng.random() < 0.7 else rng.randint(axes, dim // 2)
        cuts = sorted(rng.sample(range(1, pairs), axes - 1)) if axes > 1 else []
        sizes = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
        spectrum = rng.choice(("own", "shared"))
        if spectrum == "own":
            sizes = [2 * s for s in sizes]
        return {"op": op, "batch": batch, "tokens": tokens, "q_heads": q, "k_heads": k, "dim": dim,
                "axes": ",".join(map(str, sizes)), "spectrum": spectrum,
                "layout": rng.choice(("interleaved", "halves")), "where": rng.choice(("grid", "far", "video")),
                "qk_norm": rng.random() < 0.6, "dtype": dtype,
                "packed": rng.random() < 0.5, "head_major": rng.random() < 0.3}
    group = rng.choice((32, 64, 128))
    k = max(group, _log(rng, 256, 16384) // group * group)
    n = _log(rng, 64, max(64, min(32768, MOST_GROUPED // k)))
    return {"op": op, "m": rng.choice((1, 1, 2, 4, rng.randint(3, 16), rng.randint(17, 32))), "n": n, "k": k,
            "group": group, "zeros": rng.random() < 0.5, "bias": rng.random() < 0.5,
            "dtype": rng.choice(("bf16", "bf16", "f16"))}


# ---- inputs ---------------------------------------------------------------


def _normal(g, shape, std=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def _spectrum(case):
    """Frequency (radians for a position of one) and axis of every pair."""
    sizes = [int(s) for s in case["axes"].split(",")]
    freq, axis = [], []
    if case["spectrum"] == "own":   # every axis runs through a spectrum of its own
        for a, d in enumerate(sizes):
            freq += [THETA ** (-2.0 * i / d) for i in range(d // 2)]
            axis += [a] * (d // 2)
    else:                           # one spectrum, cut into sections
        pairs = sum(sizes)
        freq = [THETA ** (-i / pairs) for i in range(pairs)]
        for a, s in enumerate(sizes):
            axis += [a] * s
    return np.array(freq, dtype=np.float64), np.array(axis, dtype=np.int32)


def _positions(g, case, axes):
    batch, tokens = case["batch"], case["tokens"]
    if case["where"] == "far":      # integer positions late in a long sequence
        base = torch.randint(0, 1 << 19, (batch, 1, 1), generator=g, device="cuda")
        step = torch.randint(0, 1 << 10, (1, 1, axes), generator=g, device="cuda")
        return (base + step + torch.arange(tokens, device="cuda").reshape(1, -1, 1)).to(torch.int32)
    i = torch.arange(tokens, device="cuda")
    if case["where"] == "grid":     # a third of text tokens at the origin, then an image grid
        text = tokens // 3
        side = max(1, math.isqrt(max(1, tokens - text)))
        j = (i - text).clamp(min=0)
        cols = torch.stack([torch.zeros_like(j), j // side, j % side], -1)
    else:                           # frames of 32 x 32 patches, frames 1/8 second apart
        cols = torch.stack([i // 1024 * 0.125, (i // 32) % 32, i % 32], -1)
    return cols[:, 3 - axes:].float().reshape(1, tokens, axes).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DT[case["dtype"]]
    if case["op"] == "norm":
        rows, width, v, vdt = case["rows"], case["width"], case["vectors"], DT[case["vec"]]
        x = torch.randn((rows, width), generator=g, device="cuda")
        x[:, torch.randint(0, width, (max(1, width // 100),), generator=g, device="cuda")] *= 20.0
        s = {"x": x.to(dt), "y": _normal(g, (rows, width), 0.5, 0.0, dt),
             "gate": None, "scale": None, "shift": None, "weight": None, "post_weight": None}
        if v:   # one modulation output holds every vector of a batch entry side by side
            mod = _normal(g, (v, 3 * width), 0.3, 0.0, vdt)
            if case["gate"]:
                s["gate"] = mod[:, :width]
            if case["modulate"]:
                s["scale"], s["shift"] = mod[:, width:2 * width], mod[:, 2 * width:]
        if case["weight"]:
            s["weight"] = _normal(g, (width,), 0.1, 1.0, vdt)
            if case["post"] != "none":
                s["post_weight"] = _normal(g, (width,), 0.1, 1.0, vdt)
    elif case["op"] == "rope":
        b, t, hq, hk, d = case["batch"], case["tokens"], case["q_heads"], case["k_heads"], case["dim"]
        if case["packed"]:
            qkv = _normal(g, (b, t, (hq + 2 * hk) * d), 1.0, 0.0, dt)
            q = qkv[..., :hq * d].unflatten(-1, (hq, d))
            k = qkv[..., hq * d:(hq + hk) * d].unflatten(-1, (hk, d))
        else:
            q, k = _normal(g, (b, t, hq, d), 1.0, 0.0, dt), _normal(g, (b, t, hk, d), 1.0, 0.0, dt)
        freq, axis = _spectrum(case)
        s = {"q": q, "k": k, "freq": freq, "axis": axis, "positions": _positions(g, case, int(axis.max()) + 1),
             "q_weight": None, "k_weight": None}
        if case["qk_norm"]:
            s["q_weight"], s["k_weight"] = _normal(g, (d,), 0.1, 1.0, dt), _normal(g, (d,), 0.1, 1.0, dt)
    else:
        m, n, k, group = case["m"], case["n"], case["k"], case["group"]
        x = torch.randn((m, k), generator=g, device="cuda")
        x[:, torch.randint(0, k, (max(1, k // 100),), generator=g, device="cuda")] *= 20.0
        s = {"x": x.to(dt), "codes": torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8),
             "scales": ((torch.rand((n, k // group), generator=g, device="cuda") + 0.5) * 0.006).to(dt),
             "zeros": None, "bias": None}
        if case["zeros"]:
            s["zeros"] = torch.randint(5, 11, (n, k // group), generator=g, device="cuda", dtype=torch.uint8)
        if case["bias"]:
            s["bias"] = _normal(g, (n,), 0.01, 0.0, dt)
    s["case"] = case
    return s


# ---- one pass ---------------------------------------------------------------


def run(state):
    return {"norm": _run_norm, "rope": _run_rope, "grouped": _run_grouped}[state["case"]["op"]](state)


def _per_row(vec, rows):
    """A modulation vector for every row: [V, width] -> [rows, width] in 32 bits."""
    return vec.float().repeat_interleave(rows // vec.shape[0], dim=0)


def _plain_norm(z, kind):
    if kind == "layer":
        z = z - z.mean(dim=-1, keepdim=True)
    return z * torch.rsqrt((z * z).mean(dim=-1, keepdim=True) + EPS)


def _run_norm(s):
    case = s["case"]
    if own:
        from w4a4_rotated_bit_amd import binding
        return binding.convrot_residual_norm(
            s["x"], s["y"], gate=s["gate"], scale=s["scale"], shift=s["shift"], weight=s["weight"],
            post_weight=s["post_weight"], norm=case["norm"], post_norm=None if case["post"] == "none" else case["post"],
            residual_scale=case["a"], eps=EPS)
    rows, dt = case["rows"], s["x"].dtype
    z = s["y"].float()
    if case["post"] != "none":
        z = _plain_norm(z, case["post"])
        if s["post_weight"] is not None:
            z = z * s["post_weight"].float()
    if s["gate"] is not None:
        z = _per_row(s["gate"], rows) * z
    r = case["a"] * s["x"].float() + z
    h = _plain_norm(r, case["norm"])
    if s["weight"] is not None:
        h = h * s["weight"].float()
    if s["scale"] is not None:
        h = h * (1.0 + _per_row(s["scale"], rows)) + _per_row(s["shift"], rows)
    return r.to(dt), h.to(dt)


def _plain_rope(x, weight, cos, sin, layout, head_major):
    z, pairs = x.float(), cos.shape[-1]
    if weight is not None:
        z = z * torch.rsqrt((z * z).mean(dim=-1, keepdim=True) + EPS) * weight.float()
    turned, rest = z[..., :2 * pairs], z[..., 2 * pairs:]
    if layout == "interleaved":
        u, v = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([u * cos - v * sin, u * sin + v * cos], dim=-1).flatten(-2)
    else:
        u, v = turned[..., :pairs], turned[..., pairs:]
        turned = torch.cat([u * cos - v * sin, u * sin + v * cos], dim=-1)
    z = torch.cat([turned, rest], dim=-1).to(x.dtype)
    return z.transpose(1, 2).contiguous() if head_major else z


def _run_rope(s):
    case = s["case"]
    if own:
        from w4a4_rotated_bit_amd import binding
        q_out = k_out = None
        if case["head_major"]:
            b, t, d = case["batch"], case["tokens"], case["dim"]
            q_out = torch.empty((b, case["q_heads"], t, d), dtype=s["q"].dtype, device="cuda")
            k_out = torch.empty((b, case["k_heads"], t, d), dtype=s["q"].dtype, device="cuda")
            binding.convrot_rope(s["q"], s["k"], s["positions"], s["freq"], s["axis"], layout=case["layout"],
                                 qk_norm=case["qk_norm"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                                 q_out=q_out.transpose(1, 2), k_out=k_out.transpose(1, 2))
            return q_out, k_out
        return binding.convrot_rope(s["q"], s["k"], s["positions"], s["freq"], s["axis"], layout=case["layout"],
                                    qk_norm=case["qk_norm"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
    axis = torch.from_numpy(s["axis"]).to("cuda", torch.int64)
    freq = torch.from_numpy(s["freq"]).to("cuda")
    angle = s["positions"].double()[..., axis] * freq       # [batch or 1, tokens, pairs], 64 bits
    cos, sin = angle.cos().float().unsqueeze(2), angle.sin().float().unsqueeze(2)
    return (_plain_rope(s["q"], s["q_weight"], cos, sin, case["layout"], case["head_major"]),
            _plain_rope(s["k"], s["k_weight"], cos, sin, case["layout"], case["head_major"]))


def _run_grouped(s):
    case = s["case"]
    if own:
        from w4a4_rotated_bit_amd import binding
        return binding.convrot_linear_grouped(s["x"], s["codes"], s["scales"], s["zeros"], s["bias"], case["group"])
    n, k, group = case["n"], case["k"], case["group"]
    code = torch.stack([s["codes"] & 15, s["codes"] >> 4], dim=-1).reshape(n, k // group, group).float()
    if s["zeros"] is None:      # two's complement
        code = code - 16.0 * (code >= 8).float()
    else:
        code = code - s["zeros"].float().unsqueeze(-1)
    w = (code * s["scales"].float().unsqueeze(-1)).reshape(n, k)
    y = s["x"].float() @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype)


# ---- what a pass cannot do without --------------------------------------------


def work(case):
    es = SIZE[case["dtype"]]
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        vectors = case["vectors"] * ((1 if case["gate"] else 0) + (2 if case["modulate"] else 0))
        weights = (2 if case["post"] != "none" else 1) if case["weight"] else 0
        return {"bytes": 4 * n * es + (vectors + weights) * case["width"] * SIZE[case["vec"]],
                "flops": n * (10 + (8 if case["post"] != "none" else 0))}
    if case["op"] == "rope":
        n = case["batch"] * case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["dim"]
        axes = len(case["axes"].split(","))
        places = (case["batch"] if case["where"] == "far" else 1) * case["tokens"] * axes * 4
        return {"bytes": 2 * n * es + places, "flops": n * (3 + (4 if case["qk_norm"] else 0))}
    m, n, k = case["m"], case["n"], case["k"]
    groups = n * (k // case["group"])
    return {"bytes": n * k // 2 + groups * (es + (1 if case["zeros"] else 0)) + (m * k + m * n + (n if case["bias"] else 0)) * es,
            "flops": 2 * m * n * k}


# ---- the definitions in 64 bits -------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    wide = {key: v.double() for key, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    if case["op"] == "norm":
        rows, width = case["rows"], case["width"]

        def normed(z, kind, weight):
            centre = z.sum(-1, keepdim=True) / width if kind == "layer" else 0.0
            z = z - centre
            z = z / torch.sqrt(z.pow(2).sum(-1, keepdim=True) / width + EPS)
            return z if weight is None else z * weight

        per = max(1, rows // max(1, case["vectors"]))
        x, y = (wide[key].reshape(-1, per, width) for key in ("x", "y"))
        if case["post"] != "none":
            y = normed(y, case["post"], wide.get("post_weight"))
        if "gate" in wide:
            y = y * wide["gate"][:, None]
        r = x * case["a"] + y
        h = normed(r, case["norm"], wide.get("weight"))
        if "scale" in wide:
            h = h + h * wide["scale"][:, None] + wide["shift"][:, None]
        return r.reshape(rows, width), h.reshape(rows, width)
    if case["op"] == "rope":
        turns = s["positions"].double()[..., torch.from_numpy(s["axis"]).long().cuda()] * torch.from_numpy(s["freq"]).cuda()
        turn = torch.polar(torch.ones_like(turns), turns)[:, :, None]

        def rotated(x, weight):
            z = x.double()
            if weight is not None:
                z = z / torch.sqrt(z.pow(2).mean(-1, keepdim=True) + EPS) * weight.double()
            p = turn.shape[-1]
            head = z[..., :2 * p]
            head = head.unflatten(-1, (p, 2)) if case["layout"] == "interleaved" else head.unflatten(-1, (2, p)).transpose(-1, -2)
            head = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn)
            head = head if case["layout"] == "interleaved" else head.transpose(-1, -2)
            z = torch.cat([head.flatten(-2), z[..., 2 * p:]], -1)
            return z.permute(0, 2, 1, 3).contiguous() if case["head_major"] else z

        return rotated(s["q"], s["q_weight"]), rotated(s["k"], s["k_weight"])
    n, k, group = case["n"], case["k"], case["group"]
    value = torch.arange(16, dtype=torch.float64, device="cuda")
    y = torch.zeros((case["m"], n), dtype=torch.float64, device="cuda")
    if s["zeros"] is None:
        value[8:] -= 16
    even, odd = value[(s["codes"] % 16).long()], value[(s["codes"] // 16).long()]
    if s["zeros"] is not None:
        offset = s["zeros"].double().repeat_interleave(group // 2, dim=1)
        even, odd = even - offset, odd - offset
    factor = wide["scales"].repeat_interleave(group // 2, dim=1)
    y = wide["x"][:, 0::2] @ (even * factor).t() + wide["x"][:, 1::2] @ (odd * factor).t()
    return y + wide["bias"] if case["bias"] else y
