"""The operators around the linears of a block, against their formulas in
binary64: the residual update with its norms, rotary positions over several
axes, and the product with group-scaled 4-bit weights.

Tolerances are sums of what the arithmetic may lose.  u = 2^-24 is half a step
of binary32 relative to the value; an output stored in type t adds half a step
of t, finfo(t).eps / 2 of it (and half the smallest subnormal)."""
import numpy as np
import pytest
import torch

from w4a4_rotated_bit_amd import binding as B

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# additions one after the other in a row's sum: at most 64 elements a thread,
# 6 steps across a wave, 16 waves, and a few roundings of the statistics
SUM = 64 + 6 + 16 + 10


def half_step(dtype, value):
    info = torch.finfo(dtype)
    return info.eps / 2 * value.abs() + info.smallest_normal * info.eps / 2


def close(got, want, bound, what=""):
    got = got.detach().cpu().double()
    assert got.shape == want.shape
    bad = ~((got - want).abs() <= bound)
    same = (got == want) | (got.isnan() & want.isnan())
    bad &= ~same
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, first at {at}: got {got[at]}, "
                             f"want {want[at]} +- {bound[at] if bound.dim() else bound}")


def rand(shape, seed, dtype=torch.float32, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


def dev(t):
    return None if t is None else t.cuda()


# ---- residual update and norms -------------------------------------------------


def norm_of(v, e, kind, eps):
    """The norm of v (error e), and the error of its binary32 evaluation."""
    if kind is None:
        return v, e
    mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[..., :1])
    size = v.abs().mean(-1, keepdim=True)
    d = v - mean
    rstd = 1 / torch.sqrt((d * d).mean(-1, keepdim=True) + eps)
    n = d * rstd
    centred = (v.abs() + SUM * size) * U + e + e.mean(-1, keepdim=True)    # error of v - mean
    err = centred * rstd
    err = err + n.abs() * ((centred * centred).mean(-1, keepdim=True).sqrt() * rstd + SUM * U)
    return n, err


def norm_reference(x, y, gate, scale, shift, weight, post_weight, norm, post, a, eps):
    """r, h and their error bounds before the storage rounding; vectors are
    already one a row."""
    x = x.double()
    zero = torch.zeros_like(x)
    one = torch.ones_like(x)
    if y is None:
        r, er = a * x, (a * x).abs() * U
    else:
        z, ez = norm_of(y.double(), zero, post, eps)
        w = one if post_weight is None else post_weight.double()
        g = one if gate is None else gate.double()
        z, ez = z * w * g, ez * (w * g).abs()
        r = a * x + z
        er = ez + 4 * U * ((a * x).abs() + z.abs())
    h, eh = norm_of(r, er, norm, eps)
    w = one if weight is None else weight.double()
    s = zero if scale is None else scale.double()
    b = zero if shift is None else shift.double()
    n = h * w
    return r, er, n * (1 + s) + b, eh * (w * (1 + s)).abs() + 4 * U * (n.abs() * (1 + s.abs()) + b.abs())


def check_norm(rows, width, dtype="bf16", vec=None, vectors=1, norm="layer", post=None, gate=True, modulate=True,
               weight=False, y=True, a=1.0, eps=1e-6, mean=0.0, std=1.0, seed=0, strided=False):
    dt, vdt = TYPES[dtype], TYPES[vec or dtype]
    pad = 8 if strided else 0
    xs, ys = (rand((rows, width + pad), seed + i, dt, std, mean)[:, :width] for i in (0, 1))
    mods = rand((vectors, 3 * width), seed + 2, vdt, 0.4)
    g, s, b = mods[:, :width], mods[:, width:2 * width], mods[:, 2 * width:]
    ws = [rand((width,), seed + 3 + i, vdt, 0.1, 1.0) for i in (0, 1)]
    on = {"gate": g if gate and y else None, "scale": s if modulate else None, "shift": b if modulate else None,
          "weight": ws[0] if weight else None, "post_weight": ws[1] if weight and post else None}
    cuda = {k: dev(v) for k, v in on.items()}
    if strided:
        wide = dev(torch.cat([xs, ys], 1))
        cx, cy = wide[:, :width], wide[:, width:]
        cm = mods.cuda()
        for i, k in enumerate(("gate", "scale", "shift")):
            if cuda[k] is not None:
                cuda[k] = cm[:, i * width:(i + 1) * width]
    else:
        cx, cy = dev(xs), dev(ys)
    r, h = B.convrot_residual_norm(cx, cy if y else None, norm=norm, post_norm=post, residual_scale=a, eps=eps, **cuda)
    rowwise = {k: v if v is None or v.dim() == 1 else v.repeat_interleave(rows // vectors, 0) for k, v in on.items()}
    want_r, er, want_h, eh = norm_reference(xs, ys if y else None, norm=norm, post=post, a=a, eps=eps, **rowwise)
    close(r, want_r, er + half_step(dt, want_r.abs() + er), "r")
    close(h, want_h, eh + half_step(dt, want_h.abs() + eh), "h")
    return r, h


@pytest.mark.gpu
@pytest.mark.parametrize("width", [1, 7, 64, 65, 255, 512, 520, 1000, 1035, 2048, 4096, 4104, 8192, 8200, 16383, 16384])
def test_norm_widths(gpu, width):
    check_norm(5, width, norm="rms" if width == 1 else "layer", seed=width)
    check_norm(5, width, dtype="f32", norm="rms", post="rms", weight=True, seed=width + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,vec", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("norm,post", [("layer", None), ("rms", None), ("rms", "rms"), ("layer", "layer"), (None, "rms")])
def test_norm_kinds_and_types(gpu, dtype, vec, norm, post):
    for i, (width, vectors) in enumerate(((768, 1), (1024, 3), (130, 2))):
        check_norm(6, width, dtype, vec, vectors, norm, post, weight=i == 1, a=(1.0, 0.5, -2.0)[i], seed=7 * i)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,width", [("bf16", 2056), ("bf16", 4096), ("f16", 4091), ("f32", 2048), ("f32", 2045), ("f16", 1035)])
def test_norm_more_rows_than_units(gpu, dtype, width):
    check_norm(300, width, dtype, vectors=3, norm="layer", post="rms", seed=width)
    check_norm(257, width, dtype, vec="f32", norm="rms", seed=width)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 63, 1537])
def test_norm_rows_and_per_row_vectors(gpu, rows):
    check_norm(rows, 256, vectors=rows, seed=rows)       # a vector of its own for every row
    check_norm(rows, 512, "f16", vectors=1, gate=False, seed=rows)
    check_norm(rows, 384, y=False, a=3.0, seed=rows)     # a plain modulated norm


@pytest.mark.gpu
def test_norm_strided_rows(gpu):
    for width in (96, 100, 1024):
        check_norm(9, width, vectors=3, strided=True, seed=width)


@pytest.mark.gpu
def test_norm_mean_far_from_zero(gpu):
    """A mean of 1000 deviations costs the statistics nothing beyond the input's own rounding."""
    check_norm(4, 1024, "f32", mean=1000.0, std=1.0, y=False, gate=False, seed=3)
    check_norm(4, 4096, "f32", mean=-300.0, std=0.1, norm="layer", post="layer", seed=4)


@pytest.mark.gpu
def test_norm_constant_and_zero_rows(gpu):
    x = torch.full((3, 512), 2.5, dtype=torch.bfloat16, device="cuda")
    x[1] = 0
    r, h = B.convrot_residual_norm(x, norm="layer")
    assert torch.equal(r, x) and (h == 0).all()
    _, h = B.convrot_residual_norm(x, norm="rms", eps=1e-6)
    assert (h[1] == 0).all() and (h[0] == 1).all()


@pytest.mark.gpu
def test_norm_keeps_infinities_and_nans_in_their_rows(gpu):
    x = rand((4, 1024), 1, torch.bfloat16).cuda()
    y = rand((4, 1024), 2, torch.bfloat16).cuda()
    r0, h0 = B.convrot_residual_norm(x, y)
    x[1, 7], y[2, 900] = float("inf"), float("nan")
    r, h = B.convrot_residual_norm(x, y)
    for i in (0, 3):
        assert torch.equal(r[i], r0[i]) and torch.equal(h[i], h0[i])
    assert r[1, 7] == float("inf") and torch.isnan(h[1]).all() and torch.isnan(r[2, 900]) and torch.isnan(h[2]).all()
    assert torch.equal(r[1, 8:], r0[1, 8:])


@pytest.mark.gpu
def test_norm_in_place_single_outputs_and_shapes(gpu):
    x, y = (rand((2, 6, 768), s, torch.bfloat16).cuda() for s in (1, 2))
    gate, scale, shift = (rand((2, 768), s, torch.bfloat16, 0.4).cuda() for s in (3, 4, 5))
    mods = dict(gate=gate, scale=scale, shift=shift)
    r, h = B.convrot_residual_norm(x, y, **mods)
    assert r.shape == h.shape == x.shape
    # the same rows as a matrix, and vectors with a dimension of one
    r2, h2 = B.convrot_residual_norm(x.view(12, 768), y.view(12, 768), **mods)
    r3, h3 = B.convrot_residual_norm(x, y, **{k: v.unsqueeze(1) for k, v in mods.items()})
    for a, b in ((r2, h2), (r3, h3)):
        assert torch.equal(a.view_as(r), r) and torch.equal(b.view_as(h), h)
    xi, yi = x.clone(), y.clone()
    ri, hi = B.convrot_residual_norm(xi, yi, r=xi, h=yi, **mods)
    assert ri is xi and hi is yi and torch.equal(xi, r) and torch.equal(yi, h)
    only_r = B.convrot_residual_norm(x, y, gate=gate, want_h=False)
    only_h = B.convrot_residual_norm(x, y, want_r=False, **mods)
    assert only_r[1] is None and torch.equal(only_r[0], r) and only_h[0] is None and torch.equal(only_h[1], h)
    r0, h0 = B.convrot_residual_norm(x[:, :0], y[:, :0], **mods)
    assert r0.shape == h0.shape == (2, 0, 768)


@pytest.mark.gpu
def test_norm_leaves_the_gaps_of_its_outputs(gpu):
    buf = torch.full((7, 1000), 5.0, dtype=torch.bfloat16, device="cuda")
    x = rand((5, 400), 1, torch.bfloat16).cuda()
    r, h = buf[1:6, 8:408], buf[1:6, 500:900]
    B.convrot_residual_norm(x, r=r, h=h)
    assert torch.equal(r, x)
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[1:6, 8:408] = keep[1:6, 500:900] = False
    assert (buf[keep] == 5.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows_per_vec", [5, 6, 1 << 31, 1 << 32, (1 << 63) - 1])
def test_norm_one_vector_for_any_number_of_rows(gpu, rows_per_vec):
    x, gate = rand((5, 64), 1, torch.bfloat16).cuda(), rand((1, 64), 2, torch.bfloat16).cuda()
    want = B.convrot_residual_norm(x, x, gate=gate)
    r, h = torch.empty_like(x), torch.empty_like(x)
    args = norm_args(x_dev=x.data_ptr(), y_dev=x.data_ptr(), gate_dev=gate.data_ptr(), gate_stride=64, r_dev=r.data_ptr(),
                     h_dev=h.data_ptr(), rows=5, rows_per_vec=rows_per_vec)
    assert B.load().convrot_residual_norm(args, torch.cuda.current_stream().cuda_stream) == B.CONVROT_OK
    assert torch.equal(r, want[0]) and torch.equal(h, want[1])


def packed(layout, defaults, kw):
    """The bytes of an argument struct: `defaults` in the order of its fields, some replaced."""
    assert set(kw) <= set(defaults)
    return layout.pack(*[v or 0 for v in {**defaults, **kw}.values()])


def norm_args(**kw):
    return packed(B.NORM_ARGS, dict(
        x_dev=P, y_dev=P + (1 << 24), gate_dev=0, scale_dev=0, shift_dev=0, weight_dev=0, post_weight_dev=0,
        r_dev=P + (2 << 24), h_dev=P + (3 << 24), rows=4, width=64, x_stride=64, y_stride=64, r_stride=64, h_stride=64,
        gate_stride=0, scale_stride=0, shift_stride=0, rows_per_vec=1, residual_scale=1.0, eps=1e-6,
        dtype=B.CONVROT_BF16, vec_dtype=B.CONVROT_BF16, norm=B.CONVROT_NORM_LAYER, post_norm=B.CONVROT_NORM_NONE), kw)


P = 1 << 30


@pytest.mark.parametrize("kw,ok", [
    ({}, True), ({"rows": 0, "x_dev": None}, True), ({"rows": -1}, False), ({"rows": (1 << 24) + 1}, False),
    ({"width": 0}, False), ({"width": 16385}, False), ({"width": 16384, "x_stride": 16384, "y_stride": 16384,
                                                        "r_stride": 16384, "h_stride": 16384}, True),
    ({"x_dev": None}, False), ({"x_dev": P + 1}, False), ({"dtype": 0}, False), ({"dtype": 4}, False),
    ({"vec_dtype": B.CONVROT_F32}, True), ({"vec_dtype": B.CONVROT_F16}, False), ({"norm": 3}, False),
    ({"norm": 0}, True), ({"post_norm": 2}, True), ({"post_norm": -1}, False), ({"eps": -1e-6}, False),
    ({"eps": float("nan")}, False), ({"rows_per_vec": 0}, False), ({"y_dev": None}, True),
    ({"y_dev": None, "gate_dev": P}, False), ({"y_dev": None, "post_norm": 1}, False),
    ({"post_weight_dev": P}, False), ({"post_weight_dev": P, "post_norm": 1}, True),
    ({"r_dev": None}, True), ({"h_dev": None}, True), ({"r_dev": None, "h_dev": None}, False),
    ({"h_dev": None, "scale_dev": P}, False), ({"h_dev": None, "weight_dev": P}, False), ({"scale_dev": P + 1}, False),
    ({"x_stride": -64}, False), ({"x_stride": 0}, True), ({"r_stride": 0}, False), ({"r_stride": 63}, False),
    ({"r_dev": P}, True), ({"h_dev": P}, True), ({"r_dev": P, "h_dev": P}, False), ({"r_dev": P, "r_stride": 65}, False),
    ({"r_dev": P + 64}, False), ({"r_dev": P + 128, "x_stride": 128, "r_stride": 128}, True),
    ({"r_dev": P + 126, "x_stride": 128, "r_stride": 128}, False), ({"r_dev": P + 4 * 128}, True),
    ({"h_dev": P + (2 << 24) + 128}, False),
    # vectors under an output: the second of two vectors, a weight
    ({"gate_dev": P + (2 << 24) - 128, "gate_stride": 64, "rows_per_vec": 4}, True),
    ({"gate_dev": P + (2 << 24) - 128, "gate_stride": 64, "rows_per_vec": 2}, False),
    ({"weight_dev": P + (3 << 24) + 256}, False), ({"weight_dev": P + (3 << 24) + 512}, True),
])
def test_norm_refusals(kw, ok):
    rc = B.load().convrot_validate_residual_norm(norm_args(**kw))
    assert rc == (B.CONVROT_OK if ok else B.CONVROT_EINVAL)
    if not ok:
        assert B.load().convrot_residual_norm(norm_args(**kw), None) == B.CONVROT_EINVAL


@pytest.mark.parametrize("name", ["x_stride", "y_stride", "r_stride", "h_stride", "gate_stride", "scale_stride", "shift_stride"])
@pytest.mark.parametrize("rows,stride,ok", [(2, 1 << 40, True), (2, (1 << 40) + 1, False), (1 << 16, 1 << 40, True),
                                            ((1 << 16) + 2, 1 << 40, False), (1 << 24, 1 << 40, False)])
def test_norm_strides_that_reach_too_far(name, rows, stride, ok):
    places = {"x_dev": 1, "y_dev": 2, "r_dev": 3, "h_dev": 4, "gate_dev": 5, "scale_dev": 5, "shift_dev": 5}
    far = {key: i << 59 for key, i in places.items()}   # further from one another than any of them reaches
    rc = B.load().convrot_validate_residual_norm(norm_args(**far, rows=rows, **{name: stride}))
    assert rc == (B.CONVROT_OK if ok else B.CONVROT_EINVAL)


# ---- rotary positions ----------------------------------------------------------


def rope_reference(x, pos, freq, axis, layout, weight, norm, eps):
    """The rotated heads and their error bound before the storage rounding."""
    x = x.double()
    p = len(freq)
    angle = pos.double()[..., torch.from_numpy(axis).long()] * torch.from_numpy(freq)
    cos, sin = angle.cos().unsqueeze(2), angle.sin().unsqueeze(2)
    e = torch.zeros_like(x)
    if norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        x = x if weight is None else x * weight.double()
        e = x.abs() * 24 * U    # at most 8 squares a lane, 6 steps, and the roundings of root and products
    # binary64 product and reduction, the fraction rounded to binary32 (times 2 pi), then sine and cosine
    ea = (6 * U + angle.abs() * 2.0 ** -50).unsqueeze(2)
    y, ey = x.clone(), e.clone()
    u, v = (slice(0, 2 * p, 2), slice(1, 2 * p, 2)) if layout == "interleaved" else (slice(0, p), slice(p, 2 * p))
    size = x[..., u].abs() + x[..., v].abs()
    y[..., u] = x[..., u] * cos - x[..., v] * sin
    y[..., v] = x[..., u] * sin + x[..., v] * cos
    ey[..., u] = ey[..., v] = e[..., u] + e[..., v] + size * (ea + 3 * U)
    return y, ey


def check_rope(batch, tokens, hq, hk, dim, sizes, layout="interleaved", dtype="bf16", norm=False, weighted=True,
               shared=False, far=False, shared_positions=False, packed=False, head_major=False, in_place=False, seed=0):
    dt = TYPES[dtype]
    freq, axis = B.rope_frequencies(sizes, shared=shared)
    rows = 1 if shared_positions else batch
    g = torch.Generator().manual_seed(seed)
    if far:
        pos = torch.randint(-(1 << 20), 1 << 20, (rows, tokens, len(sizes)), generator=g).to(torch.int32)
    else:
        pos = torch.rand((rows, tokens, len(sizes)), generator=g) * 300 - 20
    if packed:
        qkv = rand((batch, tokens, (hq + 2 * hk) * dim), seed, dt)
        cut = lambda t: (t[..., :hq * dim].unflatten(-1, (hq, dim)), t[..., hq * dim:(hq + hk) * dim].unflatten(-1, (hk, dim)))  # noqa: E731
        (q, k), (cq, ck) = cut(qkv), cut(qkv.cuda())
    else:
        q, k = rand((batch, tokens, hq, dim), seed, dt), rand((batch, tokens, hk, dim), seed + 1, dt)
        cq, ck = dev(q), dev(k)
    weights = [rand((dim,), seed + 2 + i, dt, 0.1, 1.0) if norm and weighted else None for i in (0, 1)]
    outs = {}
    if head_major:
        outs = {"q_out": torch.empty((batch, hq, tokens, dim), dtype=dt, device="cuda").transpose(1, 2),
                "k_out": torch.empty((batch, hk, tokens, dim), dtype=dt, device="cuda").transpose(1, 2)}
    if in_place:
        outs = {"q_out": cq, "k_out": ck}
    yq, yk = B.convrot_rope(cq, ck, pos.cuda(), freq, axis, layout=layout, qk_norm=norm, q_weight=dev(weights[0]),
                            k_weight=dev(weights[1]), **outs)
    for got, x, w, what in ((yq, q, weights[0], "q"), (yk, k, weights[1], "k")):
        want, e = rope_reference(x, pos, freq, axis, layout, w, norm, 1e-6)
        close(got, want, e + half_step(dt, want.abs() + e), what)
    return yq, yk


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,sizes", [(128, (16, 56, 56)), (64, (64,)), (32, (8, 24)), (256, (64, 96, 96)), (72, (24, 24, 24)),
                                       (80, (32, 32)), (96, (32, 32, 32)), (2, (2,)), (6, (2, 2)), (65, (16, 14)),
                                       (255, (254,)), (128, (34,))])
def test_rope_heads(gpu, dim, sizes, dtype, layout):
    for i, norm in enumerate((False, True)):
        check_rope(2, 5, 3, 1, dim, sizes, layout, dtype, norm, far=bool(i), seed=dim + i)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 5, 17, 131])
@pytest.mark.parametrize("hq,hk", [(1, 1), (32, 8), (5, 5)])
def test_rope_tokens_and_head_counts(gpu, tokens, hq, hk):
    check_rope(2, tokens, hq, hk, 128, (44, 42, 42), norm=True, packed=True, seed=tokens)
    check_rope(1, tokens, hq, hk, 64, (16, 24, 24), "halves", shared=True, far=True, seed=tokens)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("dim,sizes", [(128, (16, 56, 56)), (72, (24, 24)), (50, (16, 20))])
def test_rope_strides_and_in_place(gpu, dim, sizes, layout):
    for kw in ({"packed": True}, {"packed": True, "head_major": True}, {"packed": True, "in_place": True},
               {"in_place": True, "shared_positions": True}, {"head_major": True, "weighted": False}):
        check_rope(3, 11, 6, 2, dim, sizes, layout, norm=True, seed=dim, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("tokens,hq,hk,dim,sizes,dtype", [
    (1101, 9, 3, 72, (22, 22, 20), "f16"), (1101, 9, 3, 72, (22, 22, 22), "f16"), (1100, 16, 5, 64, (64,), "bf16"),
    (2801, 13, 11, 72, (24, 24), "bf16"), (2801, 13, 11, 72, (26, 24), "f16"), (2100, 20, 20, 128, (44, 42, 42), "bf16"),
    (1701, 7, 3, 256, (256,), "f32"), (2801, 3, 3, 100, (50, 50), "f32")])
def test_rope_many_tokens(gpu, tokens, hq, hk, dim, sizes, dtype, layout):
    """A wave takes four or eight items, the last of them partly or of the other tensor."""
    check_rope(1, tokens, hq, hk, dim, sizes, layout, dtype, norm=True, packed=True, in_place=True, seed=tokens + dim)
    check_rope(2, (tokens + 1) // 2, hq, hk, dim, sizes, layout, dtype, head_major=True, seed=tokens + dim)


@pytest.mark.gpu
def test_rope_one_tensor_and_identity(gpu):
    freq, axis = B.rope_frequencies((32, 32))
    q = rand((1, 9, 4, 64), 1, torch.bfloat16).cuda()
    pos = torch.zeros((1, 9, 2), dtype=torch.int32, device="cuda")
    y, none = B.convrot_rope(q, None, pos, freq, axis)
    assert none is None and torch.equal(y, q)         # positions of zero turn nothing
    empty, _ = B.convrot_rope(q[:, :0], None, pos[:, :0], freq, axis)
    assert empty.shape == (1, 0, 4, 64)


@pytest.mark.gpu
def test_rope_negated_positions_turn_back(gpu):
    freq, axis = B.rope_frequencies((16, 24, 24))
    q = rand((2, 9, 4, 64), 1).cuda()
    pos = torch.randint(0, 1 << 18, (2, 9, 3), generator=torch.Generator().manual_seed(0), dtype=torch.int32).cuda()
    there, _ = B.convrot_rope(q, None, pos, freq, axis)
    back, _ = B.convrot_rope(there, None, -pos, freq, axis)
    # two turns of at most 9 u of |u| + |v| <= 2 max|q| each (rounding to storage included)
    assert (back - q).abs().max() <= 2 * 10 * U * 2 * q.abs().max()


@pytest.mark.gpu
def test_rope_nan_positions_stay_in_their_token(gpu):
    freq, axis = B.rope_frequencies((32, 32))
    q = rand((1, 4, 2, 64), 1, torch.bfloat16).cuda()
    pos = torch.ones((1, 4, 2), device="cuda")
    y0, _ = B.convrot_rope(q, None, pos, freq, axis)
    pos[0, 2, 1] = float("inf")
    y, _ = B.convrot_rope(q, None, pos, freq, axis)
    assert torch.isnan(y[0, 2, :, 32:]).all() and torch.equal(y[0, 2, :, :32], y0[0, 2, :, :32])
    assert torch.equal(y[0, [0, 1, 3]], y0[0, [0, 1, 3]])


def test_rope_frequencies():
    freq, axis = B.rope_frequencies((4, 6), theta=100.0)
    assert np.allclose(freq, [1, 0.1, 1, 100 ** (-1 / 3), 100 ** (-2 / 3)], rtol=1e-15) and axis.tolist() == [0, 0, 1, 1, 1]
    freq, axis = B.rope_frequencies((4, 4), theta=16.0, shared=True)
    assert np.allclose(freq, [1, 0.5, 0.25, 0.125], rtol=1e-15) and axis.tolist() == [0, 0, 1, 1]
    for bad in ((), (3,), (0, 2), (-2,)):
        with pytest.raises(ValueError):
            B.rope_frequencies(bad)


FREQ, AXIS = np.ones(32), np.zeros(32, np.int32)


def rope_args(q=None, k=None, **kw):
    FREQ[5], AXIS[5] = kw.pop("freq", 1.0), kw.pop("axis", 0)
    fields = {}
    for i, extra in ((0, q), (1, k)):
        heads = dict(in_dev=P + (4 * i + 1 << 20), out_dev=P + (4 * i + 2 << 20), weight_dev=P, heads=4,
                     in_batch_stride=768, in_token_stride=256, in_head_stride=64, out_batch_stride=768,
                     out_token_stride=256, out_head_stride=64)
        assert set(extra or {}) <= set(heads)
        fields |= {f"{key}{i}": v for key, v in {**heads, **(extra or {})}.items()}
    return packed(B.ROPE_ARGS, {**fields, **dict(
        count=2, batch=2, tokens=3, head_dim=64, pos_dev=P, pos_batch_stride=9, pos_token_stride=3,
        pos_dtype=B.CONVROT_F32, axes=3, pairs=32, freq_host=FREQ.ctypes.data, axis_host=AXIS.ctypes.data, layout=1,
        norm=B.CONVROT_NORM_RMS, dtype=B.CONVROT_BF16, eps=1e-6)}, kw)


Q, QO, K_ = P + (1 << 20), P + (2 << 20), P + (5 << 20)


@pytest.mark.parametrize("kw,ok", [
    ({}, True), ({"count": 0}, False), ({"count": 3}, False), ({"batch": -1}, False), ({"batch": 65536}, False),
    ({"tokens": 0, "pos_dev": None}, True), ({"tokens": (1 << 24) + 1}, False), ({"head_dim": 257}, False),
    ({"head_dim": 63}, False), ({"pairs": 0}, False), ({"pairs": 33}, False), ({"axes": 0}, False), ({"axes": 9}, False),
    ({"axis": 3}, False), ({"axis": -1}, False), ({"axis": 2}, True), ({"freq": float("inf")}, False),
    ({"freq": float("nan")}, False), ({"freq": -2.0}, True), ({"freq_host": None}, False), ({"axis_host": None}, False),
    ({"layout": 0}, False), ({"layout": 2}, True), ({"layout": 3}, False), ({"norm": 1}, False), ({"norm": 0}, False),
    ({"dtype": 4}, False), ({"eps": -1.0}, False), ({"pos_dtype": 1}, False), ({"pos_dtype": 4}, True),
    ({"pos_dev": None}, False), ({"pos_dev": P + 2}, False), ({"pos_token_stride": -1}, False),
    ({"q": {"heads": 0}}, False), ({"q": {"heads": 65536}}, False), ({"q": {"in_dev": None}}, False),
    ({"k": {"out_dev": None}}, False), ({"count": 1, "k": {"out_dev": None}}, True), ({"q": {"in_dev": Q + 1}}, False),
    ({"q": {"weight_dev": None}, "k": {"weight_dev": None}, "norm": 0}, True), ({"q": {"weight_dev": P + 1}}, False),
    ({"q": {"in_head_stride": 0}}, True), ({"q": {"out_head_stride": 0}}, False), ({"q": {"out_head_stride": 63}}, False),
    ({"q": {"out_dev": Q}}, True), ({"q": {"out_dev": Q, "out_head_stride": 192, "out_token_stride": 64}}, False),
    ({"q": {"out_dev": Q + 128}}, False), ({"q": {"out_dev": K_}}, False),
    ({"q": {"out_dev": QO}, "k": {"out_dev": QO}}, False),
    ({"pos_dev": QO + 1024}, False), ({"pos_dev": QO + 3072}, True), ({"k": {"weight_dev": QO + 3070}}, False),
    # heads first: [batch][heads][tokens][head_dim]
    ({"q": {"out_token_stride": 64, "out_head_stride": 192}}, True),
    # both outputs side by side in one packed buffer
    ({"q": {"out_dev": QO, "out_token_stride": 512, "out_batch_stride": 1536},
      "k": {"out_dev": QO + 512, "out_token_stride": 512, "out_batch_stride": 1536}}, True),
    ({"q": {"out_dev": QO, "out_token_stride": 512, "out_batch_stride": 1536},
      "k": {"out_dev": QO + 510, "out_token_stride": 512, "out_batch_stride": 1536}}, False),
])
def test_rope_refusals(kw, ok):
    a = rope_args(**dict(kw))
    rc = B.load().convrot_validate_rope(a)
    assert rc == (B.CONVROT_OK if ok else B.CONVROT_EINVAL)
    if not ok:
        assert B.load().convrot_rope(a, None) == B.CONVROT_EINVAL


@pytest.mark.parametrize("sizes,strides,ok", [
    ({"tokens": (1 << 16) + 1}, {"token_stride": 1 << 40}, True), ({"tokens": (1 << 16) + 2}, {"token_stride": 1 << 40}, False),
    ({"tokens": 1 << 24}, {"token_stride": 1 << 40}, False), ({"batch": 65535}, {"batch_stride": 1 << 40}, True),
    ({"heads": 65535}, {"head_stride": 1 << 40}, True), ({"heads": 4}, {"head_stride": (1 << 40) + 1}, False)])
@pytest.mark.parametrize("side", ["in", "out", "pos"])
def test_rope_strides_that_reach_too_far(side, sizes, strides, ok):
    if side == "pos" and "heads" in sizes:
        return
    strides = {f"{side}_{key}": v for key, v in strides.items()}
    n, tokens = sizes.get("heads", 4), sizes.get("tokens", 3)
    heads = dict(in_dev=1 << 60, out_dev=2 << 60, heads=n)
    for end in ("in", "out"):   # dense, but for the stride in question
        heads |= {f"{end}_head_stride": 64, f"{end}_token_stride": 64 * n, f"{end}_batch_stride": 64 * n * tokens}
    heads |= {key: v for key, v in strides.items() if side != "pos"}
    rest = {key: v for key, v in strides.items() if side == "pos"}
    a = rope_args(q=heads, count=1, pos_dev=3 << 60, tokens=tokens, batch=sizes.get("batch", 1), **rest)
    assert B.load().convrot_validate_rope(a) == (B.CONVROT_OK if ok else B.CONVROT_EINVAL)


# ---- group-scaled 4-bit weights --------------------------------------------------


def codes_of(codes, zeros, group):
    """(code - zero) as binary64 [N, K] from packed codes."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(1).double()
    if zeros is None:
        return torch.where(c >= 8, c - 16, c)
    return c - zeros.double().repeat_interleave(group, 1)


def check_grouped(m, n, k, group, zeros=False, bias=True, dtype="bf16", seed=0, exact=False):
    """exact: integer inputs and power-of-two scales, so that every sum is an
    integer below 2^24 times one scale and the result is the rounded true value."""
    dt = TYPES[dtype]
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    z = torch.randint(0, 16, (n, k // group), generator=g, dtype=torch.uint8) if zeros else None
    if exact:
        x = torch.randint(-4, 5, (m, k), generator=g).to(dt)
        scales = torch.full((n, k // group), 2.0 ** -7, dtype=dt)
        b = torch.randint(-9, 10, (n,), generator=g).to(dt) if bias else None
    else:
        x = rand((m, k), seed, dt)
        scales = ((torch.rand((n, k // group), generator=g) + 0.5) * 0.01).to(dt)
        b = rand((n,), seed + 1, dt, 0.1) if bias else None
    y = B.convrot_linear_grouped(dev(x), dev(codes), dev(scales), dev(z), dev(b), group)
    s = scales.double().repeat_interleave(group, 1)
    q = codes_of(codes, z, group)
    want = x.double() @ (q * s).t() + (0 if b is None else b.double())
    if exact:
        assert torch.equal(y.cpu(), want.to(dt))
        return y
    # products are exact; a group's two sums take at most 128 additions of one
    # rounding or truncation (2 u) each on 15 |x| and z |x|, the K / group <= 512
    # group terms and the parts of the waves add as many again of the total
    size = x.double().abs() @ s.t()
    e = (128 * 2 * 30 * U) * size + (k // group + 20) * U * 15 * size
    close(y, want, e + half_step(dt, want.abs() + e), "y")
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_grouped_exact_sums(gpu, dtype, group, zeros):
    for m, n, k in ((1, 16, group), (1, 1, 3 * group), (2, 17, 1024), (4, 100, 4096 + group), (16, 33, 2048 - group),
                    (17, 64, 640), (31, 5, 1152), (32, 48, 8192)):
        check_grouped(m, n, k, group, zeros, bias=n != 17, dtype=dtype, seed=m * n, exact=True)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 2, 3, 7, 15, 16, 17, 24, 32])
def test_grouped_rows(gpu, m):
    for group, zeros in ((32, True), (64, False), (128, True)):
        check_grouped(m, 131, 1920, group, zeros, dtype="f16" if group == 64 else "bf16", seed=m)


@pytest.mark.gpu
@pytest.mark.parametrize("n,k,group", [(1, 32, 32), (15, 96, 32), (4096, 256, 64), (7, 16384, 128), (3, 65536, 128),
                                       (2, 65504, 32), (20001, 192, 64), (1000, 4128, 32)])
def test_grouped_sizes(gpu, n, k, group):
    check_grouped(1, n, k, group, seed=n)
    check_grouped(19, n, k, group, zeros=True, dtype="f16", bias=False, seed=k)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 4, 5, 8, 12, 27])
@pytest.mark.parametrize("n", [300, 5000, 9001, 16000, 16500])
def test_grouped_tiles(gpu, m, n):
    """Every count of output tiles a workgroup, with one round of workgroups and two."""
    check_grouped(m, n, 1280, 32, zeros=True, dtype="f16", seed=n)
    check_grouped(m, n, 1152, 64, seed=n)
    check_grouped(m, n, 1408, 128, zeros=n % 2 == 1, bias=False, seed=n)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_grouped_every_code(gpu, dtype):
    """One output row for every code in all its channels, and for every zero point."""
    k, group = 128, 32
    codes = (torch.arange(16, dtype=torch.uint8) * 17).view(16, 1).expand(16, k // 2).contiguous()
    x = torch.zeros((1, k), dtype=TYPES[dtype])
    x[0, 5] = 1.0
    s = torch.ones((16, k // group), dtype=TYPES[dtype])
    y = B.convrot_linear_grouped(dev(x), dev(codes), dev(s), None, None, group)
    assert y.cpu().flatten().tolist() == [float(c - 16 * (c >= 8)) for c in range(16)]
    for z in range(16):
        zeros = torch.full((16, k // group), z, dtype=torch.uint8)
        y = B.convrot_linear_grouped(dev(x), dev(codes), dev(s), dev(zeros), None, group)
        assert y.cpu().flatten().tolist() == [float(c - z) for c in range(16)]


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
def test_grouped_every_channel_meets_its_own_code(gpu, group):
    """x a unit vector in each channel in turn (32 at a time): y is that column of W."""
    k, n = 384, 20
    g = torch.Generator().manual_seed(group)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    s = 2.0 ** torch.randint(-3, 3, (n, k // group), generator=g).to(torch.bfloat16)
    w = (codes_of(codes, None, group) * s.double().repeat_interleave(group, 1)).t()
    for k0 in range(0, k, 32):
        x = torch.zeros((32, k), dtype=torch.bfloat16)
        x[torch.arange(32), k0 + torch.arange(32)] = 1.0
        y = B.convrot_linear_grouped(dev(x), dev(codes), dev(s), None, None, group)
        assert torch.equal(y.cpu().double(), w[k0:k0 + 32])


@pytest.mark.gpu
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("k,group", [(32, 32), (96, 32), (160, 32), (192, 32), (224, 32), (544, 32), (1120, 32), (4128, 32),
                                     (4192, 32), (6240, 32), (64, 64), (192, 64), (576, 64), (1088, 64), (4160, 64), (128, 32),
                                     (1152, 64), (4224, 128)])
def test_grouped_rows_that_end_inside_a_block(gpu, k, group, zeros):
    """Whatever the next row holds stays out: every other output's scales are NaN,
    and so is the second row of x.  The rest are integers times powers of two, so
    that every sum (at most 6240 * 15 * 4 * 8 eighths, below 2^24) is exact."""
    n = 37
    g = torch.Generator().manual_seed(k)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    z = torch.randint(0, 16, (n, k // group), generator=g, dtype=torch.uint8) if zeros else None
    s = 2.0 ** torch.randint(-3, 1, (n, k // group), generator=g).to(torch.bfloat16)
    q = codes_of(codes, z, group) * s.double().repeat_interleave(group, 1)
    s[1::2] = float("nan")
    for m in (1, 3, 7, 16, 32):
        x = torch.randint(-4, 5, (m, k), generator=g).to(torch.bfloat16)
        want = (x.double() @ q.t()).to(torch.bfloat16)
        if m > 1:
            x[1] = float("nan")
        y = B.convrot_linear_grouped(dev(x), dev(codes), dev(s), dev(z), None, group).cpu()
        assert y[:, 1::2].isnan().all()
        good = torch.arange(m) != 1
        assert torch.equal(y[good][:, ::2], want[good][:, ::2]), m
        if m > 1:
            assert y[1].isnan().all()


@pytest.mark.gpu
def test_grouped_infinite_rows_stay_alone(gpu):
    x = rand((3, 256), 1, torch.bfloat16).cuda()
    codes = torch.randint(0, 256, (40, 128), generator=torch.Generator().manual_seed(1), dtype=torch.uint8).cuda()
    s = torch.full((40, 4), 0.01, dtype=torch.bfloat16, device="cuda")
    y0 = B.convrot_linear_grouped(x, codes, s, None, None, 64)
    x[1, 3] = float("inf")
    y = B.convrot_linear_grouped(x, codes, s, None, None, 64)
    assert torch.isnan(y[1]).all() and torch.equal(y[[0, 2]], y0[[0, 2]])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("asymmetric", [False, True])
def test_quantize_grouped_matches_its_definition(gpu, dtype, group, asymmetric):
    dt = TYPES[dtype]
    n, k = 37, 5 * 128
    w = rand((n, k), group, dt, 0.02, 0.01)
    w[3, :group] = 0
    w[4, :group] = 0.5      # one sign only
    w[5, 1] = float("nan")
    w[6, k - 1] = float("inf")
    codes, scales, zeros = B.convrot_quantize_weight_grouped(w.cuda(), group, asymmetric)
    v = w.float().view(n, k // group, group)
    bad = ~torch.isfinite(v).all(-1)
    if asymmetric:
        lo, hi = v.amin(-1).clamp(max=0), v.amax(-1).clamp(min=0)
        s = ((hi - lo) / 15).to(dt)
        z = torch.round(-lo / s.float()).nan_to_num(0).clamp(0, 15)
        c = (torch.round(v / s.float().unsqueeze(-1)).nan_to_num(0) + z.unsqueeze(-1)).clamp(0, 15)
    else:
        s = (v.abs().amax(-1) / 7).to(dt)
        z = torch.zeros_like(s, dtype=torch.float32)
        c = torch.round(v / s.float().unsqueeze(-1)).nan_to_num(0).clamp(-7, 7)
    s[bad], z[bad], c[bad] = float("nan"), 0, 0
    got = codes_of(codes.cpu(), torch.zeros((n, k // group), dtype=torch.uint8) if asymmetric else None, group)
    assert torch.equal(got, c.view(n, k).double())
    assert torch.equal(scales.cpu().nan_to_num(-1), s.nan_to_num(-1)) and torch.equal(scales.cpu().isnan(), bad)
    assert zeros is None if not asymmetric else torch.equal(zeros.cpu().float(), z)


@pytest.mark.parametrize("kw,ok", [
    ({}, True), ({"M": 0, "x_dev": None}, True), ({"M": 33}, False), ({"M": -1}, False), ({"N": 0}, True),
    ({"N": (1 << 24) + 1}, False), ({"K": 0}, False), ({"K": 96}, False), ({"K": 65536}, True), ({"K": 65600}, False),
    ({"group": 16}, False), ({"group": 256}, False), ({"group": 128}, True), ({"dtype": 3}, False), ({"dtype": 2}, True),
    ({"x_dev": None}, False), ({"codes_dev": None}, False), ({"scales_dev": None}, False), ({"y_dev": None}, False),
    ({"x_dev": P + 8}, False), ({"codes_dev": P + 8}, False), ({"scales_dev": P + 1}, False), ({"bias_dev": P + 1}, False),
    ({"zeros_dev": P + 1 - (1 << 20)}, True), ({"zeros_dev": P + (9 << 20)}, False), ({"bias_dev": P + (9 << 20) + 382}, False),
    ({"bias_dev": P + (9 << 20) + 384}, True), ({"codes_dev": P + (9 << 20) - 16 * 383}, False), ({"y_dev": P + (9 << 20) + 1}, False), ({"y_dev": P + 256}, False),
])
def test_grouped_refusals(kw, ok):
    a = packed(B.GROUPED_ARGS, dict(x_dev=P, codes_dev=P + (1 << 22), scales_dev=P + (1 << 23), zeros_dev=0, bias_dev=0,
                                    y_dev=P + (9 << 20), M=4, N=48, K=256, group=64, dtype=B.CONVROT_BF16), kw)
    rc = B.load().convrot_validate_linear_grouped(a)
    assert rc == (B.CONVROT_OK if ok else B.CONVROT_EINVAL)
    if not ok:
        assert B.load().convrot_linear_grouped(a, None) == B.CONVROT_EINVAL


def test_quantize_grouped_refusals():
    f = B.load().convrot_quantize_weight_grouped
    good = [P, 4, 256, 64, 1, P + (1 << 20), P + (2 << 20), None, None]
    for i, v in ((0, None), (0, P + 1), (1, -1), (1, (1 << 24) + 1), (2, 32), (2, 65600), (2, 100), (3, 48), (4, 3),
                 (5, None), (6, None), (6, P + 1)):
        args = list(good)
        args[i] = v
        assert f(*args) == B.CONVROT_EINVAL, (i, v)
    assert f(*([None, 0] + good[2:])) == B.CONVROT_OK


@pytest.mark.parametrize("codes,scales,zeros,ok", [
    (2048, 2560, 2592, True), (2047, 4096, None, False), (4096, 2046, None, False), (4096, 8192, 2047, False),
    (4096, 4096 + 510, None, False), (4096, 4096 + 512, 4096 + 512 + 31, False), (4096, 4096 - 32, None, True),
    (4096, 4096 - 30, None, False), (4096, 8192, 4096, False)])
def test_quantize_grouped_refuses_overlaps(codes, scales, zeros, ok):
    # W: 4 x 256 bf16, 2048 bytes; codes 512, scales 32, zeros 16
    args = (P, 4, 256, 64, 1, P + codes, P + scales, zeros and P + zeros)
    rc = B.load().convrot_validate_quantize_weight_grouped(*args)
    assert rc == (B.CONVROT_OK if ok else B.CONVROT_EINVAL)
    if not ok:
        assert B.load().convrot_quantize_weight_grouped(*args, None) == B.CONVROT_EINVAL


def test_host_tensors_are_refused():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        B.convrot_residual_norm(x)
    with pytest.raises(ValueError, match="device tensor"):
        B.convrot_rope(x.view(1, 2, 1, 64), None, x, [1.0], [0])
    with pytest.raises(ValueError, match="device tensor"):
        B.convrot_linear_grouped(x, x, x, None, None, 32)
    with pytest.raises(ValueError, match="device tensor"):
        B.convrot_quantize_weight_grouped(x, 32)
    with pytest.raises(TypeError):
        B.convrot_residual_norm([1.0])


@pytest.mark.gpu
def test_binding_refusals(gpu):
    x = rand((2, 6, 64), 1, torch.bfloat16).cuda()
    v = rand((64,), 2, torch.bfloat16).cuda()
    ok = dict(gate=v, y=x.clone())
    B.convrot_residual_norm(x, **ok)
    for err, kw in ((ValueError, dict(y=x[:, :5])), (ValueError, dict(y=x.float())), (ValueError, dict(y=x.cpu())),
                    (ValueError, dict(norm="batch")), (ValueError, dict(scale=v[:32])), (TypeError, dict(scale=v.half())),
                    (TypeError, dict(scale=v, shift=v.float())), (ValueError, dict(scale=v.expand(6, 64))),
                    (ValueError, dict(scale=v.expand(3, 64))), (ValueError, dict(weight=v.expand(2, 64))),
                    (ValueError, dict(scale=v.expand(2, 64), shift=v.expand(2, 6, 64))), (ValueError, dict(r=x.float())),
                    (ValueError, dict(h=x.transpose(0, 1))), (B.ConvRotError, dict(gate=v)), (B.ConvRotError, dict(r=x, h=x)),
                    (B.ConvRotError, dict(want_r=False, want_h=False)), (TypeError, dict(scale=1.0)),
                    (RuntimeError, dict(y=x.clone().requires_grad_()))):
        with pytest.raises(err):
            B.convrot_residual_norm(x, **kw)
    with torch.no_grad():
        B.convrot_residual_norm(x.clone().requires_grad_())
    with pytest.raises(ValueError):
        B.convrot_residual_norm(x.transpose(1, 2))
    with pytest.raises(TypeError):
        B.convrot_residual_norm(x.to(torch.int32))

    q, pos = x.view(2, 6, 1, 64), torch.zeros((2, 6, 1), device="cuda")
    freq, axis = B.rope_frequencies((64,))
    B.convrot_rope(q, q, pos, freq, axis)
    for err, args in ((ValueError, (x, None, pos, freq, axis)), (ValueError, (q, q[:1], pos, freq, axis)),
                      (TypeError, (q, q.float(), pos, freq, axis)), (ValueError, (q, None, pos[:, :5], freq, axis)),
                      (TypeError, (q, None, pos.double(), freq, axis)), (ValueError, (q, None, pos, freq[:5], axis)),
                      (B.ConvRotError, (q, None, pos, freq, axis + 1)), (ValueError, (q.transpose(1, 3), None, pos, freq, axis))):
        with pytest.raises(err):
            B.convrot_rope(*args)
    for err, kw in ((ValueError, dict(layout="pairs")), (B.ConvRotError, dict(q_weight=v)), (ValueError, dict(k_weight=v)),
                    (ValueError, dict(qk_norm=True, q_weight=v[:32])), (ValueError, dict(q_out=q.float()))):
        with pytest.raises(err):
            B.convrot_rope(q, None, pos, freq, axis, **kw)

    w = rand((24, 128), 3, torch.bfloat16).cuda()
    codes, scales, _ = B.convrot_quantize_weight_grouped(w, 32)
    xs = rand((2, 128), 4, torch.bfloat16).cuda()
    B.convrot_linear_grouped(xs, codes, scales, None, None, 32)
    for err, args in ((ValueError, (xs, codes, scales, None, None, 64)), (ValueError, (xs, codes, scales.half(), None, None, 32)),
                      (ValueError, (xs.half(), codes, scales, None, None, 32)), (TypeError, (xs.float(), codes, scales, None, None, 32)),
                      (ValueError, (xs.t(), codes, scales, None, None, 32)), (ValueError, (xs, codes, scales, None, v, 32)),
                      (B.ConvRotError, (rand((33, 128), 1, torch.bfloat16).cuda(), codes, scales, None, None, 32)),
                      (ValueError, (xs, codes.t(), scales, None, None, 32)), (ValueError, (xs, codes, scales, None, None, 7))):
        with pytest.raises(err):
            B.convrot_linear_grouped(*args)
    with pytest.raises(ValueError):
        B.convrot_quantize_weight_grouped(w, 48)
    with pytest.raises(TypeError):
        B.convrot_quantize_weight_grouped(w.float(), 32)
    y = B.convrot_linear_grouped(xs[:0], codes, scales, None, None, 32)
    assert y.shape == (0, 24)


# ---- streams and graphs ------------------------------------------------------------


@pytest.mark.gpu
def test_offsets_past_32_bits(gpu):
    far = (1 << 30) + 64   # elements from row to row: the third begins beyond 2^32 bytes
    buf = torch.empty(2 * far + 1024, dtype=torch.bfloat16, device="cuda")

    def spread(t):
        v = buf.as_strided(t.shape, (far, *t.stride()[1:]))
        v.copy_(t)
        return v

    x = rand((3, 64), 1, torch.bfloat16).cuda()
    want = B.convrot_residual_norm(x, x)
    got = B.convrot_residual_norm(spread(x), x, r=spread(x))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    q = rand((3, 1, 2, 64), 2, torch.bfloat16).cuda()
    pos = torch.arange(3, dtype=torch.int32, device="cuda").view(3, 1, 1)
    freq, axis = B.rope_frequencies((64,))
    want = B.convrot_rope(q, None, pos, freq, axis)[0]
    places = spread(q)
    assert torch.equal(B.convrot_rope(places, None, pos, freq, axis, q_out=places)[0], want)
    flip = lambda v: v.transpose(0, 1)   # noqa: E731  tokens as the far dimension
    places = spread(q)
    assert torch.equal(flip(B.convrot_rope(flip(places), None, flip(pos), freq, axis, q_out=flip(places))[0]), want)
    del buf, places, got
    n, k, last = (1 << 17) + 5, 65536, 5   # codes of more than 2^32 bytes
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((n, k // 128), 2.0 ** -7, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(3)
    own = torch.randint(0, 256, (last, k // 2), generator=g, dtype=torch.uint8)
    codes[-last:] = own.cuda()
    for m in (1, 17):
        x = torch.randint(-1, 2, (m, k), generator=g).to(torch.bfloat16)   # sums below 2^24
        y = B.convrot_linear_grouped(x.cuda(), codes, scales, None, None, 128)
        want = x.double() @ codes_of(own, None, 128).t() * 2.0 ** -7
        assert torch.equal(y[:, -last:].cpu(), want.to(torch.bfloat16))


def block_calls():
    """One call of each operator, in the order a block makes them, on fixed inputs."""
    vec = rand((2, 256), 1, torch.bfloat16).cuda()
    w = rand((3 * 256, 256), 2, torch.bfloat16, 0.05).cuda()
    codes, scales, zeros = B.convrot_quantize_weight_grouped(w, 64, asymmetric=True)
    x, y = (rand((2, 40, 256), s, torch.bfloat16).cuda() for s in (3, 4))
    pos = torch.arange(40, dtype=torch.int32, device="cuda").view(1, 40, 1).expand(1, 40, 2).contiguous()
    freq, axis = B.rope_frequencies((32, 32))

    def run(stream=None):
        gate, scale, shift = B.convrot_linear_grouped(vec, codes, scales, zeros, None, 64, stream=stream).chunk(3, -1)
        r, h = B.convrot_residual_norm(x, y, gate=gate, scale=scale, shift=shift, stream=stream)
        q, k = B.convrot_rope(h.view(2, 40, 4, 64), r.view(2, 40, 4, 64), pos, freq, axis, stream=stream)
        return gate, r, h, q, k

    return run, (x, y, vec)


@pytest.mark.gpu
def test_another_stream_gives_the_same(gpu):
    run, _ = block_calls()
    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    with torch.cuda.stream(side):
        again = run()
    torch.cuda.current_stream().wait_stream(side)
    for a, b, c in zip(want, got, again):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.gpu
def test_graph_replays_match_eager_calls(gpu):
    run, inputs = block_calls()
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for step in range(4):
        for i, t in enumerate(inputs):
            t.copy_(rand(t.shape, 100 * step + i, torch.bfloat16))
        want = [t.clone() for t in run()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b), step


@pytest.mark.gpu
def test_the_calls_follow_their_formulas_in_a_row(gpu):
    """The modulation linear, the gated residual with the modulated norm and the
    rotation, each checked on what the one before it returned."""
    run, (x, y, vec) = block_calls()
    gate, r, h, q, k = (t.cpu() for t in run())
    mods = {}
    out = B.convrot_linear_grouped(vec, *B.convrot_quantize_weight_grouped(rand((768, 256), 2, torch.bfloat16, 0.05).cuda(), 64, True),
                                   None, 64).cpu()
    for i, key in enumerate(("gate", "scale", "shift")):
        mods[key] = out[:, 256 * i:256 * (i + 1)].unsqueeze(1)
    assert torch.equal(mods["gate"][:, 0], gate)
    want_r, er, want_h, eh = norm_reference(x.cpu(), y.cpu(), weight=None, post_weight=None, norm="layer", post=None, a=1.0,
                                            eps=1e-6, **mods)
    close(r, want_r, er + half_step(torch.bfloat16, want_r.abs() + er), "r")
    close(h, want_h, eh + half_step(torch.bfloat16, want_h.abs() + eh), "h")
    freq, axis = B.rope_frequencies((32, 32))
    pos = torch.arange(40).view(1, 40, 1).expand(1, 40, 2)
    for got, t in ((q, h), (k, r)):
        want, e = rope_reference(t.view(2, 40, 4, 64), pos, freq, axis, "interleaved", None, False, 1e-6)
        close(got, want, e + half_step(torch.bfloat16, want.abs() + e), "rope")


# ---- modules --------------------------------------------------------------------


def test_conditioned_block_on_cpu():
    """The plain form of the block, which needs no GPU, and its positions."""
    from w4a4_rotated_bit_amd.flux_block import ConditionedBlock, picture, tokens
    blk = ConditionedBlock(128, head_dim=64).to(torch.bfloat16)
    pos = picture(30, 2)
    assert pos.shape == (2, 30, 3) and (pos[:, :10] == 0).all() and pos[0, 10:].unique(dim=0).shape[0] == 20
    assert len(blk.freq) == 32 and blk.axis.max() == 2
    x = tokens(60, 128).view(2, 30, 128)
    y = blk.plain(x, tokens(2, 128), pos)
    assert y.shape == x.shape and y.dtype == torch.bfloat16 and torch.isfinite(y.float()).all()


def test_grouped_linear_refusals():
    from w4a4_rotated_bit_amd.module import GroupedLinear
    codes, scales = torch.zeros((8, 64), dtype=torch.uint8), torch.zeros((8, 2), dtype=torch.bfloat16)
    lin = GroupedLinear(128, 8, codes, scales, None, None, 64)
    assert "group_size=64" in repr(lin)
    with pytest.raises(ValueError):
        GroupedLinear(128, 8, codes, scales, None, None, 128)
    with pytest.raises(ValueError):
        GroupedLinear(128, 8, codes, scales, scales[:4], None, 64)
    with pytest.raises(ValueError):
        GroupedLinear(100, 8, codes, scales, None, None, 64)
    with pytest.raises(ValueError):
        lin(torch.zeros(1, 64))
    with pytest.raises(ValueError):
        lin(torch.zeros(33, 128))
    with pytest.raises(ValueError):
        GroupedLinear.from_linear(torch.nn.Linear(128, 8), 64)


@pytest.mark.gpu
@pytest.mark.parametrize("asymmetric", [False, True])
def test_grouped_linear_is_its_quantized_weight(gpu, asymmetric):
    from w4a4_rotated_bit_amd.module import GroupedLinear
    dense = torch.nn.Linear(256, 96).cuda().to(torch.float16)
    lin = GroupedLinear.from_linear(dense, 64, asymmetric)
    x = rand((2, 3, 256), 1, torch.float16).cuda()
    y = lin(x)
    assert y.shape == (2, 3, 96) and y.dtype == torch.float16
    want = B.convrot_linear_grouped(x.view(6, 256), lin.codes, lin.scales, lin.zeros, lin.bias, 64)
    assert torch.equal(y.view(6, 96), want)
    # half a step of a weight is at most scale / 2, and the scale's own rounding moves it by 2^-11 of 7 (15) scales
    step = lin.scales.float().max().item() * (0.5 + 15 * 2.0 ** -11)
    off = (y.double().cpu() - dense(x).double().cpu()).abs().max()
    assert off <= step * x.double().abs().sum(-1).max().item() + 2.0 ** -10 * y.double().abs().max().item() * 2


@pytest.mark.gpu
@pytest.mark.parametrize("batch,T,hidden", [(1, 48, 256), (3, 33, 384)])
def test_conditioned_block_runs(gpu, batch, T, hidden):
    from w4a4_rotated_bit_amd.flux_block import run_conditioned
    out = run_conditioned(T, hidden, batch, group_size=64, iters=0)
    assert out["finite"]
    # with dense linears the operators and the plain form round at the same six
    # places (both h, q and k, the attended values' inputs, both sums); each may
    # fall to the other side, a step of 2^-8 of the value
    assert out["rel_err_operators"] <= 6 * 2.0 ** -8
    assert out["rel_err_operators"] < out["rel_err_block"]
