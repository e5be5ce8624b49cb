"""The operators around the linears of a block where they are easily wrong.

u = 2^-24 is half a step of binary32 relative to the value; an output stored in
type t adds half a step of t, finfo(t).eps / 2 of it."""
import pytest
import torch

from w4a4_rotated_bit_amd import binding as B

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# additions one after the other in a row's sum: at most 64 elements a thread, 6
# steps across a wave, 16 waves, and a few roundings of the statistics
SUM = 64 + 6 + 16 + 10


def rand(shape, seed, dtype=torch.float32, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


def half_step(dtype, value):
    info = torch.finfo(dtype)
    return info.eps / 2 * value.abs() + info.smallest_normal * info.eps / 2


# ---- LayerNorm far from zero -----------------------------------------------------


def layer_norm(v, eps):
    """LayerNorm of the exact rows v in binary64, and the error of a binary32
    evaluation in which a mean far from zero costs nothing: a first mean is off
    by no more than e = (SUM + 2) u mean|v|; what is left of the row is rounded
    once, has a mean of its own no larger than e that is found to SUM + 4 of its
    roundings, and that mean leaves both the row and the mean square.  The mean
    square is then off by SUM + 8 roundings of itself and of e^2."""
    d = v - v.mean(-1, keepdim=True)
    e = (SUM + 2) * U * v.abs().mean(-1, keepdim=True)
    size = d.abs().mean(-1, keepdim=True) + e
    var = (d * d).mean(-1, keepdim=True) + eps
    rstd = 1 / torch.sqrt(var)
    off = (2 * U * (d.abs() + e) + (SUM + 4) * U * size) * rstd
    # the root halves what the mean square is off by, through its own sum and
    # through the square of the second mean
    square = ((SUM + 8) * U * (1 + e * e / var) + 2 * (SUM + 4) * U * size * e / var + ((SUM + 4) * U * size) ** 2 / var)
    return d * rstd, off + (d * rstd).abs() * (square + 4 * U)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [3, 65, 255, 768, 1000, 1035, 2048, 4091, 8200, 16383])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_layer_norm_of_rows_of_one_value_is_zero(gpu, dtype, width):
    """(v - mean) is 0 whatever the value is and however its sum rounds; the norm's
    factor is 1 / sqrt(eps) = 1000 at most."""
    values = torch.tensor([20.0, 100.0, 1000.0, -1000.0, 7.7, 333.3, 60000.0]).to(TYPES[dtype])
    x = values.unsqueeze(1).expand(-1, width).contiguous().cuda()
    _, off = layer_norm(x.cpu().double(), 1e-6)
    _, h = B.convrot_residual_norm(x, norm="layer", want_r=False)
    off = off + half_step(TYPES[dtype], off)
    assert (h.cpu().double().abs() <= off).all(), h[:, 0]
    r, _ = B.convrot_residual_norm(torch.zeros_like(x), x, norm=None, post_norm="layer", want_h=False)
    assert (r.cpu().double().abs() <= off).all(), r[:, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("width", [255, 1000, 1024, 1035, 4091, 4096, 16383])
@pytest.mark.parametrize("mean,std", [(1000.0, 1.0), (-300.0, 0.1), (1e5, 3.0), (5.0, 1e-3), (0.0, 1.0)])
def test_layer_norm_far_from_zero(gpu, width, mean, std):
    x = rand((5, width), width, torch.float32, std, mean)
    want, off = layer_norm(x.double(), 1e-6)
    off = off + want.abs() * U
    for rows in (5, 300):   # fewer and more rows than units: other workgroups
        c = x.repeat(rows // 5, 1).cuda()
        _, h = B.convrot_residual_norm(c, norm="layer", want_r=False)
        r, _ = B.convrot_residual_norm(torch.zeros_like(c), c, norm=None, post_norm="layer", want_h=False)
        for got in (h, r):
            assert ((got.cpu().double() - want.repeat(rows // 5, 1)).abs() <= off.repeat(rows // 5, 1)).all()


# ---- outputs that are inputs, rows that end inside a chunk ------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("width", [65, 130, 1035, 2051, 4091, 8197, 16383])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows", [5, 300])
def test_norm_in_place_at_ragged_widths(gpu, dtype, width, rows):
    """The last chunk of a row shares elements with the one before it, which may be
    another wave's; the same bits as with outputs of their own."""
    dt = TYPES[dtype]
    x, y = rand((rows, width), 1, dt).cuda(), rand((rows, width), 2, dt).cuda()
    mods = {k: rand((width,), s, dt, 0.4).cuda() for s, k in enumerate(("gate", "scale", "shift", "weight"), 3)}
    for norm, post in (("layer", None), ("rms", "layer"), ("layer", "rms")):
        kw = dict(mods, norm=norm, post_norm=post, post_weight=mods["weight"] if post else None)
        r, h = B.convrot_residual_norm(x, y, **kw)
        for first, second in (("x", "y"), ("y", "x"), ("x", None), (None, "x"), ("y", None), (None, "y")):
            place = {"x": x.clone(), "y": y.clone()}
            got = B.convrot_residual_norm(place["x"], place["y"], r=place.get(first), h=place.get(second), **kw)
            assert torch.equal(got[0], r) and torch.equal(got[1], h), (norm, post, first, second)
            for name, t in (("x", x), ("y", y)):
                if name not in (first, second):
                    assert torch.equal(place[name], t)


# ---- the grouped linear: many blocks a wave, every count of tiles ------------------


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_grouped_scales_stay_with_their_blocks(gpu, dtype, group, zeros):
    """Rows of so many blocks that a wave hands scales, zero points, codes and x on
    from one round of four blocks to the next, with one to four output tiles a
    workgroup and with four waves.  Integers times powers of two: every sum is a
    whole number of eighths below 12544 * 2 * 15 * 8 < 2^24, so results are exact."""
    dt = TYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(group + zeros)
    # rows of whole lines, and rows that end inside a block
    for k in (4352, {32: 4128, 64: 4160, 128: 4224}[group], 12544, 8192 + group):
        for n in (40, 5000, 9001, 16000):
            codes = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
            s = (2.0 ** torch.randint(-3, 1, (n, k // group), generator=g, device="cuda")).to(dt)
            z = torch.randint(0, 16, (n, k // group), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
            b = torch.randint(-9, 10, (n,), generator=g, device="cuda").to(dt)
            c = torch.stack([codes & 15, codes >> 4], -1).view(n, k // group, group).double()
            c = torch.where(c >= 8, c - 16, c) if z is None else c - z.double().unsqueeze(-1)
            w = (c * s.double().unsqueeze(-1)).view(n, k)
            for m in (1, 4, 5, 8, 16, 32):
                x = torch.randint(-2, 3, (m, k), generator=g, device="cuda").to(dt)
                want = torch.mm(w, x.double().t().contiguous()).t() + b.double()
                got = B.convrot_linear_grouped(x, codes, s, z, b, group)
                assert torch.equal(got, want.to(dt)), (m, n, k)


@pytest.mark.gpu
@pytest.mark.parametrize("zeros", [False, True])
def test_grouped_subnormal_halves(gpu, zeros):
    """Subnormal values of x and of the scales count: whole numbers of 2^-24, exact sums."""
    g = torch.Generator().manual_seed(7)
    m, n, k, group = 5, 33, 512, 32
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    z = torch.randint(0, 16, (n, k // group), generator=g, dtype=torch.uint8) if zeros else None
    c = torch.stack([codes & 15, codes >> 4], -1).view(n, k // group, group).double()
    c = torch.where(c >= 8, c - 16, c) if z is None else c - z.double().unsqueeze(-1)
    whole = torch.randint(-9, 10, (m, k), generator=g).double()
    steps = torch.randint(1, 9, (n, k // group), generator=g).double()
    for x, s in ((whole * 2.0 ** -24, steps * 2.0 ** -3), (whole * 2.0 ** -3, steps * 2.0 ** -24)):
        want = x @ (c * s.unsqueeze(-1)).view(n, k).t()
        x, s = x.half(), s.half()
        got = B.convrot_linear_grouped(x.cuda(), codes.cuda(), s.cuda(), None if z is None else z.cuda(), None, group)
        assert torch.equal(got.cpu(), want.half())


# ---- the quantizer at the end of the range ----------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("asymmetric", [False, True])
def test_quantizer_takes_the_largest_finite_weights(gpu, dtype, asymmetric):
    """hi - lo may lie beyond binary32 where both are finite."""
    big = torch.finfo(TYPES[dtype]).max
    w = torch.zeros((2, 32), dtype=TYPES[dtype])
    w[0, :4] = torch.tensor([big, -big, big / 2, 1.0])
    w[1, :2] = torch.tensor([-big, big / 8])
    codes, scales, zeros = (None if t is None else t.cpu() for t in B.convrot_quantize_weight_grouped(w.cuda(), 32, asymmetric))
    v = w.double()
    lo, hi = v.amin(-1, keepdim=True).clamp(max=0), v.amax(-1, keepdim=True).clamp(min=0)
    s = ((hi - lo) / 15 if asymmetric else v.abs().amax(-1, keepdim=True) / 7)
    # binary32 and the type's rounding: a step and a half of either
    assert torch.isfinite(scales.double()).all() and ((scales.double() - s).abs() <= 1.5 * torch.finfo(TYPES[dtype]).eps * s).all()
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(1).double()
    c = c - zeros.double() if asymmetric else torch.where(c >= 8, c - 16, c)
    # half a scale for the code and for the zero point, and 15 scales' rounding
    assert ((c * scales.double() - v).abs() <= scales.double() * (1.0 + 15 * 2.0 ** -8)).all()


# ---- the binding's own checks, without a GPU --------------------------------------


@pytest.fixture
def host_calls(monkeypatch):
    """The binding on host tensors: its checks run, the C call is recorded instead of made."""
    B._use_torch()
    calls = []
    monkeypatch.setattr(B, "_on_gpu", lambda t, name: -1)
    monkeypatch.setattr(B, "_check_tensor", lambda t, name, device: None)
    monkeypatch.setattr(B, "_launch", lambda device, stream, call, tensors: call(0))
    monkeypatch.setattr(B, "_call", lambda name, *args: calls.append((name, args)))
    return calls


@pytest.mark.parametrize("x,v,rows_per_vec", [
    ((8,), (8,), 1), ((3, 8), (8,), 1), ((3, 8), (1, 1, 8), 1), ((6, 8), (2, 8), 3), ((6, 8), (3, 1, 8), 2), ((6, 8), (6, 8), 1),
    ((2, 3, 8), (2, 8), 3), ((2, 3, 8), (2, 1, 8), 3), ((2, 3, 8), (2, 3, 8), 1), ((2, 3, 8), (2, 3, 1, 8), 1), ((8, 8), (8, 8), 1),
    # more leading dimensions than x has, reaching into its width
    ((8,), (8, 8), None), ((3, 8), (3, 8, 8), None), ((2, 3, 8), (2, 3, 8, 8), None), ((8, 8), (8, 8, 8), None),
    ((8,), (8, 1, 8), None), ((1, 8), (8, 8), None), ((3, 8), (6, 8), None), ((3, 8), (2, 8), None), ((2, 3, 8), (3, 8), None),
    ((2, 3, 8), (6, 8), None), ((2, 3, 8), (2, 2, 8), None), ((3, 8), (0, 8), None)])
@pytest.mark.parametrize("name", ["gate", "scale", "shift"])
def test_norm_vectors_have_the_leading_dimensions_of_x(host_calls, name, x, v, rows_per_vec):
    x, v = torch.zeros(x), torch.zeros(v)
    if rows_per_vec is None:
        with pytest.raises(ValueError, match=name):
            B.convrot_residual_norm(x, x, **{name: v})
        assert not host_calls
        return
    B.convrot_residual_norm(x, x, **{name: v})
    fields = B.NORM_ARGS.unpack(host_calls[0][1][0])
    assert fields[18] == rows_per_vec
    step = fields[{"gate": 15, "scale": 16, "shift": 17}[name]]
    assert step == (8 if v.numel() > 8 else 0)


def test_tensors_with_a_tangent_are_refused(host_calls):
    """A tangent of forward differentiation would be lost as a gradient would be."""
    import torch.autograd.forward_ad as fwd
    x, q, pos = torch.zeros((2, 8)), torch.zeros((1, 2, 1, 8)), torch.zeros((1, 2, 1))
    X, codes, scales, bias = (torch.zeros(s, dtype=t) for s, t in (
        ((2, 32), torch.bfloat16), ((4, 16), torch.uint8), ((4, 1), torch.bfloat16), ((4,), torch.bfloat16)))
    freq, axis = B.rope_frequencies((8,))
    norm = dict(x=x, y=x, gate=x, scale=x, shift=x, weight=x[0], post_weight=x[0], post_norm="rms", r=torch.empty_like(x),
                h=torch.empty_like(x))
    rope = dict(q=q, k=q, positions=pos, freq=freq, axis=axis, qk_norm=True, q_weight=q[0, 0, 0], k_weight=q[0, 0, 0],
                q_out=torch.empty_like(q), k_out=torch.empty_like(q))
    grouped = dict(X=X, codes=codes, scales=scales, zeros=None, bias=bias, group=32, Y=torch.empty((2, 4), dtype=X.dtype))
    for call, args, dual in ((B.convrot_residual_norm, norm, [k for k in norm if k != "post_norm"]),
                             (B.convrot_rope, rope, ["q", "k", "positions", "q_weight", "k_weight", "q_out", "k_out"]),
                             (B.convrot_linear_grouped, grouped, ["X", "scales", "bias", "Y"])):
        with fwd.dual_level():
            call(**args)     # none of them has one
            made = len(host_calls)
            for key in dual:
                t = args[key]
                with pytest.raises(RuntimeError, match="tangent"):
                    call(**{**args, key: fwd.make_dual(t.clone(), torch.ones_like(t))})
            assert len(host_calls) == made
        call(**args)


def test_given_outputs_count_as_written(host_calls):
    """Autograd tells a saved tensor that was written since by its version."""
    x, q, pos = torch.zeros((2, 8)), torch.zeros((1, 2, 1, 8)), torch.zeros((1, 2, 1))
    X, codes, scales = (torch.zeros(s, dtype=t) for s, t in (
        ((2, 32), torch.bfloat16), ((4, 16), torch.uint8), ((4, 1), torch.bfloat16)))
    freq, axis = B.rope_frequencies((8,))
    r, h, out, y = x.clone(), x.clone(), q.clone(), X.new_zeros((2, 4))
    B.convrot_residual_norm(x, r=r, h=h)
    B.convrot_rope(q, q, pos, freq, axis, q_out=q, k_out=out)
    B.convrot_linear_grouped(X, codes, scales, None, None, 32, Y=y)
    assert [t._version for t in (r, h, q, out, y)] == [1] * 5
    assert [t._version for t in (x, pos, X, codes, scales)] == [0] * 5
    with torch.inference_mode():
        t = torch.zeros((2, 8))
        B.convrot_residual_norm(t, r=t)
    weight = torch.ones((2, 8), requires_grad=True)
    z = (weight * x).sum()      # saves x
    with torch.no_grad():
        B.convrot_residual_norm(x, r=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()


def test_tensors_of_a_call_on_another_stream_are_recorded_there(monkeypatch):
    """Memory that is freed while the stream still reads it must not be given out again."""
    from contextlib import nullcontext
    from types import SimpleNamespace
    B._use_torch()
    monkeypatch.setattr(B, "_on_gpu", lambda t, name: 0)
    monkeypatch.setattr(B, "_check_tensor", lambda t, name, device: None)
    monkeypatch.setattr(B, "_call", lambda name, *args: None)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: nullcontext())
    seen = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.append((t.data_ptr(), s)))
    side = SimpleNamespace(device=SimpleNamespace(index=0), cuda_stream=7)
    x, y, w, q, pos = torch.zeros((2, 8)), torch.zeros((2, 8)), torch.zeros(8), torch.zeros((1, 2, 1, 8)), torch.zeros((1, 2, 1))
    X, codes, scales, zeros, bias = (torch.zeros(s, dtype=t) for s, t in (
        ((2, 32), torch.bfloat16), ((4, 16), torch.uint8), ((4, 1), torch.bfloat16), ((4, 1), torch.uint8), ((4,), torch.bfloat16)))
    freq, axis = B.rope_frequencies((8,))
    r, out, Y = x.clone(), q.clone(), X.new_zeros((2, 4))
    mods = dict(gate=w.clone(), scale=w.clone(), shift=w.clone(), weight=w.clone(), post_weight=w.clone())
    k, qw = q.clone(), w.clone()
    for call, own in (
            (lambda s: B.convrot_residual_norm(x, y, post_norm="rms", r=r, stream=s, **mods), (x, y, r, *mods.values())),
            (lambda s: B.convrot_rope(q, k, pos, freq, axis, qk_norm=True, q_weight=qw, k_weight=w, q_out=out, stream=s),
             (q, k, pos, qw, w, out)),
            (lambda s: B.convrot_linear_grouped(X, codes, scales, zeros, bias, 32, Y=Y, stream=s),
             (X, codes, scales, zeros, bias, Y)),
            (lambda s: B.convrot_quantize_weight_grouped(X, 32, stream=s), (X,))):
        seen.clear()
        call(side)
        assert {at for at, _ in seen} == {t.data_ptr() for t in own} and all(s is side for _, s in seen)


@pytest.mark.gpu
def test_inputs_freed_while_another_stream_reads_them(gpu):
    side = torch.cuda.Stream()
    x = rand((64, 4096), 1, torch.bfloat16).cuda()
    want = B.convrot_residual_norm(x, x)
    torch.full_like(x, 7.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)   # the call's kernel starts after what follows here
    got = B.convrot_residual_norm(x, x, stream=side)
    at = x.data_ptr()
    del x
    others = [torch.empty((64, 4096), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    assert side.query() or all(t.data_ptr() != at for t in others)
    for t in others:
        t.fill_(7.0)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_captured_call_on_another_stream(gpu):
    """A graph whose calls run on a stream of their own, their temporaries freed during the capture."""
    side = torch.cuda.Stream()
    x, w = rand((4, 512), 1, torch.bfloat16).cuda(), rand((1024, 512), 2, torch.bfloat16, 0.05).cuda()
    codes, scales, zeros = B.convrot_quantize_weight_grouped(w, 64, asymmetric=True)

    def run(stream):
        scale, shift = B.convrot_linear_grouped(x * 0.5, codes, scales, zeros, None, 64, stream=stream).chunk(2, -1)
        return B.convrot_residual_norm(x, scale=scale, shift=shift, stream=stream)

    run(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        half = x * 0.5
        side.wait_stream(torch.cuda.current_stream())
        mods = B.convrot_linear_grouped(half, codes, scales, zeros, None, 64, stream=side)
        del half
        outs = B.convrot_residual_norm(x, scale=mods[:, :512], shift=mods[:, 512:], stream=side)
        del mods
        torch.cuda.current_stream().wait_stream(side)
    for step in range(4):
        x.copy_(rand(x.shape, step, torch.bfloat16))
        want = [t.clone() for t in run(None)]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), step


# ---- sources ------------------------------------------------------------------------


def test_lanes_pass_values_on_behind_a_fence():
    """A wave barrier alone orders nothing for the compiler's memory accesses."""
    from pathlib import Path
    csrc = Path(B.__file__).parent / "csrc"
    for name in ("norm.hip", "rope.hip", "grouped.hip", "grouped_kernel.h"):
        assert "__builtin_amdgcn_wave_barrier" not in (csrc / name).read_text(), name
    body = (csrc / "block_ops.h").read_text().split("void wave_exchange()")[1].split("}")[0]
    order = [body.index(s) for s in ("__ATOMIC_RELEASE", "__builtin_amdgcn_wave_barrier", "__ATOMIC_ACQUIRE")]
    assert order == sorted(order)
