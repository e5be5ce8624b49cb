"""Attention and the paged cache that it reads, against their formulas in binary64.

Tolerances are sums of what the arithmetic may lose.  u = 2^-24 is half a step of
binary32 relative to the value.  A score, a sum of head_dim products, is off by at
most (head_dim + 4) u of the sum of the products' magnitudes, and so is the
logarithm of its weight; a weight is rounded to the heads' type (half a step,
finfo.eps / 2 of it, and in f16 half the smallest subnormal) before it multiplies
a value; sums over n keys lose n u; an output adds half a step of its type."""
import math

import pytest
import torch

from w4a4_rotated_bit_amd import binding as B

from .test_block_ops import TYPES, U, close, half_step, packed, rand

P = 1 << 32
FORMATS = {"e4m3": (8, 3, -6, 448.0), "e2m1": (2, 1, 0, 6.0)}   # largest exponent, mantissa bits, smallest exponent, largest


# ---- the cache ------------------------------------------------------------------


def grid(kind):
    top, bits, least, most = FORMATS[kind]
    points = [m * 2.0 ** (least - bits) for m in range(1 << bits)]
    points += [(1 + m / (1 << bits)) * 2.0 ** e for e in range(least, top + 1) for m in range(1 << bits)]
    return torch.tensor([p for p in points if p <= most], dtype=torch.float64)


def power(n):
    return torch.tensor([2.0 ** i for i in range(-300, 301)], dtype=torch.float64)[n.long() + 300]


def kept(x, kind):
    """(values, scale bytes) of rows [..., dim] in a cache of this kind, from the definition."""
    x = x.double().unflatten(-1, (-1, 32))
    most = x.abs().amax(-1)
    fine = torch.isfinite(most)
    e = torch.where(fine & (most > 0), torch.frexp(most.nan_to_num(1.0, 1.0))[1] - 1, -400) - FORMATS[kind][0] + 127
    scales = torch.where(fine, e.clamp(0, 254), 255)
    unit = power(scales.clamp(max=254) - 127).unsqueeze(-1)
    g = grid(kind)
    a = (x / unit).abs().nan_to_num(0.0, 0.0).clamp(max=g[-1])
    hi = torch.searchsorted(g, a).clamp(max=len(g) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = g[hi] - a, a - g[lo]
    at = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    y = torch.sign(x).nan_to_num(0.0) * g[at] * unit
    y[~fine] = math.nan
    return y.flatten(-2), scales.to(torch.uint8)


def stored(cache, kind):
    """(k, v) values [pages, heads, page_size, dim] of a cache's bytes, in binary64."""
    out = []
    for rows, scales in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        rows = rows.cpu()
        if kind == "e2m1":
            g = torch.cat([grid(kind), -grid(kind)])
            x = torch.stack([g[(rows & 15).long()], g[(rows >> 4).long()]], -1).flatten(-2)
        else:
            x = rows.double()
        if scales is not None:
            s = scales.cpu().int()
            unit = torch.where(s == 255, math.nan, power(s.clamp(max=254) - 127))
            x = x * unit.repeat_interleave(32, -1)
        out.append(x)
    return out


def new_cache(pages, page, heads, dim, kind, dtype, seed=None):
    cache = B.new_kv_cache(pages, page, heads, dim, kind if kind in FORMATS else TYPES[dtype])
    if seed is not None:    # rows of a normal distribution
        k, v = (rand((pages * page, heads, dim), seed + i, TYPES[dtype]).cuda() for i in (0, 1))
        B.convrot_cache_write(k, v, torch.arange(pages * page, device="cuda"), cache)
    return cache


def same(got, want):
    got, want = got.cpu().double(), want.double()
    assert got.shape == want.shape
    assert ((got == want) | (got.isnan() & want.isnan())).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e2m1", "e4m3", "same"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
def test_cache_holds_what_its_format_says(gpu, kind, dtype, dim):
    dt, heads, page, pages, tokens = TYPES[dtype], 3, 16, 9, 101
    k, v = (rand((tokens, heads, dim), dim + i, dt, 3.0) for i in (0, 1))
    k[5] = 0
    k[6] *= 2.0 ** -14      # f16: subnormal
    k[7, 1, 3], k[8, 0, 0], k[9, 2, 31] = math.inf, math.nan, -math.inf
    k[10] = torch.round(k[10] * 4) / 4     # ties
    v[11, :, ::2] = -0.0
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(dim))[:tokens]
    cache = new_cache(pages, page, heads, dim, kind, dtype)
    B.convrot_cache_write(k.cuda(), v.cuda(), slots.cuda(), cache)
    got = stored(cache, kind)
    back = B.convrot_cache_read(cache, slots.cuda(), dtype=dt)
    for i, x in enumerate((k, v)):
        want, scales = (x.double(), None) if kind == "same" else kept(x, kind)
        full = torch.zeros((pages * page, heads, dim), dtype=torch.float64)
        full[slots] = want
        same(got[i], full.view(pages, page, heads, dim).transpose(1, 2))
        same(back[i], want.to(dt))
        if scales is not None:
            s = torch.zeros((pages * page, heads, dim // 32), dtype=torch.uint8)
            s[slots] = scales
            assert torch.equal((cache.k_scales, cache.v_scales)[i].cpu(), s.view(pages, page, heads, -1).transpose(1, 2))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e2m1", "e4m3"])
def test_cache_every_bf16_value(gpu, kind):
    """Every finite bf16 value beside every power of two as the block's largest: 32 x 2048 blocks
    cover all 65280 values at a scale of their own, and all values below a tie."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = bits[torch.isfinite(bits.float())]
    own = x.view(-1, 32)[torch.randperm(len(x) // 32, generator=torch.Generator().manual_seed(1))]
    mixed = x[torch.randperm(len(x), generator=torch.Generator().manual_seed(2))].view(-1, 32).clone()
    near = (torch.arange(256).float() / 16 - 8).to(torch.bfloat16).view(-1, 32)
    rows = torch.cat([own, mixed, near, near * 2.0 ** -126, near * 2.0 ** -130, near * 2.0 ** 120])
    rows = rows[:len(rows) // 4 * 4].view(-1, 1, 128)
    n = len(rows)
    cache = new_cache(-(-n // 64), 64, 1, 128, kind, "bf16")
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    B.convrot_cache_write(rows.cuda(), rows.flip(0).cuda(), slots, cache)
    k, v = B.convrot_cache_read(cache, slots)
    want, _ = kept(rows, kind)
    same(k, want.to(torch.bfloat16))
    same(v, want.to(torch.bfloat16).flip(0))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e2m1", "e4m3", "same"])
@pytest.mark.parametrize("slot_type", [torch.int32, torch.int64])
def test_cache_slots_outside_are_skipped(gpu, kind, slot_type):
    cache = new_cache(4, 8, 2, 64, kind, "bf16", seed=1)
    before = stored(cache, kind)
    x = rand((9, 2, 64), 5, torch.bfloat16).cuda()
    big = [-1, 32, 2 ** 31 - 1, -2 ** 31] + ([2 ** 40, -2 ** 62] if slot_type is torch.int64 else [33, -5])
    slots = torch.tensor(big + [31, 0, 7], dtype=slot_type, device="cuda")
    B.convrot_cache_write(x, x * 2, slots, cache)
    after = stored(cache, kind)
    touched = torch.zeros(32, dtype=torch.bool)
    touched[[31, 0, 7]] = True
    for b, a in zip(before, after):
        a, b = (t.transpose(1, 2).reshape(32, 2, 64) for t in (a, b))
        assert torch.equal(a[~touched], b[~touched]) and not torch.equal(a[touched], b[touched])
    k, v = B.convrot_cache_read(cache, slots)
    assert not k[:6].any() and not v[:6].any() and k[6:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e2m1", "e4m3", "same"])
def test_cache_strides_and_alignment(gpu, kind):
    """Rows in odd places of a wider tensor; a cache that is one layer's slice of all
    layers', its pages token by token and not head by head."""
    pages, page, heads, dim, tokens = 5, 16, 3, 96, 50
    whole = torch.zeros((tokens, 2 * heads * dim + 7), dtype=torch.bfloat16, device="cuda")
    k, v = (whole[:, 3 + i * heads * dim:][:, :heads * dim].unflatten(1, (heads, dim)) for i in (0, 1))
    k.copy_(rand(k.shape, 1, torch.bfloat16))
    v.copy_(rand(v.shape, 2, torch.bfloat16))
    plain = new_cache(pages, page, heads, dim, kind, "bf16")
    parts = []
    for t in plain:
        if t is None:
            parts.append(None)
            continue
        wide = torch.zeros((pages, 2, page, heads, t.shape[-1]), dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device="cuda")
        parts.append(wide.view(t.dtype)[:, 1].permute(0, 2, 1, 3))
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:tokens].cuda()
    B.convrot_cache_write(k.contiguous(), v.contiguous(), slots, plain)
    B.convrot_cache_write(k, v, slots, B.KVCache(*parts))
    for a, b in zip(plain, parts):
        assert a is None or torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    out = torch.zeros((tokens, 2 * heads * dim + 7), dtype=torch.bfloat16, device="cuda")
    ok, ov = (out[:, 3 + i * heads * dim:][:, :heads * dim].unflatten(1, (heads, dim)) for i in (0, 1))
    B.convrot_cache_read(B.KVCache(*parts), slots, k=ok, v=ov)
    want = B.convrot_cache_read(plain, slots)
    assert torch.equal(ok, want[0]) and torch.equal(ov, want[1])
    assert not out[:, :3].any() and not out[:, -4:].any()


@pytest.mark.gpu
def test_cache_beyond_4_gib(gpu):
    """Places whose bytes lie past 32-bit offsets, written, read and attended to."""
    page, heads, dim = 256, 8, 128
    pages = (5 << 30) // (page * heads * dim)      # 5 GiB of e4m3 keys
    rows = [torch.empty((pages, heads, page, dim), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    scales = [torch.empty((pages, heads, page, dim // 32), dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = B.KVCache(*rows, *scales)
    tokens = 300
    k, v = (rand((tokens, heads, dim), 3 + i, torch.bfloat16) for i in (0, 1))
    first = pages * page - 512
    slots = torch.arange(first, first + tokens, device="cuda")
    B.convrot_cache_write(k.cuda(), v.cuda(), slots, cache)
    got = B.convrot_cache_read(cache, slots)
    same(got[0], kept(k, "e4m3")[0])
    same(got[1], kept(v, "e4m3")[0])
    q = rand((1, heads, dim), 9, torch.bfloat16)
    table = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32, device="cuda")
    out, lse = B.convrot_attention_paged(q.cuda(), cache, table, torch.tensor([tokens], dtype=torch.int32, device="cuda"), want_lse=True)
    want, bound, want_lse, lse_bound = attended(q[0].double().unsqueeze(1), kept(k, "e4m3")[0].transpose(0, 1),
                                                kept(v, "e4m3")[0].transpose(0, 1), dim ** -0.5, None, torch.bfloat16)
    close(out[0], want[:, 0], bound[:, 0])
    close(lse[0], want_lse[:, 0], lse_bound[:, 0])


# ---- the formula ------------------------------------------------------------------


def attended(q, k, v, scale, offset, dtype):
    """out, its bound, lse, its bound; q [heads, rows, dim], k, v [heads or fewer, keys, dim] in
    binary64, row i sees keys up to i + offset (None: all)."""
    share = q.shape[0] // k.shape[0]
    k, v = (t.repeat_interleave(share, 0) for t in (k, v))
    rows, keys, dim = q.shape[1], k.shape[1], q.shape[2]
    s = (q @ k.transpose(1, 2)) * scale
    slack = (dim + 4) * U * (q.abs() @ k.abs().transpose(1, 2)) * abs(scale) + 8 * U * (1 + s.abs())
    if offset is not None:
        hidden = torch.arange(keys)[None] > torch.arange(rows)[:, None] + offset
        s = s.masked_fill(hidden, -math.inf)
        slack = slack.masked_fill(hidden, 0.0)
    if keys == 0:
        zero = torch.zeros_like(q)
        return zero, zero, torch.full(q.shape[:2], -math.inf, dtype=torch.float64), torch.zeros(q.shape[:2], dtype=torch.float64)
    none = (s == -math.inf).all(-1)
    w = torch.softmax(s, -1).masked_fill(none.unsqueeze(-1), 0.0)
    info = torch.finfo(dtype)
    # a maximum that lags by up to 2^8 leaves weights of 1 .. 2^8 at the top: a subnormal one's half step is that much of the sum
    tiny = info.smallest_normal * info.eps / 2 if dtype == torch.float16 else 0.0
    lost = slack.amax(-1, keepdim=True).expand(*s.shape[:2], 1)
    vv = torch.where(w.transpose(1, 2).amax(-1, keepdim=True) > 0, v, 0.0) if v.isnan().any() else v
    out = w @ vv
    bound = (w @ vv.abs()) * (2 * lost + info.eps / 2 + 2 * (keys + 16) * U) + tiny * keys * vv.abs().amax(1, keepdim=True)
    lse = torch.logsumexp(s, -1)
    lse_bound = lost[..., 0] + (keys + 16) * U + 4 * U * (1 + lse.abs().nan_to_num(0, 0, 0))
    return out, bound + half_step(dtype, out.abs() + bound), lse, torch.where(none, 0.0, lse_bound)


def check_paged(lengths, kind="same", dtype="bf16", q_heads=4, k_heads=2, dim=128, page=16, seed=0, q_std=1.0, scale=None,
                table_extra=1, lse=True, split_view=False):
    dt, need = TYPES[dtype], [-(-max(n, 0) // page) for n in lengths]
    pages = sum(need) + 2
    cache = new_cache(pages, page, k_heads, dim, kind, dtype, seed=seed)
    values = stored(cache, kind)
    if kind in FORMATS:     # as f16 holds them
        values = [x.to(dt).double() for x in values]
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed + 2)).int()
    table = torch.full((len(lengths), max(need, default=0) + table_extra), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    q = rand((len(lengths), q_heads, dim), seed + 3, dt, q_std)
    cq, ct = q.cuda(), table.cuda()
    if split_view:
        cq = torch.cat([cq, cq * 3], 2)[:, :, :dim]
        ct = torch.cat([ct, ct], 1)[:, :table.shape[1]]
    got = B.convrot_attention_paged(cq, cache, ct, torch.tensor(lengths, dtype=torch.int32).cuda(), scale=scale, want_lse=lse)
    out, sums = got if lse else (got, None)
    for i, n in enumerate(lengths):
        n = max(n, 0)
        rows = [x[table[i, :need[i]].long()].transpose(0, 1).reshape(k_heads, -1, dim)[:, :n] for x in values]
        want, bound, want_lse, lse_bound = attended(q[i].double().unsqueeze(1), *rows, dim ** -0.5 if scale is None else scale, None, dt)
        close(out[i], want[:, 0], bound[:, 0], f"sequence {i} of {n}")
        if lse:
            close(sums[i], want_lse[:, 0], lse_bound[:, 0], f"lse of sequence {i}")
    return out


LENGTHS = [1, 0, 31, 32, 33, 127, 128, 129, 255, 256, 257, 1000, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["same", "e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
def test_paged_dims_and_kinds(gpu, kind, dtype, dim):
    check_paged(LENGTHS, kind, dtype, dim=dim, seed=dim)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [8, 16, 24, 40, 72, 80, 120, 136, 200, 248])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_paged_odd_dims(gpu, dim, dtype):
    check_paged([300, 5, 0, 64], "same", dtype, q_heads=6, k_heads=3, dim=dim, page=8, seed=dim)


@pytest.mark.gpu
@pytest.mark.parametrize("q_heads,k_heads", [(1, 1), (3, 1), (8, 8), (16, 1), (17, 1), (40, 2), (64, 2), (96, 1), (7, 7)])
@pytest.mark.parametrize("kind", ["same", "e2m1"])
def test_paged_heads(gpu, q_heads, k_heads, kind):
    check_paged([77, 513, 1], kind, q_heads=q_heads, k_heads=k_heads, dim=64, seed=q_heads)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("kind", ["same", "e4m3", "e2m1"])
def test_paged_pages(gpu, page, kind):
    check_paged([1025, 1024, 7, 100], kind, page=page, seed=page, split_view=True)


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", [[1], [40], [200], [256], [257], [5000], [20000, 3], [1] * 200, list(range(0, 300)),
                                     [0] * 70 + [900] + [0] * 70, [0, 0, 0], [4000] * 40])
def test_paged_shares(gpu, lengths):
    """Work shared over more or fewer workgroups than there are units, sequences that
    begin and end inside a share, empty ones between, more than a wave's lanes."""
    check_paged(lengths, "e4m3", q_heads=4, k_heads=2, dim=64, page=16, seed=len(lengths))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["same", "e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_paged_short_tables(gpu, kind, dtype, dim):
    """Tables of up to 384 keys: a sequence and key head are one workgroup's, without a second launch."""
    check_paged([1, 0, 31, 33, 128, 255, 256, 257, 300], kind, dtype, q_heads=6, k_heads=3, dim=dim, seed=dim + 1)
    check_paged([350, 8, 0], kind, dtype, q_heads=20, k_heads=1, dim=dim, page=8, seed=dim + 2)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["same", "e4m3", "e2m1"])
@pytest.mark.parametrize("lengths,heads", [([700, 0, 1, 33] * 130, 2), ([450, 3, 0, 129, 64] * 120, 1), ([0] * 590 + [900], 1),
                                           ([2, 0, 385] * 400, 1)])
def test_paged_many_sequences(gpu, kind, lengths, heads):
    """More than the chip has room for, one workgroup each, and shares of several hundred."""
    check_paged(lengths, kind, q_heads=3 * heads, k_heads=heads, dim=64, page=32, seed=len(lengths))


@pytest.mark.gpu
def test_paged_large_and_ordered_scores(gpu):
    check_paged([700, 33, 128], "same", q_std=30.0, seed=1)
    check_paged([700, 33, 128], "e2m1", "f16", q_std=30.0, seed=2)
    check_paged([700, 33], "same", scale=0.0, seed=3)
    check_paged([700, 33], "same", scale=-0.2, seed=4)
    # scores that rise, and that fall, by more than the running maximum's slack with every key
    n, dim = 600, 64
    for order in (1, -1):
        k = torch.zeros((n, 1, dim), dtype=torch.bfloat16)
        k[:, 0, 0] = torch.arange(n).to(torch.bfloat16)[::1] if order == 1 else torch.arange(n).flip(0).to(torch.bfloat16)
        v = rand((n, 1, dim), 7, torch.bfloat16)
        cache = B.new_kv_cache(38, 16, 1, dim, torch.bfloat16)
        B.convrot_cache_write(k.cuda(), v.cuda(), torch.arange(n, device="cuda"), cache)
        q = torch.zeros((1, 1, dim), dtype=torch.bfloat16)
        q[0, 0, 0] = 8.0
        table = torch.arange(38, dtype=torch.int32, device="cuda")[None]
        out = B.convrot_attention_paged(q.cuda(), cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), scale=1.0)
        want, bound, _, _ = attended(q.double().transpose(0, 1), k.double().transpose(0, 1), v.double().transpose(0, 1), 1.0, None, torch.bfloat16)
        close(out[0], want[0], bound[0])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["same", "e4m3", "e2m1"])
@pytest.mark.parametrize("wide", [0, 60])      # more columns of the table: shares of the keys
def test_paged_unseen_places_stay_out(gpu, kind, wide):
    """NaN in every place that no sequence holds, in the rest of its last page, and on
    pages that its table does not name; entries that are no page hide their places."""
    page, heads, dim, n = 16, 2, 64, 83
    cache = new_cache(12, page, heads, dim, kind, "bf16")
    k, v = (rand((n, heads, dim), 1 + i, torch.bfloat16) for i in (0, 1))
    bad = torch.full((12 * page, heads, dim), math.nan, dtype=torch.bfloat16, device="cuda")
    B.convrot_cache_write(bad, bad, torch.arange(12 * page, device="cuda"), cache)
    table = torch.tensor([[7, 2, 9, -1, 4, 11, 3] + [-1] * wide], dtype=torch.int32)
    slots = torch.tensor([int(table[0, i // page]) * page + i % page if table[0, i // page] >= 0 else -1 for i in range(n)])
    B.convrot_cache_write(k.cuda(), v.cuda(), slots.cuda(), cache)
    q = rand((1, 4, dim), 5, torch.bfloat16)
    out, lse = B.convrot_attention_paged(q.cuda(), cache, table.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), want_lse=True)
    rows = [(x.double() if kind == "same" else kept(x, kind)[0])[slots >= 0].transpose(0, 1) for x in (k, v)]
    want, bound, want_lse, lse_bound = attended(q[0].double().unsqueeze(1), *rows, dim ** -0.5, None, torch.bfloat16)
    close(out[0], want[:, 0], bound[:, 0])
    close(lse[0], want_lse[:, 0], lse_bound[:, 0])
    # no page is one of the cache's; lengths beyond the table, and below zero
    none = torch.tensor([[-1, 12, 2 ** 31 - 1, -2 ** 31] + [-1] * wide] * 3, dtype=torch.int32, device="cuda")
    out, lse = B.convrot_attention_paged(q.expand(3, 4, dim).contiguous().cuda(), cache, none,
                                         torch.tensor([60, 2 ** 31 - 1, -7], dtype=torch.int32, device="cuda"), want_lse=True)
    assert not out.any() and (lse == -math.inf).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [8, 40, 64, 72, 96, 128, 136, 200, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_infinite_scores(gpu, dim, dtype):
    """Keys whose product with a query is -infinity count for nothing, in heads of any width;
    one of +infinity leaves no number, and so does a query that holds none, times a scale of 0 too."""
    dt, n, heads = TYPES[dtype], 150, 2
    q, k, v = (rand((rows, heads, dim), dim + i, dt) for i, rows in enumerate((3, n, n)))
    q[:, :, 0] = 1
    q[2, :, 0] = -1
    k[::3, :, 0] = -math.inf
    kept_keys = torch.arange(n) % 3 != 0
    want, bound, want_lse, lse_bound = attended(*(t.double().transpose(0, 1) for t in (q[:2], k[kept_keys], v[kept_keys])), dim ** -0.5,
                                                None, dt)
    table = torch.arange(10, dtype=torch.int32).expand(3, 10).contiguous()
    for extra in (0, 50):   # one workgroup a sequence, shares of the keys
        cache = new_cache(10, 16, heads, dim, "same", dtype)
        B.convrot_cache_write(k.cuda(), v.cuda(), torch.arange(n, device="cuda"), cache)
        wide = torch.cat([table, torch.full((3, extra), -1, dtype=torch.int32)], 1).cuda()
        lengths = torch.full((3,), n, dtype=torch.int32, device="cuda")
        paged = B.convrot_attention_paged(q.cuda(), cache, wide, lengths, want_lse=True)
        prompt = B.convrot_attention(q[None].cuda(), k[None].cuda(), v[None].cuda(), want_lse=True)
        for out, lse in (paged, (prompt[0][0], prompt[1][0])):
            close(out[:2].transpose(0, 1), want, bound)
            close(lse[:2].T, want_lse, lse_bound)
            assert out[2].isnan().all()
    q[1, 0, dim - 1] = math.nan
    k[::3, :, 0] = 1
    out = B.convrot_attention(q[None].cuda(), k[None].cuda(), v[None].cuda(), scale=0.0)[0]
    assert out[1, 0].isnan().all() and out.isnan().sum() == dim
    want, bound, _, _ = attended(*(t.double().transpose(0, 1) for t in (q[::2], k, v)), 0.0, None, dt)
    close(out[::2].transpose(0, 1), want, bound)


@pytest.mark.gpu
def test_paged_lengths_beyond_the_table(gpu):
    a = check_paged([64, 640], "same", page=16, table_extra=0, seed=3)
    cache = new_cache(46, 16, 2, 128, "same", "bf16", seed=3)
    order = torch.randperm(46, generator=torch.Generator().manual_seed(5)).int()
    table = torch.full((2, 40), -1, dtype=torch.int32)
    table[0, :4], table[1] = order[:4], order[4:44]
    q = rand((2, 4, 128), 6, torch.bfloat16).cuda()
    b = B.convrot_attention_paged(q, cache, table.cuda(), torch.tensor([64, 2 ** 31 - 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(a, b)


# ---- whole prompts ----------------------------------------------------------------


def check_prompt(q_lens, k_lens=None, dtype="bf16", q_heads=2, k_heads=1, dim=64, causal=True, packed_starts=True, scale=None,
                 seed=0, std=1.0, pad=0, behind=0, place=0):
    """Packed sequences, or a batch of equal ones; ``pad`` more columns a row, an odd ``place``
    of the first, and ``behind`` more rows than the sequences have."""
    dt, k_lens = TYPES[dtype], q_lens if k_lens is None else k_lens
    tensors = []
    for i, (lens, heads) in enumerate(((q_lens, q_heads), (k_lens, k_heads), (k_lens, k_heads))):
        n = sum(lens) + behind
        x = rand((n, heads, dim), seed + i, dt, std if i < 2 else 1.0)
        if behind:
            x[sum(lens):] = math.nan
        wide = torch.full((n * (heads * dim + pad) + place,), math.nan, dtype=dt, device="cuda")
        view = wide[place:].view(n, heads * dim + pad)[:, :heads * dim].unflatten(1, (heads, dim))
        view.copy_(x)
        tensors.append((x, view))
    (q, cq), (k, ck), (v, cv) = tensors
    if packed_starts:
        qs, ks = (torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32).cuda() for lens in (q_lens, k_lens))
        mark = torch.full_like(q, 7.0).cuda()
        out, lse = B.convrot_attention(cq, ck, cv, q_starts=qs, k_starts=ks, causal=causal, scale=scale, want_lse=True, out=mark)
        if behind:
            assert (out[sum(q_lens):] == 7.0).all()
    else:
        b = len(q_lens)
        out, lse = B.convrot_attention(*(t.unflatten(0, (b, -1)) for t in (cq, ck, cv)), causal=causal, scale=scale, want_lse=True)
        out, lse = out.flatten(0, 1), lse.flatten(0, 1)
    at_q = at_k = 0
    for i, (nq, nk) in enumerate(zip(q_lens, k_lens)):
        rows = [x[a:a + n].double().transpose(0, 1) for x, a, n in ((q, at_q, nq), (k, at_k, nk), (v, at_k, nk))]
        want, bound, want_lse, lse_bound = attended(*rows, dim ** -0.5 if scale is None else scale, nk - nq if causal else None, dt)
        close(out[at_q:at_q + nq].transpose(0, 1), want, bound, f"sequence {i}: {nq} x {nk}")
        close(lse[at_q:at_q + nq].transpose(0, 1), want_lse, lse_bound, f"lse of sequence {i}")
        at_q, at_k = at_q + nq, at_k + nk
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [8, 32, 40, 64, 72, 80, 96, 104, 128, 136, 160, 192, 200, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [False, True])
def test_prompt_dims(gpu, dim, dtype, causal):
    check_prompt([130, 1, 64, 0, 65], dtype=dtype, dim=dim, causal=causal, seed=dim, behind=3)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[1], [2], [31], [32], [33], [63], [64], [65], [127], [128], [129], [191], [192], [193], [255], [256],
                                  [257], [500, 3, 0, 0, 129], [0, 0], [1] * 100, list(range(70))])
@pytest.mark.parametrize("causal", [False, True])
def test_prompt_lengths(gpu, lens, causal):
    check_prompt(lens, causal=causal, seed=len(lens), dim=128 if len(lens) == 1 else 64, q_heads=8 if len(lens) < 3 else 3, behind=1)


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens,k_lens", [([5, 200], [300, 129]), ([200, 64], [5, 64]), ([1, 1, 1], [1000, 1, 0]), ([130], [0]),
                                           ([0, 3], [40, 65]), ([33], [4000]), ([300], [40]), ([128], [64]), ([2], [1])])
@pytest.mark.parametrize("causal", [False, True])
def test_prompt_other_keys(gpu, q_lens, k_lens, causal):
    """Fewer and more keys than queries: under a causal mask rows that see none."""
    check_prompt(q_lens, k_lens, causal=causal, q_heads=3, k_heads=3, seed=sum(k_lens), dim=96)


@pytest.mark.gpu
@pytest.mark.parametrize("q_heads,k_heads", [(1, 1), (8, 2), (16, 16), (12, 4), (24, 1), (9, 3)])
@pytest.mark.parametrize("packed_starts", [False, True])
def test_prompt_heads_and_batches(gpu, q_heads, k_heads, packed_starts):
    check_prompt([150] * 3, q_heads=q_heads, k_heads=k_heads, packed_starts=packed_starts, seed=q_heads)
    check_prompt([150] * 3, [70] * 3, q_heads=q_heads, k_heads=k_heads, packed_starts=packed_starts, causal=False, seed=q_heads)


@pytest.mark.gpu
@pytest.mark.parametrize("pad,place", [(8, 0), (24, 8), (1, 0), (3, 5), (0, 1), (2, 2)])
@pytest.mark.parametrize("dim", [64, 72, 128, 256])
def test_prompt_strides_and_alignment(gpu, pad, place, dim):
    check_prompt([200, 77], dim=dim, pad=pad, place=place, behind=2, seed=pad)
    check_prompt([100] * 2, dim=dim, pad=pad, place=place, packed_starts=False, causal=False, seed=pad)


@pytest.mark.gpu
def test_prompt_large_and_ordered_scores(gpu):
    for dtype in ("bf16", "f16"):
        check_prompt([300], dtype=dtype, std=6.0, seed=1)
        check_prompt([300], dtype=dtype, scale=0.0, seed=2)
        check_prompt([300], dtype=dtype, scale=-0.3, seed=3)
    n, dim = 600, 64
    for flip in (False, True):
        k = torch.zeros((1, n, 1, dim), dtype=torch.bfloat16)
        ramp = torch.arange(n).to(torch.bfloat16)
        k[0, :, 0, 0] = ramp.flip(0) if flip else ramp
        q = torch.zeros((1, n, 1, dim), dtype=torch.bfloat16)
        q[..., 0] = 8.0
        v = rand((1, n, 1, dim), 4, torch.bfloat16)
        out = B.convrot_attention(q.cuda(), k.cuda(), v.cuda(), causal=True, scale=1.0)
        want, bound, _, _ = attended(*(t[0].double().transpose(0, 1) for t in (q, k, v)), 1.0, 0, torch.bfloat16)
        close(out[0].transpose(0, 1), want, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_masked_places_stay_out(gpu, bad, where, dim):
    """A value that is no number reaches the queries that see it, and no other."""
    n, at = 400, (5, 130, 215, 399)
    q, k, v = (rand((1, n, 2, dim), 1 + i, torch.bfloat16) for i in range(3))
    clean = B.convrot_attention(q.cuda(), k.cuda(), v.cuda(), causal=True)
    for token in at:
        kk, vv = k.clone(), v.clone()
        (kk if where == "k" else vv)[0, token, 1, 3] = bad
        out = B.convrot_attention(q.cuda(), kk.cuda(), vv.cuda(), causal=True)
        assert torch.equal(out[:, :, 0], clean[:, :, 0])
        before, after = out[0, :token, 1], out[0, token:, 1]
        w = clean[0, :token, 1].double().cpu()
        # the same sums in another order, weights as they are: within a step and the sums' loss
        bound = (n + 16) * 4 * U * v[0, :, 1].double().abs().amax() + 2 * half_step(torch.bfloat16, w.abs())
        close(before, w, bound)
        if where == "v":
            assert not torch.isfinite(after[:, 3].float()).any()
            rest = [c for c in range(dim) if c != 3]
            w = clean[0, token:, 1].double().cpu()[:, rest]
            close(after[:, rest], w, (n + 16) * 4 * U * v[0, :, 1].double().abs().amax() + 2 * half_step(torch.bfloat16, w.abs()))
        elif bad != bad:
            assert after.isnan().all()


@pytest.mark.gpu
def test_prompt_starts_are_cut_to_the_rows(gpu):
    """Starts beyond the rows, descending or negative ones read and write nothing outside."""
    q, k, v = (rand((100, 2, 64), 1 + i, torch.bfloat16).cuda() for i in range(3))
    guard = torch.full((140, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for starts in ([0, 50, 2 ** 31 - 1], [-50, 40, 100], [90, 10, 100], [200, 300, 400], [0, 100, 20]):
        s = torch.tensor(starts, dtype=torch.int32, device="cuda")
        B.convrot_attention(q, k, v, q_starts=s, causal=True, out=guard[20:120])
        assert (guard[:20] == 7).all() and (guard[120:] == 7).all()
    s = torch.tensor([0, 50, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    want = B.convrot_attention(q, k, v, q_starts=torch.tensor([0, 50, 100], dtype=torch.int32, device="cuda"), causal=True)
    assert torch.equal(B.convrot_attention(q, k, v, q_starts=s, causal=True), want)


# ---- together ---------------------------------------------------------------------


@pytest.mark.gpu
def test_a_prompt_and_then_token_by_token(gpu):
    """Rotary positions, the cache and both attentions as a decoder runs them: the rows
    of a prompt's attention are those that its tokens get one by one from the cache,
    whatever the order of its pages."""
    n, hq, hk, dim, page = 150, 8, 2, 128, 16
    dt = torch.bfloat16
    qkv = rand((1, n, hq + 2 * hk, dim), 1, dt).cuda()
    freq, axis = B.rope_frequencies((dim,))
    positions = torch.arange(n, dtype=torch.int32, device="cuda").view(1, n, 1)
    q, k = B.convrot_rope(qkv[:, :, :hq], qkv[:, :, hq:hq + hk], positions, freq, axis, layout="halves")
    v = qkv[:, :, hq + hk:]
    whole = B.convrot_attention(q, k, v, causal=True)[0]
    order = torch.randperm(12, generator=torch.Generator().manual_seed(2)).cuda()
    slots = (order[:, None] * page + torch.arange(page, device="cuda")).flatten()[:n]
    table = order[None].int()
    rows = [t[0].double().cpu().transpose(0, 1) for t in (q, k, v)]
    for kind in ("same", "e4m3", "e2m1"):
        cache = B.new_kv_cache(12, page, hk, dim, dt if kind == "same" else kind)
        B.convrot_cache_write(k[0, :100], v[0, :100], slots[:100], cache)      # the prompt
        for i in range(100, n):                                                # its continuation
            B.convrot_cache_write(k[0, i:i + 1], v[0, i:i + 1], slots[i:i + 1], cache)
            out = B.convrot_attention_paged(q[0, i:i + 1], cache, table, torch.tensor([i + 1], dtype=torch.int32, device="cuda"))
            if i % 7 and i != n - 1:
                continue
            kk, vv = (r[:, :i + 1] if kind == "same" else kept(r[:, :i + 1], kind)[0] for r in rows[1:])
            want, bound, _, _ = attended(rows[0][:, i:i + 1], kk, vv, dim ** -0.5, None, dt)
            close(out[0], want[:, 0], bound[:, 0], f"{kind} token {i}")
            if kind == "same":
                close(whole[i], want[:, 0], bound[:, 0], f"row {i} of the prompt")
        got = B.convrot_cache_read(cache, slots)
        same(got[0], k[0].cpu() if kind == "same" else kept(k[0].cpu(), kind)[0])


@pytest.mark.gpu
def test_attention_graphs_streams_and_repeats(gpu):
    """The same bits from a repeated call, on a stream of its own, and from a captured graph
    replayed beside eager work; lengths and tables are read when it runs."""
    page, hk, hq, dim, b = 16, 2, 8, 128, 5
    cache = new_cache(200, page, hk, dim, "e2m1", "bf16", seed=1)
    table = torch.randperm(200, generator=torch.Generator().manual_seed(1)).int()[:b * 40].view(b, 40).cuda()
    lengths = torch.tensor([640, 3, 0, 333, 128], dtype=torch.int32, device="cuda")
    q = rand((b, hq, dim), 2, torch.bfloat16).cuda()
    new = rand((b, hk, dim), 3, torch.bfloat16).cuda()
    slots = torch.tensor([5, 77, -1, 1000, 31], device="cuda")
    pq, pk, pv = (rand((300, h, dim), 4 + i, torch.bfloat16).cuda() for i, h in enumerate((hq, hk, hk)))
    starts = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device="cuda")

    def run(stream=None):
        B.convrot_cache_write(new, new, slots, cache, stream=stream)
        return (B.convrot_attention_paged(q, cache, table, lengths, stream=stream), *B.convrot_cache_read(cache, slots, stream=stream),
                B.convrot_attention(pq, pk, pv, q_starts=starts, causal=True, stream=stream))

    want = run()
    for _ in range(3):
        assert all(torch.equal(a, w) for a, w in zip(run(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, w) for a, w in zip(got, want))
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = run()
    for step in range(4):
        lengths.copy_(torch.tensor([640 - 100 * step, 3 + step, step, 333, 128 + 200 * step], dtype=torch.int32))
        new.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in captured]
        eager = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for a, w in zip(replayed, eager)), step


@pytest.mark.gpu
def test_attention_workspaces_of_captured_graphs(gpu):
    """Calls that join partial results, captured in two graphs that are replayed in turn and
    beside eager calls, each with a workspace of its own: none meets another's."""
    page, hk, hq, dim = 64, 2, 8, 128
    cache = new_cache(130, page, hk, dim, "same", "bf16", seed=1)
    runs = []
    for g in range(2):
        table = torch.randperm(130, generator=torch.Generator().manual_seed(g)).int().view(2, 65).cuda()
        lengths = torch.tensor([4100, 777 + g], dtype=torch.int32, device="cuda")
        q = rand((2, hq, dim), 10 + g, torch.bfloat16).cuda()
        pq, pk, pv = (rand((1, n, h, dim), 20 + 3 * g + i, torch.bfloat16).cuda() for i, (n, h) in enumerate(((40, hq), (3000, hk), (3000, hk))))
        runs.append((lambda q=q, table=table, lengths=lengths: B.convrot_attention_paged(q, cache, table, lengths),
                     lambda pq=pq, pk=pk, pv=pv: B.convrot_attention(pq, pk, pv, causal=True), lengths))
    want = [(a(), b()) for a, b, _ in runs]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for a, b, _ in runs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs.append((a(), b()))
        graphs.append(graph)
    for step in range(4):
        for g in ((0, 1), (1, 0))[step % 2]:
            graphs[g].replay()
        eager = [(a(), b()) for a, b, _ in runs]
        torch.cuda.synchronize()
        for g in range(2):
            assert torch.equal(outs[g][0], eager[g][0]) and torch.equal(outs[g][1], want[g][1]) and torch.equal(eager[g][1], want[g][1])
        assert step or torch.equal(eager[0][0], want[0][0])
        runs[step % 2][2][0] = 4100 - 1000 * step      # lengths are read when a graph runs


@pytest.mark.gpu
def test_prompt_broadcast_keys(gpu):
    """Keys and values of stride 0: one token's for all, one batch entry's for all, one head's for all."""
    n, dim = 150, 64
    q, one, two = (rand(s, 1 + i, torch.bfloat16) for i, s in enumerate(((2, n, 4, dim), (1, n, 1, dim), (2, n, 1, dim))))
    for kv in (one.cuda().expand(2, n, 2, dim), one[:, :1].cuda().expand(2, n, 2, dim), two.cuda().expand(2, n, 4, dim)):
        assert 0 in kv.stride()
        for causal in (False, True):
            out = B.convrot_attention(q.cuda(), kv, kv, causal=causal)
            for b in range(2):
                rows = [t[b].double().transpose(0, 1) for t in (q, kv.cpu(), kv.cpu())]
                want, bound, _, _ = attended(*rows, dim ** -0.5, 0 if causal else None, torch.bfloat16)
                close(out[b].transpose(0, 1), want, bound)


@pytest.mark.gpu
def test_caches_keep_their_memory(gpu):
    """A handle keeps the memory that it was made of."""
    cache = B.new_kv_cache(4, 8, 2, 64, torch.bfloat16)
    x = rand((32, 2, 64), 1, torch.bfloat16).cuda()
    slots = torch.arange(32, device="cuda")
    cache.k.data = torch.empty(0, dtype=torch.bfloat16, device="cuda")
    others = [torch.full((4, 2, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    B.convrot_cache_write(x, x, slots, cache)
    assert torch.equal(B.convrot_cache_read(cache, slots)[0], x) and all((t == 7).all() for t in others)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e2m1", "same"])
def test_caches_of_resized_memory_are_refused(gpu, kind):
    x = rand((2, 2, 64), 1, torch.bfloat16).cuda()
    slots = torch.arange(2, device="cuda")
    for i in range(4 if kind == "e2m1" else 2):
        cache = new_cache(4, 8, 2, 64, kind, "bf16", seed=1)
        tuple(cache)[i].untyped_storage().resize_(0)
        for call in (lambda: B.convrot_cache_write(x, x, slots, cache), lambda: B.convrot_cache_read(cache, slots),
                     lambda: B.convrot_attention_paged(x, cache, slots.int()[:, None], slots.int())):
            with pytest.raises(ValueError):
                call()


@pytest.mark.gpu
def test_attention_outputs_and_workspaces_given(gpu):
    q, k, v = (rand((2, 90, 4, 64), 1 + i, torch.bfloat16).cuda() for i in range(3))
    wide = torch.full((2, 4, 90, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = B.convrot_attention(q, k, v)
    lse = torch.empty((2, 90, 4), device="cuda")
    version = wide._version
    got = B.convrot_attention(q, k, v, out=wide.transpose(1, 2), lse=lse)
    assert got[0].data_ptr() == wide.data_ptr() and torch.equal(got[0], out) and got[1] is lse and wide._version > version
    cache = new_cache(130, 16, 4, 64, "same", "bf16", seed=5)
    table = torch.arange(130, dtype=torch.int32, device="cuda").view(1, 130)     # wide enough for shares of the keys
    n = torch.tensor([640], dtype=torch.int32, device="cuda")
    want = B.convrot_attention_paged(q[0, :1], cache, table, n)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    assert torch.equal(B.convrot_attention_paged(q[0, :1], cache, table, n, workspace=ws, out=torch.empty_like(want)), want)
    with pytest.raises(B.ConvRotError) as e:
        B.convrot_attention_paged(q[0, :1], cache, table, n, workspace=ws[:16])
    assert e.value.status == B.CONVROT_EWORKSPACE


@pytest.mark.gpu
def test_attention_empty_calls(gpu):
    dt = torch.bfloat16
    cache = B.new_kv_cache(2, 8, 2, 64, "e4m3")
    none = torch.empty((0, 2, 64), dtype=dt, device="cuda")
    slots = torch.empty((0,), dtype=torch.int64, device="cuda")
    B.convrot_cache_write(none, none, slots, cache)
    assert B.convrot_cache_read(cache, slots)[0].shape == (0, 2, 64)
    ints = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    assert B.convrot_attention_paged(none, cache, ints, ints[:, 0].contiguous()).shape == (0, 2, 64)
    q = rand((2, 4, 64), 1, dt).cuda()
    wide = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    out, lse = B.convrot_attention_paged(q, cache, wide, torch.tensor([5, 0], dtype=torch.int32, device="cuda"), want_lse=True)
    assert not out.any() and (lse == -math.inf).all()
    assert B.convrot_attention(none[None], none[None], none[None]).shape == (1, 0, 2, 64)
    out, lse = B.convrot_attention(q[None], none[None], none[None], want_lse=True)
    assert not out.any() and (lse == -math.inf).all()
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert B.convrot_attention(q, none, none, q_starts=zero).shape == q.shape      # no sequences


@pytest.mark.gpu
@pytest.mark.parametrize("batch,T,hidden,head_dim", [(1, 130, 256, 128), (3, 77, 192, 64)])
def test_blocks_with_the_librarys_attention(gpu, batch, T, hidden, head_dim):
    """The blocks' attention against the formula on the heads that they make, and the blocks
    against themselves: the attended values, their bf16 roundings and sums are all that differ."""
    from w4a4_rotated_bit_amd.flux_block import Block, ConditionedBlock, picture, rel_err, tokens
    plain = ConditionedBlock(hidden, head_dim=head_dim).to(torch.bfloat16).cuda()
    blk = ConditionedBlock(hidden, head_dim=head_dim, attention="library").to(torch.bfloat16).cuda()
    x = tokens(batch * T, hidden).view(batch, T, hidden).cuda()
    vec, pos = tokens(batch, hidden, seed=9).cuda(), picture(T, batch).cuda()
    with torch.no_grad():
        q, k, v = blk.qkv(x).view(batch, T, 3, blk.heads, head_dim).unbind(2)
        got = B.convrot_attention(q, k, v)
        for b in range(batch):
            rows = [t[b].double().cpu().transpose(0, 1) for t in (q, k, v)]
            want, bound, _, _ = attended(*rows, head_dim ** -0.5, None, torch.bfloat16)
            close(got[b].transpose(0, 1), want, bound)
        # the attended values fall to another step of 2^-8 at most here and there, and so
        # may what is computed from them: the two sums, the norm between, the projections' outputs
        assert rel_err(blk(x, vec, pos), plain(x, vec, pos)) <= 6 * 2.0 ** -8
        one = Block(hidden, head_dim, attention="library").to(torch.bfloat16).cuda()
        two = Block(hidden, head_dim).to(torch.bfloat16).cuda()
        one.modulation, two.modulation = one.modulation.float(), two.modulation.float()
        assert rel_err(one(x[0]), two(x[0])) <= 6 * 2.0 ** -8
    with pytest.raises(ValueError):
        Block(hidden, head_dim, attention="other")


# ---- refusals ---------------------------------------------------------------------

CACHE = dict(k_rows=P, k_scales=P + (1 << 20), k_page=1 << 12, k_head=1 << 10, k_token=64, k_spage=256, k_shead=64, k_stoken=4,
             v_rows=P + (2 << 20), v_scales=P + (3 << 20), v_page=1 << 12, v_head=1 << 10, v_token=64, v_spage=256, v_shead=64, v_stoken=4,
             pages=100, page_size=16, heads=4, head_dim=128, kind=B.CONVROT_CACHE_E2M1)
SAME = dict(k_scales=0, v_scales=0, kind=1, k_page=1 << 14, k_head=1 << 12, k_token=256, v_page=1 << 14, v_head=1 << 12, v_token=256,
            v_rows=P + (2 << 20))
BAD_CACHE = [{"pages": 0}, {"pages": 1 << 31}, {"page_size": 4}, {"page_size": 24}, {"page_size": 1 << 17}, {"heads": 0}, {"heads": 65536},
             {"head_dim": 0}, {"head_dim": 48}, {"head_dim": 288}, {"kind": 3}, {"kind": 0}, {"k_rows": 0}, {"v_rows": 0},
             {"k_rows": P + 8}, {"k_scales": 0}, {"v_scales": 0}, {"k_token": 72}, {"v_head": 1000}, {"k_page": -4096}, {"k_token": -64},
             {"k_spage": -1}, {"k_page": 1 << 51}, {"k_token": (1 << 27) + 16}, {"v_stoken": (1 << 27) + 1}, {**SAME, "k_scales": P}, {**SAME, "head_dim": 12}]


@pytest.mark.parametrize("kw,write,read", [
    ({}, True, True), ({"tokens": 0, "k": 0, "v": 0, "slots": 0}, True, True), ({"dtype": 2}, True, True), ({"dtype": 3}, False, False),
    ({"slots_dtype": 4}, True, True), ({"slots_dtype": 3}, False, False), ({"tokens": -1}, False, False), ({"tokens": (1 << 24) + 1}, False, False),
    ({"k": 0}, False, False), ({"v": 0}, False, False), ({"slots": 0}, False, False), ({"k": P + (16 << 20) + 1}, False, False),
    ({"slots": P + (48 << 20) + 4}, False, False), ({"slots": P + (48 << 20) + 4, "slots_dtype": 4}, True, True),
    ({"k_head_stride": -1}, False, False), ({"v_token_stride": 1 << 50}, False, False), ({"k_token_stride": 0}, True, False),
    ({"v": P + (16 << 20) + 128}, True, False), ({"k": P + 4096}, False, False), ({"v": P + (1 << 20) + 256}, False, False),
    ({"k_token": 48}, False, True), ({"v_rows": P + 64}, False, True), ({"v_scales": P + (1 << 20) + 8}, False, True),
    ({"slots": P + (16 << 20)}, True, False), ({"slots": P + 8}, False, True),
    (SAME, True, True), ({**SAME, "dtype": 2}, False, False), ({**SAME, "kind": 2}, False, False), ({**SAME, "kind": 2, "dtype": 2}, True, True),
    ({**SAME, "head_dim": 72}, True, True), *[(kw, False, False) for kw in BAD_CACHE],
])
def test_cache_refusals(kw, write, read):
    a = packed(B.CACHE_ARGS, dict(**CACHE, k=P + (16 << 20), v=P + (32 << 20), slots=P + (48 << 20), tokens=50, k_token_stride=512,
                                  k_head_stride=128, v_token_stride=512, v_head_stride=128, slots_dtype=B.CONVROT_I64, dtype=1), kw)
    lib = B.load()
    assert lib.convrot_validate_cache_write(a) == (B.CONVROT_OK if write else B.CONVROT_EINVAL)
    assert lib.convrot_validate_cache_read(a) == (B.CONVROT_OK if read else B.CONVROT_EINVAL)
    if not write:
        assert lib.convrot_cache_write(a, None) == B.CONVROT_EINVAL
    if not read:
        assert lib.convrot_cache_read(a, None) == B.CONVROT_EINVAL


@pytest.mark.parametrize("kw,ok", [
    ({}, True), ({"batch": 0, "q": 0, "o": 0, "lengths": 0}, True), ({"batch": -1}, False), ({"batch": 65536}, False), ({"lse": 0}, True),
    ({"q_heads": 6}, False), ({"q_heads": 0}, False), ({"q_heads": 65536}, False), ({"q_heads": 4}, True), ({"dtype": 3}, False),
    ({"dtype": 2}, True), ({"reserved": 1}, False), ({"scale": float("nan")}, False), ({"scale": float("inf")}, False), ({"scale": -1.0}, True),
    ({"table_width": -1}, False), ({"table_width": (1 << 26) + 1}, False), ({"table_width": 0, "table": 0}, True), ({"table": 0}, False),
    ({"table": P + (36 << 20) + 2}, False), ({"table_stride": 0}, True), ({"table_stride": -64}, False), ({"lengths": 0}, False),
    ({"lengths": P + (40 << 20) + 1}, False), ({"q": 0}, False), ({"o": 0}, False), ({"q": P + (16 << 20) + 1}, False), ({"lse": P + (34 << 20) + 2}, False),
    ({"o_head_stride": 64}, False), ({"o_batch_stride": 0}, False), ({"q_batch_stride": 0}, True), ({"q_head_stride": -1}, False),
    ({"o": P + (16 << 20)}, False), ({"o": P}, False), ({"lse": P + (2 << 20)}, False), ({"lse": P + (32 << 20)}, False),
    ({"o": P + (36 << 20)}, False), ({"lse": P + (40 << 20)}, False),
    *[({"batch": 2048, "q_heads": n, "heads": n, "k_page": 1 << 24, "v_page": 1 << 24, "q": 1 << 40, "o": 2 << 40, "o_batch_stride": 1 << 20,
        "k_rows": 3 << 40, "v_rows": 4 << 40, "k_scales": 5 << 40, "v_scales": 6 << 40, "lse": 7 << 40}, n < 4096) for n in (4095, 4096)],
    (SAME, True), ({**SAME, "dtype": 2}, False),
    *[(kw, False) for kw in BAD_CACHE],
])
def test_paged_refusals(kw, ok):
    import ctypes
    a = packed(B.PAGED_ARGS, dict(**CACHE, q=P + (16 << 20), o=P + (32 << 20), lse=P + (34 << 20), table=P + (36 << 20), lengths=P + (40 << 20), batch=3,
                                  table_width=64, table_stride=64, q_batch_stride=1024, q_head_stride=128, o_batch_stride=1024, o_head_stride=128,
                                  q_heads=8, dtype=1, scale=0.1, reserved=0), kw)
    lib, need = B.load(), ctypes.c_size_t(0)
    rc = lib.convrot_attention_paged_workspace_bytes(a, ctypes.byref(need))
    assert rc == (B.CONVROT_OK if ok else B.CONVROT_EINVAL)
    if not ok:
        assert lib.convrot_attention_paged(a, P, 1 << 40, None) == B.CONVROT_EINVAL
        return
    assert lib.convrot_validate_attention_paged(a, P + (64 << 20), need.value) == B.CONVROT_OK
    if need.value:
        assert lib.convrot_attention_paged(a, P + (64 << 20), need.value - 1, None) == B.CONVROT_EWORKSPACE
        assert lib.convrot_attention_paged(a, None, need.value, None) == B.CONVROT_EWORKSPACE
        assert lib.convrot_attention_paged(a, P + (64 << 20) + 8, need.value, None) == B.CONVROT_EINVAL


@pytest.mark.parametrize("kw,ok", [
    ({}, True), ({"batch": 0, "q": 0, "k": 0, "v": 0, "o": 0}, True), ({"q_tokens": 0, "q": 0, "o": 0}, True), ({"batch": 65536}, False),
    ({"batch": -1}, False), ({"q_tokens": -1}, False), ({"q_tokens": (1 << 24) + 1}, False), ({"k_tokens": (1 << 24) + 1}, False),
    ({"k_tokens": 0, "k": 0, "v": 0}, True), ({"q_heads": 5}, False), ({"k_heads": 0}, False), ({"k_heads": 16}, False), ({"q_heads": 0}, False),
    ({"head_dim": 12}, False), ({"head_dim": 264}, False), ({"head_dim": 0}, False), ({"head_dim": 56}, True), ({"causal": 2}, False),
    ({"causal": 1}, True), ({"dtype": 3}, False), ({"dtype": 2}, True), ({"scale": float("nan")}, False), ({"q_starts": P + (64 << 20)}, False),
    ({"q_starts": P + (64 << 20), "k_starts": P + (65 << 20)}, True), ({"q_starts": P + (64 << 20) + 2, "k_starts": P + (65 << 20)}, False),
    ({"q": 0}, False), ({"k": 0}, False), ({"v": 0}, False), ({"o": 0}, False), ({"q": P + 1}, False), ({"k": P + (16 << 20) + 1}, False),
    ({"k": P + (16 << 20) + 2}, True), ({"lse": 0}, True), ({"lse": P + (56 << 20) + 2}, False), ({"k_token_stride": 1 << 24}, False),
    ({"v_token_stride": (1 << 24) - 1, "v": 1 << 40}, True), ({"q_token_stride": 1 << 24}, False), ({"q_token_stride": 1 << 24, "q": 1 << 40}, True), ({"o_head_stride": 32}, False),
    ({"o_token_stride": 0}, False), ({"k_head_stride": 0, "k_batch_stride": 0}, True), ({"v_batch_stride": -1}, False), ({"o": P}, False),
    ({"o": P + (16 << 20)}, False), ({"lse": P + (48 << 20)}, False), ({"lse": P}, False),
    ({"q_starts": P + (48 << 20), "k_starts": P + (65 << 20)}, False),
    *[({"batch": 4096, "q_heads": n, "k_heads": 1, "q": 1 << 40, "o": 2 << 40, "o_batch_stride": 1 << 25, "o_token_stride": 1 << 18,
        "lse": 3 << 40}, n < 4096) for n in (4095, 4096)],
])
def test_prompt_refusals(kw, ok):
    import ctypes
    a = packed(B.ATTENTION_ARGS, dict(q=P, k=P + (16 << 20), v=P + (32 << 20), o=P + (48 << 20), lse=P + (56 << 20), q_starts=0, k_starts=0, batch=2,
                                      q_tokens=100, k_tokens=70, q_batch_stride=51200, q_token_stride=512, q_head_stride=64,
                                      k_batch_stride=17920, k_token_stride=256, k_head_stride=64, v_batch_stride=17920,
                                      v_token_stride=256, v_head_stride=64, o_batch_stride=51200, o_token_stride=512, o_head_stride=64,
                                      q_heads=8, k_heads=4, head_dim=64, causal=0, dtype=1, scale=0.1), kw)
    lib, need = B.load(), ctypes.c_size_t(0)
    assert lib.convrot_attention_workspace_bytes(a, ctypes.byref(need)) == (B.CONVROT_OK if ok else B.CONVROT_EINVAL)
    if ok:
        assert lib.convrot_validate_attention(a, P + (128 << 20), need.value) == B.CONVROT_OK
    else:
        assert lib.convrot_attention(a, P + (128 << 20), 1 << 40, None) == B.CONVROT_EINVAL


def test_attention_null_arguments_are_refused():
    import ctypes
    lib, n = B.load(), ctypes.c_size_t(0)
    assert lib.convrot_cache_write(None, None) == lib.convrot_cache_read(None, None) == B.CONVROT_EINVAL
    assert lib.convrot_attention(None, None, 0, None) == lib.convrot_attention_paged(None, None, 0, None) == B.CONVROT_EINVAL
    assert lib.convrot_attention_workspace_bytes(None, ctypes.byref(n)) == B.CONVROT_EINVAL
    assert lib.convrot_attention_paged_workspace_bytes(None, ctypes.byref(n)) == B.CONVROT_EINVAL


def test_attention_needs_device_tensors():
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: B.convrot_attention(x[None], x[None], x[None]),
                 lambda: B.convrot_cache_write(x, x, torch.zeros(2, dtype=torch.int64), B.new_kv_cache(1, 8, 2, 64, device="cpu")),
                 lambda: B.convrot_attention_paged(x, B.new_kv_cache(1, 8, 2, 64, device="cpu"), None, None)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        B.convrot_attention([1.0], x, x)
    with pytest.raises(ValueError):
        B.new_kv_cache(1, 8, 2, 64, kind="int4", device="cpu")
    with pytest.raises(ValueError):
        B.new_kv_cache(1, 8, 2, 72, device="cpu")


@pytest.mark.gpu
def test_attention_binding_refusals(gpu):
    dt = torch.bfloat16
    x = torch.zeros((4, 2, 64), dtype=dt, device="cuda")
    cache, plain = B.new_kv_cache(3, 8, 2, 64, "e2m1"), B.new_kv_cache(3, 8, 2, 64, dt)
    slots = torch.arange(4, device="cuda")
    table, n = torch.zeros((4, 3), dtype=torch.int32, device="cuda"), torch.ones(4, dtype=torch.int32, device="cuda")
    four = x[None]
    starts = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    asks = x.clone().requires_grad_()
    value, kind = (ValueError, B.ConvRotError), TypeError
    for error, call in [
        (kind, lambda: B.convrot_cache_write(x.float(), x.float(), slots, cache)),
        (kind, lambda: B.convrot_cache_write(x.half(), x.half(), slots, plain)),
        (value, lambda: B.convrot_cache_write(x, x[:3], slots, cache)),
        (value, lambda: B.convrot_cache_write(x[:, :1], x, slots, cache)),
        (value, lambda: B.convrot_cache_write(x, x, slots[:3], cache)),
        (kind, lambda: B.convrot_cache_write(x, x, slots.float(), cache)),
        (value, lambda: B.convrot_cache_write(x, x, slots.cpu(), cache)),
        (value, lambda: B.convrot_cache_write(x, x, slots, cache._replace(v=cache.v[:2]))),
        (kind, lambda: B.convrot_cache_write(x, x, slots, cache._replace(k=cache.k.int(), v=cache.v.int()))),
        (value, lambda: B.convrot_cache_write(x, x, slots, cache._replace(k_scales=cache.k_scales[:2]))),
        (kind, lambda: B.convrot_cache_write(x, x, slots, cache._replace(k_scales=None))),
        (value, lambda: B.convrot_cache_write(x, x, slots, plain._replace(k_scales=cache.k_scales))),
        (value, lambda: B.convrot_cache_write(x, x, slots, plain._replace(v=plain.k))),
        (value, lambda: B.convrot_cache_write(x, x, slots, B.KVCache(x[None], x[None]))),
        (RuntimeError, lambda: B.convrot_cache_write(asks, x, slots, cache)),
        (kind, lambda: B.convrot_cache_read(plain, slots, dtype=torch.float16)),
        (kind, lambda: B.convrot_cache_read(cache, slots, dtype=torch.float32)),
        (value, lambda: B.convrot_cache_read(cache, slots, k=x[:2])),
        (value, lambda: B.convrot_cache_read(cache, slots, k=x, v=x)),
        (kind, lambda: B.convrot_attention_paged(x.half(), plain, table, n)),
        (value, lambda: B.convrot_attention_paged(x[..., :32], cache, table, n)),
        (value, lambda: B.convrot_attention_paged(torch.zeros((4, 3, 64), dtype=dt, device="cuda"), cache, table, n)),
        (kind, lambda: B.convrot_attention_paged(x, cache, table.long(), n)),
        (kind, lambda: B.convrot_attention_paged(x, cache, table, n.long())),
        (value, lambda: B.convrot_attention_paged(x, cache, table[:2], n)),
        (value, lambda: B.convrot_attention_paged(x, cache, table, n, out=x)),
        (value, lambda: B.convrot_attention_paged(x, cache, table, n, lse=torch.empty((4, 3), device="cuda"))),
        (RuntimeError, lambda: B.convrot_attention_paged(asks, cache, table, n)),
        (value, lambda: B.convrot_attention(x, x, x)),
        (value, lambda: B.convrot_attention(four, four, four, q_starts=starts)),
        (value, lambda: B.convrot_attention(four, four, four, k_starts=starts)),
        (kind, lambda: B.convrot_attention(x, x, x, q_starts=starts.long())),
        (value, lambda: B.convrot_attention(x, x, x, q_starts=starts, k_starts=starts[:1])),
        (kind, lambda: B.convrot_attention(four, four.half(), four)),
        (value, lambda: B.convrot_attention(four, four[:, :, :1], four)),
        (value, lambda: B.convrot_attention(four, four.expand(2, 4, 2, 64), four.expand(2, 4, 2, 64))),
        (value, lambda: B.convrot_attention(four, four, four, out=four)),
        (value, lambda: B.convrot_attention(four.transpose(2, 3), four.transpose(2, 3), four.transpose(2, 3))),
        (RuntimeError, lambda: B.convrot_attention(asks[None], four, four)),
    ]:
        with pytest.raises(error):
            call()
    with torch.no_grad():
        B.convrot_attention(asks[None], four, four)
