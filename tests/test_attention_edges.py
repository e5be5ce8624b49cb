"""Attention and its paged cache where they are easily wrong, against the formula in binary64.

u = 2^-24 is half a step of binary32 relative to the value; a softmax weight and an
output are each rounded to the heads' type (half a step, finfo.eps / 2 of it).  Weights
in f16 are 2^11 where the largest is 1, so the half step of its subnormals, 2^-25, is
2^-36 of that one."""
import ctypes
import math
from contextlib import nullcontext
from types import SimpleNamespace

import pytest
import torch

from w4a4_rotated_bit_amd import binding as B

from .test_attention import check_prompt, kept, new_cache, same
from .test_block_ops import TYPES, U, close, half_step, packed, rand

FLAT = {torch.float16: 2.0 ** -36, torch.bfloat16: 0.0}   # half a step of the smallest weights


def formula(q, k, v, scale, dtype, seen=None):
    """(out, its bound, lse, its bound) of q [rows, dim], k, v [keys, dim] in binary64."""
    n, dim = k.shape
    s = (q @ k.T) * scale
    slack = (dim + 4) * U * (q.abs() @ k.abs().T) * abs(scale) + 8 * U * (1 + s.abs())
    if seen is not None:
        s, slack = s.masked_fill(~seen, -math.inf), slack.masked_fill(~seen, 0.0)
    w = torch.softmax(s, -1)
    lost = slack.amax(-1, keepdim=True)
    out = w @ v
    share = torch.exp(s.amax(-1, keepdim=True) - torch.logsumexp(s, -1, keepdim=True))    # of the largest weight
    bound = (w @ v.abs()) * (2 * lost + torch.finfo(dtype).eps / 2 + 2 * (n + 16) * U)
    bound = bound + FLAT[dtype] * share * ((torch.ones_like(s) if seen is None else seen.double()) @ v.abs())
    lse = torch.logsumexp(s, -1)
    return out, bound + half_step(dtype, out.abs() + bound), lse, lost[:, 0] + (n + 16) * U + 4 * U * (1 + lse.abs())


def paged(q, k, v, scale, page=16, wide=0):
    """q [rows, dim] as that many query heads of one key head over a cache of k, v [keys, dim]."""
    n, dim = k.shape
    pages = -(-n // page)
    cache = B.new_kv_cache(pages, page, 1, dim, k.dtype)
    B.convrot_cache_write(k[:, None].cuda(), v[:, None].cuda(), torch.arange(n, device="cuda"), cache)
    table = torch.full((1, pages + wide), -1, dtype=torch.int32)
    table[0, :pages] = torch.arange(pages)
    out, lse = B.convrot_attention_paged(q[None].cuda(), cache, table.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"),
                                         scale=scale, want_lse=True)
    return out[0], lse[0]


def prompt(q, k, v, scale, causal=False):
    out, lse = B.convrot_attention(q[None, :, None].cuda(), k[None, :, None].cuda(), v[None, :, None].cuda(), scale=scale,
                                   causal=causal, want_lse=True)
    return out[0, :, 0], lse[0, :, 0]


# ---- weights far below the largest ---------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("gap", [10.0, 15.0, 17.0, 17.5, 19.0])
@pytest.mark.parametrize("where", ["first", "last", "often"])
def test_many_keys_far_below_one_of_no_value(gpu, dtype, gap, where):
    """A key that takes nearly all of the weight and whose value is zero: the output is what
    many small weights leave."""
    dt, dim = TYPES[dtype], 64
    for n, rows, call in ((32768, 5, prompt), (32768, 130, prompt), (700, 3, prompt), (380, 4, paged), (30000, 4, paged)):
        q, k = torch.zeros((rows, dim), dtype=dt), torch.zeros((n, dim), dtype=dt)
        v = (1 + rand((n, dim), 1, torch.float32, 0.25)).to(dt)
        q[:, 0], k[:, 1] = 1, rand((n,), 2, dt, 0.5)
        q[:, 1] = 1
        top = {"first": slice(0, 1), "last": slice(n - 1, n), "often": slice(0, n, 32)}[where]
        k[top, 0], k[top, 1], v[top] = gap, 0, 0
        got, lse = call(q, k, v, 1.0)
        want, bound, want_lse, lse_bound = formula(q.double(), k.double(), v.double(), 1.0, dt)
        close(got, want, bound, f"{call.__name__} of {n} keys")
        close(lse, want_lse, lse_bound, f"lse of {n} keys")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_scores_that_rise_step_by_step(gpu, dtype):
    """Steps of keys whose scores rise by less and by more than the running reference's room."""
    dt, n, dim = TYPES[dtype], 640, 64
    for rise in (1.0, 2.5, 2.75, 3.0, 5.5, 8.0, 10.25, 10.5, 11.0):    # 4, 8 and 15 in base 2 are 2.77, 5.55 and 10.4
        q, k = torch.zeros((40, dim), dtype=dt), torch.zeros((n, dim), dtype=dt)
        q[:, 0], k[:, 0] = 1, (torch.arange(n) // 64 * rise).to(dt)
        v = rand((n, dim), 3, dt)
        for call, rows in ((prompt, 40), (paged, 3)):
            got, lse = call(q[:rows], k, v, 1.0)
            want, bound, want_lse, lse_bound = formula(q[:rows].double(), k.double(), v.double(), 1.0, dt)
            close(got, want, bound, f"{call.__name__}, {rise} a step")
            close(lse, want_lse, lse_bound, f"{call.__name__}, lse")
        got, lse = prompt(q, k, v, 1.0, causal=True)
        seen = torch.arange(n)[None] <= torch.arange(40)[:, None] + n - 40
        want, bound, want_lse, lse_bound = formula(q.double(), k.double(), v.double(), 1.0, dt, seen)
        close(got, want, bound, "causal")
        close(lse, want_lse, lse_bound, "causal, lse")


# ---- scores whose steps in binary32 are large ------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,power", [(t, p) for t in ("f16", "bf16") for p in (20, 24, 27, 29, 40, 100) if p < 30 or t == "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_scores(gpu, dtype, sign, power):
    """Scores so far apart that the largest takes all of the weight, or two of one size half each;
    magnitudes at which binary32 no longer tells a score from the next whole number."""
    dt, n, dim = TYPES[dtype], 450, 64
    for seed in range(4):
        top = (7 + 53 * seed) % n
        q, k = torch.zeros((130, dim), dtype=dt), torch.zeros((n, dim), dtype=dt)
        q[:, 0] = sign * 2.0 ** (power // 2) * (1 + torch.arange(130) % 8 / 8)
        steps = torch.randint(1, 64, (n,), generator=torch.Generator().manual_seed(seed)) / 128
        k[:, 0] = 2.0 ** (power - power // 2) * (1 + (steps if sign < 0 else 0.75 - steps))
        k[top, 0] = 2.0 ** (power - power // 2) * (1.875 if sign > 0 else 1.0)
        twin = (top + 200) % n
        if seed % 2:
            k[twin] = k[top]
        v = rand((n, dim), 5 + seed, dt)
        want = ((v[top].double() + v[twin].double()) / 2 if seed % 2 else v[top].double()).expand(130, dim)
        bound = half_step(dt, want.abs()) + (4 * U + torch.finfo(dt).eps / 2) * (v[top].double().abs() + v[twin].double().abs())
        want_lse = q[:, 0].double() * k[top, 0].double() + math.log(1 + seed % 2)
        for call, rows in ((prompt, 130), (prompt, 3), (paged, 3)):
            got, lse = call(q[:rows], k, v, 1.0)
            close(got, want[:rows], bound[:rows], f"{call.__name__}, {rows} rows, key {top}")
            close(lse, want_lse[:rows], 8 * U * (1 + want_lse[:rows].abs()), "lse")
        got, lse = prompt(q, k, v, 1.0, causal=True)        # rows from the one whose last key is `top` on see it
        first = max(top if not seed % 2 else max(top, twin), n - 130) - (n - 130)
        close(got[first:], want[first:], bound[first:], f"causal, key {top}")
        close(lse[first:], want_lse[first:], 8 * U * (1 + want_lse[first:].abs()), "causal, lse")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("base", [22, 24, 25, 26, 27, 28])
def test_scores_one_step_of_binary32_apart(gpu, dtype, base):
    """Scores in base 2 of 2^base and a few steps of binary32 more: the reference of the weights
    may not lag by a rounding of its own."""
    dt, n, dim = TYPES[dtype], 384, 64
    scale = 0.6931471805599453      # times log2(e), both in binary32: 1
    assert (torch.tensor(scale) * torch.tensor(1.4426950408889634)).item() == 1.0
    step = 2.0 ** (base - 23)
    q, k = torch.zeros((3, dim), dtype=dt), torch.zeros((n, dim), dtype=dt)
    q[:, 0], q[:, 1] = 2.0 ** (base - 13), 1
    k[:, 0] = 2.0 ** 13
    for ramp in ((torch.arange(n) // 64).float(), (torch.arange(n) // 256 + 1).float(), 6 - (torch.arange(n) // 64).float()):
        k[:, 1] = ramp * step
        v = rand((n, dim), base, dt)
        w = torch.softmax(ramp.double() * step * math.log(2.0), 0)
        want = (w @ v.double()).expand(3, dim)
        bound = (w @ v.double().abs()) * (torch.finfo(dt).eps / 2 + 2 * (n + 16) * U) + FLAT[dt] * v.double().abs().sum(0)
        bound = bound + half_step(dt, want.abs() + bound)
        for call in (prompt, paged):
            close(call(q, k, v, scale)[0], want, bound, f"{call.__name__} {ramp[:2].tolist()}")


# ---- refusals ------------------------------------------------------------------------

P = 1 << 32
BF16_CACHE = dict(k_rows=P, k_scales=0, k_page=1 << 14, k_head=1 << 12, k_token=256, k_spage=0, k_shead=0, k_stoken=0,
                  v_rows=P + (2 << 20), v_scales=0, v_page=1 << 14, v_head=1 << 12, v_token=256, v_spage=0, v_shead=0, v_stoken=0,
                  pages=100, page_size=16, heads=4, head_dim=128, kind=1)


def paged_args(**kw):
    return packed(B.PAGED_ARGS, dict(**BF16_CACHE, q=P + (16 << 20), o=P + (32 << 20), lse=P + (34 << 20), table=P + (36 << 20),
                                     lengths=P + (40 << 20), batch=3, table_width=64, table_stride=64, q_batch_stride=1024, q_head_stride=128,
                                     o_batch_stride=1024, o_head_stride=128, q_heads=8, dtype=1, scale=0.1, reserved=0), kw)


def prompt_args(**kw):
    return packed(B.ATTENTION_ARGS, dict(q=P, k=P + (16 << 20), v=P + (32 << 20), o=P + (48 << 20), lse=P + (56 << 20), q_starts=P + (60 << 20),
                                         k_starts=P + (61 << 20), batch=2, q_tokens=40, k_tokens=4000, q_batch_stride=0, q_token_stride=512,
                                         q_head_stride=64, k_batch_stride=0, k_token_stride=256, k_head_stride=64, v_batch_stride=0,
                                         v_token_stride=256, v_head_stride=64, o_batch_stride=0, o_token_stride=512, o_head_stride=64,
                                         q_heads=8, k_heads=4, head_dim=64, causal=1, dtype=1, scale=0.1), kw)


CALLS = [("convrot_attention_paged", paged_args), ("convrot_attention", prompt_args)]


def workspace_bytes(lib, name, args):
    need = ctypes.c_size_t(0)
    assert getattr(lib, name + "_workspace_bytes")(args, ctypes.byref(need)) == B.CONVROT_OK
    return need.value


@pytest.mark.parametrize("name,args", CALLS)
@pytest.mark.parametrize("scale,ok", [(2.3e38, True), (-2.3e38, True), (2.4e38, False), (-2.4e38, False), (3.4e38, False), (1e-45, True)])
def test_scales_that_overflow_in_base_2_are_refused(name, args, scale, ok):
    """Scores are computed times scale log2(e), which has to be a number of binary32 too."""
    lib = B.load()
    n = workspace_bytes(lib, name, args())
    a = args(scale=scale)
    assert getattr(lib, "convrot_validate_" + name[8:])(a, P + (128 << 20), n) == (B.CONVROT_OK if ok else B.CONVROT_EINVAL)
    if not ok:
        assert getattr(lib, name)(a, P + (128 << 20), n, None) == B.CONVROT_EINVAL


@pytest.mark.parametrize("name,args", CALLS)
def test_workspaces_that_meet_a_tensor_are_refused(name, args):
    """A workspace is written while inputs are read, and read while outputs are written."""
    lib = B.load()
    a = args()
    n = workspace_bytes(lib, name, a)
    assert n
    check = getattr(lib, "convrot_validate_" + name[8:])
    if name == "convrot_attention_paged":
        tensors = [(P, 99 * (1 << 14) + 4 * (1 << 12)), (P + (2 << 20), 99 * (1 << 14) + 4 * (1 << 12)), (P + (16 << 20), 2 * 3 * 1024),
                   (P + (32 << 20), 2 * 3 * 1024), (P + (34 << 20), 4 * 3 * 8), (P + (36 << 20), 4 * 3 * 64), (P + (40 << 20), 4 * 3)]
    else:
        tensors = [(P, 2 * 40 * 512), (P + (16 << 20), 2 * 4000 * 256), (P + (32 << 20), 2 * 4000 * 256), (P + (48 << 20), 2 * 40 * 512),
                   (P + (56 << 20), 4 * 40 * 8), (P + (60 << 20), 4 * 3), (P + (61 << 20), 4 * 3)]
    far = P + (128 << 20)
    for i, (at, size) in enumerate(tensors):
        last = (at + size - 1) // 16 * 16        # the first byte of the workspace in the last of the tensor's
        for space in (at, last, (at - n) // 16 * 16 + 16):
            assert check(a, space, n) == B.CONVROT_EINVAL, (i, space)
            assert getattr(lib, name)(a, space, n, None) == B.CONVROT_EINVAL
    assert check(a, far, n) == B.CONVROT_OK
    # right behind the output, and right before the last tensor: 591360 and 1597440 bytes lie between neighbours; what
    # is longer than it needs to be may reach into it
    at, size = tensors[3]
    assert check(a, -(-(at + size) // 16) * 16, n) == B.CONVROT_OK
    end = tensors[-1][0] - -(-n // 16) * 16
    assert check(a, end, n) == check(a, end, n + 4096) == B.CONVROT_OK


# ---- the binding's checks, on host tensors -----------------------------------------------


@pytest.fixture
def host_calls(monkeypatch):
    """The binding on host tensors: its checks run, the C call is recorded instead of made."""
    B._use_torch()
    calls = []
    monkeypatch.setattr(B, "_on_gpu", lambda t, name: -1)
    monkeypatch.setattr(B, "_check_tensor", lambda t, name, device: None)
    monkeypatch.setattr(B, "_launch", lambda device, stream, call, tensors: call(0))
    monkeypatch.setattr(B, "_call", lambda name, *args: calls.append(name))
    monkeypatch.setattr(B, "_call_with_workspace", lambda name, *args: calls.append(name))
    return calls


def uses_of(cache, dtype=torch.bfloat16):
    """The three calls that take a cache of two heads of 64 channels."""
    x, slots = torch.zeros((2, 2, 64), dtype=dtype), torch.arange(2)
    return [lambda: B.convrot_cache_write(x, x, slots, cache), lambda: B.convrot_cache_read(cache, slots, dtype=dtype),
            lambda: B.convrot_attention_paged(x, cache, slots.int()[:, None], slots.int())]


@pytest.mark.parametrize("kind", ["e2m1", "same"])
@pytest.mark.parametrize("more", [-1, 1])
def test_memory_resized_in_its_place_is_refused(host_calls, kind, more):
    """A storage that got another size at the address that it had: an allocator may give the same
    place out again, and the rest of it to others."""
    class Storage:
        def __init__(self, of, more):
            self.at, self.size = of.data_ptr(), of.nbytes() + more

        def data_ptr(self):
            return self.at

        def nbytes(self):
            return self.size

    for i in range(4 if kind == "e2m1" else 2):
        cache = B.new_kv_cache(4, 8, 2, 64, "e2m1" if kind == "e2m1" else torch.bfloat16, device="cpu")
        for use in uses_of(cache):
            use()
        made = len(host_calls)
        memory = list(cache._memory)
        memory[i] = Storage(memory[i], more)
        cache._memory = tuple(memory)
        for use in uses_of(cache):
            with pytest.raises(ValueError, match="resized"):
                use()
        assert len(host_calls) == made == 3 * (i + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e2m1", "same"])
def test_smaller_memory_of_a_cache_is_refused(gpu, kind):
    x, slots = rand((2, 2, 64), 1, torch.bfloat16).cuda(), torch.arange(2, device="cuda")
    for i in range(4 if kind == "e2m1" else 2):
        cache = new_cache(64, 64, 2, 64, kind, "bf16", seed=1)
        storage = tuple(cache)[i].untyped_storage()
        size = storage.nbytes()
        for n in (0, size // 2):
            storage.resize_(n)
            for call in (lambda: B.convrot_cache_write(x, x, slots, cache), lambda: B.convrot_cache_read(cache, slots),
                         lambda: B.convrot_attention_paged(x, cache, slots.int()[:, None], slots.int())):
                with pytest.raises(ValueError, match="resized"):
                    call()


@pytest.mark.parametrize("kind", ["e2m1", "same"])
@pytest.mark.parametrize("swapped", [False, True])
def test_memory_of_a_call_on_another_stream_is_recorded_there(monkeypatch, kind, swapped):
    """What the kernels read and write is kept until the stream is done: the memory that a cache's
    handle was made of, also where one of its tensors was set to other memory since."""
    B._use_torch()
    monkeypatch.setattr(B, "_on_gpu", lambda t, name: 0)
    monkeypatch.setattr(B, "_check_tensor", lambda t, name, device: None)
    monkeypatch.setattr(B, "_call", lambda name, *args: None)
    monkeypatch.setattr(B, "_call_with_workspace", lambda name, *args: None)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: nullcontext())
    seen = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.append((t.untyped_storage().data_ptr(), s)))
    side = SimpleNamespace(device=SimpleNamespace(index=0), cuda_stream=7)
    cache = B.new_kv_cache(4, 8, 2, 64, "e2m1" if kind == "e2m1" else torch.bfloat16, device="cpu")
    held = [t.untyped_storage().data_ptr() for t in cache if t is not None]
    if swapped:
        cache.k.data = torch.empty_like(cache.k)
    x, y, out = (torch.zeros((2, 2, 64), dtype=torch.bfloat16) for _ in range(3))
    slots = torch.arange(2)
    lse, table, lengths = torch.zeros((2, 2)), slots.int()[:, None].clone(), slots.int()
    work, starts, ends = torch.zeros(16, dtype=torch.uint8), torch.tensor([0, 2], dtype=torch.int32), torch.tensor([0, 2], dtype=torch.int32)
    z = torch.zeros_like(x)
    for call, own in (
            (lambda: B.convrot_cache_write(x, y, slots, cache, stream=side), (x, y, slots)),
            (lambda: B.convrot_cache_read(cache, slots, k=x, v=y, stream=side), (slots, x, y)),
            (lambda: B.convrot_attention_paged(x, cache, table, lengths, out=out, lse=lse, workspace=work, stream=side),
             (x, table, lengths, out, lse, work)),
            (lambda: B.convrot_attention(x, y, z, q_starts=starts, k_starts=ends, out=out, lse=lse, workspace=work, stream=side),
             (x, y, z, starts, ends, out, lse, work))):
        seen.clear()
        call()
        want = {t.untyped_storage().data_ptr() for t in own}
        if len(own) < 8:
            want |= set(held)
        assert {at for at, _ in seen} == want and all(s is side for _, s in seen)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e2m1", "same"])
@pytest.mark.parametrize("swapped", [False, True])
def test_caches_freed_while_another_stream_reads_them(gpu, kind, swapped):
    """The last reference to a cache goes while a stream of its own is still to read it; what is
    allocated next is written at once."""
    side = torch.cuda.Stream()
    slots = torch.arange(2048, device="cuda")
    gate = rand((4096, 4096), 3).cuda()
    for _ in range(3):
        cache = new_cache(32, 64, 8, 128, kind, "bf16", seed=1)
        want = B.convrot_cache_read(cache, slots)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):
                gate @ gate         # the read waits behind these
        if swapped:
            cache.k.data, cache.v.data = (torch.zeros_like(t) for t in (cache.k, cache.v))
        got = B.convrot_cache_read(cache, slots, stream=side)
        del cache
        others = [torch.full((32, 8, 64, 128 if kind == "same" else 64), 77, dtype=torch.bfloat16 if kind == "same" else torch.uint8,
                             device="cuda") for _ in range(6)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and all((t == 77).all() for t in others)


def test_empty_heads_are_refused(host_calls):
    """No heads and heads of no channels reach the library's own check."""
    none, x, n = torch.zeros((1, 2, 2, 0), dtype=torch.bfloat16), torch.zeros((2, 2, 64), dtype=torch.bfloat16), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="heads"):
        B.convrot_attention_paged(x, B.KVCache(*(torch.zeros((4, 0, 8, 64), dtype=torch.bfloat16) for _ in range(2))), n[:, None], n)
    assert not host_calls
    B.convrot_attention_paged(x[..., :0], B.KVCache(*(torch.zeros((4, 2, 8, 0), dtype=torch.bfloat16) for _ in range(2))), n[:, None], n)
    B.convrot_attention(none, none, none)
    assert host_calls == ["convrot_attention_paged", "convrot_attention"]
    lib = B.load()
    for name, args in CALLS:
        assert getattr(lib, name)(args(head_dim=0), P + (128 << 20), 1 << 30, None) == B.CONVROT_EINVAL


@pytest.mark.parametrize("kind", ["e4m3", "same"])
@pytest.mark.parametrize("which", [0, 1])
def test_caches_that_ask_for_a_gradient_are_refused(host_calls, monkeypatch, kind, which):
    """8-bit floating point rows can ask for one as 16-bit rows can."""
    def check(t, name, device):
        if t.requires_grad and torch.is_grad_enabled():
            raise RuntimeError(f"{name} requires a gradient")

    monkeypatch.setattr(B, "_check_tensor", check)
    cache = B.new_kv_cache(4, 8, 2, 64, "e4m3" if kind == "e4m3" else torch.bfloat16, device="cpu")
    (cache.k, cache.v)[which].requires_grad_()
    for use in uses_of(cache):
        with pytest.raises(RuntimeError, match="gradient"):
            use()
    assert not host_calls
    with torch.no_grad():
        for use in uses_of(cache)[1:]:
            use()
    assert len(host_calls) == 2


def test_tangents_are_refused(host_calls):
    """A tangent of forward differentiation would be lost as a gradient would be."""
    import torch.autograd.forward_ad as fwd
    cache = B.new_kv_cache(4, 8, 2, 64, torch.bfloat16, device="cpu")
    x, slots, lse = torch.zeros((2, 2, 64), dtype=torch.bfloat16), torch.arange(2), torch.zeros((2, 2))
    n = slots.int()
    calls = [(lambda k, v, c: B.convrot_cache_write(k, v, slots, c), (x, x)),
             (lambda k, v, c: B.convrot_cache_read(c, slots, k=k, v=v), (x, x)),
             (lambda q, out, lse, c: B.convrot_attention_paged(q, c, n[:, None], n, out=out, lse=lse), (x, x.clone(), lse)),
             (lambda q, k, v, out, lse, c: B.convrot_attention(q[None], k[None], v[None], out=out[None], lse=lse[None]),
              (x, x, x, x.clone(), lse))]
    for i, (call, args) in enumerate(calls):
        with fwd.dual_level():
            call(*args, cache)
            made = len(host_calls)
            for at in range(len(args)):
                dual = fwd.make_dual(args[at].clone(), torch.ones_like(args[at]))
                with pytest.raises(RuntimeError, match="tangent"):
                    call(*args[:at], dual, *args[at + 1:], cache)
            for name in ("k", "v") if i < 3 else ():
                other = B.KVCache(cache.k, cache.v)
                setattr(other, name, fwd.make_dual(getattr(cache, name).clone(), torch.ones_like(cache.k)))
                with pytest.raises(RuntimeError, match="tangent"):
                    call(*args, other)
            assert len(host_calls) == made
        call(*args, cache)


def test_given_outputs_and_caches_count_as_written(host_calls):
    """Autograd tells a saved tensor that was written since by its version."""
    for kind in ("e2m1", "e4m3", torch.bfloat16):
        cache = B.new_kv_cache(4, 8, 2, 64, kind, device="cpu")
        x, slots, k, v, out, lse = (torch.zeros((2, 2, 64), dtype=torch.bfloat16), torch.arange(2), *(torch.zeros((2, 2, 64),
                                    dtype=torch.bfloat16) for _ in range(3)), torch.zeros((2, 2)))
        n = slots.int()
        B.convrot_cache_write(x, x, slots, cache)
        assert all(t is None or t._version == 1 for t in cache)
        B.convrot_cache_read(cache, slots, k=k, v=v)
        B.convrot_attention_paged(x, cache, n[:, None], n, out=out, lse=lse)
        assert [t._version for t in (x, slots, k, v, out, lse)] == [0, 0, 1, 1, 1, 1] and all(t is None or t._version == 1 for t in cache)
        B.convrot_attention(x[None], k[None], v[None], out=out[None], lse=lse[None])
        assert [t._version for t in (x, k, v, out, lse)] == [0, 1, 1, 2, 2]


# ---- prompts whose keys are shared, and joined -----------------------------------------------


def parts_of(q_lens, k_lens, q_heads, k_heads, dim, packed_starts=True):
    """How many workgroups share a tile's keys, from the workspace that a call asks for."""
    lib, need = B.load(), ctypes.c_size_t(0)
    batch, nq, nk = len(q_lens), sum(q_lens), sum(k_lens)
    rows = nq * q_heads
    if not packed_starts:
        nq, nk = nq // batch, nk // batch
    a = prompt_args(batch=batch, q_tokens=nq, k_tokens=nk, q_heads=q_heads, k_heads=k_heads, head_dim=dim, q_token_stride=q_heads * dim,
                    q_head_stride=dim, o_token_stride=q_heads * dim, o_head_stride=dim, k_token_stride=k_heads * dim, k_head_stride=dim,
                    v_token_stride=k_heads * dim, v_head_stride=dim, q=1 << 40, k=2 << 40, v=3 << 40, o=4 << 40, lse=5 << 40,
                    **{} if packed_starts else dict(q_starts=0, k_starts=0, q_batch_stride=nq * q_heads * dim, o_batch_stride=nq * q_heads * dim,
                                                    k_batch_stride=nk * k_heads * dim, v_batch_stride=nk * k_heads * dim))
    assert lib.convrot_attention_workspace_bytes(a, ctypes.byref(need)) == B.CONVROT_OK
    return need.value // (rows * (dim + 2) * 4) or 1


SHARED = [   # queries and keys of each sequence, query heads, key heads, packed one behind the other, pad, place
    ([40] * 2, [3000] * 2, 4, 2, False, 0, 0), ([40] * 3, [2000] * 3, 3, 3, False, 1, 0), ([130] * 2, [2500] * 2, 2, 1, False, 0, 3),
    ([5, 33, 0], [6000, 300, 40], 6, 2, True, 0, 0), ([33, 0, 200], [2000, 2000, 199], 4, 1, True, 8, 0), ([3, 1], [4000, 5], 3, 1, True, 3, 5),
    ([1] * 9, [30, 5000, 0, 64, 4000, 1, 300, 65, 900], 4, 2, True, 0, 1), ([1], [20000], 2, 1, True, 0, 0)]


@pytest.mark.parametrize("dim", [8, 64, 256])
@pytest.mark.parametrize("case", SHARED)
def test_shared_keys_are_shared(case, dim):
    q_lens, k_lens, hq, hk, packed_starts, _, _ = case
    assert parts_of(q_lens, k_lens, hq, hk, dim, packed_starts) > 1


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [8, 40, 64, 96, 128, 136, 200, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", SHARED)
def test_prompts_of_shared_keys(gpu, case, dtype, dim):
    q_lens, k_lens, hq, hk, packed_starts, pad, place = case
    for causal in (False, True):
        check_prompt(q_lens, k_lens, dtype, hq, hk, dim, causal, packed_starts, seed=dim + len(q_lens), pad=pad, place=place,
                     behind=2 if packed_starts else 0)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 200])
def test_masked_places_of_shared_keys_stay_out(gpu, bad, dtype, dim):
    """A value that is no number reaches the queries that see it and no other, in whichever part it lies."""
    dt, nq, n = TYPES[dtype], 150, 3000
    assert parts_of([nq], [n], 1, 1, dim) > 1
    q, k, v = rand((nq, dim), 1, dt), rand((n, dim), 2, dt), rand((n, dim), 3, dt)
    seen = torch.arange(n)[None] <= torch.arange(nq)[:, None] + n - nq
    scale = dim ** -0.5
    want, bound, want_lse, lse_bound = formula(q.double(), k.double(), v.double(), scale, dt, seen)
    others = [c for c in range(dim) if c != 3]
    for at in (n - 1, n - 2, n - 64, n - 130, n - 149, n - 150):
        x = v.clone()
        x[at, 3] = bad
        out, lse = prompt(q, k, x, scale, causal=True)
        sees = seen[:, at]
        assert int(sees.sum()) == n - max(at, n - nq)
        close(out[:, others], want[:, others], bound[:, others], f"key {at}")
        close(out[~sees, 3], want[~sees, 3], bound[~sees, 3], f"key {at}, channel 3")
        got = out[sees, 3].cpu().float()
        assert got.isnan().all() if bad != bad else (got == bad).all()
        close(lse, want_lse, lse_bound, "lse")
        y = k.clone()
        y[at, 3] = math.nan
        out = prompt(q, y, v, scale, causal=True)[0]
        close(out[~sees], want[~sees], bound[~sees], f"key {at} of NaN")
        assert out[sees].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_shared_keys_of_large_and_small_scores(gpu, dtype):
    """Parts whose references are far apart, too large for whole numbers, or of keys that all count for nothing."""
    dt, nq, n, dim = TYPES[dtype], 20, 4000, 64
    q, k, v = torch.zeros((nq, dim), dtype=dt), torch.zeros((n, dim), dtype=dt), rand((n, dim), 3, dt)
    q[:, 0] = 1
    for column in ((torch.arange(n) // 500).float() * 3, 20 - (torch.arange(n) // 300).float() * 4, (torch.arange(n) % 2 - 1).float() * 300):
        k[:, 0] = column.to(dt)
        for causal in (False, True):
            seen = torch.arange(n)[None] <= torch.arange(nq)[:, None] + n - nq if causal else None
            want, bound, want_lse, lse_bound = formula(q.double(), k.double(), v.double(), 1.0, dt, seen)
            out, lse = prompt(q, k, v, 1.0, causal=causal)
            close(out, want, bound)
            close(lse, want_lse, lse_bound)
    k[:, 0] = -math.inf
    k[1234, 0] = 1
    out, lse = prompt(q, k, v, 1.0)
    assert torch.equal(out.cpu(), v[1234].expand(nq, dim))
    # a score of log2(e): half a step of it and of the scale (2 u), of its difference of 11 from an f16 reference (8 u),
    # a step of the exponential and of the logarithm (4 u), and of the product with ln 2 (2 u)
    close(lse, torch.ones(nq, dtype=torch.float64), torch.tensor(16 * U))
    top = 2.0 ** 14
    q[:, 0], k[:, 0] = top, -top
    k[2000, 0] = top
    out, lse = prompt(q, k, v, 1.0)     # 2^28 and -2^28
    assert torch.equal(out.cpu(), v[2000].expand(nq, dim))


# ---- ends of the ranges -----------------------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_cache_blocks_of_every_exponent(gpu, kind, dtype):
    """Every exponent of the type as that of a block's largest value, the others up to 12 binades
    below it; read in bf16, and in f16 where they were f16, the values are the format's own."""
    dt, g = TYPES[dtype], torch.Generator().manual_seed(5)
    exponents, bits = (255, 7) if dtype == "bf16" else (31, 10)
    n = 32 if dtype == "bf16" else 256     # blocks of an exponent
    e = torch.arange(exponents).repeat_interleave(n)[:, None] - torch.randint(0, 13, (exponents * n, 32), generator=g)
    at = torch.randint(0, 32, (exponents * n, 1), generator=g)
    e = e.scatter(1, at, torch.arange(exponents).repeat_interleave(n)[:, None]).clamp(min=0)
    words = torch.randint(0, 2, e.shape, generator=g) << 15 | e << bits | torch.randint(0, 1 << bits, e.shape, generator=g)
    x = (words - (words >> 15 << 16)).to(torch.int16).view(dt)
    assert torch.isfinite(x.float()).all()
    rows = x[:len(x) // 4 * 4].view(-1, 1, 128)
    cache = B.new_kv_cache(-(-len(rows) // 64), 64, 1, 128, kind)
    slots = torch.arange(len(rows), device="cuda")
    B.convrot_cache_write(rows.cuda(), rows.flip(0).cuda(), slots, cache)
    want, scales = kept(rows, kind)
    assert torch.equal(cache.k_scales.cpu().view(-1, 4)[:len(rows)], scales.view(-1, 4))
    for t in {torch.bfloat16, dt}:
        k, v = B.convrot_cache_read(cache, slots, dtype=t)
        same(k, want.to(t))
        same(v, want.to(t).flip(0))
        exact = want.to(t).double() == want
        # beyond bf16's range only: 448 or 6 times the scale of the largest exponent
        assert exact[want.abs() < 2.0 ** 127].all() and (t == torch.bfloat16 or exact.all())


@pytest.mark.gpu
@pytest.mark.parametrize("place", [0, 1])      # copied straight to shared memory, and by way of registers
def test_prompts_past_32_bit_offsets(gpu, place):
    """Rows whose bytes lie past 32-bit offsets: queries, keys, values and outputs of a token 16 MB apart."""
    n, heads, dim, step = 330, 2, 64, 1 << 23
    memory = torch.empty(n * step + 1024, dtype=torch.bfloat16, device="cuda")
    at = [torch.as_strided(memory, (n, heads, dim), (step, dim, 1), place + i * 128) for i in range(4)]
    rows = [rand((n, heads, dim), 1 + i, torch.bfloat16) for i in range(3)]
    for t, x in zip(at, rows):
        t.copy_(x)
    starts = torch.tensor([0, 130, n], dtype=torch.int32, device="cuda")
    out = B.convrot_attention(*at[:3], q_starts=starts, causal=True, out=at[3])
    for a, b in ((0, 130), (130, n)):
        seen = torch.arange(b - a)[None] <= torch.arange(b - a)[:, None]
        for h in range(heads):
            want, bound, _, _ = formula(*(x[a:b, h].double() for x in rows), dim ** -0.5, torch.bfloat16, seen)
            close(out[a:b, h], want, bound, f"rows from {a}, head {h}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,std", [("bf16", 2.0 ** 20), ("bf16", 2.0 ** 45), ("f16", 2.0 ** 12)])
@pytest.mark.parametrize("dim", [8, 72, 128, 200])
def test_large_scores_of_packed_and_unaligned_rows(gpu, dtype, std, dim):
    """Rows computed once more, of several sequences and heads, copied straight to shared memory and by
    way of registers: the same bits, and the value of the key with the largest score."""
    dt, lens, heads = TYPES[dtype], [200, 1, 0, 333], 2
    n = sum(lens)
    q, k, v = (rand((n, heads, dim), 1 + i, dt, std if i < 2 else 1.0) for i in range(3))
    starts = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    for causal in (False, True):
        outs = []
        for pad, place in ((0, 0), (1, 0), (8, 3)):
            views = []
            for x in (q, k, v):
                wide = torch.full((n * (heads * dim + pad) + place,), math.nan, dtype=dt, device="cuda")
                views.append(wide[place:].view(n, heads * dim + pad)[:, :heads * dim].unflatten(1, (heads, dim)))
                views[-1].copy_(x)
            outs.append(B.convrot_attention(*views, q_starts=starts, causal=causal, want_lse=True))
        assert all(torch.equal(a, b) for o in outs[1:] for a, b in zip(o, outs[0]))
        out, lse = (t.cpu().double() for t in outs[0])
        at = clear = 0
        for m in lens:
            for h in range(heads if m else 0):
                qq, kk = q[at:at + m, h].double(), k[at:at + m, h].double()
                s = qq @ kk.T * dim ** -0.5
                lost = (dim + 4) * U * (qq.abs() @ kk.abs().T) * dim ** -0.5 + 8 * U * s.abs()
                if causal:
                    hidden = torch.ones(m, m, dtype=torch.bool).triu(1)
                    s, lost = s.masked_fill(hidden, -math.inf), lost.masked_fill(hidden, 0.0)
                best = s.argmax(-1)
                top = s.gather(1, best[:, None])[:, 0]
                others = (s + lost).scatter(1, best[:, None], -math.inf).amax(-1)
                alone = top - lost.gather(1, best[:, None])[:, 0] - others > 40     # the others' weights sum to less than 2^-40
                clear += int(alone.sum())
                # up to 2^24 the exact score is what the weight is taken from, and the reference a rounded one: the weight is
                # a power of two within half a binary place, rounded to the type (half a step of it), as the output is
                want = v[at:at + m, h][best].double()
                bound = (torch.finfo(dt).eps / 2 + 2 * (n + 16) * U) * want.abs() + 2.0 ** -39
                close(out[at:at + m, h][alone], want[alone], (bound + half_step(dt, want.abs() + bound))[alone])
                assert ((lse[at:at + m, h] - top).abs() <= lost.amax(-1) + 8 * U * top.abs()).all()
            at += m
        assert clear > 0.9 * n * heads


@pytest.mark.gpu
@pytest.mark.parametrize("place", [0, 1])
def test_masked_places_of_packed_and_unaligned_rows(gpu, place):
    """Values that are no numbers in a packed sequence reach its own later rows alone."""
    lens, heads, dim = [70, 130, 260], 2, 72
    n = sum(lens)
    q, k, v = (rand((n, heads, dim), 1 + i, torch.bfloat16) for i in range(3))
    starts = torch.tensor([0, 70, 200, 460], dtype=torch.int32, device="cuda")
    memory = torch.empty(3 * n * heads * dim + place, dtype=torch.bfloat16, device="cuda")[place:].view(3, n, heads, dim)
    for at in (0, 69, 70, 133, 199, 330, 459):
        x = v.clone()
        x[at, 1, 5] = math.nan
        for to, t in zip(memory, (q, k, x)):
            to.copy_(t)
        out = B.convrot_attention(*memory, q_starts=starts, causal=True)
        for a, b in ((0, 70), (70, 200), (200, 460)):
            seen = torch.arange(b - a)[None] <= torch.arange(b - a)[:, None]
            for h in range(heads):
                want, bound, _, _ = formula(*(t[a:b, h].double() for t in (q, k, v)), dim ** -0.5, torch.bfloat16, seen)
                if h == 1 and a <= at < b:
                    assert out[at:b, h, 5].isnan().all()
                    want[at - a:, 5] = math.nan
                close(out[a:b, h], want, bound, f"rows from {a}, head {h}, key {at}")
