"""A synthetic FLUX-shaped transformer block, run dense and with its linears
swapped for ConvRotLinear.

The pages measure ConvRot inside FLUX.1 Dev image generation (convrot-mlx
README, "Why this repository exists"); no FLUX weights, prompts or runtime are
used here.  This harness builds one block of the same shape with random
weights (N(0, 0.02), biases N(0, 0.01)) and synthetic tokens (N(0, 1) with a
few outlier channels scaled up), and runs it twice: with plain bf16
``nn.Linear`` layers, and after ``convert_linears`` has replaced every linear
by a ConvRotLinear (the module swap of the convrot-mlx README, "What is
included").  It reports the relative Frobenius error of the block output and
the time per block of both.

Block, hidden size H, heads of 128, T tokens:
    h = LayerNorm(x) * (1 + scale) + shift       (random modulation)
    q, k, v = qkv(h)                             H -> 3H
    x = x + proj(softmax(q k^T / sqrt(128)) v)   H -> H
    x = x + down(gelu_tanh(up(LayerNorm(x))))    H -> 4H -> H
The norms and the attention run in float32 torch ops around the linears;
they are the harness, not the path.

ConditionedBlock is the same block as a diffusion transformer conditions and
positions it, with the library's operators between its linears:
    shift1, scale1, gate1, shift2, scale2, gate2 = modulation(silu(vec))
    h = LayerNorm(x) * (1 + scale1) + shift1
    q, k turned by the tokens' (index, row, column), after a norm of each head
    x = x + gate1 * proj(attention);  h = LayerNorm(x) * (1 + scale2) + shift2
    x = x + gate2 * down(gelu_tanh(up(h)))
The modulation runs in GroupedLinear, each residual update and the norm after
it in one call, the norm and rotation of all heads in another; the attention
and the GELU stay the harness.

    python -m w4a4_rotated_bit_amd.flux_block [--tokens 1536] [--hidden 3072]
        [--rotation sylvester|regular] [--group-size 256] [--iters 20]
        [--conditioned] [--batch 1]
"""
from __future__ import annotations

import argparse
import copy
import json
import sys

import torch

from . import binding, synth
from .module import ConvRotLinear, GroupedLinear, convert_linears


class Block(torch.nn.Module):
    def __init__(self, hidden: int, head_dim: int = 128, seed: int = 0):
        super().__init__()
        if hidden % head_dim:
            raise ValueError("hidden must be a multiple of the head size")
        self.hidden, self.head_dim, self.heads = hidden, head_dim, hidden // head_dim
        self.qkv = torch.nn.Linear(hidden, 3 * hidden)
        self.proj = torch.nn.Linear(hidden, hidden)
        self.up = torch.nn.Linear(hidden, 4 * hidden)
        self.down = torch.nn.Linear(4 * hidden, hidden)
        for i, lin in enumerate((self.qkv, self.proj, self.up, self.down)):
            n, k = lin.weight.shape
            w = synth.random_bf16((n, k), seed=seed * 16 + 2 * i, std=0.02)
            b = synth.random_bf16((n,), seed=seed * 16 + 2 * i + 1, std=0.01)
            lin.weight.data = torch.from_numpy(synth.bf16_bits_to_f32(w)).to(torch.bfloat16)
            lin.bias.data = torch.from_numpy(synth.bf16_bits_to_f32(b)).to(torch.bfloat16)
        mod = synth.random_bf16((2, hidden), seed=seed * 16 + 9, std=0.1)
        self.register_buffer("modulation", torch.from_numpy(synth.bf16_bits_to_f32(mod)))

    @staticmethod
    def _norm(x: torch.Tensor) -> torch.Tensor:
        return torch.nn.functional.layer_norm(x.float(), (x.shape[-1],), eps=1e-6)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """x: bf16 [T, hidden] -> bf16 [T, hidden]."""
        T, H = x.shape
        shift, scale = self.modulation[0], self.modulation[1]
        h = (self._norm(x) * (1 + scale) + shift).to(torch.bfloat16)
        qkv = self.qkv(h).float().reshape(T, 3, self.heads, self.head_dim)
        q, k, v = (qkv[:, i].transpose(0, 1).contiguous() for i in range(3))   # [heads, T, D] each
        s = torch.bmm(q, k.transpose(1, 2).contiguous()) / self.head_dim ** 0.5
        a = torch.bmm(torch.softmax(s, dim=-1), v).transpose(0, 1).reshape(T, H)
        x = (x.float() + self.proj(a.to(torch.bfloat16)).float()).to(torch.bfloat16)
        u = torch.nn.functional.gelu(self.up(self._norm(x).to(torch.bfloat16)).float(), approximate="tanh")
        return (x.float() + self.down(u.to(torch.bfloat16)).float()).to(torch.bfloat16)


class ConditionedBlock(Block):
    """Block with a modulation of each batch entry, gates, and positioned heads."""

    def __init__(self, hidden: int, head_dim: int = 128, seed: int = 0, axes=None):
        super().__init__(hidden, head_dim, seed)
        if axes is None:    # an eighth for the index, the rest halved for row and column
            index = head_dim // 16 * 2
            row = (head_dim - index) // 4 * 2
            axes = (index, row, head_dim - index - row)
        self.freq, self.axis = binding.rope_frequencies(axes)
        self.modulation_linear = torch.nn.Linear(hidden, 6 * hidden)
        w = synth.random_bf16((6 * hidden, hidden), seed=seed * 16 + 10, std=0.02)
        b = synth.random_bf16((6 * hidden,), seed=seed * 16 + 11, std=0.1)
        self.modulation_linear.weight.data = torch.from_numpy(synth.bf16_bits_to_f32(w)).to(torch.bfloat16)
        self.modulation_linear.bias.data = torch.from_numpy(synth.bf16_bits_to_f32(b)).to(torch.bfloat16)
        for i, name in enumerate(("q_weight", "k_weight")):
            w = synth.random_bf16((head_dim,), seed=seed * 16 + 12 + i, std=0.1)
            self.register_buffer(name, (1 + torch.from_numpy(synth.bf16_bits_to_f32(w))).to(torch.bfloat16))

    def _attend(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor) -> torch.Tensor:
        """q, k, v: [B, T, heads, D] -> bf16 [B, T, H]."""
        B, T = q.shape[:2]
        q, k, v = (t.float().transpose(1, 2).reshape(-1, T, self.head_dim).contiguous() for t in (q, k, v))
        s = torch.softmax(torch.bmm(q, k.transpose(1, 2).contiguous()) / self.head_dim ** 0.5, dim=-1)
        a = torch.bmm(s, v).reshape(B, self.heads, T, self.head_dim).transpose(1, 2).reshape(B, T, self.hidden)
        return a.to(torch.bfloat16)

    def _feed_forward(self, h: torch.Tensor) -> torch.Tensor:
        u = torch.nn.functional.gelu(self.up(h).float(), approximate="tanh")
        return self.down(u.to(torch.bfloat16))

    def _modulation(self, vec: torch.Tensor):
        return self.modulation_linear(torch.nn.functional.silu(vec.float()).to(torch.bfloat16)).chunk(6, -1)

    def forward(self, x: torch.Tensor, vec: torch.Tensor, positions: torch.Tensor) -> torch.Tensor:
        """x: bf16 [B, T, H]; vec: [B, H]; positions: int32 or float32 [B or 1, T, 3]."""
        B, T, H = x.shape
        shift1, scale1, gate1, shift2, scale2, gate2 = self._modulation(vec)
        _, h = binding.convrot_residual_norm(x, scale=scale1, shift=shift1, want_r=False)
        q, k, v = self.qkv(h).view(B, T, 3, self.heads, self.head_dim).unbind(2)
        q, k = binding.convrot_rope(q, k, positions, self.freq, self.axis, qk_norm=True, q_weight=self.q_weight,
                                    k_weight=self.k_weight)
        x, h = binding.convrot_residual_norm(x, self.proj(self._attend(q, k, v)), gate=gate1, scale=scale2, shift=shift2)
        return binding.convrot_residual_norm(x, self._feed_forward(h), gate=gate2, want_h=False)[0]

    def plain(self, x: torch.Tensor, vec: torch.Tensor, positions: torch.Tensor) -> torch.Tensor:
        """The same block with float32 torch operations between its linears."""
        B, T, H = x.shape
        bf16 = torch.bfloat16
        shift1, scale1, gate1, shift2, scale2, gate2 = (m.float().unsqueeze(1) for m in self._modulation(vec))
        q, k, v = self.qkv((self._norm(x) * (1 + scale1) + shift1).to(bf16)).view(B, T, 3, self.heads, self.head_dim).unbind(2)
        axis = torch.from_numpy(self.axis).long().to(x.device)
        angle = (positions.double()[..., axis] * torch.from_numpy(self.freq).to(x.device)).unsqueeze(2)
        cos, sin = angle.cos().float(), angle.sin().float()

        def turned(t, weight):
            t = t.float()
            t = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * weight.float()
            a, b = t[..., 0::2], t[..., 1::2]
            return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2).to(bf16)

        x = x.float() + gate1 * self.proj(self._attend(turned(q, self.q_weight), turned(k, self.k_weight), v)).float()
        h = (self._norm(x) * (1 + scale2) + shift2).to(bf16)
        return (x.to(bf16).float() + gate2 * self._feed_forward(h).float()).to(bf16)


def picture(T: int, batch: int = 1) -> torch.Tensor:
    """Positions float32 [batch, T, 3] of a picture: a third of the tokens are
    text at the origin, the rest a grid of (0, row, column)."""
    text = T // 3
    side = max(1, int((T - text) ** 0.5))
    j = (torch.arange(T) - text).clamp(min=0)
    return torch.stack([torch.zeros_like(j), j // side, j % side], -1).float().expand(batch, T, 3).contiguous()


def tokens(T: int, hidden: int, seed: int = 7) -> torch.Tensor:
    """Synthetic bf16 tokens: N(0, 1), 1% of the channels scaled by 20."""
    bits = synth.random_bf16((T, hidden), seed=seed, outliers=max(1, round(0.01 * hidden)))
    return torch.from_numpy(synth.bf16_bits_to_f32(bits)).to(torch.bfloat16)


def rel_err(y: torch.Tensor, ref: torch.Tensor) -> float:
    y, ref = y.detach().double(), ref.detach().double()
    return float(torch.linalg.vector_norm(y - ref) / torch.linalg.vector_norm(ref))


def time_ms(fn, x: torch.Tensor, iters: int) -> float:
    for _ in range(3):
        fn(x)
    torch.cuda.synchronize()
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(iters):
        fn(x)
    stop.record()
    torch.cuda.synchronize()
    return start.elapsed_time(stop) / iters


@torch.no_grad()
def run(T: int = 1536, hidden: int = 3072, group_size: int = 256, rotation: str = "sylvester",
        iters: int = 20) -> dict:
    dense = Block(hidden).cuda().to(torch.bfloat16)
    dense.modulation = dense.modulation.float()
    quant = copy.deepcopy(dense)
    swapped = convert_linears(quant, group_size, rotation)
    if sorted(swapped) != ["down", "proj", "qkv", "up"]:
        raise RuntimeError(f"unexpected linears swapped: {swapped}")
    assert all(isinstance(getattr(quant, n), ConvRotLinear) for n in swapped)
    x = tokens(T, hidden).cuda()
    y_dense, y_quant = dense(x), quant(x)
    torch.cuda.synchronize()
    out = {
        "tokens": T, "hidden": hidden, "group_size": group_size, "rotation": rotation,
        "swapped": sorted(swapped),
        "rel_err_block": rel_err(y_quant, y_dense),
        "rel_err_update": rel_err(y_quant.float() - x.float(), y_dense.float() - x.float()),
        "finite": bool(torch.isfinite(y_quant.float()).all()),
    }
    if iters > 0:
        out["dense_ms"] = time_ms(dense, x, iters)
        out["convrot_ms"] = time_ms(quant, x, iters)
    return out


@torch.no_grad()
def run_conditioned(T: int = 1536, hidden: int = 3072, batch: int = 1, group_size: int = 256,
                    rotation: str = "sylvester", iters: int = 20) -> dict:
    dense = ConditionedBlock(hidden).cuda().to(torch.bfloat16)
    quant = copy.deepcopy(dense)
    swapped = convert_linears(quant, group_size, rotation, include=lambda name: name != "modulation_linear")
    if sorted(swapped) != ["down", "proj", "qkv", "up"]:
        raise RuntimeError(f"unexpected linears swapped: {swapped}")
    quant.modulation_linear = GroupedLinear.from_linear(quant.modulation_linear, 128)   # of heads of 128
    x = tokens(batch * T, hidden).view(batch, T, hidden).cuda()
    vec = torch.from_numpy(synth.bf16_bits_to_f32(synth.random_bf16((batch, hidden), seed=8))).to(torch.bfloat16).cuda()
    inputs = (x, vec, picture(T, batch).cuda())
    y, y_dense, y_plain = quant(*inputs), dense(*inputs), dense.plain(*inputs)
    torch.cuda.synchronize()
    out = {
        "tokens": T, "hidden": hidden, "batch": batch, "group_size": group_size, "rotation": rotation,
        "rel_err_operators": rel_err(y_dense, y_plain),   # dense linears, the operators against torch operations
        "rel_err_block": rel_err(y, y_plain),
        "finite": bool(torch.isfinite(y.float()).all()),
    }
    if iters > 0:
        out["operators_ms"] = time_ms(lambda a: quant(*a), inputs, iters)
        out["plain_ms"] = time_ms(lambda a: quant.plain(*a), inputs, iters)
    return out


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--tokens", type=int, default=1536)
    ap.add_argument("--hidden", type=int, default=3072)
    ap.add_argument("--group-size", type=int, default=256, choices=(64, 256))
    ap.add_argument("--rotation", default="sylvester", choices=("sylvester", "regular"))
    ap.add_argument("--iters", type=int, default=20)
    ap.add_argument("--conditioned", action="store_true", help="the modulated, gated and positioned block")
    ap.add_argument("--batch", type=int, default=1, help="batch entries of the conditioned block")
    args = ap.parse_args(argv)
    if not torch.cuda.is_available():
        print("a GPU is required", file=sys.stderr)
        return 2
    if args.conditioned:
        print(json.dumps(run_conditioned(args.tokens, args.hidden, args.batch, args.group_size, args.rotation, args.iters)))
        return 0
    print(json.dumps(run(args.tokens, args.hidden, args.group_size, args.rotation, args.iters)))
    return 0


if __name__ == "__main__":
    sys.exit(main())
