"""ConvRotLinear: a torch module around the library's W4A4 (or W4A16) linear,
and GroupedLinear: one around its group-scaled 4-bit linear for a few rows.

The weight is rotated, quantized and packed once, on construction from an
``nn.Linear`` (the offline step; convrot-mlx README, "What is included": the
conversion of eligible linears and the ConvRotLinear layer that replaces
them).  ``forward`` flattens the leading dimensions of x to M rows, runs
``convrot_linear`` (or ``convrot_linear_w4a16``) on the current stream and
restores them.  Every step of the linear runs in the library's kernels; the
module only holds buffers and reshapes.
"""
from __future__ import annotations

import torch

from . import binding


class ConvRotLinear(torch.nn.Module):
    """y = x W^T + b with the ConvRot rotation and INT4 weights.

    group_size: 64 or 256; rotation: "sylvester" or "regular"; path: "w4a4"
    (activations quantized to INT4) or "w4a16" (bf16 rotated activations,
    M <= 32 rows per call)."""

    def __init__(self, in_features: int, out_features: int, image: torch.Tensor, sw: torch.Tensor,
                 bias: torch.Tensor | None, group_size: int = 256, rotation: str = "sylvester", path: str = "w4a4"):
        super().__init__()
        if rotation not in ("sylvester", "regular"):
            raise ValueError(f"unknown rotation {rotation!r}")
        if path not in ("w4a4", "w4a16"):
            raise ValueError(f"unknown path {path!r}")
        self.in_features, self.out_features = in_features, out_features
        self.group_size, self.rotation, self.path = group_size, rotation, path
        self.g = group_size | (binding.CONVROT_REGULAR_HADAMARD if rotation == "regular" else 0)
        self.register_buffer("image", image)
        self.register_buffer("sw", sw)
        self.register_buffer("bias", bias)

    @classmethod
    @torch.no_grad()
    def from_linear(cls, linear: torch.nn.Linear, group_size: int = 256, rotation: str = "sylvester",
                    path: str = "w4a4") -> "ConvRotLinear":
        if not linear.weight.is_cuda:
            raise ValueError("the linear must be on the GPU")
        w = linear.weight.detach().to(torch.bfloat16).contiguous()
        g = group_size | (binding.CONVROT_REGULAR_HADAMARD if rotation == "regular" else 0)
        image, sw = binding.convrot_prepare_weight(w, g)
        b = None if linear.bias is None else linear.bias.detach().to(torch.bfloat16).contiguous()
        return cls(linear.in_features, linear.out_features, image, sw, b, group_size, rotation, path)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.in_features:
            raise ValueError(f"last dimension {x.shape[-1]} != in_features {self.in_features}")
        lead = x.shape[:-1]
        x2 = x.reshape(-1, self.in_features).to(torch.bfloat16).contiguous()
        if self.path == "w4a16":
            y = binding.convrot_linear_w4a16(x2, self.image, self.sw, self.bias, self.out_features, self.g)
        else:
            y = binding.convrot_linear(x2, self.image, self.sw, self.bias, self.out_features, self.g)
        return y.reshape(*lead, self.out_features)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, bias={self.bias is not None}, "
                f"group_size={self.group_size}, rotation={self.rotation}, path={self.path}")


class GroupedLinear(torch.nn.Module):
    """y = x W^T + b for at most 32 rows, W in 4 bits with a scale (and zero
    point) for every ``group_size`` input channels: the modulation linear of a
    conditioned block, or a decoder's linear at a few tokens.

    codes: uint8 [out_features, in_features / 2], the low nibble the even
    channel, unsigned with zeros and two's complement without; scales: bf16 or
    f16 [out_features, in_features / group_size]; zeros: uint8 of that shape."""

    def __init__(self, in_features: int, out_features: int, codes: torch.Tensor, scales: torch.Tensor,
                 zeros: torch.Tensor | None, bias: torch.Tensor | None, group_size: int = 128):
        super().__init__()
        if group_size not in (32, 64, 128) or in_features % group_size:
            raise ValueError(f"group_size must be 32, 64 or 128 and divide {in_features}, got {group_size}")
        shape = (out_features, in_features // group_size)
        if tuple(codes.shape) != (out_features, in_features // 2) or tuple(scales.shape) != shape:
            raise ValueError("codes and scales do not fit the features and the group size")
        if zeros is not None and tuple(zeros.shape) != shape:
            raise ValueError("zeros must have the shape of scales")
        self.in_features, self.out_features, self.group_size = in_features, out_features, group_size
        self.register_buffer("codes", codes)
        self.register_buffer("scales", scales)
        self.register_buffer("zeros", zeros)
        self.register_buffer("bias", bias)

    @classmethod
    @torch.no_grad()
    def from_linear(cls, linear: torch.nn.Linear, group_size: int = 128, asymmetric: bool = False) -> "GroupedLinear":
        if not linear.weight.is_cuda:
            raise ValueError("the linear must be on the GPU")
        w = linear.weight.detach()
        w = (w if w.dtype == torch.float16 else w.to(torch.bfloat16)).contiguous()
        codes, scales, zeros = binding.convrot_quantize_weight_grouped(w, group_size, asymmetric)
        b = None if linear.bias is None else linear.bias.detach().to(w.dtype).contiguous()
        return cls(linear.in_features, linear.out_features, codes, scales, zeros, b, group_size)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.in_features:
            raise ValueError(f"last dimension {x.shape[-1]} != in_features {self.in_features}")
        lead = x.shape[:-1]
        x2 = x.reshape(-1, self.in_features).to(self.scales.dtype).contiguous()
        if x2.shape[0] > 32:
            raise ValueError(f"{x2.shape[0]} rows: a GroupedLinear takes at most 32")
        y = binding.convrot_linear_grouped(x2, self.codes, self.scales, self.zeros, self.bias, self.group_size)
        return y.reshape(*lead, self.out_features)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, bias={self.bias is not None}, "
                f"group_size={self.group_size}, asymmetric={self.zeros is not None}")


def eligible(linear: torch.nn.Linear, group_size: int = 256) -> bool:
    """Whether the library takes this linear: K a multiple of 8 whose rotated
    width fits, and N within the row limit."""
    K, N = linear.in_features, linear.out_features
    return K % 8 == 0 and binding.rotated_width(K, group_size) <= binding.MAX_K and 1 <= N <= binding.MAX_ROWS


@torch.no_grad()
def convert_linears(model: torch.nn.Module, group_size: int = 256, rotation: str = "sylvester", path: str = "w4a4",
                    include=None) -> list[str]:
    """Replace, in place, every eligible ``nn.Linear`` of ``model`` (and whose
    qualified name ``include(name)`` accepts, when given) by a ConvRotLinear
    built from it -- the module swap of the convrot-mlx README, "What is
    included".  Returns the names of the replaced linears."""
    done = []
    for name, parent in list(model.named_modules()):
        for child_name, child in list(parent.named_children()):
            full = f"{name}.{child_name}" if name else child_name
            if type(child) is not torch.nn.Linear or not eligible(child, group_size):
                continue
            if include is not None and not include(full):
                continue
            setattr(parent, child_name, ConvRotLinear.from_linear(child, group_size, rotation, path))
            done.append(full)
    return done
