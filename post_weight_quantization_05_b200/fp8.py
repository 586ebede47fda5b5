"""Layers that hold their weights in the 8-bit floating-point form (note "Model
Quantization", "주요 양자화 기법": FP8 among the post-training forms), for
inference: torch modules over api.fp8_quantize_weight, fp8_quantize_rows,
fp8_gemm and fp8_gated.  A weight is quantized once, when the layer is made;
each call quantizes its inputs, a scale per token and 128 channels, and
multiplies codes with codes.  The float weights are not kept.

A weight or an input that holds a NaN or an infinity is recorded in the library's
status word (a token's outputs are then NaN): api.get_status() reads and clears it.
"""
from __future__ import annotations

import torch
from torch import nn
from torch.autograd import forward_ad

from . import api


def _pitched(x: torch.Tensor) -> torch.Tensor:
    """A matrix whose rows may be pitched, but neither strided inside nor over one another."""
    return x if x.stride(1) == 1 and (x.shape[0] <= 1 or x.stride(0) >= x.shape[1]) else x.contiguous()


def _rows(x: torch.Tensor) -> torch.Tensor:
    """[..., d] as such a matrix."""
    if torch.is_grad_enabled() and x.requires_grad:
        raise RuntimeError("the 8-bit layers are for inference: their inputs' gradients are not computed")
    if forward_ad.unpack_dual(x).tangent is not None:
        raise RuntimeError("the 8-bit layers are for inference: no tangents are computed")
    return _pitched(x.reshape(-1, x.shape[-1]))


def _activations(x: torch.Tensor):
    m, d = x.shape
    codes = api.fp8_codes(m, d, device=x.device)
    scales = torch.empty((api.fp8_blocks(d), m), dtype=torch.float32, device=x.device)
    api.fp8_quantize_rows(x, codes, scales)
    return codes, scales


class _Fp8Module(nn.Module):
    """Holds weights as codes (uint8, rows padded to whole 16 bytes) and fp32
    scales, which a change of the module's float type leaves as they are."""

    def _add_weight(self, name: str, weight: torch.Tensor):
        w = weight.detach()
        n, d = w.shape
        codes = torch.zeros((n, -(-d // 16) * 16), dtype=torch.uint8, device=w.device)
        scales = torch.empty((api.fp8_blocks(n), api.fp8_blocks(d)), dtype=torch.float32, device=w.device)
        api.fp8_quantize_weight(_pitched(w), codes[:, :d], scales)
        self.register_buffer(name, codes)
        self.register_buffer(name + "_scales", scales)

    def _weight(self, name: str, d: int):
        codes = getattr(self, name)
        return codes if codes.shape[1] == d else codes[:, :d], getattr(self, name + "_scales")

    def _apply(self, fn, recurse=True):
        scales = {k: v for k, v in self._buffers.items() if k.endswith("_scales")}
        super()._apply(fn, recurse)
        for k, v in scales.items():
            if self._buffers[k].dtype != torch.float32:
                self._buffers[k] = v.to(self._buffers[k].device)
        return self


class Fp8Linear(_Fp8Module):
    """nn.Linear's product from the 8-bit form; outputs in the inputs' type
    (fp32, bf16 or fp16)."""

    @staticmethod
    def check(linear: nn.Linear):
        """Raises ValueError if `linear` has no 8-bit form."""
        w = linear.weight
        if not w.is_cuda or w.dtype not in (torch.float32, torch.bfloat16, torch.float16) or not (
                1 <= w.shape[0] <= 1 << 22 and 1 <= w.shape[1] <= 1 << 18):
            raise ValueError("the 8-bit form needs a weight of fp32, bf16 or fp16 on a GPU, of at most 2^22 x 2^18, "
                             f"got {tuple(w.shape)} of {w.dtype} on {w.device}")

    def __init__(self, linear: nn.Linear):
        super().__init__()
        self.check(linear)
        self.out_features, self.in_features = linear.weight.shape
        self._add_weight("codes", linear.weight)
        self.register_buffer("bias", None if linear.bias is None else linear.bias.detach().clone())

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        rows = _rows(x)
        y = torch.empty((rows.shape[0], self.out_features), dtype=x.dtype, device=x.device)
        if rows.shape[0]:
            api.fp8_gemm(*_activations(rows), *self._weight("codes", self.in_features), y)
        if self.bias is not None:
            y += self.bias
        return y.reshape(*x.shape[:-1], self.out_features)


class Fp8GatedMLP(_Fp8Module):
    """down(act(gate(x)) * up(x)) from the 8-bit form: one kernel for the gated
    pair, whose output leaves as the down projection's codes.  act "silu" or
    "gelu"; linears without bias."""

    def __init__(self, gate: nn.Linear, up: nn.Linear, down: nn.Linear, act: str = "silu"):
        super().__init__()
        if any(m.bias is not None for m in (gate, up, down)):
            raise ValueError("a gated feed-forward layer with biases is not supported")
        if gate.weight.shape != up.weight.shape or down.in_features != gate.out_features:
            raise ValueError("gate and up must have one shape, and down must take their outputs")
        self.hidden, self.out_features, self.act = gate.out_features, down.out_features, act
        self.in_features = gate.in_features
        for name, m in (("gate", gate), ("up", up), ("down", down)):
            self._add_weight(name, m.weight)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        rows = _rows(x)
        m = rows.shape[0]
        y = torch.empty((m, self.out_features), dtype=x.dtype, device=x.device)
        if m:
            h = api.fp8_codes(m, self.hidden, device=x.device)
            hs = torch.empty((api.fp8_blocks(self.hidden), m), dtype=torch.float32, device=x.device)
            api.fp8_gated(*_activations(rows), *self._weight("gate", self.in_features),
                          *self._weight("up", self.in_features), h, hs, act=self.act)
            api.fp8_gemm(h, hs, *self._weight("down", self.hidden), y)
        return y.reshape(*x.shape[:-1], self.out_features)


# Modules of torch that in inference hand their linears' weights to a function of
# their own, past the linears' forward.
_READS_WEIGHTS = (nn.TransformerEncoderLayer,)


def quantize_linears(module: nn.Module, exclude=None) -> nn.Module:
    """Replace every nn.Linear inside `module` by its 8-bit form, in place (a
    linear layer itself: the form is returned).  A linear that the module holds
    in several places keeps doing so, as one form.  Either all are replaced or,
    if one has no such form (ValueError), none.

    The form has no `weight`, so a linear whose weight someone else reads has to
    stay: subclasses of nn.Linear do, and those of an nn.TransformerEncoderLayer.
    For others exclude(name, linear) says so by returning True, asked for every
    place that holds a linear, with the place's name as module.named_modules()
    spells it."""
    def taken(name, linear):
        if type(linear) is not nn.Linear or (exclude is not None and exclude(name, linear)):
            return False
        Fp8Linear.check(linear)
        return True
    if type(module) is nn.Linear:
        return Fp8Linear(module) if taken("", module) else module
    places = [(parent, name, child)
              for prefix, parent in module.named_modules() if not isinstance(parent, _READS_WEIGHTS)
              for name, child in parent._modules.items() if taken(f"{prefix}.{name}" if prefix else name, child)]
    forms: dict[nn.Module, Fp8Linear] = {}
    for parent, name, linear in places:
        if linear not in forms:
            forms[linear] = Fp8Linear(linear)
        setattr(parent, name, forms[linear])
    return module
