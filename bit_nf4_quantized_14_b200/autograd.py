"""PyTorch autograd glue for the QLoRA linear layer: the frozen NF4 weight and the trainable LoRA adapters
as one torch.autograd.Function and an nn.Module around it; and for the two operators beside it in a decoder,
the rotary positions of queries and keys (`rotary`) and the vocabulary loss (`vocab_loss`).

The adapters are fp32 parameters (the pages keep the adapters in full precision for training: PEFT page,
zerotofrontier.app/sft/peft, "Paged optimizers, and QLoRA end to end"); each call hands bf16 copies to the
library, which computes Y = X W_hat^T + (alpha/r) (X A^T) B^T in its kernels and returns fp32 gradients of
A and B (written straight into the parameters' .grad by autograd). The frozen weight gets no gradient
(QLoRA explainer, prism.theerrors.in, "Putting it together"). No arithmetic of the layer happens here.
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import NF4Weight, RotaryConfig, _aligned, linear_bwd, linear_fwd, quantize
from . import rotary as _rotary
from . import vocab_loss as _vocab_loss


class QLoRALinearFn(torch.autograd.Function):
    """y = x W_hat^T + (alpha / r) (x A^T) B^T for x of shape (..., K); returns (..., N) bf16."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, w: NF4Weight, alpha: float):
        K = x.shape[-1]
        x2 = x.reshape(-1, K).to(torch.bfloat16).contiguous()
        a16 = A.detach().to(torch.bfloat16).contiguous()
        b16 = B.detach().to(torch.bfloat16).contiguous()
        y, u = linear_fwd(x2, w, a16, b16, alpha)
        ctx.save_for_backward(x2, a16, b16, u)
        ctx.w, ctx.alpha, ctx.in_shape = w, alpha, x.shape
        return y.view(*x.shape[:-1], w.rows)

    @staticmethod
    def backward(ctx, dy: torch.Tensor):
        x2, a16, b16, u = ctx.saved_tensors
        dy2 = dy.reshape(-1, ctx.w.rows).to(torch.bfloat16).contiguous()
        need_dx = ctx.needs_input_grad[0]
        dx, dA, dB = linear_bwd(dy2, x2, ctx.w, a16, b16, ctx.alpha, U=u, need_dx=need_dx)
        dx = dx.view(ctx.in_shape) if need_dx else None
        return dx, dA, dB, None, None


class QLoRALinear(torch.nn.Module):
    """A frozen weight (N x K, out x in) stored as NF4 with double-quantized constants, plus a LoRA adapter
    of rank r: A (r x K) initialised like a Kaiming-uniform linear, B (N x r) at zero, so the layer starts
    as the quantized base layer."""

    def __init__(self, weight: torch.Tensor, r: int = 64, alpha: float = 16.0,
                 generator: torch.Generator | None = None):
        super().__init__()
        if weight.dim() != 2 or not weight.is_cuda:
            raise ValueError("QLoRALinear: weight must be a 2-D CUDA tensor (out x in)")
        N, K = weight.shape
        self.w = quantize(weight.contiguous())
        self.r, self.alpha = r, float(alpha)
        bound = 1.0 / math.sqrt(K)
        a = torch.empty(r, K, device=weight.device, dtype=torch.float32).uniform_(-bound, bound, generator=generator)
        self.A = torch.nn.Parameter(a)
        self.B = torch.nn.Parameter(torch.zeros(N, r, device=weight.device, dtype=torch.float32))

    @property
    def in_features(self) -> int:
        return self.w.cols

    @property
    def out_features(self) -> int:
        return self.w.rows

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return QLoRALinearFn.apply(x, self.A, self.B, self.w, self.alpha)


class RotaryFn(torch.autograd.Function):
    """(q', k') of bit_nf4_quantized_14_b200.rotary; the gradients are the same rotations turned back."""

    @staticmethod
    def forward(ctx, q: torch.Tensor, k: torch.Tensor | None, config: RotaryConfig, positions, offset: int):
        ctx.save_for_backward(positions)
        ctx.config, ctx.offset = config, offset
        return _rotary(_aligned(q), _aligned(k), config, positions, offset)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        (positions,) = ctx.saved_tensors
        dq, dk = (_aligned(g if g is None or g.stride(-1) == 1 else g.contiguous()) for g in (dq, dk))
        dq, dk = _rotary(dq, dk, ctx.config, positions, ctx.offset, inverse=True)
        return dq, dk, None, None, None


def rotary(q: torch.Tensor, k: torch.Tensor | None, config: RotaryConfig, positions: torch.Tensor | None = None,
           offset: int = 0):
    """Differentiable rotary positions (see bit_nf4_quantized_14_b200.rotary): returns (q', k'). Heads, or gradients,
    that do not begin on 16 bytes (a part of a head behind an odd prefix) are copied first."""
    return RotaryFn.apply(q, k, config, positions, offset)


class VocabLossFn(torch.autograd.Function):
    """Cross entropy of x W^T. A mean or a sum leaves dX with the loss itself, kept until the backward scales it
    by the gradient of the loss; per-token losses are differentiated in the backward, once their gradients
    are known (the logits are formed again then)."""

    @staticmethod
    def forward(ctx, x, head, targets, ignore_index: int, reduction: str):
        x2 = _aligned(x.reshape(-1, x.shape[-1]).to(torch.bfloat16).contiguous())
        need = ctx.needs_input_grad[0] and reduction != "none"
        loss, dx = _vocab_loss(x2, head, targets.reshape(-1).contiguous(), ignore_index, reduction, need_dx=need)
        ctx.ignore_index, ctx.reduction, ctx.like = ignore_index, reduction, x.shape
        if reduction == "none":
            ctx.save_for_backward(x2, head, targets)
            return loss.view(targets.shape)
        ctx.save_for_backward(dx)
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        if not ctx.needs_input_grad[0]:
            return None, None, None, None, None
        if ctx.reduction == "none":
            x2, head, targets = ctx.saved_tensors
            _, dx = _vocab_loss(x2, head, targets.reshape(-1).contiguous(), ctx.ignore_index, "none",
                                dloss=dloss.reshape(-1).float().contiguous())
        else:
            dx = ctx.saved_tensors[0] * dloss        # fp32 product, rounded once more to bf16
        return dx.view(ctx.like), None, None, None, None


def vocab_loss(x: torch.Tensor, head: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
               reduction: str = "mean") -> torch.Tensor:
    """Differentiable vocabulary loss of hidden states x (..., K) with a frozen bf16 head (V x K) and targets
    (...): the cross entropy of x head^T without its logits (see bit_nf4_quantized_14_b200.vocab_loss). x is taken
    in bf16, copied where it does not begin on 16 bytes. A head that wants a gradient is refused: it would get none."""
    if head.requires_grad and torch.is_grad_enabled():
        raise ValueError("vocab_loss: the head is frozen and gets no gradient (detach it)")
    return VocabLossFn.apply(x, head, targets, ignore_index, reduction)
