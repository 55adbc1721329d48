"""Rows of a language model moved by an index: the embedding lookup with a scale
and its gradient, and a mixture of experts' tokens sorted by expert, dispatched
and combined. Tensor-level calls of the C ABI (rmsnorm_embedding_*,
rmsnorm_expert_* in include/rmsnorm.h), in the manner of ``image_ops``: checks,
outputs from PyTorch, ``RMSNormError`` on a non-OK status, the tensors' own
device, its current stream or ``stream`` as if that were the current one.
``autograd`` holds the differentiable forms.

Sums are fp32 in an order that the sizes and the alignment alone fix, without
floating-point atomics: the same bits on every run, gradients included.
"""
from __future__ import annotations

from typing import NamedTuple

from . import image_ops
from .image_ops import _binding, _handle


class ExpertRows(NamedTuple):
    """Where a router's choices go once sorted by expert (all int32)."""

    position: object  #: [..., K]: the row of each choice, -1 if dropped
    source: object  #: [R]: the choice (token * K + k) of each row, -1 of rows without one
    offsets: object  #: [E + 1]: the first row of each expert, and behind the last one's
    counts: object  #: [E]: choices of each expert


def embedding_forward(ids, table, scale: float = 1.0, out_dtype=None, stream=None):
    """scale * table[ids]: ids int32 or int64 of any shape (up to two strides:
    tokens[:, :-1] is one), table [V, H] with dense rows; ids outside [0, V) give
    rows of zeros. out_dtype: the table's type, or a 16-bit one beside an fp32 table."""
    return (image_ops._bound or _binding()).embedding_forward(ids, table, scale, out_dtype,
                                                              _handle(stream))


def embedding_backward(ids, dy, num_embeddings: int, scale: float = 1.0, padding_idx=None,
                       grad_dtype=None, out=None, accumulate: bool = False, stream=None):
    """The table's gradient [num_embeddings, H] from dy [*ids.shape, H]: of each row
    the scaled sum over its tokens. Ids outside the table or equal to padding_idx
    (negative: from the end) count for nothing. grad_dtype: dy's type or fp32. `out` gives
    the tensor to write (rows without a token become zero); with `accumulate` the
    gradient is added to it."""
    return (image_ops._bound or _binding()).embedding_backward(
        ids, dy, num_embeddings, scale, padding_idx, grad_dtype, out, accumulate, _handle(stream))


def expert_sort(experts, num_experts: int, align: int = 1, stream=None) -> ExpertRows:
    """The choices experts [..., K] (int32 or int64; outside [0, num_experts): dropped)
    sorted by expert, in their order within an expert, every expert's first row a
    multiple of `align`. The rows number R = rmsnorm_expert_rows(...), however the
    choices fall. The four tensors share one allocation."""
    return ExpertRows._make((image_ops._bound or _binding()).expert_sort(experts, num_experts, align,
                                                                        _handle(stream)))


def expert_dispatch_forward(x, position, source, stream=None):
    """rows [R, H] of x [..., H]: each token's row at the positions of its choices,
    zeros where a row has no choice."""
    return (image_ops._bound or _binding()).expert_dispatch_forward(x, position, source,
                                                                    _handle(stream))


def expert_dispatch_backward(drows, position, stream=None):
    """dx [..., H]: the sum of drows [R, H] over each token's choices."""
    return (image_ops._bound or _binding()).expert_dispatch_backward(drows, position,
                                                                     _handle(stream))


def expert_combine_forward(rows, position, weights=None, residual=None, stream=None):
    """y [..., H]: residual (None: 0) and each token's weighted sum of its choices'
    rows [R, H]; weights [..., K] in the rows' type or fp32 (None: 1)."""
    return (image_ops._bound or _binding()).expert_combine_forward(rows, position, weights,
                                                                   residual, _handle(stream))


def expert_combine_backward(dy, rows, position, source, weights=None, stream=None):
    """drows [R, H] and dweights [..., K] (fp32; None without weights) of the combine.
    The residual's gradient is dy."""
    return (image_ops._bound or _binding()).expert_combine_backward(dy, rows, position, source,
                                                                    weights, _handle(stream))
