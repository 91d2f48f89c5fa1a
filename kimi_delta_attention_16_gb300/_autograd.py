"""What the differentiable operations share: the choice of how inputs are kept for the backward pass,
and the check that a call inside a stream capture can be differentiated there."""
from __future__ import annotations

import torch

SAVED = ("io", "e4m3")  # how a layer keeps its large inputs for its backward pass
_STREAM = "kda_stream"


def check_saved(saved: str) -> None:
    if saved not in SAVED:
        raise ValueError(f"saved must be one of {SAVED}, got {saved!r}")


def apply(function, where: str, *args):
    """function.apply(*args), refusing a capture that could not be differentiated.

    A leaf tensor has one gradient accumulator for all graphs that are alive, and it belongs to the stream on
    which the first of them was built.  A backward pass captured on another stream would wait on that one, which
    the capture forbids and which ends the process.  So each call marks its leaves' accumulators with its stream,
    and a call that is being captured raises when it meets another stream's mark: an eager graph of that leaf is
    still alive."""
    leaves = [a for a in args if isinstance(a, torch.Tensor) and a.requires_grad and a.is_leaf and a.is_cuda]
    if not leaves or not torch.is_grad_enabled():
        return function.apply(*args)
    stream = torch.cuda.current_stream().cuda_stream
    capturing = torch.cuda.is_current_stream_capturing()
    # held until the call is part of the graph, which keeps the accumulators (and their marks) alive
    nodes = [torch.autograd.graph.get_gradient_edge(a).node for a in leaves]
    for node in nodes:
        mark = node.metadata.setdefault(_STREAM, stream)
        if capturing and mark != stream:
            raise RuntimeError(f"{where} is being captured while a graph of one of its leaves, built on another stream, "
                               "is alive: drop that graph (its outputs and losses) before the capture, or capture the "
                               "forward and backward calls that this layer is made of")
    return function.apply(*args)
