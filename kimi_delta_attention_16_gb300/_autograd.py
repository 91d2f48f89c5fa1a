"""What the differentiable operations share: the choice of how inputs are kept for the backward pass,
and the checks that a step inside a stream capture can be differentiated there.

A leaf tensor has one gradient accumulator for all graphs that are alive, and it belongs to the stream on which the
first of them was built.  A captured backward pass makes that stream wait for the capture.  Another stream of the
program joins the capture by that; the default stream must not, and the attempt ends the process.  So each call marks its
leaves' accumulators with its stream, and a capture that meets the default stream's mark raises: an eager graph of that
leaf, or whatever else holds its accumulator (hooks, a data-parallel wrapper), is still alive."""
from __future__ import annotations

import torch

SAVED = ("io", "e4m3")  # how a layer keeps its large inputs for its backward pass
_STREAM = "kda_stream"
_DEFAULT = 0  # the handle of the default stream


def check_saved(saved: str) -> None:
    if saved not in SAVED:
        raise ValueError(f"saved must be one of {SAVED}, got {saved!r}")


def _raise(where: str) -> None:
    raise RuntimeError(f"{where} is being captured while a gradient accumulator of one of its leaves, made on the default "
                       "stream, is alive: before the capture drop the eager graphs of that leaf (their outputs and losses) "
                       "and what holds accumulators (hooks, wrappers), or build them on another stream")


def apply(function, where: str, *args, early: bool = True):
    """function.apply(*args), with its leaves' accumulators marked.  early: inside a capture, refuses what its backward
    pass could not do in the same capture before anything is recorded (a forward pass that is captured alone runs
    under torch.no_grad())."""
    leaves = [a for a in args if isinstance(a, torch.Tensor) and a.requires_grad and a.is_leaf and a.is_cuda]
    if not leaves or not torch.is_grad_enabled():
        return function.apply(*args)
    stream = torch.cuda.current_stream().cuda_stream
    capturing = torch.cuda.is_current_stream_capturing()
    # held until the call is part of the graph, which keeps the accumulators (and their marks) alive
    nodes = [torch.autograd.graph.get_gradient_edge(a).node for a in leaves]
    for node in nodes:
        mark = node.metadata.setdefault(_STREAM, stream)
        if early and capturing and mark == _DEFAULT:
            _raise(where)
    return function.apply(*args)


def check_backward(ctx, where: str) -> None:
    """Inside a function's backward: raises where the pass is being captured and would go on to an accumulator of the
    default stream."""
    if torch.cuda.is_current_stream_capturing():
        for node, _ in ctx.next_functions:
            if node is not None and node.metadata.get(_STREAM) == _DEFAULT:
                _raise(where)
