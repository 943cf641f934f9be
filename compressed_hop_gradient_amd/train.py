"""Autograd forms of the training-step operators: dropout from the
counter-based generator, and the expert router with its balance loss.

A data-parallel step computes these per worker before its gradients go through
a round (``dq.Plan.allreduce``, or ``ddp_hook`` in DDP).  ``rnd`` is the round
index of the step and ``worker`` the worker's, as for the plan: masks differ
between workers, steps and call sites, and a recomputed forward pass draws the
same mask again.  Gradients are computed by kernels and cannot be
differentiated again.
"""
from collections import namedtuple

import torch
from torch.autograd.function import once_differentiable

from . import dq

Routing = namedtuple("Routing", "ids gates loss counts coef")


def _by_rows(t):
    """``t``, copied if its rows do not lie at one stride (as an expanded
    gradient's may not)."""
    if t.is_contiguous() or t.dim() == 2 and t.stride(1) == 1:
        return t
    return t.contiguous()


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, rnd, worker, site):
        ctx.args = (p, seed, worker, site)
        ctx.rnd = None if isinstance(rnd, torch.Tensor) else rnd
        if ctx.rnd is None:
            # a saved tensor: changing it before the backward pass, which would
            # draw another mask, is an error
            ctx.save_for_backward(rnd)
        return dq.dropout(_by_rows(x), p, None if residual is None else _by_rows(residual), seed, rnd, worker, site)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        dx = None
        if ctx.needs_input_grad[0]:
            p, seed, worker, site = ctx.args
            rnd = ctx.saved_tensors[0] if ctx.rnd is None else ctx.rnd
            dx = dq.dropout_backward(_by_rows(dout), p, seed, rnd, worker, site)
        return dx, dout if ctx.needs_input_grad[1] else None, None, None, None, None, None


def dropout(x, p, residual=None, training=True, seed=1, rnd=0, worker=0, site=0):
    """``residual + dropout(x)`` or ``dropout(x)``, differentiable by both; the
    mask is drawn again in the backward pass.  Arguments as ``dq.dropout``;
    without ``training`` nothing is dropped."""
    if not training:
        if residual is None:
            return x
        p = 0.0
    return _Dropout.apply(x, residual, p, seed, rnd, worker, site)


class _Route(torch.autograd.Function):
    """loss, *gates; ids, counts and coef, which have no gradient, go into
    ``found``."""

    @staticmethod
    def forward(ctx, top_k, renorm, masks, reduce, found, *logits):
        logits = [_by_rows(l) for l in logits]
        ids, gates, stats = dq.route(logits, top_k, renorm, masks)
        if reduce is not None:
            stats = stats.fold()
            reduce(stats)
        loss, coef, counts = dq.balance(stats, top_k)
        found += (ids, counts, coef)
        ctx.renorm = renorm
        ctx.save_for_backward(coef, *logits, *ids, *masks)
        ctx.set_materialize_grads(False)
        return (loss, *gates)

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, *dgates):
        coef, *saved = ctx.saved_tensors
        n = len(dgates)
        grads = [None] * n
        # without the loss, only the workers whose gates were used
        at = [w for w, dg in enumerate(dgates) if ctx.needs_input_grad[5 + w] and (dloss is not None or dg is not None)]
        if at:
            dgs = [dgates[w] if dgates[w] is None else dgates[w].contiguous() for w in at]
            for w, d in zip(at, dq.route_backward([saved[w] for w in at], [saved[n + w] for w in at], dgs,
                                                  None if dloss is None else coef, dloss, ctx.renorm,
                                                  [saved[2 * n + w] for w in at])):
                grads[w] = d
        return (None, None, None, None, None, *grads)


def route(logits, top_k, renorm=True, masks=None, reduce=None):
    """Expert choices of all workers' tokens and the balance loss of them
    together: ``Routing(ids, gates, loss, counts, coef)``.

    ``logits`` is one [tokens, experts] tensor, or a list with one per worker;
    ``ids`` and ``gates`` come in the same form, ``masks`` goes in so.  ``gates`` and
    ``loss`` are differentiable by the logits.  See ``dq.route`` and
    ``dq.balance``.  ``reduce`` is called with the statistics of these workers
    before the loss is computed: where the other workers are other processes,
    ``torch.distributed.all_reduce`` makes it the loss over all of them (the
    gradient stays that of the whole loss by the local logits, so ranks' gradients
    are to be summed, not averaged)."""
    one = isinstance(logits, torch.Tensor)
    ls = [logits] if one else list(logits)
    ms = [masks] * len(ls) if masks is None or one else list(masks)
    found = []
    loss, *gates = _Route.apply(top_k, renorm, ms, reduce, found, *ls)
    ids, counts, coef = found
    return Routing(ids[0] if one else ids, gates[0] if one else gates, loss, counts, coef)
