"""64-bit definitions behind the tests of the router's training side: the balance loss, the gates
and the combine, as functions that autograd and finite differences can take apart."""
from __future__ import annotations

import torch

EPS = 2.0 ** -24  # half a unit in the last place of an fp32 value near 1, relative


def affinity(logits, router):
    """Affinities of float64 logits: sigmoid (0) or sqrt(softplus) (1)."""
    if router:
        return torch.logaddexp(logits, torch.zeros_like(logits)).sqrt()
    return torch.sigmoid(logits)


def logits_of(scores, router):
    """The float64 logits whose affinities are `scores`, where 0 < scores (< 1 for sigmoid)."""
    s = scores.double()
    return torch.log(torch.expm1(s * s)) if router else torch.log(s) - torch.log1p(-s)


def spans(seq_offsets, T):
    if seq_offsets is None:
        return [(0, T)]
    o = [int(v) for v in seq_offsets]
    return list(zip(o[:-1], o[1:]))


def counts(topk_idx, seq_offsets, E):
    T = topk_idx.shape[0]
    return torch.stack([torch.bincount(topk_idx[lo:hi].flatten().long(), minlength=E)
                        for lo, hi in spans(seq_offsets, T)])


def balance_loss(scores, n, seq_offsets, alpha, K):
    """(prob [n_seq, E], loss [n_seq]) of float64 affinities and the counts n [n_seq, E]."""
    T, E = scores.shape
    prob, loss = [], []
    for s, (lo, hi) in enumerate(spans(seq_offsets, T)):
        total = scores[lo:hi].sum(1, keepdim=True)
        p = scores[lo:hi] / torch.where(total == 0, torch.ones_like(total), total)
        prob.append(p.sum(0) / max(1, hi - lo))
        loss.append(alpha * E / (K * max(1, hi - lo)) * (n[s].double() * prob[-1]).sum())
    return torch.stack(prob), torch.stack(loss)


def gates(scores, topk_idx):
    chosen = scores.gather(1, topk_idx.long())
    return chosen / chosen.sum(1, keepdim=True)


def router_goal(scores, topk_idx, d_topk_w, seq_offsets, n, d_loss, alpha):
    """The scalar whose gradient moe_route_backward computes."""
    goal = scores.new_zeros(())
    if d_topk_w is not None:
        goal = goal + (gates(scores, topk_idx) * d_topk_w.double()).sum()
    if d_loss is not None:
        _, loss = balance_loss(scores, n, seq_offsets, alpha, topk_idx.shape[1])
        goal = goal + (loss * d_loss.double()).sum()
    return goal
