"""The measured operators: the router's balance loss and gradients, and the experts in 8-bit integers.

Five operators, each with its plain form (elementary torch operations) and the call of
``combine_expert_ffn_b200`` that a user makes:

  balance_loss      per-expert counts, mean normalised affinities and the sequence-wise balance
                    loss of a router's affinities            -> ``moe_balance_loss``
  route_backward    gradient of the gates and of that loss with respect to the router's logits
                                                             -> ``moe_route_backward``
  combine_backward  gradient of the gate-weighted combine: the expert outputs' and the gates'
                                                             -> ``moe_combine_backward``
  dispatch_int8     counting-sort dispatch of the token copies with one int8 scale per token
                                                             -> ``moe_dispatch_int8``
  expert_ffn_int8   grouped SwiGLU experts as int8 matrix products, a scale for each token row and
                    each weight channel                      -> ``moe_expert_ffn_int8``

A case is a dict of plain values; ``op`` names the operator, the other keys are its sizes.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # a fine-tuning micro-batch: latency of the loss and its gradient
        {"name": "balance_micro", "op": "balance_loss", "T": 520, "E": 40, "K": 6, "n_seq": 3},
        # a pre-training step of the 256-expert router on packed documents of very unlike lengths
        {"name": "balance_docs", "op": "balance_loss", "T": 262144, "E": 256, "K": 8, "n_seq": 61},
        # router gradient of one batch of the 256-expert layer, sigmoid affinities
        {"name": "router_grad_batch", "op": "route_backward", "T": 8192, "E": 256, "K": 8,
         "n_seq": 4, "router": 0},
        # ... of a long accumulated batch of a 64-expert layer, sqrt(softplus) affinities
        {"name": "router_grad_long", "op": "route_backward", "T": 196601, "E": 64, "K": 6,
         "n_seq": 48, "router": 1},
        # combine's gradient, a mid-sized layer and the widest one
        {"name": "combine_grad_mid", "op": "combine_backward", "T": 1021, "d": 2048, "K": 6},
        {"name": "combine_grad_wide", "op": "combine_backward", "T": 8192, "d": 7168, "K": 8},
        # serving: a decode batch's dispatch, and a prefill batch's
        {"name": "dispatch_decode", "op": "dispatch_int8", "T": 128, "d": 7168, "E": 256, "K": 8,
         "skew": 0.0},
        {"name": "dispatch_prefill", "op": "dispatch_int8", "T": 8192, "d": 7168, "E": 256, "K": 8,
         "skew": 1.2},
        # serving: a single token, a decode batch, prefill of a mid-sized and of the widest layer
        {"name": "experts_token", "op": "expert_ffn_int8", "T": 1, "d": 7168, "E": 256, "K": 8,
         "d_ff": 2048, "n_shared": 1, "d_ff_shared": 2048, "skew": 0.0},
        {"name": "experts_decode", "op": "expert_ffn_int8", "T": 128, "d": 7168, "E": 256, "K": 8,
         "d_ff": 2048, "n_shared": 1, "d_ff_shared": 2048, "skew": 0.0},
        {"name": "experts_mid", "op": "expert_ffn_int8", "T": 4096, "d": 2048, "E": 64, "K": 6,
         "d_ff": 1408, "n_shared": 2, "d_ff_shared": 1408, "skew": 0.6},
        {"name": "experts_prefill", "op": "expert_ffn_int8", "T": 8192, "d": 7168, "E": 256,
         "K": 8, "d_ff": 2048, "n_shared": 1, "d_ff_shared": 2048, "skew": 0.0},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance_loss", "route_backward", "combine_backward", "dispatch_int8",
                     "expert_ffn_int8", "expert_ffn_int8"])
    if op in ("balance_loss", "route_backward"):
        E = rng.choice([rng.randint(2, 64), rng.randint(65, 300), 64, 128, 256, 1024])
        T = _log(rng, 1, min(262144, (1 << 26) // E))
        c = {"op": op, "T": T, "E": E, "K": rng.randint(1, min(16, E)),
             "n_seq": _log(rng, 1, max(1, min(T, 512)))}
        if op == "route_backward":
            c["router"] = rng.randint(0, 1)
        return c
    if op == "combine_backward":
        d = 64 * _log(rng, 1, 112)
        K = rng.randint(1, 10)
        return {"op": op, "T": _log(rng, 1, min(32768, 8192 * 7168 * 8 // (d * K))), "d": d, "K": K}
    E = rng.choice([rng.randint(4, 64), rng.randint(65, 256), 64, 256])
    K = rng.randint(1, min(8, E))
    skew = rng.choice([0.0, 0.0, 0.6, 1.2])
    if op == "dispatch_int8":
        d = 64 * _log(rng, 1, 112)
        return {"op": op, "T": _log(rng, 1, min(32768, 8192 * 7168 * 8 // (d * K))), "d": d,
                "E": E, "K": K, "skew": skew}
    d, d_ff = 64 * _log(rng, 2, 112), 64 * _log(rng, 1, 32)
    n_shared = rng.randint(0, 2)
    return {"op": op, "T": _log(rng, 1, 8192), "d": d, "E": E, "K": K, "d_ff": d_ff,
            "n_shared": n_shared, "d_ff_shared": d_ff if n_shared else 0, "skew": skew}


# ------------------------------------------------------------------------------ inputs
def _popularity(E, skew):
    p = np.arange(1, E + 1, dtype=np.float64) ** -skew
    return p / p.sum()


def _routing(T, E, K, skew, g):
    """[T, K] int32: K distinct experts a token, sampled without replacement by popularity."""
    p = torch.from_numpy(_popularity(E, skew)).to(DEV, torch.float32)
    p = p[torch.randperm(E, device=DEV, generator=g)]
    u = torch.rand(T, E, device=DEV, generator=g).clamp_min_(1e-30)
    return torch.topk(u.log_().div_(p), K, dim=1).indices.to(torch.int32)


def _bounds(T, n_seq, g):
    """[n_seq + 1] int32 sequence starts: ragged, some empty, a few padding tokens at the end."""
    end = T - T // 97
    cut = torch.randint(0, end + 1, (n_seq - 1,), device=DEV, generator=g).sort().values
    ends = torch.tensor([end], device=DEV)
    return torch.cat([ends * 0, cut, ends]).to(torch.int32)


def _codes(shape, g):
    """int8 codes of a bell-like spread over -126 .. 126."""
    a = torch.randint(-63, 64, shape, dtype=torch.int8, device=DEV, generator=g)
    return a.add_(torch.randint(-63, 64, shape, dtype=torch.int8, device=DEV, generator=g))


def _scales(n, mean, g):
    return (torch.rand(n, device=DEV, generator=g) + 0.5).mul_(mean)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s, op = {"case": case}, case["op"]
    T, K, E = case["T"], case["K"], case.get("E", 0)
    if op in ("balance_loss", "route_backward"):
        logits = torch.randn(T, E, device=DEV, generator=g)
        logits += 1.5 * torch.randn(E, device=DEV, generator=g)  # experts differ in popularity
        if case.get("router"):
            s["scores"] = torch.nn.functional.softplus(logits).sqrt_()
        else:
            s["scores"] = torch.sigmoid(logits)
        s["topk_idx"] = torch.topk(s["scores"], K, dim=1).indices.to(torch.int32)
        s["seq_offsets"] = _bounds(T, case["n_seq"], g)
        s["alpha"] = 1e-3
        if op == "route_backward":
            s["d_topk_w"] = torch.randn(T, K, device=DEV, generator=g)
            s["d_loss"] = torch.rand(case["n_seq"], device=DEV, generator=g) * 1e4
            s["counts"] = _counts(s["topk_idx"], s["seq_offsets"], E)
    elif op == "combine_backward":
        s["d_out"] = torch.randn(T, case["d"], device=DEV, generator=g).to(torch.bfloat16)
        s["y_perm"] = torch.randn(T * K, case["d"], device=DEV, generator=g).to(torch.bfloat16)
        s["inv_perm"] = torch.randperm(T * K, device=DEV, generator=g).to(torch.int32).view(T, K)
        w = torch.rand(T, K, device=DEV, generator=g) + 0.05
        s["topk_w"] = w / w.sum(1, keepdim=True)
    elif op == "dispatch_int8":
        row = torch.rand(T, 1, device=DEV, generator=g) + 0.5  # tokens differ in magnitude
        s["x"] = torch.randn(T, case["d"], device=DEV, generator=g).mul_(row).to(torch.bfloat16)
        s["topk_idx"] = _routing(T, E, K, case["skew"], g)
    else:
        d, ff, ffs = case["d"], case["d_ff"], case["n_shared"] * case["d_ff_shared"]
        idx = _routing(T, E, K, case["skew"], g)
        n = torch.bincount(idx.flatten().long(), minlength=E).tolist()
        s["segments"] = [0] + np.cumsum(n).tolist()
        s["offsets"] = torch.tensor(s["segments"], dtype=torch.int32, device=DEV)
        s["x_perm_q"] = _codes((T * K, d), g)
        s["x_scale"] = _scales(T * K, 0.02, g)
        s["x"] = torch.randn(T, d, device=DEV, generator=g).to(torch.bfloat16)
        s["w"] = {"w_gate": _codes((E, ff, d), g), "w_up": _codes((E, ff, d), g),
                  "w_down": _codes((E, d, ff), g)}
        # weights of variance 1 / fan-in: the codes' own spread is 52
        for name, rows, fan in (("w_gate", ff, d), ("w_up", ff, d), ("w_down", d, ff)):
            s["w"][name + "_scale"] = _scales((E, rows), fan ** -0.5 / 52, g)
        if ffs:
            ns, fs = case["n_shared"], case["d_ff_shared"]
            s["w"] |= {"ws_gate": _codes((ns, fs, d), g), "ws_up": _codes((ns, fs, d), g),
                       "ws_down": _codes((ns, d, fs), g),
                       "ws_gate_scale": _scales((ns, fs), d ** -0.5 / 52, g),
                       "ws_up_scale": _scales((ns, fs), d ** -0.5 / 52, g),
                       "ws_down_scale": _scales(d, ffs ** -0.5 / 52, g)}
    if own:
        _kept(s)
    return s


def _kept(s):
    """The workspace and output buffers that a program keeps from call to call."""
    import combine_expert_ffn_b200 as moe

    c = s["case"]
    s["moe"], op, T, K, E = moe, c["op"], c["T"], c["K"], c.get("E", 16)
    cfg = s["cfg"] = moe.MoeConfig(T, c.get("d", 64), max(E, K), 1, K, 1, c.get("d_ff", 64),
                                   c.get("n_shared", 0), c.get("d_ff_shared", 0),
                                   c.get("router", 0), 0)

    def new(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=DEV)

    if op == "balance_loss":
        s["ws"] = moe.alloc_workspace(cfg)
        s["out"] = {"counts": new(c["n_seq"], E, dtype=torch.int32), "prob": new(c["n_seq"], E),
                    "loss": new(c["n_seq"])}
    elif op == "route_backward":
        s["out"] = {"d_logits": new(T, E)}
    elif op == "combine_backward":
        s["out"] = {"d_y_perm": new(T * K, c["d"], dtype=torch.bfloat16), "d_topk_w": new(T, K)}
    elif op == "dispatch_int8":
        s["ws"] = moe.alloc_workspace(cfg)
        s["send"] = new(1, 1, dtype=torch.int32)
        s["out"] = {"counts": new(E, dtype=torch.int32), "offsets": new(E + 1, dtype=torch.int32),
                    "perm_token": new(T * K, dtype=torch.int32),
                    "inv_perm": new(T, K, dtype=torch.int32),
                    "x_perm_q": new(T * K, c["d"], dtype=torch.int8), "x_scale": new(T * K)}
    else:
        s["weights"] = moe.Int8Weights(**s["w"])
        s["ws"] = moe.alloc_int8_workspace(cfg)
        s["out"] = {"y_perm": new(T * K, c["d"], dtype=torch.bfloat16)}
        if c["n_shared"]:
            s["out"]["y_shared"] = new(T, c["d"], dtype=torch.bfloat16)


# ------------------------------------------------------------------------------ the pass
def run(state):
    op = state["case"]["op"]
    return _own_run(state, op) if own else _PLAIN[op](state)


def _own_run(s, op):
    moe, cfg, o = s["moe"], s["cfg"], s["out"]
    if op == "balance_loss":
        moe.moe_balance_loss(cfg, s["scores"], s["topk_idx"], s["seq_offsets"], s["alpha"],
                             o["counts"], o["prob"], o["loss"], s["ws"])
    elif op == "route_backward":
        moe.moe_route_backward(cfg, s["scores"], s["topk_idx"], s["d_topk_w"], s["seq_offsets"],
                               s["counts"], s["d_loss"], s["alpha"], o["d_logits"])
    elif op == "combine_backward":
        moe.moe_combine_backward(cfg, s["d_out"], s["y_perm"], s["inv_perm"], s["topk_w"],
                                 o["d_y_perm"], o["d_topk_w"])
    elif op == "dispatch_int8":
        moe.moe_dispatch_int8(cfg, s["x"], s["topk_idx"], o["counts"], o["offsets"], s["send"],
                              None, o["perm_token"], o["inv_perm"], o["x_perm_q"], o["x_scale"],
                              s["ws"])
    else:
        moe.moe_expert_ffn_int8(cfg, s["x_perm_q"], s["x_scale"], s["offsets"], s["weights"],
                                o["y_perm"], s["x"], o.get("y_shared"), s["ws"])
    return o


# ------------------------------------------------------------------------------ plain forms
def _sequence(T, seq_offsets):
    """The sequence of each token; the number of sequences for a token in none."""
    n = seq_offsets.numel() - 1
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    q = torch.searchsorted(seq_offsets[1:], t, right=True)
    return torch.where(t >= seq_offsets[0], q, n)


def _counts(topk_idx, seq_offsets, E):
    T, K = topk_idx.shape
    n = seq_offsets.numel() - 1
    c = torch.zeros((n + 1) * E, dtype=torch.int32, device=DEV)
    at = _sequence(T, seq_offsets)[:, None] * E + topk_idx
    c.index_add_(0, at.flatten(), torch.ones(T * K, dtype=torch.int32, device=DEV))
    return c.view(n + 1, E)[:n].contiguous()


def _normalised(scores):
    """Each row over its sum; a row of zeros stays one."""
    total = scores.sum(1, keepdim=True)
    return scores / total.masked_fill(total == 0, 1.0), total


def _plain_balance_loss(s):
    scores, idx, offs = s["scores"], s["topk_idx"], s["seq_offsets"]
    E, K = scores.shape[1], idx.shape[1]
    counts = _counts(idx, offs, E)
    p, _ = _normalised(scores)
    # sums over up to T tokens, as differences of running sums in 64 bits
    upto = torch.nn.functional.pad(p.t().double().cumsum(1), (1, 0))
    total = (upto[:, offs[1:].long()] - upto[:, offs[:-1].long()]).t()
    length = (offs[1:] - offs[:-1]).double().clamp_min(1.0)[:, None]
    prob = total / length
    loss = s["alpha"] * (counts * (E / K) / length * prob).sum(1)
    return {"counts": counts, "prob": prob.float(), "loss": loss.float()}


def _plain_route_backward(s):
    scores, idx, offs = s["scores"], s["topk_idx"].long(), s["seq_offsets"]
    (T, E), K = scores.shape, idx.shape[1]
    # the balance loss: counts less their mean, in 64 bits (balanced experts nearly cancel)
    length = (offs[1:] - offs[:-1]).double().clamp_min(1.0)
    pull = s["d_loss"].double() * s["alpha"] * E / (K * length * length)
    excess = pull[:, None] * (s["counts"] - s["counts"].double().mean(1, keepdim=True))
    excess = torch.cat([excess, excess.new_zeros(1, E)])[_sequence(T, offs)]
    p, total = _normalised(scores.double())
    d = (excess - (excess * p).sum(1, keepdim=True)) / total.masked_fill(total == 0, math.inf)
    # the gates: each chosen affinity over the sum of the chosen
    chosen = scores.gather(1, idx)
    w, both = _normalised(chosen)
    dw = s["d_topk_w"]
    gate = (dw - (dw * w).sum(1, keepdim=True)) / both.masked_fill(both == 0, math.inf)
    d.scatter_add_(1, idx, gate.double())
    sd = scores.double()
    if s["case"]["router"]:  # s = sqrt(softplus(L)): sigmoid(L) / (2 s), sigmoid(L) = 1 - e^(-s^2)
        d *= torch.where(sd > 0, -torch.expm1(-sd * sd) / (2 * sd), 0.0)
    else:
        d *= sd * (1 - sd)
    return {"d_logits": d.float()}


def _plain_combine_backward(s):
    d_out, rows = s["d_out"].float(), s["inv_perm"].long()
    y = s["y_perm"].float()[rows.flatten()].view(*rows.shape, -1)
    d_w = (y * d_out[:, None]).sum(2)
    d_y = torch.empty_like(s["y_perm"])
    d_y[rows.flatten()] = (s["topk_w"][:, :, None] * d_out[:, None]).to(d_y.dtype).flatten(0, 1)
    return {"d_y_perm": d_y, "d_topk_w": d_w}


def _quantise(x):
    """Codes and scales of the rows of x: the row's largest magnitude becomes 127. The scale is a
    32-bit number, and the quotient is rounded to 32 bits before it is rounded to a code (64-bit
    division and one rounding: the correctly rounded quotient)."""
    scale = (x.abs().amax(1, keepdim=True).double() / 127).float()
    q = (x.double() / scale.masked_fill(scale == 0, 1.0).double()).float().round()
    return q, scale


def _plain_dispatch_int8(s):
    x, idx, E = s["x"], s["topk_idx"], s["case"]["E"]
    T, K = idx.shape
    order = idx.flatten().argsort(stable=True)
    counts = torch.zeros(E, dtype=torch.int32, device=DEV)
    counts.index_add_(0, idx.flatten(), torch.ones(T * K, dtype=torch.int32, device=DEV))
    offsets = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
    inv = torch.empty(T * K, dtype=torch.int32, device=DEV)
    inv[order] = torch.arange(T * K, dtype=torch.int32, device=DEV)
    tok = order // K
    q, scale = _quantise(x.float())
    return {"counts": counts, "offsets": offsets, "perm_token": tok.to(torch.int32),
            "inv_perm": inv.view(T, K), "x_perm_q": q.to(torch.int8)[tok],
            "x_scale": scale.flatten()[tok]}


def _plain_expert(q, scale, gate, gate_s, up, up_s, down, down_s):
    """One expert on rows of codes q with scales [rows, 1]."""
    a = (q @ gate.float().t()) * scale * gate_s
    b = (q @ up.float().t()) * scale * up_s
    hq, hs = _quantise(a / (1 + torch.exp(-a)) * b)
    return ((hq @ down.float().t()) * hs * down_s).to(torch.bfloat16)


def _plain_expert_ffn_int8(s):
    w, seg = s["w"], s["segments"]
    y = torch.empty(s["x_perm_q"].shape, dtype=torch.bfloat16, device=DEV)
    for e in range(len(seg) - 1):
        lo, hi = seg[e], seg[e + 1]
        if hi > lo:
            y[lo:hi] = _plain_expert(
                s["x_perm_q"][lo:hi].float(), s["x_scale"][lo:hi, None], w["w_gate"][e],
                w["w_gate_scale"][e], w["w_up"][e], w["w_up_scale"][e], w["w_down"][e],
                w["w_down_scale"][e])
    out = {"y_perm": y}
    if "ws_gate" in w:  # the shared experts are one expert of their summed width
        q, scale = _quantise(s["x"].float())
        out["y_shared"] = _plain_expert(
            q, scale, w["ws_gate"].flatten(0, 1), w["ws_gate_scale"].flatten(),
            w["ws_up"].flatten(0, 1), w["ws_up_scale"].flatten(),
            w["ws_down"].permute(1, 0, 2).flatten(1), w["ws_down_scale"])
    return out


_PLAIN = {"balance_loss": _plain_balance_loss, "route_backward": _plain_route_backward,
          "combine_backward": _plain_combine_backward, "dispatch_int8": _plain_dispatch_int8,
          "expert_ffn_int8": _plain_expert_ffn_int8}


# ------------------------------------------------------------------------------ cost
def work(case):
    T, K = case["T"], case["K"]
    op, E, d = case["op"], case.get("E", 0), case.get("d", 0)
    if op == "balance_loss":
        return {"bytes": 4 * T * (E + K) + 4 * case["n_seq"] * (2 * E + 2), "flops": 3 * T * E}
    if op == "route_backward":
        return {"bytes": 8 * T * (E + K) + 4 * case["n_seq"] * (E + 2), "flops": 8 * T * E}
    if op == "combine_backward":
        return {"bytes": 2 * T * d * (1 + 2 * K) + 12 * T * K, "flops": 3 * T * K * d}
    if op == "dispatch_int8":
        return {"bytes": 2 * T * d + T * K * (d + 4) + 12 * T * K + 8 * E, "flops": 3 * T * d}
    ff, ffs = case["d_ff"], case["n_shared"] * case["d_ff_shared"]
    hit = np.minimum(1.0, K * _popularity(E, case["skew"]))
    active = float((1 - (1 - hit) ** T).sum())  # experts that some token chose
    weights = (active * ff + ffs) * d * 3
    rows = T * K * (3 * d + 4) + (4 * T * d if ffs else 0)
    return {"bytes": weights + rows, "flops": 6 * d * T * (K * ff + ffs)}


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s)


def _slices(offsets):
    o = offsets.tolist()
    return [(o[i], o[i + 1]) for i in range(len(o) - 1)]


def _exact_balance_loss(s):
    (_, E), K = s["scores"].shape, s["topk_idx"].shape[1]
    prob, loss = [], []
    for lo, hi in _slices(s["seq_offsets"]):
        a = s["scores"][lo:hi].double()
        n = max(1, hi - lo)
        f = torch.zeros(E, dtype=torch.float64, device=DEV)
        f.scatter_add_(0, s["topk_idx"][lo:hi].flatten().long(),
                       torch.ones((hi - lo) * K, dtype=torch.float64, device=DEV))
        prob.append((a / a.sum(1, keepdim=True)).sum(0) / n)
        loss.append(s["alpha"] * (f * E / (K * n)).dot(prob[-1]))
    return {"counts": None, "prob": torch.stack(prob), "loss": torch.stack(loss)}


def _exact_route_backward(s):
    """By differentiation of the definition in 64 bits: loss and gates as functions of the
    affinities, the affinities as functions of the logits that give them."""
    a0 = s["scores"].double()
    if s["case"]["router"]:
        logits = torch.log(torch.expm1(a0 * a0))
    else:
        logits = torch.log(a0 / (1 - a0))
    logits.requires_grad_()
    a = (torch.logaddexp(logits, torch.zeros_like(logits)).sqrt() if s["case"]["router"]
         else torch.sigmoid(logits))
    E, K = a.shape[1], s["topk_idx"].shape[1]
    goal = a.new_zeros(())
    share = a / a.sum(1, keepdim=True)
    for i, (lo, hi) in enumerate(_slices(s["seq_offsets"])):
        if hi > lo:
            f = s["counts"][i].double() * E / (K * (hi - lo))
            goal = goal + s["d_loss"][i].double() * s["alpha"] * f.dot(share[lo:hi].mean(0))
    chosen = a.gather(1, s["topk_idx"].long())
    gates = chosen / chosen.sum(1, keepdim=True)
    goal = goal + (gates * s["d_topk_w"].double()).sum()
    return {"d_logits": torch.autograd.grad(goal, logits)[0]}


def _exact_combine_backward(s):
    T, K = s["inv_perm"].shape
    d_out = s["d_out"].double()
    slot = torch.empty(T * K, dtype=torch.long, device=DEV)
    slot[s["inv_perm"].flatten().long()] = torch.arange(T * K, device=DEV)
    d_w = torch.empty(T * K, dtype=torch.float64, device=DEV)
    d_y = torch.empty(s["y_perm"].shape, dtype=torch.float64, device=DEV)
    for rows in torch.arange(T * K, device=DEV).split(8192):
        at = slot[rows]
        g = d_out[at // K]
        d_w[at] = torch.einsum("rc,rc->r", g, s["y_perm"][rows].double())
        d_y[rows] = g * s["topk_w"].flatten()[at].double()[:, None]
    return {"d_y_perm": d_y, "d_topk_w": d_w.view(T, K)}


def _exact_dispatch_int8(s):
    tok = torch.sort(s["topk_idx"].flatten().long(), stable=True).indices // s["case"]["K"]
    scale = s["x"].double().abs().max(1).values / 127
    return {"counts": None, "offsets": None, "perm_token": None, "inv_perm": None,
            "x_perm_q": None, "x_scale": scale[tok]}


def _exact_expert(rows, scale, gate, up, down):
    """In 64 bits; `gate`, `up` and `down` are (codes, channel scales)."""
    x = rows.double() * scale.double()[:, None]
    a, b = (x @ (m[0].double() * m[1].double()[:, None]).t() for m in (gate, up))
    h = a * torch.sigmoid(a) * b
    step = h.abs().max(1, keepdim=True).values / 127
    h = torch.where(step > 0, torch.round(h / step) * step, 0.0)
    return h @ (down[0].double() * down[1].double()[:, None]).t()


def _exact_expert_ffn_int8(s):
    w, out = s["w"], {}
    parts = []
    for e, (lo, hi) in enumerate(_slices(s["offsets"])):
        if hi > lo:
            parts.append(_exact_expert(s["x_perm_q"][lo:hi], s["x_scale"][lo:hi],
                                       *((w[k][e], w[k + "_scale"][e])
                                         for k in ("w_gate", "w_up", "w_down"))))
    out["y_perm"] = torch.cat(parts)
    if "ws_gate" in w:
        # the shared experts' codes as the operator defines them: 32-bit scales and quotients,
        # which settle the many exact ties of 8-bit mantissas over a common divisor
        x = s["x"].double()
        step = (x.abs().max(1).values / 127).float().double()
        q = torch.round((x / torch.where(step > 0, step, 1.0)[:, None]).float().double())
        down = torch.cat(list(w["ws_down"]), dim=1)
        out["y_shared"] = _exact_expert(
            q, step, *((w[k].reshape(-1, x.shape[1]), w[k + "_scale"].reshape(-1))
                       for k in ("ws_gate", "ws_up")), (down, w["ws_down_scale"]))
    return out


_EXACT = {"balance_loss": _exact_balance_loss, "route_backward": _exact_route_backward,
          "combine_backward": _exact_combine_backward, "dispatch_int8": _exact_dispatch_int8,
          "expert_ffn_int8": _exact_expert_ffn_int8}
