"""64-bit definition of the int8 experts, and how far a correct kernel may be from it.

Codes of a row: s = fp32(amax / 127), q = rint(fp32(x / s)).  The integer products are exact, so a
kernel differs by (1) fp32 roundings of the scaled products and of SiLU, (2) codes of h that lie on
the border of two integers in exact arithmetic and fall to the other side, (3) the final rounding to
bf16.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24


def quantize(x):
    """(codes float64, scale float64 [rows, 1]) of the rows of x, as the kernels define them."""
    x = x.double()
    amax = x.abs().amax(1, keepdim=True)
    s = (amax / 127).float().double()
    q = (x / torch.where(s == 0, 1.0, s)).float().double().round().clamp(-127, 127)
    bad = ~amax.isfinite()
    q = torch.where(bad | (s == 0), 0.0, q)
    return q, torch.where(bad, float("nan"), s)


# relative error of h in fp32: the products' conversion, two scale products each (3 u), the product
# of the two and the reciprocal (3 u), and 1 + e^-g: e^-g by the hardware exponential is within
# 2^-21 for |g| <= 20 (2^-22.5 of its base-2 argument, up to 29, times ln 2, plus 2 ulp), and it
# enters SiLU with a weight of at most 1
H_REL = 12 * U + 2.0 ** -18


def expert(xq, xs, gate, up, down):
    """(y, bound) of rows of codes xq with scales xs [rows, 1]; gate, up, down: (codes, scales)."""
    gq, gs, uq, us, dq, ds = (t.double() for t in (*gate, *up, *down))
    xq, xs = xq.double(), xs.double()
    g, u = (xq @ gq.t()) * xs * gs, (xq @ uq.t()) * xs * us
    h = g * torch.sigmoid(g) * u
    step = h.abs().amax(1, keepdim=True) / 127
    real = h / torch.where(step == 0, 1.0, step)
    q = real.round()
    y = (q @ dq.t()) * step * ds  # the integer sum first: it is exact, zeros among it
    # a code may fall to either side where the exact quotient is this near a half
    near = (real - real.floor() - 0.5).abs() <= real.abs() * 2 * H_REL + 4 * 127 * U
    flips = near.double() @ dq.abs().t() * step * ds
    # before the last rounding the kernel's value v has |v - y| <= off (the scale carries h's
    # relative error, and so does the size of a flip); rounding to bf16 then moves v by at most
    # 2^-8 |v| <= 2^-8 (|y| + off), so |bf16(v) - y| <= off + 2^-8 (|y| + off)
    off = (y.abs() + flips) * (H_REL + 8 * U) + flips
    return y, off + 2.0 ** -8 * (y.abs() + off) + 1e-30


def ffn(case, xq, xs, offsets, w, x):
    """((y_perm, bound), (y_shared, bound) or None) of the layer's experts."""
    parts = []
    o = [int(v) for v in offsets]
    for e in range(len(o) - 1):
        lo, hi = o[e], o[e + 1]
        if hi > lo:
            parts.append(expert(xq[lo:hi], xs[lo:hi, None],
                                *((w[k][e], w[k + "_scale"][e])
                                  for k in ("w_gate", "w_up", "w_down"))))
    routed = tuple(torch.cat([p[i] for p in parts]) for i in range(2))
    if not case.n_shared:
        return routed, None
    sq, ss = quantize(x)
    down = w["ws_down"].permute(1, 0, 2).flatten(1)
    flat = {k: (w[k].flatten(0, 1), w[k + "_scale"].flatten()) for k in ("ws_gate", "ws_up")}
    return routed, expert(sq, ss, flat["ws_gate"], flat["ws_up"], (down, w["ws_down_scale"]))
