"""The balance loss, the router's gradient and the combine's gradient on the GPU against their
64-bit definitions.

Tolerances are bounds of fp32 arithmetic, with u = 2^-24 the relative error of one operation. A
row's sum of E non-negative affinities is at most 32 additions in a lane and 5 shuffles; with the
reciprocal and the product, p is off by at most 40 u. prob adds at most tile / 16 + 2 of them in a
lane, 1 + 16 across a block and tiles / 8 + 8 across blocks, all non-negative, so its relative error
is the number of additions times u.
"""
import ctypes as C
import os
import subprocess
import sys
import threading

import pytest
import torch

import combine_expert_ffn_b200 as moe
from tests import training_ref as R

pytestmark = pytest.mark.gpu
U = R.EPS
DEV = "cuda"


def cfg_of(T, E, K, router=0, d=64):
    return moe.MoeConfig(T, d, E, 1, K, 1, 64, 0, 0, router, 0)


def tile(T):  # tokens of a block
    return max(32, -(-T // (8 if T <= 1024 else 296)))


def inputs(T, E, K, router=0, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + 7 * T + E)
    logits = torch.randn(T, E, device=DEV, generator=g) + torch.randn(E, device=DEV, generator=g)
    s = R.affinity(logits.double(), router).float()
    idx = torch.topk(s, K, dim=1).indices.int() if T else torch.zeros(0, K, dtype=torch.int32,
                                                                     device=DEV)
    return s, idx, g


def offsets(o):
    return None if o is None else torch.tensor(o, dtype=torch.int32, device=DEV)


def balance(cfg, s, idx, o, alpha, ws=None, stream=None):
    n = 1 if o is None else o.numel() - 1
    out = (torch.full((n, cfg.E), -7, dtype=torch.int32, device=DEV),
           torch.full((n, cfg.E), float("nan"), device=DEV), torch.full((n,), float("nan"),
                                                                        device=DEV))
    ws = moe.alloc_workspace(cfg) if ws is None else ws
    moe.moe_balance_loss(cfg, s, idx, o, alpha, *out, ws, stream=stream)
    return *out, ws


SEQ = {  # sequence starts for a batch of T tokens
    "none": lambda T: None,
    "one": lambda T: [0, T],
    "padded": lambda T: [T // 5, T // 5, T // 2, T - T // 7],  # front, back, an empty sequence
    "singles": lambda T: list(range(T + 1)),
    "tiles": lambda T: [0] + list(range(32, T, 32)) + [T],
    "straddle": lambda T: sorted({0, min(T, 31), min(T, 33), min(T, 95), T}),
    "all_empty": lambda T: [T, T, T],
    "no_sequence": lambda T: [0],
}
SIZES = [(1, 4, 1), (1, 7, 7), (2, 64, 6), (31, 12, 4), (33, 100, 5), (97, 30, 3), (256, 256, 8),
         (520, 40, 6), (700, 128, 32), (1200, 256, 8), (257, 250, 8), (130, 384, 8),
         (100, 1024, 16), (65, 1022, 31), (40, 514, 2)]


@pytest.mark.parametrize("seq", list(SEQ))
@pytest.mark.parametrize("T,E,K", SIZES)
def test_balance_loss(T, E, K, seq):
    cfg, alpha = cfg_of(T, E, K), 0.25
    s, idx, _ = inputs(T, E, K)
    o = SEQ[seq](T)
    n, p, loss, ws = balance(cfg, s, idx, offsets(o), alpha)
    assert moe.moe_read_device_status(ws) == moe.MOE_OK
    if o is not None and len(o) == 1:
        return  # nothing to write
    ref_n = R.counts(idx, o, E)
    assert torch.equal(n.long(), ref_n)
    ref_p, ref_loss = R.balance_loss(s.double(), ref_n, o, alpha, K)
    bound = (40 + tile(T) / 16 + 2 + 17 + T / tile(T) / 8 + 9) * U
    assert ((p.double() - ref_p).abs() <= bound * ref_p).all()
    assert ((loss.double() - ref_loss).abs() <= (bound + 4 * U) * ref_loss).all()


def test_counts_of_one_sequence_are_the_dispatch_counts():
    T, E, K = 515, 48, 4
    cfg = cfg_of(T, E, K)
    s, idx, _ = inputs(T, E, K)
    n, *_ = balance(cfg, s, idx, None, 1.0)
    i32 = dict(dtype=torch.int32, device=DEV)
    got, off = torch.empty(E, **i32), torch.empty(E + 1, **i32)
    moe.moe_dispatch(cfg, None, idx, got, off, torch.empty(1, 1, **i32), None,
                     torch.empty(T * K, **i32), torch.empty(T, K, **i32), None,
                     moe.alloc_workspace(cfg))
    assert torch.equal(n[0], got)


def test_balance_loss_long_batch_is_deterministic():
    T, E, K = 30011, 64, 6
    cfg = cfg_of(T, E, K)
    s, idx, _ = inputs(T, E, K)
    o = offsets([0, 9, 12000, 12001, 29000])
    a, b = balance(cfg, s, idx, o, 1e-3), balance(cfg, s, idx, o, 1e-3)
    for x, y in zip(a[:3], b[:3]):
        assert torch.equal(x, y)
    ref_n = R.counts(idx, o.tolist(), E)
    ref_p, ref_loss = R.balance_loss(s.double(), ref_n, o.tolist(), 1e-3, K)
    bound = (40 + tile(T) / 16 + 2 + 17 + T / tile(T) / 8 + 9) * U
    assert torch.equal(a[0].long(), ref_n)
    assert ((a[1].double() - ref_p).abs() <= bound * ref_p).all()
    assert ((a[2].double() - ref_loss).abs() <= (bound + 4 * U) * ref_loss).all()


@pytest.mark.parametrize("E", [64, 30])
def test_balance_loss_rows_of_zeros_tiny_rows_and_padding_that_holds_nan(E):
    T, K = 200, 3
    cfg = cfg_of(T, E, K)
    s, idx, _ = inputs(T, E, K)
    s[3] = 0.0
    s[50] *= 2.0 ** -130   # subnormal: their digits are few, but exact
    s[51] *= 2.0 ** -100
    s[180:] = float("nan")
    o = [0, 40, 180]
    n, p, loss, ws = balance(cfg, s, idx, offsets(o), 1.0)
    ref_n = R.counts(idx, o, E)
    ref_p, ref_loss = R.balance_loss(s.double(), ref_n, o, 1.0, K)
    assert torch.equal(n.long(), ref_n)
    assert ((p.double() - ref_p).abs() <= 80 * U * ref_p).all()
    assert ((loss.double() - ref_loss).abs() <= 84 * U * ref_loss).all()
    assert moe.moe_read_device_status(ws) == moe.MOE_OK
    s[7, 2] = float("nan")  # in a sequence it shows, there alone
    _, p, loss, _ = balance(cfg, s, idx, offsets(o), 1.0)
    assert p[0].isnan().all() and loss[0].isnan() and not p[1].isnan().any()


def test_balance_loss_of_no_tokens_writes_zeros():
    cfg = cfg_of(0, 16, 2)
    e = torch.empty(0, device=DEV)
    n, p, loss, _ = balance(cfg, e, e.int(), offsets([0, 0, 0]), 1.0, moe.alloc_workspace(cfg))
    assert not n.any() and not p.any() and not loss.any()


def test_balance_loss_flags_bad_ids_and_offsets():
    T, E, K = 300, 32, 4
    cfg = cfg_of(T, E, K)
    s, idx, _ = inputs(T, E, K)
    bad = idx.clone()
    bad[5, 1], bad[299, 3] = E, -1
    n, *_, ws = balance(cfg, s, bad, None, 1.0)
    assert moe.moe_read_device_status(ws) == moe.MOE_ERR_DEVICE_FAULT
    assert int(n.sum()) == T * K - 2
    for o in ([0, 200, 100, 300], [-5, 300], [0, 301], [2 ** 31 - 1, -2 ** 31]):
        *_, ws = balance(cfg, s, idx, offsets(o), 1.0)
        assert moe.moe_read_device_status(ws) == moe.MOE_ERR_DEVICE_FAULT, o


# ------------------------------------------------------------------ router gradient
def route_bound(s, idx, dw, pull, router):
    """Element bound: 60 u on each of the products r p (pull - mean) and r w (dw - mean)."""
    S = s.double()
    p = S / S.sum(1, keepdim=True)
    b = p * 2 * pull.abs().amax(1, keepdim=True)
    if dw is not None:
        w = R.gates(S, idx)
        b.scatter_add_(1, idx.long(), w * 2 * dw.double().abs().amax(1, keepdim=True))
    # 1 - s loses at most u of 1, and r is at most 1; 1e-12: the 64-bit reference's own
    # cancellation where all counts are equal
    return 60 * U * b + 1e-12


def reference(s, idx, dw, o, n, dl, alpha, router):
    x = R.logits_of(s, router).requires_grad_()
    return torch.autograd.grad(R.router_goal(R.affinity(x, router), idx, dw, o, n, dl, alpha), x)[0]


def pull_of(n, o, dl, alpha, K, T, E):
    pull = torch.zeros(T, E, dtype=torch.float64, device=DEV)
    for q, (lo, hi) in enumerate(R.spans(o, T)):
        if hi > lo:
            c = n[q].double()
            pull[lo:hi] = dl[q].double() * alpha * E / (K * (hi - lo) ** 2) * (c - c.mean())
    return pull


@pytest.mark.parametrize("router", [0, 1])
@pytest.mark.parametrize("seq", ["none", "padded", "singles", "straddle"])
@pytest.mark.parametrize("T,E,K", SIZES)
def test_route_backward(T, E, K, seq, router):
    cfg, alpha = cfg_of(T, E, K, router), 0.1
    s, idx, g = inputs(T, E, K, router)
    o = SEQ[seq](T)
    n = R.counts(idx, o, E)
    dl = torch.randn(n.shape[0], device=DEV, generator=g) * T
    dw = torch.randn(T, K, device=DEV, generator=g)
    out = torch.full((T, E), float("nan"), device=DEV)
    fault = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_route_backward(cfg, s, idx, dw, offsets(o), n.int(), dl, alpha, out, fault)
    ref = reference(s, idx, dw, o, n, dl, alpha, router)
    pull = pull_of(n, o, dl, alpha, K, T, E)
    assert int(fault) == 0
    assert ((out.double() - ref).abs() <= route_bound(s, idx, dw, pull, router)).all()
    # each part alone
    moe.moe_route_backward(cfg, s, idx, None, offsets(o), n.int(), dl, alpha, out)
    ref = reference(s, idx, None, o, n, dl, alpha, router)
    assert ((out.double() - ref).abs() <= route_bound(s, idx, None, pull, router)).all()
    moe.moe_route_backward(cfg, s, idx, dw, None, None, None, alpha, out)
    ref = reference(s, idx, dw, o, n, None, alpha, router)
    assert ((out.double() - ref).abs() <= route_bound(s, idx, dw, pull * 0, router)).all()


@pytest.mark.parametrize("router", [0, 1])
def test_route_backward_against_differences(router):
    T, E, K = 24, 12, 3
    cfg, alpha = cfg_of(T, E, K, router), 0.5
    s, idx, g = inputs(T, E, K, router)
    o = [0, 10, 24]
    n = R.counts(idx, o, E)
    dl, dw = torch.tensor([3.0, -4.0], device=DEV), torch.randn(T, K, device=DEV, generator=g)
    out = torch.empty(T, E, device=DEV)
    moe.moe_route_backward(cfg, s, idx, dw, offsets(o), n.int(), dl, alpha, out)
    x = R.logits_of(s, router)

    def goal(v):
        return R.router_goal(R.affinity(v, router), idx, dw, o, n, dl, alpha)

    h = 1e-4  # truncation h^2 |f'''| / 6 <= 1e-8, cancellation 1e-15 / h = 1e-11
    for t in range(0, T, 5):
        for i in range(E):
            e = torch.zeros_like(x)
            e[t, i] = h
            diff = float(goal(x + e) - goal(x - e)) / (2 * h)
            assert abs(diff - float(out[t, i])) <= 1e-7 + 1e-5 * abs(diff)


@pytest.mark.parametrize("router", [0, 1])
def test_route_backward_at_the_ends_of_the_range(router):
    """Affinities of 0, near the smallest floats, at 1 and large; tokens in no sequence."""
    T, E, K = 64, 16, 2
    cfg = cfg_of(T, E, K, router)
    s, idx, g = inputs(T, E, K, router)
    s[0] = 0.0
    s[1] *= 2.0 ** -110
    s[2, idx[2].long()] = 1.0 if router == 0 else 40.0
    s[3, idx[3].long()] = 0.0
    s[60:] = float("nan")
    o = [0, 60]
    n = R.counts(idx, o, E)
    dl = torch.tensor([50.0], device=DEV)
    dw = torch.randn(T, K, device=DEV, generator=g)
    out = torch.full((T, E), 9.0, device=DEV)
    moe.moe_route_backward(cfg, s, idx, dw, offsets(o), n.int(), dl, 0.1, out)
    S = s[:60].double()
    tot = S.sum(1, keepdim=True)
    p = S / torch.where(tot == 0, 1.0, tot)
    pull = pull_of(n, o, dl, 0.1, K, T, E)[:60]
    chosen = S.gather(1, idx[:60].long())
    z = chosen.sum(1, keepdim=True)
    w = chosen / torch.where(z == 0, 1.0, z)
    ref = p * (pull - (pull * p).sum(1, keepdim=True))
    ref.scatter_add_(1, idx[:60].long(), w * (dw[:60] - (dw[:60] * w).sum(1, keepdim=True)))
    ref *= torch.where(S > 0, -torch.expm1(-S * S) / (2 * S * S), 0.5) if router else 1 - S
    bound = 60 * U * 2 * (p * pull.abs().max() + dw.abs().max())
    assert ((out[:60].double() - ref).abs() <= bound).all()
    moe.moe_route_backward(cfg, s, idx, None, offsets(o), n.int(), dl, 0.1, out)
    assert not out[60:].any()  # no sequence and no gate: zero, whatever the row holds


def test_route_backward_bad_and_repeated_ids():
    T, E, K = 70, 16, 4
    cfg = cfg_of(T, E, K)
    s, idx, g = inputs(T, E, K)
    dw = torch.randn(T, K, device=DEV, generator=g)
    bad = idx.clone()
    bad[9, 0], bad[69, 3] = -1, E
    fault = torch.zeros(1, dtype=torch.int32, device=DEV)
    good, out = torch.empty(T, E, device=DEV), torch.empty(T, E, device=DEV)
    moe.moe_route_backward(cfg, s, idx, dw, None, None, None, 0.0, good)
    moe.moe_route_backward(cfg, s, bad, dw, None, None, None, 0.0, out, fault)
    assert int(fault) == moe.MOE_ERR_DEVICE_FAULT
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[[9, 69]] = False
    assert torch.equal(good[keep], out[keep]) and out.isfinite().all()
    twice = idx.clone()
    twice[:, 1] = twice[:, 0]
    moe.moe_route_backward(cfg, s, twice, dw, None, None, None, 0.0, out)
    ref = reference(s, twice, dw, None, None, None, 0.0, 0)
    zero = torch.zeros(T, E, dtype=torch.float64, device=DEV)
    assert ((out.double() - ref).abs() <= 2 * route_bound(s, twice, dw, zero, 0) + 1e-30).all()


@pytest.mark.parametrize("router", [0, 1])
@pytest.mark.parametrize("T,E,K", [(70, 64, 1), (33, 256, 1), (50, 30, 1), (40, 1024, 1), (64, 64, 6),
                                   (40, 24, 12), (21, 254, 31)])
def test_route_backward_of_equal_gate_gradients_is_the_balance_losss(T, E, K, router):
    """Gates sum to 1: a gradient that all gates of a token share (any, with a single gate) moves
    nothing, and must not leave its rounding behind beside a much smaller balance gradient."""
    cfg, alpha = cfg_of(T, E, K, router), 1e-6
    s, idx, g = inputs(T, E, K, router)
    o = [0, T // 3, T]
    n = R.counts(idx, o, E).int()
    dl = torch.ones(2, device=DEV)
    dw = 1e3 * torch.randn(T, 1, device=DEV, generator=g).expand(T, K).contiguous()
    both, alone = torch.empty(T, E, device=DEV), torch.empty(T, E, device=DEV)
    moe.moe_route_backward(cfg, s, idx, dw, offsets(o), n, dl, alpha, both)
    moe.moe_route_backward(cfg, s, idx, None, offsets(o), n, dl, alpha, alone)
    assert torch.equal(both, alone)


@pytest.mark.parametrize("T,E,K", [(40, 16, 4), (33, 256, 17), (20, 30, 9)])
@pytest.mark.parametrize("slot", [0, 2])
def test_route_backward_does_not_read_the_gradient_of_a_skipped_gate(T, E, K, slot):
    cfg = cfg_of(T, E, K)
    s, idx, g = inputs(T, E, K)
    idx[5, slot], idx[T - 1, slot] = E, -1
    dw = torch.randn(T, K, device=DEV, generator=g)
    dw[5, slot] = dw[T - 1, slot] = 0.0
    want, out = torch.empty(T, E, device=DEV), torch.empty(T, E, device=DEV)
    moe.moe_route_backward(cfg, s, idx, dw, None, None, None, 0.0, want)
    dw[5, slot], dw[T - 1, slot] = float("nan"), 1e30
    moe.moe_route_backward(cfg, s, idx, dw, None, None, None, 0.0, out)
    assert torch.equal(want, out) and want.isfinite().all()


@pytest.mark.parametrize("T,E,K", [(40, 24, 12), (33, 256, 17), (20, 30, 9)])
def test_route_backward_repeated_ids_in_long_choices(T, E, K):
    """Two gates of one expert where a lane holds several of a token's gates."""
    cfg = cfg_of(T, E, K)
    s, idx, g = inputs(T, E, K)
    idx = idx.clone()
    idx[:, K - 1] = idx[:, 0]
    dw = torch.randn(T, K, device=DEV, generator=g)
    out = torch.empty(T, E, device=DEV)
    moe.moe_route_backward(cfg, s, idx, dw, None, None, None, 0.0, out)
    ref = reference(s, idx, dw, None, None, None, 0.0, 0)
    zero = torch.zeros(T, E, dtype=torch.float64, device=DEV)
    assert ((out.double() - ref).abs() <= 2 * route_bound(s, idx, dw, zero, 0)).all()


def test_more_affinities_than_2_to_the_31():
    T, E, K = (1 << 21) + 37, 1024, 2
    cfg, alpha = cfg_of(T, E, K), 1.0
    g = torch.Generator(device=DEV).manual_seed(11)
    s = torch.rand(T, E, device=DEV, generator=g) * 0.9 + 0.05
    a = torch.randint(0, E, (T,), device=DEV, generator=g)
    idx = torch.stack([a, (a + 1 + a % 7) % E], 1).int()
    cut = T - 300
    o = [0, 1000, cut, T]
    n, p, loss, ws = balance(cfg, s, idx, offsets(o), alpha)
    assert moe.moe_read_device_status(ws) == moe.MOE_OK
    assert torch.equal(n.long(), R.counts(idx, o, E))
    tail = R.balance_loss(s[cut:].double(), n[2:], [0, 300], alpha, K)
    assert ((p[2].double() - tail[0][0]).abs() <= 200 * U * tail[0][0]).all()
    assert abs(float(loss[2]) - float(tail[1][0])) <= 204 * U * float(tail[1][0])
    # the long sequence's shares add up to 1, each within its own relative error
    bound = (40 + tile(T) / 16 + 2 + 17 + T / tile(T) / 8 + 9) * U
    assert abs(float(p[1].double().sum()) - 1) <= bound
    dl = torch.tensor([1.0, 1.0, 300.0], device=DEV)
    dw = torch.randn(T, K, device=DEV, generator=g)
    out = torch.empty(T, E, device=DEV)
    moe.moe_route_backward(cfg, s, idx, dw, offsets(o), n, dl, alpha, out)
    sub, o2 = slice(cut, T), [0, 300]
    ref = reference(s[sub], idx[sub], dw[sub], o2, n[2:].long(), dl[2:], alpha, 0)
    pull = pull_of(n[2:], o2, dl[2:], alpha, K, 300, E)
    assert ((out[sub].double() - ref).abs() <= route_bound(s[sub], idx[sub], dw[sub], pull, 0)).all()


def test_many_short_sequences():
    """Every token a sequence of its own, more of them than one tile's search probes at once."""
    T, E, K = 20000, 24, 3
    cfg = cfg_of(T, E, K)
    s, idx, _ = inputs(T, E, K)
    o = list(range(0, T + 1))
    n, p, loss, _ = balance(cfg, s, idx, offsets(o), 1.0)
    want = torch.zeros(T, E, device=DEV).scatter_(1, idx.long(), 1.0)
    assert torch.equal(n.float(), want)
    share = s.double() / s.double().sum(1, keepdim=True)
    assert ((p.double() - share).abs() <= 60 * U * share).all()
    ref = (share * want.double()).sum(1) * E / K
    assert ((loss.double() - ref).abs() <= 64 * U * ref).all()


@pytest.mark.parametrize("T,E,K", [(1000, 40, 6), (300, 256, 8), (70000, 30, 2)])
def test_a_long_sequence_among_short_ones(T, E, K):
    """Short tiles for the many short ones, and so many shares of the long one.  Its p is a sum of
    at most tile terms a lane, of a block's, and of the tiles in as many chains as the join's 1024
    threads allow; each addition of fp32 is off by U of a sum of positive terms."""
    cfg, alpha = cfg_of(T, E, K), 0.5
    s, idx, _ = inputs(T, E, K)
    o = [*range(0, T // 8), *range(T // 8, T // 4, 5), T // 4, T - T // 8, *range(T - T // 8 + 3, T, 7), T]
    n, p, loss, ws = balance(cfg, s, idx, offsets(o), alpha)
    assert moe.moe_read_device_status(ws) == moe.MOE_OK
    ref_n = R.counts(idx, o, E)
    assert torch.equal(n.long(), ref_n)
    ref_p, ref_loss = R.balance_loss(s.double(), ref_n, o, alpha, K)
    short = max(8, T // (len(o) - 1), T // 2048)
    bound = (40 + short / 8 + 2 + 17 + T / short / (1024 // (-(-E // 32) * 32)) + 41) * U
    assert ((p.double() - ref_p).abs() <= bound * ref_p).all()
    assert ((loss.double() - ref_loss).abs() <= (bound + 4 * U) * ref_loss).all()


# ------------------------------------------------------------------ combine gradient
COMBINE = [(1, 64, 1), (1, 7168, 8), (3, 320, 5), (40, 128, 32), (300, 2048, 6), (700, 576, 8),
           (2500, 64, 1), (9, 8256, 3)]


def combine_inputs(T, d, K, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + T + d)
    r = dict(device=DEV, generator=g)
    return (torch.randn(T, d, **r).bfloat16(), torch.randn(T * K, d, **r).bfloat16(),
            torch.randperm(T * K, **r).int().view(T, K), torch.rand(T, K, **r))


@pytest.mark.parametrize("T,d,K", COMBINE)
def test_combine_backward(T, d, K):
    cfg = cfg_of(T, max(K, 4), K, d=d)
    g, y, inv, w = combine_inputs(T, d, K)
    dy, dw = torch.empty_like(y), torch.empty_like(w)
    moe.moe_combine_backward(cfg, g, y, inv, w, dy, dw)
    rows = inv.flatten().long()
    ref_dy = torch.empty(T * K, d, dtype=torch.float64, device=DEV)
    ref_dy[rows] = (w.double()[:, :, None] * g.double()[:, None]).flatten(0, 1)
    # one fp32 product and one rounding to bf16, each by at most half a step
    assert ((dy.double() - ref_dy).abs() <= (2.0 ** -8 + 2 * U) * ref_dy.abs()).all()
    prod = g.double()[:, None] * y.double()[rows].view(T, K, d)
    n = 8 * -(-d // 256) + 5 + 8  # additions in a lane, a warp and a block
    assert ((dw.double() - prod.sum(2)).abs() <= n * U * prod.abs().sum(2)).all()
    one, two = torch.empty_like(y), torch.empty_like(w)
    moe.moe_combine_backward(cfg, g, None, inv, w, one, None)
    moe.moe_combine_backward(cfg, g, y, inv, None, None, two)
    assert torch.equal(one, dy) and torch.equal(two, dw)


@pytest.mark.parametrize("T", [20, 700])
def test_combine_backward_skips_rows_that_no_copy_names(T):
    d, K = 192, 4
    cfg = cfg_of(T, 8, K, d=d)
    g, y, inv, w = combine_inputs(T, d, K)
    inv = inv.clone()
    gone = [int(inv[3, 1]), int(inv[T - 1, 0])]
    inv[3, 1], inv[T - 1, 0] = -1, T * K
    dy, dw = torch.full_like(y, 5.0), torch.full_like(w, 5.0)
    moe.moe_combine_backward(cfg, g, y, inv, w, dy, dw)
    assert float(dw[3, 1]) == 0.0 and float(dw[T - 1, 0]) == 0.0
    assert (dy[gone] == 5.0).all()
    assert int((dy == 5.0).all(1).sum()) == 2


def test_combine_backward_is_the_combines_gradient():
    """Against the combine itself: d_topk_w against differences of moe_combine in one gate, the
    dispatch's gradient (combine with gates of 1) against the sum of the rows."""
    T, d, K = 12, 128, 3
    cfg = cfg_of(T, 4, K, d=d)
    g, y, inv, w = combine_inputs(T, d, K)
    dy, dw = torch.empty_like(y), torch.empty_like(w)
    moe.moe_combine_backward(cfg, g, y, inv, w, dy, dw)
    for t, j in ((0, 0), (5, 2), (11, 1)):
        w2 = w.clone()
        w2[t, j] += 4.0
        a, b = (torch.empty(T, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        moe.moe_combine(cfg, y, inv, w, None, a)
        moe.moe_combine(cfg, y, inv, w2, None, b)
        diff = ((b.double() - a.double()) * g.double()).sum() / 4
        # both outputs are rounded to bf16
        room = ((a.double().abs() + b.double().abs()) * g.double().abs()).sum() * 2.0 ** -8 / 4
        assert abs(float(diff) - float(dw[t, j])) <= float(room)


# ------------------------------------------------------------------ together
def test_router_training_step_streams_and_graph():
    """route -> dispatch -> combine, then the gradients back to the logits and the router weights,
    on a stream of its own, then captured and replayed on new inputs."""
    T, d, E, G, K, M = 264, 320, 12, 4, 4, 2
    cfg = moe.MoeConfig(T, d, E, G, K, M, 64, 0, 0, 0, 0)
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(T, d, device=DEV, generator=g).bfloat16()
    rw = torch.randn(E, d, device=DEV, generator=g) * d ** -0.5
    y = torch.randn(T * K, d, device=DEV, generator=g).bfloat16()
    up = torch.randn(T, d, device=DEV, generator=g).bfloat16()
    o = offsets([0, 100, 240])
    dl = torch.tensor([1.0, 1.0], device=DEV)
    alpha = 0.05
    i32 = dict(dtype=torch.int32, device=DEV)
    b = {"idx": torch.empty(T, K, **i32), "w": torch.empty(T, K, device=DEV),
         "s": torch.empty(T, E, device=DEV), "n": torch.empty(E, **i32),
         "off": torch.empty(E + 1, **i32), "send": torch.empty(G, G, **i32),
         "tok": torch.empty(T * K, **i32), "inv": torch.empty(T, K, **i32),
         "out": torch.empty(T, d, dtype=torch.bfloat16, device=DEV),
         "c": torch.empty(2, E, **i32), "p": torch.empty(2, E, device=DEV),
         "loss": torch.empty(2, device=DEV), "dw": torch.empty(T, K, device=DEV),
         "dy": torch.empty_like(y), "dlogits": torch.empty(T, E, device=DEV)}
    ws = moe.alloc_workspace(cfg)
    torch.cuda.synchronize()

    def step():
        moe.moe_route(cfg, x, rw, None, None, b["idx"], b["w"], b["s"], ws)
        moe.moe_dispatch(cfg, None, b["idx"], b["n"], b["off"], b["send"], None, b["tok"],
                         b["inv"], None, ws)
        moe.moe_combine(cfg, y, b["inv"], b["w"], None, b["out"])
        moe.moe_balance_loss(cfg, b["s"], b["idx"], o, alpha, b["c"], b["p"], b["loss"], ws)
        moe.moe_combine_backward(cfg, up, y, b["inv"], b["w"], b["dy"], b["dw"])
        moe.moe_route_backward(cfg, b["s"], b["idx"], b["dw"], o, b["c"], dl, alpha, b["dlogits"])

    def check():
        torch.cuda.synchronize()
        assert moe.moe_read_device_status(ws) == moe.MOE_OK
        s, idx = b["s"], b["idx"]
        logits = R.logits_of(s, 0).requires_grad_()
        a = R.affinity(logits, 0)
        rows = y.double()[b["inv"].long().flatten()].view(T, K, d)
        out = (R.gates(a, idx)[:, :, None] * rows).sum(1)
        goal = (out * up.double()).sum()
        n = R.counts(idx, o.tolist(), E)
        goal = goal + R.balance_loss(a, n, o.tolist(), alpha, K)[1].sum()
        ref = torch.autograd.grad(goal, logits)[0]
        # the gates' gradients are fp32 sums over d of |up y|
        mag = (up.double()[:, None] * rows).abs().sum(2).amax(1, keepdim=True)
        bound = torch.zeros_like(ref)
        bound.scatter_add_(1, idx.long(), (R.gates(s.double(), idx) * 2 * mag))
        bound += s.double() / s.double().sum(1, keepdim=True) * alpha * E * 2
        assert ((b["dlogits"].double() - ref).abs() <= (60 + 8 * 2 + 13) * U * bound).all()

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(torch.randn(T, d, device=DEV, generator=g))
    y.copy_(torch.randn(T * K, d, device=DEV, generator=g))
    graph.replay()
    check()


def test_two_streams_with_a_workspace_each():
    T, E, K = 5000, 64, 6
    cfg = cfg_of(T, E, K)
    s, idx, _ = inputs(T, E, K)
    s2, idx2, _ = inputs(T, E, K, seed=1)
    want, want2 = balance(cfg, s, idx, None, 1.0)[:3], balance(cfg, s2, idx2, None, 1.0)[:3]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    ws = [moe.alloc_workspace(cfg) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(a):
            got = balance(cfg, s, idx, None, 1.0, ws[0])[:3]
        with torch.cuda.stream(b):
            got2 = balance(cfg, s2, idx2, None, 1.0, ws[1])[:3]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert all(torch.equal(x, y) for x, y in zip(got2, want2))


def test_python_entry_points_refuse_wrong_tensors():
    T, E, K = 8, 8, 2
    cfg = cfg_of(T, E, K)
    s, idx, _ = inputs(T, E, K)
    n, p, loss, ws = balance(cfg, s, idx, None, 1.0)
    out = torch.empty(T, E, device=DEV)
    dw = torch.zeros(T, K, device=DEV)
    for args in [(s.double(), idx, None, 1.0, n, p, loss, ws), (s.t(), idx, None, 1.0, n, p, loss, ws),
                 (s.cpu(), idx, None, 1.0, n, p, loss, ws), (s, idx.long(), None, 1.0, n, p, loss, ws),
                 (s[:7], idx, None, 1.0, n, p, loss, ws), (s, idx, None, float("nan"), n, p, loss, ws),
                 (s, idx, offsets([0, 4, 8]), 1.0, n, p, loss, ws)]:
        with pytest.raises(moe.MoeError):
            moe.moe_balance_loss(cfg, *args)
    with pytest.raises(moe.MoeError):
        moe.moe_route_backward(cfg, s, idx, None, None, None, None, 1.0, out)
    with pytest.raises(moe.MoeError):
        moe.moe_route_backward(cfg, s, idx, dw.half(), None, None, None, 1.0, out)
    with pytest.raises(moe.MoeError):
        moe.moe_route_backward(cfg_of(T, E, K, moe.MOE_ROUTER_HASH), s, idx, dw, None, None, None,
                               1.0, out)


# ------------------------------------------------------------------ sizes that need more shared memory
def child(call):
    """Runs ``call``, a line of this module, in a process of its own: what an earlier call of this one
    did to the kernels' settings must not matter."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", f"import tests.test_gpu_router_training as t; t.{call}"],
                       cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def check_balance(T, E, K):
    """Both of the loss's kernels at (T, E, K): one sequence, and some that cross tiles."""
    cfg, alpha = cfg_of(T, E, K), 0.25
    s, idx, _ = inputs(T, E, K)
    for o in (None, SEQ["straddle"](T)):
        n, p, loss, ws = balance(cfg, s, idx, offsets(o), alpha)
        assert moe.moe_read_device_status(ws) == moe.MOE_OK
        ref_n = R.counts(idx, o, E)
        assert torch.equal(n.long(), ref_n)
        ref_p, ref_loss = R.balance_loss(s.double(), ref_n, o, alpha, K)
        bound = (40 + tile(T) / 16 + 2 + 17 + T / tile(T) / 8 + 9) * U
        assert ((p.double() - ref_p).abs() <= bound * ref_p).all()
        assert ((loss.double() - ref_loss).abs() <= (bound + 4 * U) * ref_loss).all()


def balance_sizes():
    for E in (655, 658, 659, 660, 704, 721, 722, 723, 724, 1023, 1024):  # ascending: no earlier call
        for T in (20, 40, 1000, 1300):                                   # asked for more
            check_balance(T, E, 4)


def test_balance_loss_of_many_experts_in_a_fresh_process():
    """68 bytes of shared memory an expert and what the kernels declare besides (4352 bytes where
    the batch is one cluster) pass 48 KB from 659 experts on."""
    child("balance_sizes()")


def balance_from_two_threads():
    """Sizes of one row layout, each in a thread of its own: neither call's setting is the other's."""
    fails = []

    def work(E):
        try:
            cfg = cfg_of(64, E, 2)
            s, idx, _ = inputs(64, E, 2)
            with torch.cuda.stream(torch.cuda.Stream()):
                torch.cuda.synchronize()
                n, p, loss, ws = balance(cfg, s, idx, None, 0.25)
                for _ in range(20000):
                    moe.moe_balance_loss(cfg, s, idx, None, 0.25, n, p, loss, ws)
            torch.cuda.synchronize()
        except Exception as e:  # (for the test's own thread)
            fails.append(repr(e))

    threads = [threading.Thread(target=work, args=(E,)) for E in (732, 1024)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not fails, fails


def test_balance_loss_from_two_threads():
    child("balance_from_two_threads()")


def right_call_after_a_refused_launch():
    """A launch that CUDA refuses on the host (on the legacy stream while a stream that it would have
    to wait for is capturing) is that call's error and no other's."""
    T, E, K = 64, 16, 2
    cfg = cfg_of(T, E, K)
    s, idx, g = inputs(T, E, K)
    n, p, loss, ws = balance(cfg, s, idx, None, 1.0)
    g, y, inv, w = combine_inputs(T, 64, K)
    out, want = torch.empty_like(g), torch.empty_like(g)
    moe.moe_combine(cfg, y, inv, w, None, want)
    torch.cuda.synchronize()
    path = next(line.split()[-1] for line in open("/proc/self/maps") if "libcudart" in line)
    rt, stream, graph = C.CDLL(path), C.c_void_p(), C.c_void_p()
    assert rt.cudaStreamCreate(C.byref(stream)) == 0
    assert rt.cudaStreamBeginCapture(stream, 0) == 0
    with pytest.raises(moe.MoeError) as e:
        moe.moe_balance_loss(cfg, s, idx, None, 1.0, n, p, loss, ws, stream=0)
    assert e.value.status == moe.MOE_ERR_CUDA
    assert rt.cudaStreamEndCapture(stream, C.byref(graph)) != 0  # the capture is lost
    rt.cudaGetLastError()
    moe.moe_combine(cfg, y, inv, w, None, out)  # raises where the error above is still there
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_refused_launch_is_not_the_next_calls_error():
    child("right_call_after_a_refused_launch()")


# ------------------------------------------------------------------ digits of the router gradient
def gate_bound(s, idx, dw, router):
    """Element bound of the gates' gradient r w_j (dw_j - m), m = sum_k dw_k w_k, that does not scale
    with the largest gradient.  Taken off every dw is that of a gate whose weight is the largest (by
    2^-18 of it at most), so at least 1 / K: its size is at most K A, A = sum_k |dw_k| w_k, and each
    of 60 roundings (7 a sum, the slope's 20 among them) is one of |dw_j| or of at most (K + 1) A."""
    w, K = R.gates(s.double(), idx), idx.shape[1]
    a = (w * dw.double().abs()).sum(1, keepdim=True)
    b = torch.zeros(s.shape, dtype=torch.float64, device=DEV)
    b.scatter_add_(1, idx.long(), w * (dw.double().abs() + 1.001 * (K + 1) * a))
    return 60 * U * b + 1e-30


@pytest.mark.parametrize("router", [0, 1])
@pytest.mark.parametrize("T,E,K", [(64, 16, 4), (64, 64, 8), (50, 64, 6), (40, 256, 8), (33, 256, 17),
                                   (21, 24, 12), (20, 30, 9), (20, 1024, 32), (9, 254, 31), (7, 40, 1)])
def test_route_backward_of_a_small_gate_with_a_large_gradient(T, E, K, router):
    """One gate of each token, in every slot in turn, is 1e-3 to 1e-12 of the others and has a
    gradient of the inverse size: it hardly enters the others' gradients, which keep their digits."""
    cfg = cfg_of(T, E, K, router)
    s, idx, g = inputs(T, E, K, router)
    t = torch.arange(T, device=DEV)
    slot = t % K
    small = 10.0 ** -(3 + 9 * torch.rand(T, device=DEV, generator=g))
    s[t, idx[t, slot].long()] *= small
    dw = torch.randn(T, K, device=DEV, generator=g)
    dw[t, slot] /= small
    out = torch.empty(T, E, device=DEV)
    moe.moe_route_backward(cfg, s, idx, dw, None, None, None, 0.0, out)
    ref = reference(s, idx, dw, None, None, None, 0.0, router)
    off = (out.double() - ref).abs()
    bound = gate_bound(s, idx, dw, router)
    assert (off <= bound).all(), float((off / bound).max())


@pytest.mark.parametrize("router", [0, 1])
@pytest.mark.parametrize("T,E,K", [(96, 64, 6), (70, 256, 8), (33, 30, 3), (40, 1024, 4), (24, 1022, 2)])
@pytest.mark.parametrize("seq", ["none", "padded", "singles", "straddle"])
def test_route_backward_of_counts_summed_over_ranks(T, E, K, seq, router):
    """Counts of a step's eight ranks: large and nearly equal, their mean far from this rank's
    K N / E.  What is left of them beside their own mean is the gradient, to fp32's digits of it."""
    cfg, alpha = cfg_of(T, E, K, router), 1.0
    s, idx, g = inputs(T, E, K, router)
    o = SEQ[seq](T)
    n = 8 * R.counts(idx, o, E) + 100_000
    n += torch.randint(0, 50, n.shape, device=DEV, generator=g)
    dl = torch.randn(n.shape[0], device=DEV, generator=g)
    out = torch.empty(T, E, device=DEV)
    moe.moe_route_backward(cfg, s, idx, None, offsets(o), n.int(), dl, alpha, out)
    pull = pull_of(n, o, dl, alpha, K, T, E)
    S = s.double()
    p = S / S.sum(1, keepdim=True)
    ref = p * (pull - (pull * p).sum(1, keepdim=True))
    ref *= -torch.expm1(-S * S) / (2 * S * S) if router else 1 - S
    off = (out.double() - ref).abs()
    bound = route_bound(s, idx, None, pull, router)
    assert (off <= bound).all(), float((off / bound).max())


# ------------------------------------------------------------------ what another stream writes
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("T", [200, 3000])
def test_affinities_that_another_stream_writes(T, captured):
    """Loss and gradient behind an event of the stream that writes all they read, with a round of
    the same calls right before it; eager, and as the branches of a graph."""
    E, K, alpha = 64, 6, 0.5
    cfg = cfg_of(T, E, K)
    s, idx, g = inputs(T, E, K)
    s2, idx2, _ = inputs(T, E, K, seed=9)
    dw, dw2 = (torch.randn(T, K, device=DEV, generator=g) for _ in range(2))
    o, o2 = offsets([0, T // 3, T]), offsets([0, T // 2, T - 5])
    dl, dl2 = torch.tensor([1.0, 2.0], device=DEV), torch.tensor([3.0, -1.0], device=DEV)
    ws, fault = moe.alloc_workspace(cfg), torch.zeros(1, dtype=torch.int32, device=DEV)

    def calls(s, idx, dw, o, dl, out):
        moe.moe_balance_loss(cfg, s, idx, o, alpha, *out[:3], ws)
        moe.moe_route_backward(cfg, s, idx, dw, o, out[0], dl, alpha, out[3], fault)

    def outs():
        return (torch.full((2, E), -7, dtype=torch.int32, device=DEV), torch.zeros(2, E, device=DEV),
                torch.zeros(2, device=DEV), torch.zeros(T, E, device=DEV))

    want, out = outs(), outs()
    calls(s2, idx2, dw2, o2, dl2, want)
    pairs = [(s, s2), (idx, idx2), (dw, dw2), (o, o2), (dl, dl2)]
    first = [a.clone() for a, _ in pairs]
    side = torch.cuda.Stream()

    def run():
        here = torch.cuda.current_stream()
        calls(s, idx, dw, o, dl, out)
        side.wait_stream(here)
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
            for a, b in pairs:
                a.copy_(b)
        here.wait_stream(side)
        calls(s, idx, dw, o, dl, out)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
    for _ in range(3):
        for (a, _), b in zip(pairs, first):
            a.copy_(b)
        graph.replay() if captured else run()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    assert moe.moe_read_device_status(ws) == moe.MOE_OK and int(fault) == 0
