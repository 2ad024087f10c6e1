"""The int8 experts on the GPU: codes and scales bit for bit, the products against 64 bits."""
import os
import subprocess
import sys

import pytest
import torch

import combine_expert_ffn_b200 as moe
import synth
from tests import harness as H
from tests import int8_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def config(T, d, E, K, d_ff, n_shared=0, d_ff_shared=0, G=1, M=1, router=0):
    return moe.MoeConfig(T, d, E, G, K, M, d_ff, n_shared, d_ff_shared, router, 0)


def routing(T, E, K, g, skew=0.0):
    p = torch.arange(1, E + 1, device=DEV).float() ** -skew
    u = torch.rand(T, E, device=DEV, generator=g).clamp_min(1e-30)
    return torch.topk(u.log() / p, K, dim=1).indices.int()


def dispatch(cfg, x, idx, ws):
    i32, rows = dict(dtype=torch.int32, device=DEV), cfg.T * cfg.K
    o = {"counts": torch.empty(cfg.E, **i32), "offsets": torch.empty(cfg.E + 1, **i32),
         "send": torch.empty(cfg.G, cfg.G, **i32), "send_tok": torch.empty(cfg.G, cfg.G, **i32),
         "perm_token": torch.empty(rows, **i32), "inv_perm": torch.empty(cfg.T, cfg.K, **i32)}
    q = torch.full((rows, cfg.d), 77, dtype=torch.int8, device=DEV)
    s = torch.full((rows,), -1.0, device=DEV)
    moe.moe_dispatch_int8(cfg, x, idx, *o.values(), q, s, ws)
    return o, q, s


def same(a, b):
    """Equal bits, any NaN equal to any other."""
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


def random_weights(cfg, g):
    """int8 codes over the whole range with -128 among them, scales of a layer of unit variance."""
    def codes(*shape):
        return torch.randint(-128, 128, shape, dtype=torch.int8, device=DEV, generator=g)

    def scales(fan, *shape):
        return (torch.rand(shape, device=DEV, generator=g) + 0.5) * fan ** -0.5 / 74

    E, d, ff, ns, fs = cfg.E, cfg.d, cfg.d_ff, cfg.n_shared, cfg.d_ff_shared
    w = {"w_gate": codes(E, ff, d), "w_up": codes(E, ff, d), "w_down": codes(E, d, ff),
         "w_gate_scale": scales(d, E, ff), "w_up_scale": scales(d, E, ff),
         "w_down_scale": scales(ff, E, d)}
    if ns:
        w |= {"ws_gate": codes(ns, fs, d), "ws_up": codes(ns, fs, d), "ws_down": codes(ns, d, fs),
              "ws_gate_scale": scales(d, ns, fs), "ws_up_scale": scales(d, ns, fs),
              "ws_down_scale": scales(ns * fs, d)}
    return w


# ------------------------------------------------------------------ codes
@pytest.mark.parametrize("T,d,E,K", [(1, 64, 4, 1), (1, 7168, 16, 8), (37, 128, 8, 8),
                                     (130, 2048, 12, 3), (64, 2112, 8, 2), (300, 576, 40, 6),
                                     (9, 8192, 4, 2), (9, 8256, 4, 2), (5, 16448, 4, 3)])
def test_dispatch_int8(T, d, E, K):
    cfg, g = config(T, d, E, K, 64), gen(T + d)
    x = (torch.randn(T, d, device=DEV, generator=g)
         * torch.exp(2 * torch.randn(T, 1, device=DEV, generator=g))).bfloat16()
    if T > 8:
        x[2] = 0.0
        x[3, 5] = float("nan")
        x[4, 7] = float("-inf")
        x[5] = 2.0 ** -133               # the smallest bf16
        x[6, :] = 0.0
        x[6, d - 1] = -3.0e38
        x[7] = x[7, 0]                    # one value: every code +-127
    idx = routing(T, E, K, g)
    ws = moe.alloc_workspace(cfg)
    o, q, s = dispatch(cfg, x, idx, ws)
    plain = {k: torch.empty_like(v) for k, v in o.items()}
    moe.moe_dispatch(cfg, None, idx, *plain.values(), None, ws)
    for k in o:
        assert torch.equal(o[k], plain[k]), k
    rq, rs = R.quantize(x.float())
    tok = o["perm_token"].long()
    assert torch.equal(q.double(), rq[tok]) and same(s.double(), rs[tok, 0])
    assert moe.moe_read_device_status(ws) == moe.MOE_OK


@pytest.mark.parametrize("T,d,E,G,K,M", [(4, 64, 16, 4, 4, 2), (64, 128, 16, 4, 4, 2),
                                         (256, 192, 256, 8, 8, 4), (256, 64, 1024, 64, 32, 32),
                                         (128, 64, 1024, 64, 32, 32),
                                         (255, 8256, 40, 5, 6, 2), (257, 320, 12, 1, 4, 1),
                                         (264, 320, 12, 4, 4, 2), (1, 64, 1, 1, 1, 1)])
@pytest.mark.parametrize("bad", [False, True])
def test_dispatch_int8_plan_is_moe_dispatchs(T, d, E, G, K, M, bad):
    """Every output of the plan, in batches of one launch (up to 256 tokens) and of several; with
    ids out of range and an expert listed twice too, which are flagged and skipped alike."""
    cfg, g = config(T, d, E, K, 64, G=G, M=M), gen(T + E)
    x = torch.randn(T, d, device=DEV, generator=g).bfloat16()
    idx = routing(T, E, K, g, 1.0)
    if bad:
        idx[T // 2, 0] = E
        idx[T - 1, K - 1] = -7
        if K > 1:
            idx[0, 1] = idx[0, 0]
    ws = moe.alloc_workspace(cfg)
    o, q, s = dispatch(cfg, x, idx, ws)
    assert moe.moe_read_device_status(ws) == (moe.MOE_ERR_DEVICE_FAULT if bad else moe.MOE_OK)
    plain = {k: torch.full_like(v, -3) for k, v in o.items()}
    moe.moe_dispatch(cfg, None, idx, *plain.values(), None, moe.alloc_workspace(cfg))
    n = int(plain["offsets"][-1])
    for k in o:
        a, b = (o[k][:n], plain[k][:n]) if k == "perm_token" else (o[k], plain[k])
        assert torch.equal(a, b), k
    rq, rs = R.quantize(x.float())
    tok = o["perm_token"][:n].long()
    assert torch.equal(q[:n].double(), rq[tok]) and torch.equal(s[:n].double(), rs[tok, 0])
    assert (q[n:] == 77).all() and (s[n:] == -1).all()  # rows of no copy, as they were


def test_exact_ties_round_to_the_even_code():
    T, d = 2, 64
    cfg = config(T, d, 4, 1, 64)
    x = torch.arange(-32, 32, device=DEV).float() / 2  # steps of half a code: amax 16 -> no tie
    x = torch.stack([x, torch.cat([torch.tensor([63.5], device=DEV), x[1:]])]).bfloat16()
    _, q, s = dispatch(cfg, x, torch.zeros(T, 1, dtype=torch.int32, device=DEV),
                       moe.alloc_workspace(cfg))
    rq, rs = R.quantize(x.float())
    assert torch.equal(q.double(), rq) and torch.equal(s.double(), rs[:, 0])
    assert float(s[1]) == 0.5 and (q[1, 1:].double() == (x[1, 1:].double() / 0.5).round()).all()


@pytest.mark.parametrize("d,d_ff,ns,fs", [(64, 64, 0, 0), (192, 2112, 1, 64), (2112, 128, 2, 64),
                                          (320, 192, 3, 2880)])
def test_quantize_weights(d, d_ff, ns, fs):
    cfg, g = config(8, d, 3, 1, d_ff, ns, fs), gen(d)
    sizes = {"w_gate": (3, d_ff, d), "w_up": (3, d_ff, d), "w_down": (3, d, d_ff)}
    if ns:
        sizes |= {"ws_gate": (ns, fs, d), "ws_up": (ns, fs, d), "ws_down": (ns, d, fs)}
    w = {k: torch.randn(v, device=DEV, generator=g).bfloat16() for k, v in sizes.items()}
    out = moe.quantize_weights_int8(cfg, *w.values()).tensors
    for k, v in w.items():
        if k == "ws_down":
            q, s = R.quantize(v.permute(1, 0, 2).flatten(1).float())
            q = q.view(d, ns, fs).permute(1, 0, 2)
        else:
            q, s = R.quantize(v.flatten(0, 1).float())
            q = q.view(v.shape)
        assert torch.equal(out[k].double(), q), k
        assert torch.equal(out[k + "_scale"].double().flatten(), s.flatten()), k


# ------------------------------------------------------------------ products
FFN = [  # T, d, E, K, d_ff, n_shared, d_ff_shared, skew
    (1, 64, 1, 1, 64, 0, 0, 0.0), (1, 7168, 16, 8, 192, 1, 64, 0.0), (2, 128, 8, 2, 128, 2, 64, 0.0),
    (64, 192, 4, 4, 64, 3, 192, 0.0), (127, 128, 1, 1, 256, 0, 0, 0.0),
    (128, 256, 1, 1, 320, 1, 128, 0.0), (129, 64, 2, 1, 192, 1, 320, 0.0),
    (264, 320, 12, 4, 192, 1, 128, 0.0), (520, 192, 40, 6, 128, 2, 64, 1.2),
    (300, 2048, 64, 6, 1408, 2, 1408, 0.6), (33, 576, 1024, 8, 64, 0, 0, 0.0),
    (1000, 448, 6, 2, 576, 1, 576, 2.0), (16, 4096, 3, 3, 2112, 1, 4160, 0.0),
    (700, 1024, 5, 4, 1024, 1, 512, 0.0)]


def check_ffn(cfg, x_perm_q, x_scale, offsets, w, x, y, y_shared):
    routed, shared = R.ffn(cfg, x_perm_q, x_scale, offsets, w, x)
    for got, want in ((y, routed), (y_shared, shared)):
        if want is not None:
            off = (got.double() - want[0]).abs()
            assert (off <= want[1]).all(), float((off / want[1]).max())


def ffn_inputs(case, seed=0):
    T, d, E, K, d_ff, ns, fs, skew = case
    cfg, g = config(T, d, E, K, d_ff, ns, fs), gen(seed + sum(case[:6]))
    idx = routing(T, E, K, g, skew)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.bincount(idx.flatten().long(), minlength=E).cumsum(0)
    xq = torch.randint(-128, 128, (T * K, d), dtype=torch.int8, device=DEV, generator=g)
    xs = (torch.rand(T * K, device=DEV, generator=g) + 0.5) / 74
    x = torch.randn(T, d, device=DEV, generator=g).bfloat16()
    return cfg, xq, xs, offsets, random_weights(cfg, g), x


def run_ffn(cfg, xq, xs, offsets, w, x, ws=None, stream=None):
    y = torch.full(xq.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    sh = torch.full(x.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = moe.alloc_int8_workspace(cfg) if ws is None else ws
    moe.moe_expert_ffn_int8(cfg, xq, xs, offsets, moe.Int8Weights(**w), y, x,
                            sh if cfg.n_shared else None, ws, stream=stream)
    return y, sh, ws


@pytest.mark.parametrize("case", FFN, ids=str)
def test_expert_ffn_int8(case):
    cfg, xq, xs, offsets, w, x = ffn_inputs(case)
    y, sh, ws = run_ffn(cfg, xq, xs, offsets, w, x)
    assert moe.moe_read_device_status(ws) == moe.MOE_OK
    check_ffn(cfg, xq, xs, offsets, w, x, y, sh)
    again, sh2, _ = run_ffn(cfg, xq, xs, offsets, w, x)
    assert torch.equal(again, y) and (not cfg.n_shared or torch.equal(sh, sh2))


def test_integer_sums_are_exact():
    """Sums of small integers behind partial sums of 127 * 127 * 8191 > 2^26, which 24-bit
    arithmetic would round away: g = u = 1, 2, 3, and the whole range of codes in w_down."""
    T, d, d_ff = 3, 16384, 64
    cfg = config(T, d, 1, 1, d_ff)
    xq = torch.full((T, d), 127, dtype=torch.int8, device=DEV)
    xq[:, -1] = torch.arange(1, T + 1, device=DEV)
    row = torch.full((d,), 127, dtype=torch.int8, device=DEV)
    row[8191:] = -127
    row[-2], row[-1] = 0, 1
    one = torch.ones(1, d_ff, device=DEV)
    w = {"w_gate": row.expand(1, d_ff, d).contiguous(), "w_up": row.expand(1, d_ff, d).contiguous(),
         "w_down": torch.zeros(1, d, d_ff, dtype=torch.int8, device=DEV),
         "w_gate_scale": one, "w_up_scale": one.clone(),
         "w_down_scale": torch.ones(1, d, device=DEV)}
    w["w_down"][0, :, 0] = torch.arange(-128, 128, device=DEV).repeat(d // 256).to(torch.int8)
    off = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    y, _, _ = run_ffn(cfg, xq, torch.ones(T, device=DEV), off, w, x)
    g = torch.arange(1, T + 1, device=DEV).double()[:, None]
    want = g * torch.sigmoid(g) * g * w["w_down"][0, :, 0].double()
    # h's row is constant: its code is 127 and its scale h / 127
    assert ((y.double() - want).abs() <= (2.0 ** -8 + 2 * R.H_REL) * want.abs()).all()


def test_gate_and_up_in_either_order_of_addresses():
    cfg, xq, xs, offsets, w, x = ffn_inputs((90, 192, 3, 2, 192, 2, 64, 0.0))
    y, sh, _ = run_ffn(cfg, xq, xs, offsets, w, x)
    for first, second in (("gate", "up"), ("up", "gate")):
        v = dict(w)
        for k in ("w_", "ws_"):
            both = torch.stack([w[k + first], w[k + second]])
            v[k + first], v[k + second] = both[0], both[1]
        y2, sh2, _ = run_ffn(cfg, xq, xs, offsets, v, x)
        assert torch.equal(y, y2) and torch.equal(sh, sh2)
    check_ffn(cfg, xq, xs, offsets, w, x, y, sh)


def test_tiles_of_more_than_256_tokens_give_the_same_bits():
    """152 experts of 4096 x 4160 with 0 to 700 tokens take tiles of up to 512 tokens in both
    products (the averages and lengths that choose them); 8 or 16 experts of them at a time do not.
    Integer sums and the same roundings: equal bits, the shared experts' among them."""
    E, K, T, d, ff = 152, 8, 4864, 4096, 4160
    cfg, g = config(T, d, E, K, ff, 1, 128), gen(21)
    counts = [0, 1, 255, 256, 257, 288, 289, 320, 384, 415, 416, 480, 511, 512, 513, 700]
    rest = T * K - sum(counts) - 40  # (40 rows in no segment)
    counts += [rest // (E - 16)] * (E - 17)
    counts += [T * K - 40 - sum(counts)]
    offsets = torch.tensor([0] + counts).cumsum(0).int().to(DEV)
    xq = torch.randint(-127, 128, (T * K, d), dtype=torch.int8, device=DEV, generator=g)
    xs = torch.rand(T * K, device=DEV, generator=g) / 74 + 1e-3
    x = torch.randn(T, d, device=DEV, generator=g).bfloat16()
    w = random_weights(cfg, g)
    y, sh, ws = run_ffn(cfg, xq, xs, offsets, w, x)
    assert not y[:-40].isnan().any() and y[-40:].isnan().all()
    for e, n in ((0, 8), (8, 8), (136, 16)):
        lo, hi = int(offsets[e]), int(offsets[e + n])
        part = config(-(-(hi - lo) // K), d, n, K, ff, 1, 128)
        rows = part.T * K
        pad = lambda t: torch.cat([t[lo:hi], t[:rows - (hi - lo)]])
        some = {k: v if k.startswith("ws_") else v[e:e + n].clone() for k, v in w.items()}
        seg = (offsets[e:e + n + 1] - lo).contiguous()
        y2, sh2, _ = run_ffn(part, pad(xq), pad(xs), seg, some, x[:part.T].contiguous())
        assert torch.equal(y[lo:hi], y2[:hi - lo]) and torch.equal(sh[:part.T], sh2)
    assert moe.moe_read_device_status(ws) == moe.MOE_OK


def test_rows_behind_the_2_to_the_31st_byte():
    """Dispatch, experts and the combine's gradient at 300,032 rows of 7168: codes pass 2^31 bytes,
    bf16 rows 2^32.  The last rows against their definition, the dispatch in full."""
    T, d, E, K, d_ff = 37504, 7168, 8, 8, 64
    cfg, g = config(T, d, E, K, d_ff), gen(9)
    x = torch.randn(T, d, device=DEV, generator=g).bfloat16()
    idx = torch.rand(T, E, device=DEV, generator=g).argsort(1).int()
    ws = moe.alloc_int8_workspace(cfg)
    o, q, s = dispatch(cfg, x, idx, ws)
    rq, rs = R.quantize(x.float())
    rq = rq.to(torch.int8)
    for rows in torch.arange(T * K, device=DEV).split(50000):
        tok = o["perm_token"][rows].long()
        assert torch.equal(q[rows], rq[tok]) and torch.equal(s[rows].double(), rs[tok, 0])
    w = random_weights(cfg, g)
    y, _, _ = run_ffn(cfg, q, s, o["offsets"], w, x, ws)
    assert moe.moe_read_device_status(ws) == moe.MOE_OK
    tail = 200
    last = {k: v[E - 1:] for k, v in w.items()}
    seg = torch.tensor([0, tail], dtype=torch.int32)
    check_ffn(cfg, q[-tail:], s[-tail:], seg, last, None, y[-tail:], None)
    up = torch.randn(T, d, device=DEV, generator=g).bfloat16()
    gate = torch.rand(T, K, device=DEV, generator=g)
    dy, dw = torch.empty_like(y), torch.empty(T, K, device=DEV)
    moe.moe_combine_backward(cfg, up, y, o["inv_perm"], gate, dy, dw)
    t = torch.arange(T - 50, T, device=DEV)
    rows = o["inv_perm"][t].long()
    want = gate[t].double()[:, :, None] * up[t].double()[:, None]
    assert ((dy[rows].double() - want).abs() <= (2.0 ** -8 + 2 * R.U) * want.abs()).all()
    prod = up[t].double()[:, None] * y[rows].double()
    n = 8 * -(-d // 256) + 13
    assert ((dw[t].double() - prod.sum(2)).abs() <= n * R.U * prod.abs().sum(2)).all()


def test_a_row_with_a_nan_scale_is_nan_and_no_other():
    cfg, xq, xs, offsets, w, x = ffn_inputs((70, 128, 4, 2, 192, 1, 64, 0.0))
    y, sh, _ = run_ffn(cfg, xq, xs, offsets, w, x)
    xs[33] = float("nan")
    x[11, 3] = float("inf")
    y2, sh2, _ = run_ffn(cfg, xq, xs, offsets, w, x)
    assert y2[33].isnan().all() and sh2[11].isnan().all()
    keep = torch.arange(140, device=DEV) != 33
    assert torch.equal(y[keep], y2[keep])
    keep = torch.arange(70, device=DEV) != 11
    assert torch.equal(sh[keep], sh2[keep])


def test_rows_of_zeros_give_zeros():
    cfg, xq, xs, offsets, w, x = ffn_inputs((20, 64, 2, 1, 64, 1, 64, 0.0))
    xs[4] = 0.0
    xq[5] = 0
    x[6] = 0.0
    y, sh, _ = run_ffn(cfg, xq, xs, offsets, w, x)
    assert not y[4].any() and not y[5].any() and not sh[6].any()


def test_empty_experts_and_rows_outside_the_segments_are_left_alone():
    cfg, xq, xs, offsets, w, x = ffn_inputs((50, 128, 8, 1, 64, 0, 0, 0.0))
    off = torch.tensor([0, 0, 7, 7, 7, 30, 30, 41, 41], dtype=torch.int32, device=DEV)
    y, _, ws = run_ffn(cfg, xq, xs, off, w, x)
    assert moe.moe_read_device_status(ws) == moe.MOE_OK
    check_ffn(cfg, xq, xs, off, w, x, y[:41], None)
    assert y[41:].isnan().all()  # as they were


def test_bad_offsets_are_flagged_and_skipped():
    cfg, xq, xs, offsets, w, x = ffn_inputs((50, 128, 4, 1, 64, 0, 0, 0.0))
    for off in ([0, 10, 5, 20, 50], [-3, 10, 20, 30, 50], [0, 10, 20, 30, 51],
                [0, 2 ** 31 - 1, 20, 30, 50]):
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        _, _, ws = run_ffn(cfg, xq, xs, o, w, x)
        assert moe.moe_read_device_status(ws) == moe.MOE_ERR_DEVICE_FAULT, off


# ------------------------------------------------------------------ the layer
def layer(sh, router=0):
    inp = synth.make_inputs(sh, DEV)
    cfg = moe.MoeConfig.of(sh, router=router)
    w = moe.quantize_weights_int8(cfg, *(inp[k] for k in ("w_gate", "w_up", "w_down", "ws_gate",
                                                          "ws_up", "ws_down")))
    return inp, cfg, w


@pytest.mark.parametrize("name,router", [("tiny", 0), ("ragged", 0), ("ragged2", 1),
                                         ("noshared", 0), ("ragged", 2)])
def test_forward_int8_is_its_stages(name, router):
    sh = H.shape(name)
    inp, cfg, w = layer(sh, router)
    ws = moe.alloc_int8_workspace(cfg)
    o = moe.forward_outputs(cfg)
    moe.moe_forward_int8(cfg, inp["x"], inp["router_w"], None, inp["bias"], w, **o, ws=ws)
    assert moe.moe_read_device_status(ws) == moe.MOE_OK
    ws2 = moe.alloc_int8_workspace(cfg)
    bf = moe.forward_outputs(cfg)
    moe.moe_forward(cfg, inp["x"], inp["router_w"], None, inp["bias"], inp["w_gate"], inp["w_up"],
                    inp["w_down"], inp["ws_gate"], inp["ws_up"], inp["ws_down"], **bf, ws=ws2)
    for k in ("topk_idx", "topk_w", "counts", "offsets", "send", "send_tok"):
        assert torch.equal(o[k], bf[k]), k
    d, q, s = dispatch(cfg, inp["x"], o["topk_idx"], ws2)
    y, shared, _ = run_ffn(cfg, q, s, d["offsets"], w.tensors, inp["x"], ws2)
    out = torch.empty_like(o["out"])
    moe.moe_combine(cfg, y, d["inv_perm"], o["topk_w"], shared if cfg.n_shared else None, out)
    assert torch.equal(out, o["out"])
    check_ffn(cfg, q, s, d["offsets"], w.tensors, inp["x"], y, shared)


def test_forward_int8_is_near_the_bf16_layer():
    """Codes are off by half a step, s / 2 = amax / 254, at most: uniform over the step, a row of
    near-normal values (amax about 4 sigma, 6 for h) has a relative error of about
    4 / (127 sqrt 12) = 0.9 % a factor, 1.4 % for h; of the five factors of an output (x twice, its
    two weights, h, w_down) the squares add up to 2.5 %.  Twice that is allowed."""
    sh = H.shape("ragged")
    inp, cfg, w = layer(sh)
    ws = moe.alloc_int8_workspace(cfg)
    a, b = moe.forward_outputs(cfg), moe.forward_outputs(cfg)
    moe.moe_forward_int8(cfg, inp["x"], inp["router_w"], None, inp["bias"], w, a["out"], ws=ws)
    moe.moe_forward(cfg, inp["x"], inp["router_w"], None, inp["bias"], inp["w_gate"], inp["w_up"],
                    inp["w_down"], inp["ws_gate"], inp["ws_up"], inp["ws_down"], b["out"], ws=ws)
    frob, _ = H.compare_out(a["out"], H.bf16_to_f64(b["out"]))
    assert frob < 0.05


def test_forward_int8_of_one_token():
    sh = H.shape("v3").replace(T=1, G=1, M=1, E=16, d=1024, d_ff=512, d_ff_shared=512)
    inp, cfg, w = layer(sh)
    ws = moe.alloc_int8_workspace(cfg)
    o = moe.forward_outputs(cfg)
    moe.moe_forward_int8(cfg, inp["x"], inp["router_w"], None, inp["bias"], w, **o, ws=ws)
    assert moe.moe_read_device_status(ws) == moe.MOE_OK
    d, q, s = dispatch(cfg, inp["x"], o["topk_idx"], ws)
    y, shared, _ = run_ffn(cfg, q, s, d["offsets"], w.tensors, inp["x"], ws)
    check_ffn(cfg, q, s, d["offsets"], w.tensors, inp["x"], y, shared)


def test_forward_int8_streams_and_graph():
    sh = H.shape("ragged2")
    inp, cfg, w = layer(sh)
    ws = [moe.alloc_int8_workspace(cfg) for _ in range(2)]
    o = [moe.forward_outputs(cfg) for _ in range(2)]
    x2 = inp["x"].flip(0).contiguous()

    def call(x, out, wsp):
        moe.moe_forward_int8(cfg, x, inp["router_w"], None, inp["bias"], w, **out, ws=wsp)

    want = []
    for x in (inp["x"], x2):
        call(x, o[0], ws[0])
        want.append({k: v.clone() for k, v in o[0].items()})
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):  # two calls at once, a workspace each
        for s, x, out, wsp in zip(streams, (inp["x"], x2), o, ws):
            with torch.cuda.stream(s):
                call(x, out, wsp)
    torch.cuda.synchronize()
    for out, ref in zip(o, want):
        assert all(torch.equal(out[k], ref[k]) for k in ref)
    x = inp["x"].clone()
    graphs = []
    for i in range(2):  # two graphs that share a workspace, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(x, o[i], ws[0])
        graphs.append(graph)
    for _ in range(3):
        x.copy_(inp["x"])
        graphs[0].replay()
        x.copy_(x2)
        graphs[1].replay()
    torch.cuda.synchronize()
    for out, ref in zip(o, want):
        assert all(torch.equal(out[k], ref[k]) for k in ref)


def test_python_entry_points_refuse_wrong_tensors():
    cfg, xq, xs, offsets, w, x = ffn_inputs((8, 64, 2, 1, 64, 1, 64, 0.0))
    ws = moe.alloc_int8_workspace(cfg)
    y, sh = torch.empty_like(xq, dtype=torch.bfloat16), torch.empty_like(x)
    good = moe.Int8Weights(**w)
    for args in [(xq.float(), xs, offsets, good, y, x, sh, ws), (xq, xs.half(), offsets, good, y, x, sh, ws),
                 (xq, xs, offsets.long(), good, y, x, sh, ws), (xq[:4], xs, offsets, good, y, x, sh, ws),
                 (xq, xs, offsets, good, y, None, sh, ws), (xq, xs, offsets, good, y, x, None, ws),
                 (xq.cpu(), xs, offsets, good, y, x, sh, ws), (xq, xs, offsets, good, y, x, sh, None),
                 (xq, xs, offsets, good, y, x, sh, ws[:4096]),
                 (xq, xs, offsets, moe.Int8Weights(**{**w, "w_up": w["w_up"][:1]}), y, x, sh, ws),
                 (xq, xs, offsets, moe.Int8Weights(**{**w, "w_up": None}), y, x, sh, ws)]:
        with pytest.raises(moe.MoeError):
            moe.moe_expert_ffn_int8(cfg, *args)
    with pytest.raises(TypeError):
        moe.Int8Weights(w_gate=w["w_gate_scale"])
    with pytest.raises(TypeError):
        moe.Int8Weights(w_gate=w["w_gate"].transpose(1, 2))
    with pytest.raises(TypeError):
        moe.Int8Weights(gate=w["w_gate"])


# ------------------------------------------------------------------ short kernels one behind the other
@pytest.mark.parametrize("d,d_ff", [(64, 64), (128, 64), (704, 320), (768, 768), (832, 1472)])
def test_short_pair_kernels_behind_one_another(d, d_ff):
    """Tiles of 1 to 13 k blocks on a ring of six stages, from one tile up to several a pair, three
    hundred calls without a pause: a block's last stages are still being released when the next
    kernel's blocks want its place."""
    for T, E, K in ((1, 1, 1), (3, 5, 2), (64, 24, 4)):
        cfg, xq, xs, offsets, w, x = ffn_inputs((T, d, E, K, d_ff, 1, 64, 0.0))
        y, sh, ws = run_ffn(cfg, xq, xs, offsets, w, x)
        weights, y2, sh2 = moe.Int8Weights(**w), torch.empty_like(y), torch.empty_like(sh)
        for _ in range(300):
            moe.moe_expert_ffn_int8(cfg, xq, xs, offsets, weights, y2, x, sh2, ws)
        assert torch.equal(y, y2) and torch.equal(sh, sh2)
        assert moe.moe_read_device_status(ws) == moe.MOE_OK
        check_ffn(cfg, xq, xs, offsets, w, x, y, sh)


# ------------------------------------------------------------------ sizes that need more shared memory
def dispatch_sizes():
    for T, E, G, K, M in ((118, 590, 59, 4, 2), (118, 649, 59, 4, 2), (256, 1024, 64, 8, 4)):
        cfg, g = config(T, 64, E, K, 64, G=G, M=M), gen(E)
        x, idx = torch.randn(T, 64, device=DEV, generator=g).bfloat16(), routing(T, E, K, g)
        o, q, s = dispatch(cfg, x, idx, moe.alloc_workspace(cfg))
        plain = {k: torch.empty_like(v) for k, v in o.items()}
        moe.moe_dispatch(cfg, None, idx, *plain.values(), None, moe.alloc_workspace(cfg))
        assert all(torch.equal(o[k], plain[k]) for k in o), (E, G)
        rq, rs = R.quantize(x.float())
        tok = o["perm_token"].long()
        assert torch.equal(q.double(), rq[tok]) and torch.equal(s.double(), rs[tok, 0])


def test_dispatch_int8_of_many_experts_and_groups_in_a_fresh_process():
    """590 experts in 59 groups take 49092 bytes of shared memory, which with the 192 that the
    kernel declares are more than 48 KB; nothing before this call asked for more."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", "import tests.test_gpu_int8 as t; t.dispatch_sizes()"],
                       cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------------------------ the rows of bad segments
@pytest.mark.parametrize("n_shared", [0, 1])
def test_bad_segments_are_neither_computed_nor_written(n_shared):
    """Segments that leave the buffer or have a negative length are empty; the others are computed,
    and rows of no valid segment stay as they were."""
    cfg, xq, xs, offsets, w, x = ffn_inputs((50, 128, 4, 1, 64, n_shared, 64 * n_shared, 0.0))
    for off in ([0, 10, 20, 30, 51], [-3, 10, 20, 30, 50], [0, 2 ** 31 - 1, 20, 30, 50],
                [12, 12, 5, 20, -1], [0, 10, 5, 20, 50]):
        y, sh, ws = run_ffn(cfg, xq, xs, torch.tensor(off, dtype=torch.int32, device=DEV), w, x)
        assert moe.moe_read_device_status(ws) == moe.MOE_ERR_DEVICE_FAULT, off
        owners = torch.zeros(50, dtype=torch.int64, device=DEV)
        valid = [(e, lo, hi) for e, (lo, hi) in enumerate(zip(off, off[1:])) if 0 <= lo <= hi <= 50]
        for _, lo, hi in valid:
            owners[lo:hi] += 1
        for e, lo, hi in valid:
            one = owners[lo:hi] == 1  # a row of two segments has either's value
            if hi == lo or not one.any():
                continue
            some = {k: v if k.startswith("ws_") else v[e:e + 1] for k, v in w.items()}
            want, room = R.ffn(config(50, 128, 1, 1, 64), xq[lo:hi], xs[lo:hi], [0, hi - lo], some,
                               None)[0]
            assert ((y[lo:hi].double() - want).abs() <= room)[one].all(), (off, e)
        assert y[owners == 0].isnan().all() and not y[owners > 0].isnan().any(), off
        if n_shared:
            want, room = R.ffn(cfg, xq, xs, [0, 50, 50, 50, 50], w, x)[1]
            assert ((sh.double() - want).abs() <= room).all()


# ------------------------------------------------------------------ the codes of h
def test_codes_of_h_are_those_of_the_product_with_the_reciprocal():
    """h's codes by their rule, rint(h * fp32(1 / s)) of the exact product, where a division gives
    others: rows whose h lies on every half between two codes, for scales of inexact reciprocal.
    g = 128, whose SiLU is 128 itself (e^-128 adds nothing to 1), u = j m with whole j and m, so
    h = 128 j m exactly; its largest is 128 * 254 m, s = 256 m, and h / s = j / 2.  w_down copies
    code c to channel c, in units."""
    d = d_ff = 512
    ms = [m for m in range(3, 128, 2)]
    T = len(ms)
    cfg = config(T, d, 1, 1, d_ff)
    j = torch.cat([torch.arange(-254, 255), torch.tensor([254, 1, -1])])  # 512 values, 254 among them
    xq = torch.zeros(T, d, dtype=torch.int8)
    xq[:, 0] = xq[:, 1] = torch.tensor(ms)
    xq[:, 2] = 1
    up, gate = torch.zeros(1, d_ff, d, dtype=torch.int8), torch.zeros(1, d_ff, d, dtype=torch.int8)
    up[0, :, 0] = torch.div(j, 2, rounding_mode="floor")
    up[0, :, 1] = j - torch.div(j, 2, rounding_mode="floor")
    gate[0, :, 2] = 64
    one = torch.ones(1, d_ff, device=DEV)
    w = {"w_gate": gate.to(DEV), "w_up": up.to(DEV),
         "w_down": torch.eye(d, dtype=torch.int8, device=DEV)[None].contiguous(),
         "w_gate_scale": 2 * one, "w_up_scale": one.clone(), "w_down_scale": torch.ones(1, d, device=DEV)}
    off = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    y, _, ws = run_ffn(cfg, xq.to(DEV), torch.ones(T, device=DEV), off, w, x)
    assert moe.moe_read_device_status(ws) == moe.MOE_OK
    m = torch.tensor(ms, dtype=torch.float64)[:, None]
    h, s = 128 * j.double() * m, 256 * m
    inv = (1 / s).float().double()               # fp32(1 / s): 53 bits first, which is no tie of 24
    want = (h * inv).round()                     # 24 + 24 bits: exact in 64
    divided = (h / s).round()
    assert int((want != divided).sum()) > 1000   # the two rules differ here
    # y = bf16(code * s), an 8-bit code times s and one rounding: the nearest code is the code
    got = (y.double().cpu() / s).round()
    assert torch.equal(got, want)


# ------------------------------------------------------------------ what another stream writes
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("T", [100, 300])
def test_operands_that_another_stream_writes(T, captured):
    """Every operand of the dispatch and of the experts -- offsets and weights too, which a product
    may read while the kernel before it still runs -- comes from another stream, which the calls'
    stream waits for between two rounds of calls; eager, and as the branches of a graph."""
    cfg, xq, xs, offsets, w, x = ffn_inputs((T, 192, 12, 4, 320, 1, 128, 0.0))
    _, xq2, xs2, offsets2, w2, x2 = ffn_inputs((T, 192, 12, 4, 320, 1, 128, 0.0), seed=77)
    g = gen(5)
    idx, idx2 = routing(T, 12, 4, g), routing(T, 12, 4, g)
    ws = [moe.alloc_int8_workspace(cfg) for _ in range(2)]
    want = (*run_ffn(cfg, xq2, xs2, offsets2, w2, x2)[:2], *dispatch(cfg, x2, idx2, ws[0]))
    weights = moe.Int8Weights(**w)
    pairs = [(xq, xq2), (xs, xs2), (offsets, offsets2), (x, x2), (idx, idx2)] + [(w[k], w2[k]) for k in w]
    y, sh = torch.empty(xq.shape, dtype=torch.bfloat16, device=DEV), torch.empty_like(x)
    first = [a.clone() for a, _ in pairs]
    o, q, s = dispatch(cfg, x, idx, ws[0])
    side = torch.cuda.Stream()

    def calls():
        moe.moe_dispatch_int8(cfg, x, idx, *o.values(), q, s, ws[1])
        moe.moe_expert_ffn_int8(cfg, xq, xs, offsets, weights, y, x, sh, ws[0])

    def run():
        here = torch.cuda.current_stream()
        calls()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
            for a, b in pairs:
                a.copy_(b)
        here.wait_stream(side)
        calls()

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
    for _ in range(3):
        for (a, _), b in zip(pairs, first):
            a.copy_(b)
        y.fill_(float("nan"))
        q.fill_(77)
        graph.replay() if captured else run()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(sh, want[1])
        assert all(torch.equal(o[k], want[2][k]) for k in o)
        assert torch.equal(q, want[3]) and torch.equal(s, want[4])
    for wsp in ws:
        assert moe.moe_read_device_status(wsp) == moe.MOE_OK


@pytest.mark.parametrize("T,E,G,K,M", [(129, 64, 1, 32, 1), (192, 256, 8, 24, 8), (256, 256, 8, 32, 8),
                                       (256, 40, 1, 17, 1), (256, 32, 1, 32, 1)])
def test_dispatch_int8_of_one_block_and_many_copies(T, E, G, K, M):
    """Batches of one launch with more than 4096 copies: up to 8192, every expert of a token's."""
    cfg, g = config(T, 320, E, K, 64, G=G, M=M), gen(T + K)
    x, idx = torch.randn(T, 320, device=DEV, generator=g).bfloat16(), routing(T, E, K, g, 0.6)
    ws = moe.alloc_workspace(cfg)
    before = moe.moe_launch_count()
    o, q, s = dispatch(cfg, x, idx, ws)
    assert moe.moe_launch_count() - before == 1
    assert moe.moe_read_device_status(ws) == moe.MOE_OK
    plain = {k: torch.empty_like(v) for k, v in o.items()}
    moe.moe_dispatch(cfg, None, idx, *plain.values(), None, ws)
    assert all(torch.equal(o[k], plain[k]) for k in o)
    rq, rs = R.quantize(x.float())
    tok = o["perm_token"].long()
    assert torch.equal(q.double(), rq[tok]) and torch.equal(s.double(), rs[tok, 0])
