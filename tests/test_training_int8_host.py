"""Host-side checks of the balance loss, the gradients and the int8 experts that need no GPU: every
call here is refused by argument validation before a kernel is launched."""
import ctypes as C

import pytest
import torch

import synth

P = 1 << 20  # a 256-byte aligned address that no call reads


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__ as g
    g._builder().build()
    import combine_expert_ffn_b200 as m
    return m


def cfg(moe, **kw):
    return moe.MoeConfig.of(synth.config("tiny").replace(**kw))


def refused(moe, fn, *args):
    with pytest.raises(moe.MoeError) as e:
        fn(*args)
    return e.value.status


class WS:
    """Stands for a workspace tensor of n bytes."""
    def __init__(self, n, ptr=P):
        self.n, self.ptr = n, ptr

    def data_ptr(self):
        return self.ptr

    def numel(self):
        return self.n

    def element_size(self):
        return 1


def test_balance_loss_arguments(moe):
    c = cfg(moe)
    n = moe.moe_workspace_size(c)
    lib = moe._lib.moe_balance_loss

    def call(scores=P, idx=P, seq=P, n_seq=2, alpha=0.1, counts=P, prob=P, loss=P, ws=P, wn=n, c=c):
        return lib(C.byref(c), scores, idx, seq, n_seq, alpha, counts, prob, loss, ws, wn, None)

    for kw in (dict(scores=None), dict(idx=None), dict(seq=None), dict(n_seq=-1), dict(counts=None),
               dict(prob=None), dict(loss=None), dict(ws=None), dict(scores=P + 4), dict(ws=P + 16),
               dict(alpha=float("inf")), dict(alpha=float("nan"))):
        assert call(**kw) == moe.MOE_ERR_INVALID_ARG, kw
    assert call(wn=n - 1) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    assert call(c=cfg(moe, T=63)) == moe.MOE_ERR_UNSUPPORTED_SHAPE
    assert lib(None, P, P, P, 2, 0.1, P, P, P, P, n, None) == moe.MOE_ERR_INVALID_ARG


def test_balance_tiles_fit_the_workspace(moe):
    """The tiles' shares, 16 E bytes a tile, against the 4 T E bytes of the affinities' region."""
    for T in [*range(1, 2000), 9472, 9473, 262144, 2 ** 26 - 1]:
        tile = max(32, -(-T // (8 if T <= 1024 else 296)))
        tiles = -(-T // tile)
        assert tiles == 1 or 4 * tiles <= T


def test_balance_tiles_of_short_sequences_fit_the_workspace(moe):
    """The same for tiles of an average sequence, 8 tokens or more."""
    for T in [*range(1, 400), 1024, 1025, 262144]:
        for n_seq in {1, 2, T // 40 + 1, T // 9 + 1, T, 2 * T, 2 ** 20}:
            tile, average = max(32, -(-T // (8 if T <= 1024 else 296))), max(8, T // n_seq, T // 2048)
            tile = average if 2 * average <= tile else tile
            tiles = -(-T // tile)
            assert tiles == 1 or 4 * tiles <= T


def test_route_backward_arguments(moe):
    c = cfg(moe)
    lib = moe._lib.moe_route_backward

    def call(scores=P, idx=P, dw=P, seq=P, n_seq=2, counts=P, dl=P, alpha=0.1, out=P, c=c):
        return lib(C.byref(c), scores, idx, dw, seq, n_seq, counts, dl, alpha, out, None, None)

    hashed = moe.MoeConfig.of(synth.config("tiny"), router=moe.MOE_ROUTER_HASH)
    for kw in (dict(scores=None), dict(idx=None), dict(dw=None, dl=None), dict(seq=None),
               dict(n_seq=-1), dict(counts=None), dict(out=None), dict(scores=P + 8),
               dict(out=P + 4), dict(alpha=float("nan")), dict(c=hashed)):
        assert call(**kw) == moe.MOE_ERR_INVALID_ARG, kw
    assert call(c=cfg(moe, K=3)) == moe.MOE_ERR_UNSUPPORTED_SHAPE


def test_combine_backward_arguments(moe):
    c = cfg(moe)
    lib = moe._lib.moe_combine_backward

    def call(g=P, y=P, inv=P, w=P, dy=P, dw=P, c=c):
        return lib(C.byref(c), g, y, inv, w, dy, dw, None)

    for kw in (dict(g=None), dict(y=None), dict(inv=None), dict(w=None), dict(dy=None, dw=None),
               dict(g=P + 2), dict(y=P + 8), dict(dy=P + 4)):
        assert call(**kw) == moe.MOE_ERR_INVALID_ARG, kw
    assert call(c=cfg(moe, d=100)) == moe.MOE_ERR_UNSUPPORTED_SHAPE


def weights(moe, **kw):
    w = moe.Int8Weights()
    for n, _ in w._fields_:
        setattr(w, n, kw.get(n, P + 4096 * (n in ("w_up", "ws_up"))))
    return w


def test_int8_sizes(moe):
    for name in synth.CONFIGS:
        c = moe.MoeConfig.of(synth.config(name))
        T, rows, ffs = c.T, c.T * c.K, c.n_shared * c.d_ff_shared

        def up(v):
            return (v + 255) // 256 * 256

        extra = up(4 * rows * c.d_ff) + up(4 * T * ffs) + up(T * c.d) + up(4 * T)
        assert moe.moe_int8_workspace_size(c) == moe.moe_workspace_size(c) + extra
    assert moe.moe_int8_workspace_size(cfg(moe, T=63)) == 0
    for kw in (dict(d=131072), dict(d_ff=131072), dict(n_shared=2, d_ff_shared=65536)):
        assert moe.moe_check_config(cfg(moe, **kw)) == moe.MOE_OK
        assert moe.moe_int8_workspace_size(cfg(moe, **kw)) == 0
    sizes = [moe.moe_int8_workspace_size(cfg(moe, T=T)) for T in range(0, 1000, 4)]
    assert sizes == sorted(sizes)
    with pytest.raises(moe.MoeError):
        moe.alloc_int8_workspace(cfg(moe, d=131072), "cpu")


def test_quantize_weights_arguments(moe):
    c = cfg(moe)
    lib, w = moe._lib.moe_quantize_weights_int8, weights(moe)
    ptrs = [P] * 6
    for i in range(6):
        assert lib(C.byref(c), *ptrs[:i], None, *ptrs[i + 1:], C.byref(w), None) == \
            moe.MOE_ERR_INVALID_ARG
        assert lib(C.byref(c), *ptrs[:i], P + 2, *ptrs[i + 1:], C.byref(w), None) == \
            moe.MOE_ERR_INVALID_ARG
    for n, _ in w._fields_:
        for bad in (None, P + 4):
            b = weights(moe, **{n: bad})
            assert lib(C.byref(c), *ptrs, C.byref(b), None) == moe.MOE_ERR_INVALID_ARG, n
    assert lib(C.byref(c), *ptrs, None, None) == moe.MOE_ERR_INVALID_ARG
    assert lib(C.byref(cfg(moe, d_ff=131072)), *ptrs, C.byref(w), None) == \
        moe.MOE_ERR_UNSUPPORTED_SHAPE


def test_dispatch_int8_arguments(moe):
    c = cfg(moe)
    n = moe.moe_workspace_size(c)
    lib = moe._lib.moe_dispatch_int8
    args = [P] * 10  # x, topk_idx, counts, offsets, send, send_tok, perm_token, inv_perm, codes, scales
    for i in (0, 1, 2, 3, 4, 6, 7, 8, 9):
        bad = [*args]
        bad[i] = None
        assert lib(C.byref(c), *bad, P, n, None) == moe.MOE_ERR_INVALID_ARG, i
    for i in (0, 8, 9):
        bad = [*args]
        bad[i] = P + 4
        assert lib(C.byref(c), *bad, P, n, None) == moe.MOE_ERR_INVALID_ARG, i
    assert lib(C.byref(c), *args, P, n - 1, None) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    assert lib(C.byref(c), *args, P + 8, n, None) == moe.MOE_ERR_INVALID_ARG
    assert lib(C.byref(c), *args, None, n, None) == moe.MOE_ERR_INVALID_ARG


def test_expert_ffn_int8_arguments(moe):
    c = cfg(moe)
    n = moe.moe_int8_workspace_size(c)
    lib = moe._lib.moe_expert_ffn_int8

    def call(xq=P, xs=P, off=P, w=weights(moe), y=P, x=P, sh=P, ws=P, wn=n, c=c):
        return lib(C.byref(c), xq, xs, off, C.byref(w) if w else None, y, x, sh, ws, wn, None)

    for kw in (dict(xq=None), dict(xs=None), dict(off=None), dict(w=None), dict(y=None),
               dict(x=None), dict(sh=None), dict(ws=None), dict(xq=P + 8), dict(y=P + 2),
               dict(x=P + 4), dict(sh=P + 8), dict(ws=P + 64)):
        assert call(**kw) == moe.MOE_ERR_INVALID_ARG, kw
    for f, _ in moe.Int8Weights._fields_:
        for bad in (None, P + 4):
            assert call(w=weights(moe, **{f: bad})) == moe.MOE_ERR_INVALID_ARG, f
    for pair in ("w", "ws"):  # gate and up: two buffers, less than 2^40 bytes apart
        for gate, up in ((P, P), (P, P + (1 << 40)), (P + (1 << 40), P)):
            assert call(w=weights(moe, **{pair + "_gate": gate, pair + "_up": up})) == \
                moe.MOE_ERR_INVALID_ARG
    assert call(wn=n - 1) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    assert call(wn=moe.moe_workspace_size(c)) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    assert call(c=cfg(moe, d=131072)) == moe.MOE_ERR_UNSUPPORTED_SHAPE


def test_forward_int8_arguments(moe):
    c = cfg(moe)
    n = moe.moe_int8_workspace_size(c)
    lib = moe._lib.moe_forward_int8

    def call(x=P, rw=P, w=weights(moe), out=P, ws=P, wn=n, c=c):
        return lib(C.byref(c), x, rw, None, None, None, C.byref(w) if w else None, out, None, None,
                   None, None, None, None, ws, wn, None)

    for kw in (dict(x=None), dict(rw=None), dict(w=None), dict(out=None), dict(ws=None),
               dict(x=P + 2), dict(out=P + 2), dict(ws=P + 128),
               dict(w=weights(moe, ws_down_scale=None))):
        assert call(**kw) == moe.MOE_ERR_INVALID_ARG, kw
    assert call(wn=n - 1) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    fp8 = moe.MoeConfig.of(synth.config("tiny"), payload=moe.MOE_PAYLOAD_FP8)
    assert call(c=fp8) == moe.MOE_ERR_UNSUPPORTED_SHAPE


def test_python_layer_refuses_host_tensors_and_wrong_types(moe):
    c = cfg(moe)
    T, E, K = c.T, c.E, c.K
    s, idx = torch.zeros(T, E), torch.zeros(T, K, dtype=torch.int32)
    out = (torch.zeros(1, E, dtype=torch.int32), torch.zeros(1, E), torch.zeros(1))
    ws = WS(moe.moe_workspace_size(c))
    assert refused(moe, moe.moe_balance_loss, c, s, idx, None, 0.1, *out, ws) == \
        moe.MOE_ERR_INVALID_ARG
    assert refused(moe, moe.moe_balance_loss, c, s, idx, torch.zeros(0, dtype=torch.int32), 0.1,
                   *out, ws) == moe.MOE_ERR_INVALID_ARG
    assert refused(moe, moe.moe_route_backward, c, s, idx, torch.zeros(T, K), None, None, None, 0.1,
                   s.clone()) == moe.MOE_ERR_INVALID_ARG
    b = torch.zeros(T, c.d, dtype=torch.bfloat16)
    assert refused(moe, moe.moe_combine_backward, c, b, b, idx, s, b, None) == \
        moe.MOE_ERR_INVALID_ARG
    w = moe.Int8Weights(w_gate=torch.zeros(4, dtype=torch.int8))
    assert refused(moe, moe.moe_expert_ffn_int8, c, None, None, None, w, None, None, None, ws) == \
        moe.MOE_ERR_INVALID_ARG
    with pytest.raises(TypeError):
        moe.Int8Weights(w_gate=torch.zeros(4))
    with pytest.raises(TypeError):
        moe.Int8Weights(w_gate_scale=torch.zeros(4, 4).t())


def test_python_layer_refuses_weights_that_are_missing_or_of_another_type(moe):
    c = cfg(moe)
    for w in (None, {}, torch.zeros(4, dtype=torch.int8)):
        assert refused(moe, moe.moe_quantize_weights_int8, c, P, P, P, P, P, P, w, 0) == \
            moe.MOE_ERR_INVALID_ARG
        assert refused(moe, moe.moe_expert_ffn_int8, c, P, P, P, w, P, P, P, None, 0) == \
            moe.MOE_ERR_INVALID_ARG
        assert refused(moe, moe.moe_forward_int8, c, P, P, None, None, w, P, None, None, None, None,
                       None, None, None, 0) == moe.MOE_ERR_INVALID_ARG
