"""The gated experts' fused entry points and the 8-bit checkpoints refuse bad
arguments on the host, before anything is enqueued (no GPU needed)."""
import ctypes as C

import pytest
import torch

import unpermute_count_expert_amd as moe

P = [C.c_void_p(0x10000000 * (i + 1)) for i in range(14)]   # far apart, never dereferenced
ODD = C.c_void_p(0x10000008)
OK, ARG, SHAPE = 0, 1, 2


def L():
    return moe.load()


def inside(p, by):
    return C.c_void_p(p.value + by)


def fwd(a=P[0], w=P[1], off=P[2], cnt=P[3], El=4, cap=64, n=64, k=64, act=P[4], h=None, hs=None):
    return L().moe_grouped_gemm_bf16_silu_mul(a, w, off, cnt, El, cap, n, k, 0, act, h, hs, None)


def bwd(a=P[0], w=P[1], off=P[2], cnt=P[3], El=4, cap=64, n=64, k=64, h=P[5], hs=None, rw=None, dh=P[4], act=None,
        dots=None):
    return L().moe_grouped_gemm_bf16_dgrad_silu_mul(a, w, off, cnt, El, cap, k, n, 0, h, hs, rw, dh, act, dots, None)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("kw,status", [
    (dict(El=0), SHAPE), (dict(El=1025), SHAPE), (dict(cap=-1), SHAPE), (dict(cap=1 << 31), SHAPE),
    (dict(n=0), SHAPE), (dict(n=12), SHAPE), (dict(n=32776), SHAPE), (dict(k=-8), SHAPE), (dict(k=100), SHAPE),
    (dict(k=65544), SHAPE), (dict(off=None), ARG), (dict(cnt=None), ARG), (dict(off=ODD), ARG), (dict(cnt=ODD), ARG),
    (dict(a=None), ARG), (dict(a=ODD), ARG), (dict(w=None), ARG), (dict(w=ODD), ARG),
    (dict(h=P[5], hs=P[6], n=40), SHAPE), (dict(h=None, hs=P[6]), ARG), (dict(h=P[5], hs=ODD), ARG),
    (dict(h=ODD), ARG)])
def test_gated_products_refuse(call, kw, status):
    assert call(**kw) == status
    assert L().moe_last_error()


def test_gated_products_refuse_overlap():
    b = 64 * 64 * 2   # act, and the rows
    for o in (P[0], P[1], P[2], P[3], inside(P[0], b - 16), inside(P[1], 4 * 2 * b - 16), None, ODD):
        assert fwd(act=o) == ARG
    for o in (P[0], P[1], P[4], inside(P[4], b - 16)):
        assert fwd(h=o) == ARG
    assert fwd(h=P[5], hs=P[5]) == ARG and fwd(h=P[5], hs=P[4]) == ARG and fwd(h=P[5], hs=inside(P[0], 16)) == ARG
    for o in (P[0], P[1], P[2], P[3], inside(P[1], 4 * b - 16), inside(P[5], 16), None, ODD):
        assert bwd(dh=o) == ARG
    assert bwd(hs=P[6], dh=P[5]) == ARG and bwd(hs=P[6], dh=P[6]) == ARG   # in place: bf16 only
    assert bwd(h=None) == ARG
    for name in ("act", "dots"):
        for o in (P[0], P[1], P[2], P[4], P[5], inside(P[4], 2 * b - 16), ODD):
            assert bwd(**{name: o}) == ARG
    assert bwd(act=P[7], dots=P[7]) == ARG
    assert bwd(rw=ODD) == ARG and bwd(rw=P[4]) == ARG and bwd(rw=P[7], dots=P[7]) == ARG
    assert bwd(act=P[5], dh=P[5]) == ARG                                   # act in the in-place rows


def test_gated_products_without_rows_do_nothing():
    assert fwd(cap=0, a=None, w=None, act=None) == OK
    assert bwd(cap=0, a=None, w=None, h=None, dh=None) == OK


def ckpt(x=P[0], rows=8, width=64, q=P[1], s=P[2]):
    return L().moe_checkpoint(x, rows, width, q, s, None)


def restore(q=P[0], s=P[1], M=8, width=64, inv=P[2], topk=2, out=P[3], rows=16):
    return L().moe_checkpoint_restore(q, s, M, width, inv, topk, out, rows, None)


def rows(x=P[0], inv=P[1], tw=None, M=8, K=64, topk=2, out=P[2], n=16, rw=None):
    return L().moe_permute_rows(x, inv, tw, M, K, topk, out, n, rw, None)


def dots(d=P[0], nd=3, n=16, inv=P[1], M=8, topk=2, dw=P[2]):
    return L().moe_topk_weights_bwd(d, nd, n, inv, M, topk, dw, None)


@pytest.mark.parametrize("call,kw,status", [
    (ckpt, dict(rows=-1), SHAPE), (ckpt, dict(rows=1 << 31), SHAPE), (ckpt, dict(width=0), SHAPE),
    (ckpt, dict(width=48), SHAPE), (ckpt, dict(width=65568), SHAPE), (ckpt, dict(x=None), ARG), (ckpt, dict(x=ODD), ARG),
    (ckpt, dict(q=None), ARG), (ckpt, dict(s=None), ARG), (ckpt, dict(s=ODD), ARG), (ckpt, dict(q=P[0]), ARG),
    (ckpt, dict(s=P[0]), ARG), (ckpt, dict(s=P[1]), ARG), (ckpt, dict(q=inside(P[0], 1008)), ARG),
    (restore, dict(M=-1), SHAPE), (restore, dict(rows=-1), SHAPE), (restore, dict(rows=1 << 31), SHAPE),
    (restore, dict(width=48), SHAPE), (restore, dict(topk=0), SHAPE), (restore, dict(topk=257), SHAPE),
    (restore, dict(M=1 << 30), SHAPE), (restore, dict(q=None), ARG), (restore, dict(s=None), ARG),
    (restore, dict(inv=ODD), ARG), (restore, dict(out=None), ARG), (restore, dict(out=P[0]), ARG),
    (restore, dict(out=P[1]), ARG), (restore, dict(out=P[2]), ARG),
    (rows, dict(M=-1), SHAPE), (rows, dict(n=1 << 31), SHAPE), (rows, dict(K=12), SHAPE), (rows, dict(K=65544), SHAPE),
    (rows, dict(topk=0), SHAPE), (rows, dict(topk=257), SHAPE), (rows, dict(M=1 << 30), SHAPE), (rows, dict(x=None), ARG),
    (rows, dict(inv=None), ARG), (rows, dict(out=None), ARG), (rows, dict(out=P[0]), ARG), (rows, dict(out=P[1]), ARG),
    (rows, dict(tw=P[3]), ARG), (rows, dict(rw=P[3]), ARG), (rows, dict(tw=P[3], rw=P[3]), ARG),
    (rows, dict(tw=P[3], rw=P[2]), ARG), (rows, dict(tw=P[3], rw=ODD), ARG), (rows, dict(tw=P[2], rw=P[3]), ARG),
    (dots, dict(nd=0), SHAPE), (dots, dict(nd=1025), SHAPE), (dots, dict(n=-1), SHAPE), (dots, dict(M=1 << 30), SHAPE),
    (dots, dict(topk=0), SHAPE), (dots, dict(d=None), ARG), (dots, dict(inv=None), ARG), (dots, dict(dw=None), ARG),
    (dots, dict(dw=P[0]), ARG), (dots, dict(dw=P[1]), ARG), (dots, dict(dw=ODD), ARG)])
def test_rows_refuse(call, kw, status):
    assert call(**kw) == status
    assert L().moe_last_error()


def test_rows_without_work_do_nothing():
    assert ckpt(rows=0, x=None, q=None, s=None) == OK
    assert restore(M=0, q=None, s=None, out=None) == OK and restore(rows=0, out=None) == OK
    assert rows(M=0, x=None, inv=None, out=None) == OK and rows(n=0, out=None) == OK
    assert dots(M=0, inv=None, dw=None) == OK


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def u(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def f(*shape):
    return torch.zeros(shape)


def test_binding_checks():
    a, w13, w2, o, c, act, h = t(16, 64), t(2, 64, 64), t(2, 64, 32), i(3), i(2), t(16, 32), t(16, 64)
    up, down = moe.moe_grouped_gemm_bf16_silu_mul, moe.moe_grouped_gemm_bf16_dgrad_silu_mul
    for fits in (lambda: up(a, w13, o, c, act), lambda: up(a, w13, o, c, act, h), lambda: up(a, w13, o, c, act, u(16, 64), u(16, 2)),
                 lambda: down(a, w2, o, c, h, t(16, 64)),
                 lambda: down(a, w2, o, c, u(16, 64), t(16, 64), act, u(16, 2), f(16), f(16, 1)),
                 lambda: moe.moe_checkpoint(a, u(16, 64), u(16, 2)),
                 lambda: moe.moe_checkpoint_restore(u(16, 64), u(16, 2), a),
                 lambda: moe.moe_permute_rows(a, i(16, 2), t(40, 64), f(16, 2), f(40)),
                 lambda: moe.moe_topk_weights_bwd(f(40, 3), i(16, 2), f(16, 2))):
        with pytest.raises(ValueError, match="current CUDA device|needs tensors on"):
            fits()                                                     # everything fits, but on the CPU
    for bad, err in ((lambda: up(a, t(2, 63, 64), o, c, act), ValueError), (lambda: up(a, w13, o, c, h), ValueError),
                     (lambda: up(a, w13, o, c, act, u(16, 64)), TypeError),              # codes without scales
                     (lambda: up(a, w13, o, c, act, h, u(16, 2)), TypeError),            # scales for bf16
                     (lambda: up(a, w13, o, c, act, u(16, 64), u(16, 1)), ValueError),
                     (lambda: up(a, w13, o, c, act, None, u(16, 2)), ValueError),
                     (lambda: up(a.t(), w13, o, c, act), ValueError),
                     (lambda: down(a, w2, o, c, None, h), ValueError), (lambda: down(a, w2, o, c, h, act), ValueError),
                     (lambda: down(a, w2, o, c, h, t(16, 64), row_weights=f(15)), ValueError),
                     (lambda: down(a, w2, o, c, h, t(16, 64), dots=f(16, 2)), ValueError),
                     (lambda: down(a, w2, o, c, h, t(16, 64), dots=t(16, 1)), TypeError),
                     (lambda: moe.moe_checkpoint(t(16, 48), u(16, 48), u(16, 2)), ValueError),
                     (lambda: moe.moe_checkpoint(f(16, 64), u(16, 64), u(16, 2)), TypeError),
                     (lambda: moe.moe_checkpoint_restore(u(16, 64), u(16, 2), t(15, 64)), ValueError),
                     (lambda: moe.moe_checkpoint_restore(u(16, 64), u(16, 2), a, i(15, 2)), ValueError),
                     (lambda: moe.moe_permute_rows(a, i(16, 2), t(40, 32)), ValueError),
                     (lambda: moe.moe_permute_rows(a, i(16, 2), t(40, 64), f(16, 3), f(40)), ValueError),
                     (lambda: moe.moe_topk_weights_bwd(f(40, 3), i(16, 2), f(16, 3)), ValueError)):
        with pytest.raises(err):
            bad()


def test_layer_checks_its_checkpoint():
    with pytest.raises(ValueError, match="checkpoint"):
        moe.MoeTrainLayer(t(2, 256, 128), t(2, 128, 128), 2, checkpoint="fp8")
    for kept in (None, "bf16", "e4m3"):
        layer = moe.MoeTrainLayer(t(2, 256, 128), t(2, 128, 128), 2, checkpoint=kept)
        for call in (layer.forward, layer.infer):
            with pytest.raises(TypeError):
                call(t(4, 128), torch.zeros(4, 2, dtype=torch.int64), f(4, 2))
            with pytest.raises(ValueError, match="CUDA"):
                call(t(4, 128), i(4, 2), f(4, 2))
