"""The bf16 experts' entry points refuse bad arguments on the host, before
anything is enqueued (no GPU needed)."""
import ctypes as C

import pytest
import torch

import unpermute_count_expert_amd as moe
from unpermute_count_expert_amd import _lib

P = [C.c_void_p(0x10000000 * (i + 1)) for i in range(8)]   # far apart, never dereferenced
ODD = C.c_void_p(0x10000008)
OK, ARG, SHAPE, SMALL = 0, 1, 2, 3


def L():
    return moe.load()


def fwd(a=P[0], w=P[1], off=P[2], cnt=P[3], El=4, cap=64, n=64, k=64, out=P[4]):
    return L().moe_grouped_gemm_bf16(a, w, off, cnt, El, cap, n, k, 0, out, None)


def dgrad(a=P[0], w=P[1], off=P[2], cnt=P[3], El=4, cap=64, n=64, k=64, out=P[4]):
    return L().moe_grouped_gemm_bf16_dgrad(a, w, off, cnt, El, cap, n, k, 0, out, None)


def wgrad(a=P[0], w=P[1], off=P[2], cnt=P[3], El=4, cap=64, n=64, k=64, out=P[4], dt=1, acc=0):
    return L().moe_grouped_gemm_bf16_wgrad(a, w, off, cnt, El, cap, n, k, 0, dt, acc, out, None)


@pytest.mark.parametrize("call", [fwd, dgrad, wgrad])
@pytest.mark.parametrize("kw,status", [
    (dict(El=0), SHAPE), (dict(El=1025), SHAPE), (dict(cap=-1), SHAPE), (dict(cap=1 << 31), SHAPE),
    (dict(n=0), SHAPE), (dict(n=12), SHAPE), (dict(n=65544), SHAPE), (dict(k=-8), SHAPE), (dict(k=100), SHAPE),
    (dict(k=65544), SHAPE), (dict(off=None), ARG), (dict(cnt=None), ARG), (dict(off=ODD), ARG), (dict(cnt=ODD), ARG),
    (dict(a=None), ARG), (dict(a=ODD), ARG), (dict(w=None), ARG), (dict(w=ODD), ARG), (dict(out=None), ARG),
    (dict(out=ODD), ARG), (dict(out=P[0]), ARG), (dict(out=P[1]), ARG),
    (dict(out=C.c_void_p(0x10000000 + 64 * 64 * 2 - 16)), ARG),
])
def test_products_refuse(call, kw, status):
    assert call(**kw) == status
    assert L().moe_last_error()


def test_products_without_rows_do_nothing():
    assert fwd(cap=0, a=None, w=None, out=None) == OK
    assert dgrad(cap=0, a=None, w=None, out=None) == OK


@pytest.mark.parametrize("kw", [dict(dt=2), dict(dt=-1), dict(acc=2), dict(acc=-1), dict(dt=0, acc=1)])
def test_wgrad_refuses_types(kw):
    assert wgrad(**kw) == ARG


def silu(h=P[0], rows=8, n=64, off=None, cnt=None, El=0, act=P[1]):
    return L().moe_silu_mul(h, rows, n, off, cnt, El, act, None)


def silu_bwd(h=P[0], d=P[1], rows=8, n=64, off=None, cnt=None, El=0, dh=P[2]):
    return L().moe_silu_mul_bwd(h, d, rows, n, off, cnt, El, dh, None)


@pytest.mark.parametrize("call", [silu, silu_bwd])
@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(n=0), SHAPE), (dict(n=4), SHAPE), (dict(n=65544), SHAPE),
    (dict(off=P[5]), ARG), (dict(cnt=P[5]), ARG), (dict(off=P[5], cnt=P[6], El=0), SHAPE),
    (dict(off=ODD, cnt=P[6], El=2), ARG), (dict(h=None), ARG), (dict(h=ODD), ARG)])
def test_silu_refuses(call, kw, status):
    assert call(**kw) == status


def test_silu_refuses_overlap():
    assert silu(act=P[0]) == ARG
    assert silu_bwd(dh=C.c_void_p(0x10000010)) == ARG     # part of h, but not h
    assert silu_bwd(dh=P[1]) == ARG
    assert silu_bwd(d=None) == ARG and silu_bwd(dh=None) == ARG
    assert silu(rows=0, h=None, act=None) == OK and silu_bwd(rows=0, h=None, d=None, dh=None) == OK


def unp(dout=P[0], y=P[1], rows=16, inv=P[2], tw=P[3], M=4, K=128, topk=2, dy=P[4], dw=P[5]):
    return L().moe_unpermute_weight_reduce_bwd(dout, y, rows, inv, tw, M, K, topk, dy, dw, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(K=64), SHAPE), (dict(K=0), SHAPE),
    (dict(topk=0), SHAPE), (dict(topk=257), SHAPE), (dict(M=1 << 31), SHAPE), (dict(dout=None), ARG),
    (dict(y=None), ARG), (dict(inv=None), ARG), (dict(tw=None), ARG), (dict(dy=None), ARG), (dict(dw=None), ARG),
    (dict(dy=P[1]), ARG), (dict(dy=P[0]), ARG), (dict(dy=ODD), ARG), (dict(K=65664), SHAPE), (dict(dw=P[3]), ARG),
    (dict(dw=P[2]), ARG), (dict(dw=P[0]), ARG), (dict(dw=P[1]), ARG), (dict(dw=P[4]), ARG), (dict(dy=P[3]), ARG),
    (dict(dy=P[2]), ARG)])
def test_unpermute_bwd_refuses(kw, status):
    assert unp(**kw) == status


def perm(x=P[0], ids=P[1], M=10, K=256, topk=2, emap=None, Eg=8, El=8, align=128, cap=None, a=P[2], cnt=P[3], off=P[4],
         inv=P[5], src=P[6], ws=P[7], wsb=1 << 20):
    cap = moe.moe_max_rows(10, 2, 8, 128) if cap is None else cap
    return L().moe_permute_bf16(x, ids, M, K, topk, emap, Eg, El, align, cap, a, cnt, off, inv, src, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(K=192), SHAPE), (dict(K=65664), SHAPE), (dict(topk=0), SHAPE), (dict(El=9), SHAPE),
    (dict(align=8), SHAPE), (dict(cap=5), SMALL), (dict(wsb=0), SMALL), (dict(x=None), ARG), (dict(ids=None), ARG),
    (dict(a=None), ARG), (dict(a=ODD), ARG), (dict(a=P[0]), ARG), (dict(inv=None), ARG), (dict(src=None), ARG),
    (dict(cnt=None), ARG), (dict(off=None), ARG), (dict(ws=None), ARG), (dict(emap=ODD), ARG)])
def test_permute_refuses(kw, status):
    assert perm(**kw) == status


class T(C.Structure):
    _fields_ = [("grad", C.c_void_p), ("out", C.c_void_p), ("numel", C.c_int64), ("dtype", C.c_int32),
                ("reserved", C.c_int32)]


def clip(*tensors, num=None, sumsq=P[6], norm=P[7], max_norm=1.0):
    arr = (T * max(1, len(tensors)))(*[T(*t) for t in tensors])
    return L().moe_grad_clip(arr, len(tensors) if num is None else num, sumsq, max_norm, norm, None)


def sumsq(*tensors, num=None, out=P[6], ws=P[7], wsb=1 << 20):
    arr = (T * max(1, len(tensors)))(*[T(*t) for t in tensors])
    return L().moe_grad_sumsq(arr, len(tensors) if num is None else num, out, ws, wsb, None)


G = 0x20000000


def test_grad_lists_refuse():
    good = (G, G, 100, 1, 0)
    for call in (clip, sumsq):
        assert call(good, num=-1) == SHAPE
        assert call((G, G, -1, 1, 0)) == SHAPE and call((G, G, 1 << 41, 1, 0)) == SHAPE
        assert call((G, G, 100, 2, 0)) == ARG and call((G, G, 100, 1, 1)) == ARG
        assert call((None, G, 100, 1, 0)) == ARG and call((G + 2, G, 100, 1, 0)) == ARG
        assert call((G + 1, G, 100, 0, 0)) == ARG
    assert clip(good, max_norm=-1.0) == ARG and clip(good, max_norm=float("nan")) == ARG
    assert clip(good, sumsq=None) == ARG and clip(good, norm=ODD) == ARG
    assert clip((G, None, 100, 1, 0)) == ARG and clip((G, G + 2, 100, 1, 0)) == ARG
    assert sumsq(good, out=None) == ARG and sumsq(good, ws=None) == ARG and sumsq(good, wsb=8) == SMALL
    assert L().moe_grad_clip(None, 1, P[6], 1.0, None, None) == ARG


def test_clip_refuses_overlapping_memory():
    assert clip((G, G + 4, 100, 1, 0)) == ARG                               # out overlaps its own grad
    assert clip((G, G, 100, 1, 0), (G, G, 100, 1, 0)) == ARG                # one tensor twice, in place
    assert clip((G, 2 * G, 100, 1, 0), (3 * G, 2 * G + 396, 9, 1, 0)) == ARG   # two outs
    assert clip((G, 2 * G, 100, 1, 0), (2 * G + 396, 3 * G, 9, 1, 0)) == ARG   # an out over another's grad
    assert clip((2 * G + 40, 3 * G, 9, 1, 0), (G, 2 * G, 100, 1, 0)) == ARG    # inside, listed first
    assert clip((G, 2 * G, 100, 1, 0), norm=P[6]) == ARG                       # the norm over the sum
    assert clip((G, 2 * G, 100, 1, 0), sumsq=C.c_void_p(2 * G + 16)) == ARG    # an out over the sum
    assert clip((G, G, 100, 1, 0), norm=C.c_void_p(G + 16)) == ARG             # the norm in a tensor


def test_sumsq_refuses_to_write_over_a_gradient():
    need = moe.moe_grad_workspace_size(1)
    at = lambda p: C.c_void_p(p)
    inside = (G, None, 100, 1, 0)   # 400 bytes
    assert sumsq(inside, out=at(G)) == ARG and sumsq(inside, out=at(G + 384)) == ARG
    assert sumsq((G + 4, None, 1, 1, 0), out=at(G)) == ARG                       # the double's second half
    assert sumsq(inside, ws=at(G)) == ARG and sumsq(inside, ws=at(G + 384)) == ARG
    assert sumsq(inside, ws=at(G - need + 16)) == ARG                            # the workspace's last bytes
    assert sumsq((3 * G, None, 5, 0, 0), inside, ws=at(G - need + 16)) == ARG    # any tensor of the list


def test_workspace_size():
    assert moe.moe_grad_workspace_size(0) == moe.moe_grad_workspace_size(1) > 0
    assert moe.moe_grad_workspace_size(1000) > moe.moe_grad_workspace_size(100)
    with pytest.raises(moe.MoeError):
        moe.moe_grad_workspace_size(-1)


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_checks_dtype_shape_and_layout():
    ok = dict(a=t(16, 64), w=t(2, 8, 64), o=i(3), c=i(2), out=t(16, 8))
    call = lambda **kw: (lambda d: moe.moe_grouped_gemm_bf16(d["a"], d["w"], d["o"], d["c"], d["out"]))({**ok, **kw})
    with pytest.raises(ValueError, match="current CUDA device|needs tensors on"):
        call()                                                       # everything fits, but on the CPU
    for kw, err in ((dict(a=t(16, 64, dtype=torch.float32)), TypeError), (dict(a=t(16, 32)), ValueError),
                    (dict(w=t(2, 8, 64).transpose(1, 2)), ValueError), (dict(o=i(2)), ValueError),
                    (dict(c=torch.zeros(2, dtype=torch.int64)), TypeError), (dict(out=t(15, 8)), ValueError)):
        with pytest.raises(err):
            call(**kw)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm_bf16_dgrad(t(16, 9), ok["w"], ok["o"], ok["c"], t(16, 64))
    with pytest.raises(TypeError):
        moe.moe_grouped_gemm_bf16_wgrad(t(16, 8), ok["a"], ok["o"], ok["c"], t(2, 8, 64, dtype=torch.float64))
    with pytest.raises(ValueError):
        moe.moe_silu_mul(t(4, 32), 8, t(4, 8))
    with pytest.raises(ValueError):
        moe.moe_silu_mul_bwd(t(4, 16), t(4, 9), 8, t(4, 16))
    with pytest.raises(ValueError):
        moe.moe_unpermute_weight_reduce_bwd(t(4, 128), t(9, 128), i(4, 2), torch.zeros(4, 3), t(9, 128), torch.zeros(4, 2))
    with pytest.raises(TypeError):
        moe.moe_grad_sumsq([t(3, dtype=torch.float64)], torch.zeros(1, dtype=torch.float64), torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError):
        moe.moe_grad_sumsq([t(4, 4).t()[1:]], torch.zeros(1, dtype=torch.float64), torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError):
        moe.moe_grad_clip([t(3)], [t(3), t(3)], torch.zeros(1, dtype=torch.float64), 1.0)


def test_train_layer_checks_weights():
    with pytest.raises(TypeError):
        moe.MoeTrainLayer(t(2, 256, 128, dtype=torch.float32), t(2, 128, 128), 2)
    with pytest.raises(ValueError):
        moe.MoeTrainLayer(t(2, 200, 128), t(2, 128, 100), 2)
    with pytest.raises(ValueError):
        moe.MoeTrainLayer(t(2, 256, 128), t(2, 128, 256), 2)
    layer = moe.MoeTrainLayer(t(2, 256, 128), t(2, 128, 128), 2)
    with pytest.raises(TypeError):
        layer.forward(t(4, 128), torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        layer.forward(t(4, 128), i(4, 2), torch.zeros(4, 2))
