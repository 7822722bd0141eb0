"""The bf16 experts' operators on the GPU against plain 64-bit implementations.

Tolerances, derived before the first run.  A sum of C products of bf16 values
(each product exact in fp32) accumulated in fp32 in any order is off by at
most C * 2^-23 * T, T the sum of the products' magnitudes (2^-24 a step for
rounding to nearest, 2^-23 should the matrix unit truncate); rounding the
result to bf16 adds 2^-8 relative (2^-24 for fp32).  Both bounds are added.
"""
import ctypes as C

import numpy as np
import pytest
import torch

import unpermute_count_expert_amd as moe
from tests.gpu_helpers import announce

DEV = "cuda:0"
BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
EPS = {BF: 2.0 ** -8, F32: 2.0 ** -24}
TINY = 2.0 ** -133   # half the smallest bf16 denormal's spacing


def gen(seed):
    return torch.Generator().manual_seed(seed)


def bf(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(BF)


def segments(counts, align, cap_extra=5):
    off = [0]
    for c in counts:
        off.append(off[-1] + -(-c // align) * align)
    return off, off[-1] + cap_extra


def valid_mask(counts, off, cap):
    m = torch.zeros(cap, dtype=torch.bool)
    for e, c in enumerate(counts):
        m[off[e]:off[e] + c] = True
    return m


def poison(t, mask):
    t = t.clone()
    t[~mask] = float("nan")
    return t


def close(got, ref, mag, terms, what=""):
    got = got.double().cpu()
    tol = EPS[BF if what.endswith("bf16") else F32] * ref.abs() + terms * 2.0 ** -23 * mag + TINY
    bad = ~((got - ref).abs() <= tol * (1 + 2.0 ** -7))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off; worst " \
                          f"{float(((got - ref).abs() / tol).nan_to_num(1e30).max()):.3g} tolerances"


def i32(v):
    return torch.tensor(v, dtype=I32, device=DEV)


SENT = 0x7b7b   # a bf16 bit pattern that no result here has


def sentinel(shape):
    return torch.full(shape, SENT, dtype=torch.int16, device=DEV).view(BF)


def untouched(t, mask):
    return bool((t.cpu().view(torch.int16)[~mask] == SENT).all())


COUNTS = {
    "none": [0, 0, 0],
    "one": [0, 1, 0, 0],
    "few": [1, 0, 3, 16, 2, 0, 17],
    "ragged": [63, 0, 65, 1, 130, 128, 15],
    "long": [300, 0, 257, 7],
    "single_expert": [200],
}


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("n,k", [(8, 8), (64, 128), (40, 136), (264, 1000), (520, 72), (1000, 264)])
@pytest.mark.parametrize("hint", [1, 0, 1 << 20])
def test_products(counts, n, k, hint):
    announce("products", counts, n, k, hint)
    cs = COUNTS[counts]
    E = len(cs)
    off, cap = segments(cs, 16)
    mask = valid_mask(cs, off, cap)
    g = gen(n * 7 + k + len(cs))
    a, dy, w = bf((cap, k), g), bf((cap, n), g, 0.1), bf((E, n, k), g, 0.05)
    A, D, W = (poison(a, mask).to(DEV), poison(dy, mask).to(DEV), w.to(DEV))
    O, Cn = i32(off), i32(cs)
    out, dx = sentinel((cap, n)), sentinel((cap, k))
    dwf = torch.full((E, n, k), 3.25, device=DEV)
    dwb = sentinel((E, n, k))
    moe.moe_grouped_gemm_bf16(A, W, O, Cn, out, hint)
    moe.moe_grouped_gemm_bf16_dgrad(D, W, O, Cn, dx, hint)
    moe.moe_grouped_gemm_bf16_wgrad(D, A, O, Cn, dwf, 0, hint)
    moe.moe_grouped_gemm_bf16_wgrad(D, A, O, Cn, dwb, 0, hint)
    acc = torch.full((E, n, k), 3.25, device=DEV)
    moe.moe_grouped_gemm_bf16_wgrad(D, A, O, Cn, acc, 1, hint)
    torch.cuda.synchronize()
    assert untouched(out, mask) and untouched(dx, mask)
    for e, c in enumerate(cs):
        r = slice(off[e], off[e] + c)
        ae, de, we = a[r].double(), dy[r].double(), w[e].double()
        close(out[r], ae @ we.T, ae.abs() @ we.abs().T, k, "out bf16")
        close(dx[r], de @ we, de.abs() @ we.abs(), n, "dx bf16")
        ref, mag = de.T @ ae, de.abs().T @ ae.abs()
        close(dwf[e], ref, mag, c, "dw f32")
        close(dwb[e], ref, mag, c, "dw bf16")
        close(acc[e], ref + 3.25, mag + 3.25, c + 1, "dw accumulated f32")


def run_products(a, dy, w, off, cs, hint=0):
    cap, k = a.shape
    E, n, _ = w.shape
    O, Cn = i32(off), i32(cs)
    out, dx = sentinel((cap, n)), sentinel((cap, k))
    dw = torch.empty((E, n, k), device=DEV)
    A, D, W = a.to(DEV), dy.to(DEV), w.to(DEV)
    moe.moe_grouped_gemm_bf16(A, W, O, Cn, out, hint)
    moe.moe_grouped_gemm_bf16_dgrad(D, W, O, Cn, dx, hint)
    moe.moe_grouped_gemm_bf16_wgrad(D, A, O, Cn, dw, 0, hint)
    torch.cuda.synchronize()
    return out.cpu(), dx.cpu(), dw.cpu()


def test_products_inconsistent_segments_are_cut():
    """A count past its slot is cut at the next segment and at the buffer; a negative one is empty."""
    off, cap = [0, 16, 32, 40], 44
    g = gen(5)
    a, dy, w = bf((cap, 64), g), bf((cap, 40), g), bf((3, 40, 64), g)
    for hint in (1, 1 << 20):
        got = run_products(a, dy, w, off, [100, -3, 900], hint)
        want = run_products(a, dy, w, off, [16, 0, 8], hint)
        for x, y in zip(got, want):
            assert torch.equal(x.view(torch.int16 if x.dtype == BF else I32), y.view(torch.int16 if y.dtype == BF else I32))
        # offsets past the buffer and out of order: in bounds, no valid row beyond the buffer
        run_products(a, dy, w, [0, 500, 20, 44], [4, 9, 30], hint)
        run_products(a, dy, w, [-7, 44, 44, 10], [50, 9, 30], hint)


@pytest.mark.parametrize("hint", [1, 1 << 20])
def test_products_non_finite_values_stay_in_their_rows(hint):
    """Infinities and NaN of one expert's rows or weights reach only the outputs that contain them."""
    cs, n, k = [20, 3, 40], 72, 104
    off, cap = segments(cs, 16)
    g = gen(6)
    a, dy, w = bf((cap, k), g), bf((cap, n), g), bf((3, n, k), g)
    base = run_products(a, dy, w, off, cs, hint)
    a2, dy2 = a.clone(), dy.clone()
    a2[off[1] + 1, 5] = float("inf")
    dy2[off[1] + 2, 7] = float("nan")
    out, dx, dw = run_products(a2, dy2, w, off, cs, hint)
    rows = torch.ones(cap, dtype=torch.bool)
    rows[off[1] + 1] = False
    assert torch.equal(out.view(torch.int16)[rows], base[0].view(torch.int16)[rows])
    assert not torch.isfinite(out[off[1] + 1].float()).any()
    rows = torch.ones(cap, dtype=torch.bool)
    rows[off[1] + 2] = False
    assert torch.equal(dx.view(torch.int16)[rows], base[1].view(torch.int16)[rows])
    assert torch.isnan(dx[off[1] + 2].float()).all()
    assert torch.equal(dw[[0, 2]], base[2][[0, 2]])
    ref = dy2[off[1]:off[1] + 3].double().T @ a2[off[1]:off[1] + 3].double()
    assert torch.equal(torch.isfinite(dw[1]), torch.isfinite(ref))


def test_products_many_experts():
    """1024 experts, most without rows."""
    g = gen(7)
    cs = [0] * 1024
    for e, c in ((0, 2), (1, 1), (511, 40), (777, 5), (1023, 3)):
        cs[e] = c
    off, cap = segments(cs, 16, 0)
    a, dy, w = bf((cap, 32), g), bf((cap, 16), g), bf((1024, 16, 32), g)
    for hint in (1, 1 << 24):
        out, dx, dw = run_products(a, dy, w, off, cs, hint)
        for e in (0, 1, 2, 511, 777, 1023):
            r = slice(off[e], off[e] + cs[e])
            ae, de, we = a[r].double(), dy[r].double(), w[e].double()
            close(out[r], ae @ we.T, ae.abs() @ we.abs().T, 32, "out bf16")
            close(dx[r], de @ we, de.abs() @ we.abs(), 16, "dx bf16")
            close(dw[e], de.T @ ae, de.abs().T @ ae.abs(), cs[e], "dw f32")


def test_products_match_differences():
    """The products are linear: moving the rows (weights) by an exactly representable step moves <out, dy> by the
    step's inner product with dx (dw), here in integers, where every rounding is exact."""
    g = gen(8)
    cs = [5, 0, 18]
    off, cap = segments(cs, 16)
    mask = valid_mask(cs, off, cap)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g).to(BF)
    a, dy, w, da, dw_ = ints(cap, 24), ints(cap, 16), ints(3, 16, 24), ints(cap, 24), ints(3, 16, 24)
    f = lambda aa, ww: (run_products(aa, dy, ww, off, cs)[0].double()[mask] * dy.double()[mask]).sum()
    _, dx, dw = run_products(a, dy, w, off, cs)
    assert f(a + da, w) - f(a - da, w) == 2 * (dx.double()[mask] * da.double()[mask]).sum()
    assert f(a, w + dw_) - f(a, w - dw_) == 2 * (dw.double() * dw_.double()).sum()


# ---- permute -----------------------------------------------------------------------
@pytest.mark.parametrize("M,topk,Eg,El,align,K", [
    (1, 1, 4, 4, 16, 128), (7, 3, 8, 8, 32, 256), (130, 8, 128, 64, 128, 384), (1500, 4, 60, 60, 16, 128),
    (0, 2, 4, 4, 16, 128), (33, 2, 3000, 40, 64, 128)])
def test_permute_rows(M, topk, Eg, El, align, K):
    announce("permute_bf16", M, topk, Eg, El, align, K)
    g = gen(M + K)
    x = bf((M, K), g)
    ids = torch.randint(-1, Eg, (M, topk), generator=g, dtype=torch.int64).to(I32)   # the same expert twice too
    emap = None
    if El < Eg:
        emap = torch.full((Eg,), -1, dtype=I32)
        emap[torch.randperm(Eg, generator=g)[:El]] = torch.arange(El, dtype=I32)
    cap = moe.moe_max_rows(M, topk, El, align) + 3
    a = sentinel((cap, K))
    counts, off, inv = i32([9] * El), i32([9] * (El + 1)), torch.empty((M, topk), dtype=I32, device=DEV)
    src = torch.empty((cap,), dtype=I32, device=DEV)
    ws = torch.empty(moe.moe_permute_workspace_size(M, topk, El), dtype=torch.uint8, device=DEV)
    moe.moe_permute_bf16(x.to(DEV), ids.to(DEV), None if emap is None else emap.to(DEV), Eg, El, align, cap, a,
                         counts, off, inv, src, ws)
    torch.cuda.synchronize()
    loc = [[(-1 if i < 0 else i if emap is None else int(emap[i])) for i in row] for row in ids.tolist()]
    want_c = [sum(l == e for row in loc for l in row) for e in range(El)]
    want_o, _ = segments(want_c, align)
    nxt, want_inv, want_src = list(want_o), [], [-1] * cap
    for t, row in enumerate(loc):
        for l in row:
            want_inv.append(nxt[l] if l >= 0 else -1)
            if l >= 0:
                want_src[nxt[l]] = t
                nxt[l] += 1
    assert counts.tolist() == want_c and off.tolist() == want_o
    assert inv.reshape(-1).tolist() == want_inv and src.tolist() == want_src
    rows = torch.tensor([s >= 0 for s in want_src])
    assert torch.equal(a.cpu()[rows], x[[s for s in want_src if s >= 0]])
    assert untouched(a, rows)


# ---- SiLU-mul ----------------------------------------------------------------------
def silu_ref(h, d):
    n = h.shape[1] // 2
    g, u = h[:, :n].double(), h[:, n:].double()
    s = 1 / (1 + torch.exp(-g))
    return g * s * u, d * u * s * (1 + g * (1 - s)), d * g * s


def test_silu_reference_matches_differences():
    g = gen(3)
    h = torch.randn(5, 12, generator=g, dtype=F64) * 3
    d = torch.randn(5, 6, generator=g, dtype=F64)
    _, dg, du = silu_ref(h, d)
    step = 1e-6
    for c in range(12):
        hp, hm = h.clone(), h.clone()
        hp[:, c] += step
        hm[:, c] -= step
        num = ((silu_ref(hp, d)[0] - silu_ref(hm, d)[0]) * d).sum(1) / (2 * step)
        ref = dg[:, c] if c < 6 else du[:, c - 6]
        assert torch.allclose(num, ref, rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("counts,n", [("none", 8), ("one", 128), ("few", 40), ("ragged", 1000), ("long", 4096),
                                      (None, 8), (None, 264)])
@pytest.mark.parametrize("in_place", [False, True])
def test_silu_mul(counts, n, in_place):
    announce("silu", counts, n, in_place)
    if counts is None:
        cap, off, cs = 37, None, None
        mask = torch.ones(cap, dtype=torch.bool)
        args = ()
    else:
        cs = COUNTS[counts]
        off, cap = segments(cs, 16)
        mask = valid_mask(cs, off, cap)
        args = (i32(off), i32(cs), len(cs))
    g = gen(n)
    h, d = bf((cap, 2 * n), g, 4.0), bf((cap, n), g)
    H, D = poison(h, mask).to(DEV), poison(d, mask).to(DEV)
    act = sentinel((cap, n))
    moe.moe_silu_mul(H, n, act, *args)
    if in_place:
        H[~mask.to(DEV)] = sentinel((1, 1))
        dh = H
    else:
        dh = sentinel((cap, 2 * n))
    moe.moe_silu_mul_bwd(H, D, n, dh, *args)
    torch.cuda.synchronize()
    assert untouched(act, mask) and untouched(dh, mask)
    ra, rg, ru = silu_ref(h[mask], d[mask].double())
    # e^-g from the hardware exp2 of -g log2(e) rounded in fp32: at most 2^-22 (2 + |g|) relative; s inherits it,
    # 1 - s is off by 2^-24 absolute on top of s's error, and each of at most five further operations adds 2^-24
    gg = h[mask][:, :n].double()
    rel = 2.0 ** -22 * (4 + gg.abs())
    for got, ref, extra in ((act[mask], ra, 0), (dh[mask][:, n:], ru, 0),
                            (dh[mask][:, :n], rg,
                             (d[mask].double() * h[mask][:, n:].double()).abs() * (1 + gg.abs()) * rel)):
        err = (got.double().cpu() - ref).abs()
        tol = (2.0 ** -8 + rel) * ref.abs() + extra + TINY
        assert (err <= tol * (1 + 2.0 ** -7)).all(), float((err / tol).max())


def test_silu_mul_extremes():
    """Large gates of either sign, zeros, infinities and NaN: as the formula in 64 bits says, where it has a value."""
    gates = [0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 87.0, -87.0, 300.0, -300.0, 1e30, -1e30, 3e38, -3e38,
             float("inf"), float("nan")]
    n = len(gates)
    h = torch.tensor([gates + [1.5] * n]).to(BF)
    d = torch.full((1, n), 0.5, dtype=BF)
    act, dh = sentinel((1, n)), sentinel((1, 2 * n))
    moe.moe_silu_mul(h.to(DEV), n, act)
    moe.moe_silu_mul_bwd(h.to(DEV), d.to(DEV), n, dh)
    act, dh = act.cpu().double()[0], dh.cpu().double()[0]
    for i, g in enumerate(h[0, :n].double().tolist()):
        if g != g:
            assert act[i].isnan() and dh[i].isnan() and dh[n + i].isnan()
            continue
        s = 1 / (1 + np.exp(-g)) if g > -700 else 0.0
        want = (g * s * 1.5, 0.5 * 1.5 * s * (1 + (g * (1 - s) if np.isfinite(g) else 0.0)), 0.5 * g * s)
        for j, (got, ref) in enumerate(zip((act[i], dh[i], dh[n + i]), want)):
            if g == float("inf") and j == 1:
                continue   # inf * 0 in the formula
            # past the largest bf16, (2 - 2^-7) 2^127, by half a step and more: infinity
            ref = float("inf") if ref >= (2 - 2.0 ** -8) * 2.0 ** 127 else ref
            # below 2^-126 the fp32 sigmoid may be flushed: |g| s is under 2^-118 there
            assert abs(got - ref) <= 2.0 ** -7 * abs(ref) + 2.0 ** -118 or got == ref, (g, float(got), ref)


# ---- weighted unpermute's gradient -----------------------------------------------------
@pytest.mark.parametrize("M,topk,K,rows", [(1, 1, 128, 4), (5, 8, 640, 60), (130, 3, 2048, 500), (3000, 2, 128, 7000),
                                           (2, 256, 256, 600), (4, 2, 128, 0)])
def test_unpermute_bwd(M, topk, K, rows):
    announce("unpermute_bwd", M, topk, K, rows)
    g = gen(M + K)
    y, dout = bf((rows, K), g), bf((M, K), g)
    tw = torch.rand((M, topk), generator=g)
    place = torch.randperm(max(rows, M * topk), generator=g)[:M * topk].reshape(M, topk).to(I32)   # some >= rows
    place[torch.rand((M, topk), generator=g) < 0.3] = -1
    place[-1] = -1   # a token with no row
    dy = sentinel((rows, K))
    dtw = torch.full((M, topk), 7.0, device=DEV)
    moe.moe_unpermute_weight_reduce_bwd(dout.to(DEV), y.to(DEV), place.to(DEV), tw.to(DEV), dy, dtw)
    torch.cuda.synchronize()
    ok = (place >= 0) & (place < rows)
    t, k = ok.nonzero(as_tuple=True)
    r = place[t, k].long()
    named = torch.zeros(rows, dtype=torch.bool)
    named[r] = True
    assert untouched(dy, named)
    yd, dd = y[r].double(), dout[t].double()
    close(dtw.cpu()[t, k], (yd * dd).sum(1), (yd * dd).abs().sum(1), K, "dweights f32")
    assert (dtw.cpu()[~ok] == 0).all()
    ref = tw[t, k, None].double() * dd
    close(dy.cpu()[r], ref, ref.abs(), 1, "dy bf16")


def test_unpermute_bwd_many_tokens():
    """More tokens (4.3 M) than one launch has waves for: each wave takes several."""
    M, K = (1 << 22) + 100_001, 128
    announce("unpermute_bwd", M, 1, K, "many tokens")
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device=DEV, dtype=torch.int8)   # exact in small integers
    y, dout, tw = ints(M, K).to(BF), ints(M, K).to(BF), ints(M, 1).float()
    inv = torch.randperm(M, generator=g, device=DEV).to(I32)[:, None]
    inv[7] = -1
    row7 = torch.ones(M, dtype=torch.bool, device=DEV).index_fill_(0, inv[inv >= 0].long(), False).nonzero()[0, 0]
    dy, dtw = torch.full((M, K), 9.0, dtype=BF, device=DEV), torch.full((M, 1), 9.0, device=DEV)
    moe.moe_unpermute_weight_reduce_bwd(dout, y, inv, tw, dy, dtw)
    torch.cuda.synchronize()
    assert (dy[row7] == 9).all() and dtw[7, 0] == 0
    dy[row7] = 0
    tw[7], inv[7, 0] = 0, row7
    want = dout * tw.to(BF)
    assert torch.equal(dy[inv[:, 0].long()], want)
    dtw[7, 0] = (y[row7].float() * dout[7].float()).sum()
    assert torch.equal(dtw[:, 0], (y[inv[:, 0].long()].float() * dout.float()).sum(1))


def test_unpermute_bwd_matches_differences():
    """out is linear in y and in the weights: exact in small integers."""
    g = gen(4)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g).float()
    M, topk, K, rows = 6, 2, 128, 12
    y, dout, tw = ints(rows, K).to(BF), ints(M, K).to(BF), ints(M, topk)
    inv = torch.randperm(rows, generator=g).reshape(M, topk).to(I32)

    def f(yy, ww):
        out = torch.empty((M, K), dtype=BF, device=DEV)
        moe.moe_unpermute_weight_reduce(yy.to(DEV), inv.to(DEV), ww.to(DEV), 0, out)
        return (out.cpu().double() * dout.double()).sum()

    dy, dtw = torch.empty((rows, K), dtype=BF, device=DEV), torch.empty((M, topk), device=DEV)
    moe.moe_unpermute_weight_reduce_bwd(dout.to(DEV), y.to(DEV), inv.to(DEV), tw.to(DEV), dy, dtw)
    sy, sw = ints(rows, K).to(BF), ints(M, topk)
    assert f(y + sy, tw) - f(y - sy, tw) == 2 * (dy.cpu().double() * sy.double()).sum()
    assert f(y, tw + sw) - f(y, tw - sw) == 2 * (dtw.cpu().double() * sw.double()).sum()


# ---- global norm and clipping ------------------------------------------------------------
def clip(grads, outs, max_norm):
    s = torch.full((1,), -1.0, dtype=F64, device=DEV)
    nrm = torch.full((1,), -1.0, device=DEV)
    ws = torch.empty(moe.moe_grad_workspace_size(len(grads)), dtype=torch.uint8, device=DEV)
    moe.moe_grad_sumsq(grads, s, ws)
    moe.moe_grad_clip(grads, outs, s, max_norm, nrm)
    torch.cuda.synchronize()
    return float(s), float(nrm)


def flat_views(sizes, skew, g, scale=1.0):
    """Tensors end to end in one buffer a type, so most start off 16-byte alignment."""
    out = []
    for i, m in enumerate(sizes):
        dt = BF if (i + skew) % 2 else F32
        buf = (torch.randn(m + skew, generator=g) * scale).to(dt).to(DEV)
        out.append(buf[skew:])
    return out


@pytest.mark.parametrize("sizes", [[1], [0, 3, 0], [5000, 0, 9], [7, 8, 9, 15, 16, 17], [4097, 1, 100000, 8191],
                                   [5] * 200, [3_000_001, 17], []])
@pytest.mark.parametrize("skew", [0, 1, 3])
@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9])
def test_clip(sizes, skew, max_norm):
    announce("clip", len(sizes), skew, max_norm)
    grads = flat_views(sizes, skew, gen(len(sizes) + skew))
    before = [t.cpu() for t in grads]
    ref = sum(float((t.double() ** 2).sum()) for t in before)
    for mode in ("same skew", "other skew", "in place"):
        if mode == "in place":
            outs = None
        else:
            sk = skew if mode == "same skew" else skew + 1
            outs = [torch.full((t.numel() + sk + 9,), 5.0, dtype=t.dtype, device=DEV)[sk:sk + t.numel()] for t in grads]
        s, nrm = clip(grads, outs, max_norm)
        # fp64 sums of exact squares: n 2^-53 relative; the norm is rounded once to fp32
        assert abs(s - ref) <= max(1, sum(sizes)) * 2.0 ** -52 * ref
        assert abs(nrm - ref ** 0.5) <= 2.0 ** -24 * ref ** 0.5 * 1.01
        c = min(1.0, max_norm / (ref ** 0.5 + 1e-6))
        for i, t in enumerate(before):
            got = (grads if outs is None else outs)[i].cpu().double()
            want = t.double() * c
            # c: the norm's rounding, the sum, the quotient and the product, 2^-24 each, then the rounding to t's type
            tol = (4 * 2.0 ** -24 + EPS[t.dtype]) * want.abs() + TINY
            assert ((got - want).abs() <= tol * (1 + 2.0 ** -7)).all()
        if outs is not None:
            for o in outs:   # nothing past the end
                end = o.storage_offset() + o.numel()
                assert (torch.as_strided(o, (9 if o.numel() else 1,), (1,), end) == 5.0).all()


def test_clip_extreme_values():
    for v in (1e30, 1e-30, 3e38):   # squares far outside fp32
        t = torch.full((1000,), v, device=DEV)
        s, nrm = clip([t], None, 1.0)
        want = float(torch.tensor(v).double()) * 1000 ** 0.5
        assert abs(s - want ** 2) <= 1e-12 * want ** 2 and (abs(nrm - want) <= 1e-6 * want or want > 3.4e38)
    t = torch.tensor([1.0, float("inf"), 2.0], device=DEV)
    _, nrm = clip([t], None, 1.0)
    assert nrm == float("inf") and t[0] == 0 and t[2] == 0 and t[1].isnan()
    t = torch.tensor([1.0, float("nan"), 2.0], device=DEV)
    _, nrm = clip([t], None, 1.0)
    assert nrm != nrm and t.isnan().all()


def test_clip_is_reproducible():
    grads = flat_views([123457, 65, 999999], 1, gen(1))
    first = clip(grads, [torch.empty_like(t) for t in grads], 0.1)
    for _ in range(3):
        assert clip(grads, [torch.empty_like(t) for t in grads], 0.1) == first


# ---- the operators together ---------------------------------------------------------------
def make_layer(seed, Eg=8, El=8, K=256, N=128):
    g = gen(seed)
    w13, w2 = bf((El, 2 * N, K), g, 0.08).to(DEV), bf((El, K, N), g, 0.08).to(DEV)
    emap = None
    if El < Eg:
        emap = torch.full((Eg,), -1, dtype=I32)
        emap[Eg - El:] = torch.arange(El, dtype=I32)
        emap = emap.to(DEV)
    return moe.MoeTrainLayer(w13, w2, Eg, emap)


def batch(seed, M, K=256, Eg=8, topk=2):
    g = gen(seed)
    x, dout = bf((M, K), g), bf((M, K), g, 0.1)
    ids = torch.stack([torch.randperm(Eg, generator=g)[:topk] for _ in range(max(M, 1))])[:M].to(I32)
    return x.to(DEV), ids.to(DEV).reshape(M, topk), torch.rand((M, topk), generator=g).to(DEV), dout.to(DEV)


def layer_ref(layer, x, ids, tw, dout):
    """The layer and its gradients in 64 bits, token by token pair, no roundings in between; with every quantity
    the sum of its terms' magnitudes, which bounds how far one relative 2^-8 in each factor moves it."""
    d = lambda t: t.detach().cpu().double()
    w13, w2, X, TW, G = d(layer.w13).requires_grad_(), d(layer.w2).requires_grad_(), d(x).requires_grad_(), \
        d(tw).requires_grad_(), d(dout)
    emap = None if layer.expert_map is None else layer.expert_map.tolist()
    N = layer.N
    out = torch.zeros(x.shape, dtype=F64)
    rows = []
    for t, picks in enumerate(ids.tolist()):
        acc = torch.zeros(x.shape[1], dtype=F64)
        for k, i in enumerate(picks):
            e = i if emap is None else emap[i]
            if e >= 0:
                h = w13[e] @ X[t]
                acc = acc + TW[t, k] * (w2[e] @ (torch.nn.functional.silu(h[:N]) * h[N:]))
        rows.append(acc)
    if rows:
        out = torch.stack(rows)
        (out * G).sum().backward()
    z = lambda t: t.grad if t.grad is not None else torch.zeros_like(t)
    return out.detach(), z(X), z(TW), z(w13), z(w2)


def rel(got, ref):
    got = got.double().cpu()
    return float((got - ref).norm() / ref.norm().clamp(min=1e-30)) if ref.numel() else 0.0


@pytest.mark.parametrize("M,Eg,El,topk", [(1, 8, 8, 2), (37, 8, 8, 2), (64, 8, 4, 3), (300, 8, 8, 1), (0, 8, 8, 2)])
def test_layer_forward_backward(M, Eg, El, topk):
    """Against the whole layer in 64 bits.  At most six bf16 roundings (2^-8 each, most far below) lie between the
    inputs and any output, and each enters linearly, so the 2-norm of the difference stays below 6 * 2^-8 of the
    result's."""
    announce("layer", M, Eg, El, topk)
    layer = make_layer(M + 1, Eg, El)
    x, ids, tw, dout = batch(M + 2, M, Eg=Eg, topk=topk)
    out, saved = layer.forward(x, ids, tw)
    dx, dtw = layer.backward(dout, saved)
    torch.cuda.synchronize()
    ref = layer_ref(layer, x, ids, tw, dout)
    for got, want, what in zip((out, dx, dtw, layer.grad_w13, layer.grad_w2), ref, ("out", "dx", "dtw", "dw13", "dw2")):
        assert got.shape == want.shape
        assert rel(got, want) <= 6 * 2.0 ** -8, (what, rel(got, want))
    # a second batch adds to the weights' gradients: the fp32 sum goes on from the first's, so by the bound above
    # (c terms and the start, magnitudes |start| + T) it is within (c + 1) 2^-23 (|start| + T) of twice the first
    before = layer.grad_w2.clone()
    dy, off, cnt = torch.zeros_like(saved.y), saved.expert_offsets.tolist(), saved.counts.tolist()
    moe.moe_unpermute_weight_reduce_bwd(dout, saved.y, saved.inv_perm, tw, dy, torch.empty_like(tw))
    layer.backward(dout, saved)
    for e, c in enumerate(cnt):
        r = slice(off[e], off[e] + c)
        mag = before[e].double().abs() + dy[r].double().abs().T.contiguous() @ saved.act[r].double().abs()
        err = (layer.grad_w2[e].double() - 2 * before[e].double()).abs()
        assert (err <= (c + 1) * 2.0 ** -23 * mag).all(), e
    # and the clip scales both to the norm asked for
    norm = float(layer.clip_gradients(0.25))
    total = float((layer.grad_w13.double() ** 2).sum() + (layer.grad_w2.double() ** 2).sum()) ** 0.5
    if M:
        assert norm > 0.25 and abs(total - 0.25) <= 0.25 * 2.0 ** -18
    else:
        assert norm == 0.0 and total == 0.0


def test_layer_interleaved_forwards():
    """Two forwards before their backwards equal one after the other, bit for bit."""
    b1, b2 = batch(1, 40), batch(2, 23)
    l1, l2 = make_layer(9), make_layer(9)
    o1, s1 = l1.forward(*b1[:3])
    o2, s2 = l1.forward(*b2[:3])
    g1, g2 = l1.backward(b1[3], s1), l1.backward(b2[3], s2)
    p1, t1 = l2.forward(*b1[:3])
    q1 = l2.backward(b1[3], t1)
    p2, t2 = l2.forward(*b2[:3])
    q2 = l2.backward(b2[3], t2)
    for a, b in ((o1, p1), (o2, p2), *zip(g1, q1), *zip(g2, q2), (l1.grad_w13, l2.grad_w13), (l1.grad_w2, l2.grad_w2)):
        assert torch.equal(a, b)


def test_layer_on_another_stream():
    layer = make_layer(3)
    x, ids, tw, dout = batch(4, 50)
    want, saved = layer.forward(x, ids, tw)
    wdx, wdt = layer.backward(dout, saved)
    ww = layer.grad_w13.clone()
    layer.zero_grad()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        out, saved = layer.forward(x, ids, tw)
        dx, dt = layer.backward(dout, saved)
    st.synchronize()
    assert torch.equal(out, want) and torch.equal(dx, wdx) and torch.equal(dt, wdt) and torch.equal(layer.grad_w13, ww)


def test_layer_in_a_graph():
    """Forward, backward and clip captured once and replayed on new inputs, eager work between the replays."""
    layer, eager = make_layer(5), make_layer(5)
    x, ids, tw, dout = batch(6, 48)

    def step(l, *b):
        l.zero_grad()
        out, s = l.forward(*b[:3])
        dx, dt = l.backward(b[3], s)
        n = l.clip_gradients(0.5)
        return out, dx, dt, n, l.grad_w13, l.grad_w2

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step(layer, x, ids, tw, dout)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(layer, x, ids, tw, dout)
    for seed in (6, 7, 8, 9):
        new = batch(seed, 48)
        for dst, src in zip((x, ids, tw, dout), new):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        want = step(eager, *new)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), seed


# ---- the products over longer walks, other layouts, and side by side ---------------------
def check_products_on_gpu(cs, n, k, off, cap, hints, seed):
    """All three products against 64-bit products on the GPU, every expert."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    a, dy, w = rn(cap, k).to(BF), (rn(cap, n) * 0.1).to(BF), (rn(len(cs), n, k) * 0.05).to(BF)
    O, Cn = i32(off), i32(cs)
    mask = valid_mask(cs, off, cap).to(DEV)
    for hint in hints:
        out, dx = sentinel((cap, n)), sentinel((cap, k))
        dwf, dwb = torch.empty((len(cs), n, k), device=DEV), torch.empty((len(cs), n, k), dtype=BF, device=DEV)
        moe.moe_grouped_gemm_bf16(a, w, O, Cn, out, hint)
        moe.moe_grouped_gemm_bf16_dgrad(dy, w, O, Cn, dx, hint)
        moe.moe_grouped_gemm_bf16_wgrad(dy, a, O, Cn, dwf, 0, hint)
        moe.moe_grouped_gemm_bf16_wgrad(dy, a, O, Cn, dwb, 0, hint)
        assert untouched(out, mask.cpu()) and untouched(dx, mask.cpu())
        for e, c in enumerate(cs):
            r = slice(off[e], off[e] + c)
            ae, de, we = a[r].double(), dy[r].double(), w[e].double()
            wt, dt = we.T.contiguous(), de.T.contiguous()
            for got, ref, mag, terms, eps in ((out[r], ae @ wt, ae.abs() @ wt.abs(), k, EPS[BF]),
                                              (dx[r], de @ we, de.abs() @ we.abs(), n, EPS[BF]),
                                              (dwf[e], dt @ ae, dt.abs() @ ae.abs(), c, EPS[F32]),
                                              (dwb[e], dt @ ae, dt.abs() @ ae.abs(), c, EPS[BF])):
                tol = (eps * ref.abs() + terms * 2.0 ** -23 * mag + TINY) * (1 + 2.0 ** -7)
                assert ((got.double() - ref).abs() <= tol).all(), (hint, e)


@pytest.mark.parametrize("cs,n,k", [
    ([5000, 0, 1, 777, 2048], 1544, 776),             # many tiles a block, experts of unlike length, odd edges
    ([257, 256, 255, 0, 1, 128, 129, 64, 65], 264, 520),
    ([40] * 60, 512, 192),                            # experts not a multiple of eight, all of one class
    ([0, 0, 900], 8, 4096)])
def test_products_long_walks(cs, n, k):
    announce("long walks", cs[:9], n, k)
    off, cap = segments(cs, 32)
    check_products_on_gpu(cs, n, k, off, cap, (1, 50 * len(cs), 1 << 20), n + k)


@pytest.mark.parametrize("n,k", [(504, 520), (504, 576), (512, 40), (520, 1032)])
def test_products_every_kernel(n, k):
    """Enough experts that the row count given picks each kernel in turn (a few rows; 128-row tiles; 256-row tiles
    with staggered and with common starts of the contraction), 256-row tiles of weight gradients, and widths whose
    gradient rows are whole 128-byte lines in both, one or neither type."""
    announce("every kernel", n, k)
    g = torch.Generator().manual_seed(n + k)
    cs = torch.randint(0, 30, (128,), generator=g).tolist()
    cs[3], cs[64], cs[127] = 0, 150, 290
    off, cap = segments(cs, 16)
    check_products_on_gpu(cs, n, k, off, cap, (1, 40 * 128, 120 * 128, 1 << 20), n + 2 * k)
    # accumulating: fp32 sums that start at what is there, in rows that start inside a line
    g = torch.Generator(device=DEV).manual_seed(7)
    rn = lambda *sh: torch.randn(sh, generator=g, device=DEV)
    a, dy, start = rn(cap, k).to(BF), (rn(cap, n) * 0.1).to(BF), rn(128, n, k)
    dw = torch.empty(128 * n * k + 4, device=DEV)[4:].view(128, n, k).copy_(start)   # 16 bytes past a line
    moe.moe_grouped_gemm_bf16_wgrad(dy, a, i32(off), i32(cs), dw, 1, 0)
    for e, c in enumerate(cs):
        r = slice(off[e], off[e] + c)
        ae, dt = a[r].double(), dy[r].double().T.contiguous()
        mag = dt.abs() @ ae.abs() + start[e].double().abs()
        err = (dw[e].double() - (dt @ ae + start[e].double())).abs()
        assert (err <= ((c + 1) * 2.0 ** -23 * mag + TINY)).all(), e


@pytest.mark.parametrize("n,k", [(65536, 8), (8, 65536), (72, 30000)])
def test_products_widest(n, k):
    announce("widest", n, k)
    cs = [3, 0, 20]
    off, cap = segments(cs, 16)
    check_products_on_gpu(cs, n, k, off, cap, (1, 1 << 20), 5)


def test_products_on_slots():
    """Slots of a fixed size, most of each unused (a batched, masked layout)."""
    cs = [0, 7, 300, 1, 64]
    check_products_on_gpu(cs, 136, 200, [i * 320 for i in range(6)], 1600, (1, 1 << 20), 6)


def test_products_side_by_side():
    """The same kernels on two streams at once, each with its own tensors."""
    g = gen(11)
    cs = [300, 20, 0, 150]
    off, cap = segments(cs, 16)
    sets = [(bf((cap, 320), g).to(DEV), bf((cap, 264), g).to(DEV), bf((4, 264, 320), g).to(DEV)) for _ in range(2)]
    O, Cn = i32(off), i32(cs)

    def run(s, hint):
        a, dy, w = s
        out, dx, dw = sentinel((cap, 264)), sentinel((cap, 320)), torch.empty((4, 264, 320), device=DEV)
        moe.moe_grouped_gemm_bf16(a, w, O, Cn, out, hint)
        moe.moe_grouped_gemm_bf16_dgrad(dy, w, O, Cn, dx, hint)
        moe.moe_grouped_gemm_bf16_wgrad(dy, a, O, Cn, dw, 0, hint)
        return out.view(torch.int16), dx.view(torch.int16), dw

    want = [[run(s, h) for h in (1, 1 << 20)] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append([run(s, h) for h in (1, 1 << 20)])
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            for p, q in zip(x, y):
                assert all(torch.equal(a, b) for a, b in zip(p, q))


def test_clip_many_tensors_in_a_graph():
    """Past one launch's list, captured once; the list is not needed after the call."""
    g = torch.Generator(device=DEV).manual_seed(2)
    grads = [torch.randn(1 + 37 * i % 5000, generator=g, device=DEV) for i in range(300)]
    outs = [torch.empty_like(t) for t in grads]
    s, nrm = torch.zeros(1, dtype=F64, device=DEV), torch.zeros(1, device=DEV)
    ws = torch.empty(moe.moe_grad_workspace_size(300), dtype=torch.uint8, device=DEV)

    def step():
        moe.moe_grad_sumsq(list(grads), s, ws)
        moe.moe_grad_clip(list(grads), list(outs), s, 1.0, nrm)

    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for scale in (1.0, 0.25, 3.0):
        for t in grads:
            t.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        ref = sum(float((t.double() ** 2).sum()) for t in grads)
        assert abs(float(s) - ref) <= 1e-12 * ref
        c = min(1.0, 1.0 / (ref ** 0.5 + 1e-6))
        for t, o in zip(grads, outs):
            want = t.double() * c
            assert ((o.double() - want).abs() <= 5 * 2.0 ** -24 * want.abs()).all()


@pytest.mark.parametrize("experts,n,k", [(5, 72, 136), (5, 72, 128), (128, 512, 40), (128, 512, 64)])
def test_wgrad_adds_its_finished_sum(experts, n, k):
    """accumulate rounds once, however many rows an expert has: the rows are small integers, so that every order of
    their sum is exact, and start + sum needs more bits than fp32 has (start: multiples of 2^-20 below 2^3; sums: up
    to some hundreds) but no more than fp64, which rounds to the one fp32 answer.  128-row and 256-row tiles, rows of
    whole 128-byte lines and not."""
    announce("wgrad accumulated", experts, n, k)
    g = torch.Generator().manual_seed(experts + n + k)
    cs = [1300, 0, 1, 64, 700] + torch.randint(0, 200, (experts - 5,), generator=g).tolist()
    off, cap = segments(cs, 16)
    mask = valid_mask(cs, off, cap)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g).to(BF)
    a, dy = ints(cap, k), ints(cap, n)
    start = (torch.randint(-2 ** 23, 2 ** 23, (experts, n, k), generator=g).double() * 2.0 ** -20).float()
    A, D, dw = poison(a, mask).to(DEV), poison(dy, mask).to(DEV), start.to(DEV)
    want, rounded = start.clone(), 0
    for _ in range(3):
        moe.moe_grouped_gemm_bf16_wgrad(D, A, i32(off), i32(cs), dw, 1, 0)
        for e, c in enumerate(cs):
            r = slice(off[e], off[e] + c)
            exact = want[e].double() + dy[r].double().T.contiguous() @ a[r].double()
            want[e] = exact.float()
            rounded += int((want[e].double() != exact).sum())
        assert torch.equal(dw.cpu(), want)
    assert rounded > n * k


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("value,max_norm", [(3e38, 1.0), (3e38, 1e30), (1e38, 1e-6), (1e30, 1.0), (1e30, 1e-30),
                                            (1e-30, 1.0), (1e-30, 1e-32), (1e20, 0.0)])
def test_clip_far_from_one(value, max_norm, dtype):
    """Norms past the largest fp32 value and factors below the smallest: finite gradients come out as the formula
    says.  The factor and the product are rounded to fp32 (2^-24 each; 2^-150 where the product is a denormal), then
    the result to its type."""
    announce("clip far from one", value, max_norm, dtype)
    sign = torch.where(torch.rand(1003, generator=gen(1)) < 0.5, -1.0, 1.0)
    before = (sign * value).to(dtype)
    norm = float((before.double() ** 2).sum()) ** 0.5
    want = before.double() * min(1.0, max_norm / (norm + 1e-6))
    for skew in (0, 1):   # the output aligned as the gradient, and not
        out = torch.full((1003 + 8,), 5.0, dtype=dtype, device=DEV)
        s, nrm = clip([before.to(DEV)], [out[skew:skew + 1003]], max_norm)
        assert abs(s - norm ** 2) <= 1e-12 * norm ** 2
        assert nrm == float("inf") if norm > 3.41e38 else abs(nrm - norm) <= 2.0 ** -23 * norm
        got = out[skew:skew + 1003].cpu().double()
        tol = (2 * 2.0 ** -24 + EPS[dtype]) * want.abs() + 2.0 ** -149 + (TINY if dtype == BF else 0)
        assert ((got - want).abs() <= tol * (1 + 2.0 ** -7)).all(), (skew, got[0], want[0])


def test_clip_in_one_buffer():
    """Workspace, sum and gradients side by side, with the workspace longer than what is needed."""
    need = moe.moe_grad_workspace_size(2)
    buf = torch.zeros(need + 16 + 4 * 3000, dtype=torch.uint8, device=DEV)
    ws, s, flat = buf[:need], buf[need:need + 8].view(F64), buf[need + 16:].view(F32)
    flat.copy_(torch.arange(3000) % 7 - 3)
    grads, before = [flat[:1111], flat[1111:]], flat.clone()
    moe.moe_grad_sumsq(grads, s, ws)
    assert float(s) == float((before.double() ** 2).sum()) and torch.equal(flat, before)
    s.zero_()
    moe.moe_grad_sumsq(grads[:1], s, buf[-16 - need:].clone())   # another workspace, any contents
    assert float(s) == float((before[:1111].double() ** 2).sum())


# ---- the layer in a model that autograd trains ---------------------------------------------
def explicit(layer, x, ids, tw, dout):
    """Gradients through backward(), from zeroed sums: what autograd has to give."""
    layer.zero_grad()
    with torch.no_grad():
        out, rows = layer.forward(x, ids, tw)
        grads = layer.backward(dout, rows)
    want = (out, *grads, layer.grad_w13.clone(), layer.grad_w2.clone())
    layer.zero_grad()
    return want


@pytest.mark.parametrize("leaves", ["x", "tw", "w13", "w2", "x tw w13 w2"])
def test_layer_through_autograd(leaves):
    announce("layer autograd", leaves)
    layer = make_layer(31)
    x, ids, tw, dout = batch(32, 45)
    want = explicit(layer, x, ids, tw, dout)
    names = leaves.split()
    x, tw = (t.clone().requires_grad_(n in names) for t, n in ((x, "x"), (tw, "tw")))
    for n in ("w13", "w2"):
        getattr(layer, n).requires_grad_(n in names)
    # neither input is a leaf of the layer's own node, and the gradient arrives in another layout
    out, rows = layer.forward(x * 1, ids, tw * 1)
    assert out.requires_grad and torch.equal(out, want[0])
    (out.t() * 1).backward(dout.t().contiguous())
    got = (out, x.grad, tw.grad, layer.grad_w13, layer.grad_w2)
    for a, b, n in zip(got, want, ("out", "x", "tw", "w13", "w2")):
        assert torch.equal(a, b) if a is not None else n not in names, n
    assert layer.w13.grad is None and layer.w2.grad is None
    # backward() on the same rows adds once more
    dx, dtw = layer.backward(dout, rows)
    assert torch.equal(dx, want[1]) and torch.equal(dtw, want[2]) and not torch.equal(layer.grad_w2, want[4])


def test_layers_chained_through_autograd():
    first, second = make_layer(33), make_layer(34)
    x, ids, tw, dout = batch(35, 30)
    h, r1 = first.forward(x, ids, tw)
    _, r2 = second.forward(h, ids, tw)
    dh, _ = second.backward(dout, r2)
    dx, _ = first.backward(dh, r1)
    want = [t.clone() for t in (dx, first.grad_w13, first.grad_w2, second.grad_w13, second.grad_w2)]
    first.zero_grad(), second.zero_grad()
    x.requires_grad_()
    second.forward(first.forward(x, ids, tw)[0], ids, tw)[0].backward(dout)
    for a, b in zip((x.grad, first.grad_w13, first.grad_w2, second.grad_w13, second.grad_w2), want):
        assert torch.equal(a, b)


def test_layer_without_gradients_has_no_graph():
    layer = make_layer(36)
    x, ids, tw, dout = batch(37, 9)
    assert not layer.forward(x, ids, tw)[0].requires_grad
    x.requires_grad_()
    layer.w2.requires_grad_()
    with torch.no_grad():
        assert not layer.forward(x, ids, tw)[0].requires_grad


@pytest.mark.parametrize("what", ["w13", "w2", "tw"])
def test_layer_refuses_weights_changed_before_the_backward(what):
    layer = make_layer(38)
    x, ids, tw, dout = batch(39, 9)
    out, _ = layer.forward(x.requires_grad_(), ids, tw)
    (tw if what == "tw" else getattr(layer, what)).mul_(0.5)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.backward(dout)


def test_layer_autograd_in_a_graph():
    """Forward and autograd's backward captured while an eager graph of the same layer lives, replayed on new inputs."""
    layer, eager = make_layer(40), make_layer(40)
    layer.w13.requires_grad_()
    x, ids, tw, dout = batch(41, 33)
    alive = layer.forward(x, ids, tw)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())

    def step():
        layer.zero_grad()
        out, _ = layer.forward(x, ids, tw)
        out.backward(dout)
        return out.detach()

    with torch.cuda.stream(st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (42, 43, 44):
        new = batch(seed, 33)
        for dst, src in zip((x, ids, tw, dout), new):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        want = explicit(eager, *new)
        for a, b in zip((got, layer.grad_w13, layer.grad_w2), (want[0], want[3], want[4])):
            assert torch.equal(a, b), seed
    assert alive[0].requires_grad


def test_wgrad_does_not_depend_on_the_hint():
    g = gen(51)
    cs = [300, 0, 20, 1000]
    off, cap = segments(cs, 16)
    a, dy = bf((cap, 264), g).to(DEV), bf((cap, 136), g).to(DEV)
    got = []
    for hint in (0, 1, 77, 1 << 20, -5):
        dw = torch.zeros((4, 136, 264), device=DEV)
        moe.moe_grouped_gemm_bf16_wgrad(dy, a, i32(off), i32(cs), dw, 1, hint)
        got.append(dw)
    assert all(torch.equal(got[0], t) for t in got[1:])


# ---- exact sums over the longest contractions, large permutes, a layer of real width --------
@pytest.mark.parametrize("n,k", [(65536, 8), (8, 65536), (72, 30000), (30000, 72), (4104, 4168)])
def test_products_of_small_integers_are_exact(n, k):
    """Operands in -2 .. 2: every partial sum is an integer below 2^18 + 2^2, exact in fp32 in any order, so the one
    rounding to bf16 is all that may happen.  A step of the contraction left out, read twice or wrapped wrongly
    changes most outputs, which the bound on random rounding does not notice at these lengths."""
    announce("exact products", n, k)
    g = torch.Generator(device=DEV).manual_seed(n + 3 * k)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device=DEV, dtype=torch.int8).to(BF)
    cs = [3, 0, 20, 150]
    off, cap = segments(cs, 16)
    mask = valid_mask(cs, off, cap).to(DEV)
    a, dy, w, start = ints(cap, k), ints(cap, n), ints(len(cs), n, k), ints(len(cs), n, k).float()
    a[~mask], dy[~mask] = float("nan"), float("nan")
    O, Cn = i32(off), i32(cs)
    for hint in (1, 64 * len(cs), 150 * len(cs), 1 << 20):
        out, dx, dw = sentinel((cap, n)), sentinel((cap, k)), start.clone()
        moe.moe_grouped_gemm_bf16(a, w, O, Cn, out, hint)
        moe.moe_grouped_gemm_bf16_dgrad(dy, w, O, Cn, dx, hint)
        moe.moe_grouped_gemm_bf16_wgrad(dy, a, O, Cn, dw, 1)
        dwb = torch.empty((len(cs), n, k), dtype=BF, device=DEV)
        moe.moe_grouped_gemm_bf16_wgrad(dy, a, O, Cn, dwb)
        assert untouched(out, mask.cpu()) and untouched(dx, mask.cpu())
        for e, c in enumerate(cs):
            r = slice(off[e], off[e] + c)
            ae, de, we = a[r].double(), dy[r].double(), w[e].double()
            dt = de.T.contiguous()
            assert torch.equal(out[r], (ae @ we.T.contiguous()).to(BF)), (hint, e)
            assert torch.equal(dx[r], (de @ we).to(BF)), (hint, e)
            assert torch.equal(dw[e], (dt @ ae + start[e].double()).float()), (hint, e)
            assert torch.equal(dwb[e], (dt @ ae).to(BF)), (hint, e)


@pytest.mark.parametrize("M,topk,K", [(16500, 8, 1152),   # one slice of all columns a pair block, several batches a wave
                                      (20000, 4, 2048), (250, 8, 8320),   # slices of three groups, the last of one
                                      (5, 2, 65536), (700, 8, 65536)])
def test_permute_large_rows(M, topk, K):
    announce("permute_bf16 large", M, topk, K)
    Eg, El, align = 128, 100, 32
    g = torch.Generator(device=DEV).manual_seed(M)
    x = torch.randint(-2 ** 15, 2 ** 15, (M, K), generator=g, device=DEV, dtype=torch.int32).to(torch.int16)
    ids = torch.randint(-1, Eg, (M, topk), generator=g, device=DEV, dtype=I32)
    emap = torch.full((Eg,), -1, dtype=I32, device=DEV)
    emap[torch.randperm(Eg, generator=g, device=DEV)[:El]] = torch.arange(El, dtype=I32, device=DEV)
    cap = moe.moe_max_rows(M, topk, El, align)
    a = torch.full((cap, K), SENT, dtype=torch.int16, device=DEV)
    counts, off, inv, src = (torch.empty(s, dtype=I32, device=DEV) for s in ((El,), (El + 1,), (M, topk), (cap,)))
    ws = torch.empty(moe.moe_permute_workspace_size(M, topk, El), dtype=torch.uint8, device=DEV)
    moe.moe_permute_bf16(x, ids, emap, Eg, El, align, cap, a, counts, off, inv, src, ws)
    loc = torch.where(ids < 0, -1, emap[ids.clamp(min=0).long()]).reshape(-1).cpu().long()
    want_c = torch.bincount(loc[loc >= 0], minlength=El)
    want_o = torch.cat([torch.zeros(1, dtype=torch.int64), ((want_c + align - 1) // align * align).cumsum(0)])
    order = torch.sort(torch.where(loc < 0, El, loc), stable=True).indices[:int(want_c.sum())]
    first = want_c.cumsum(0) - want_c
    rows = want_o[loc[order]] + torch.arange(len(order)) - first[loc[order]]
    want_inv, want_src = torch.full((M * topk,), -1), torch.full((cap,), -1)
    want_inv[order], want_src[rows] = rows, order // topk
    assert torch.equal(counts.cpu().long(), want_c) and torch.equal(off.cpu().long(), want_o)
    assert torch.equal(inv.reshape(-1).cpu().long(), want_inv) and torch.equal(src.cpu().long(), want_src)
    valid = (want_src >= 0).to(DEV)
    assert torch.equal(a[valid], x[want_src.to(DEV)[valid]]) and bool((a[~valid] == SENT).all())


def layer_ref_by_expert(layer, x, ids, tw, dout):
    """layer_ref, one expert's rows at a time on the GPU."""
    d = lambda t: t.detach().double().requires_grad_()
    w13, w2, X, TW = d(layer.w13), d(layer.w2), d(x), d(tw)
    N, out = layer.N, torch.zeros(x.shape, dtype=F64, device=DEV)
    local = ids.long() if layer.expert_map is None else layer.expert_map[ids.long()].long()
    for e in range(layer.El):
        t, k = (local == e).nonzero(as_tuple=True)
        h = X[t] @ w13[e].T
        out = out.index_add(0, t, TW[t, k, None] * ((torch.nn.functional.silu(h[:, :N]) * h[:, N:]) @ w2[e].T))
    (out * dout.double()).sum().backward()
    return out.detach().cpu(), X.grad.cpu(), TW.grad.cpu(), w13.grad.cpu(), w2.grad.cpu()


@pytest.mark.parametrize("M,Eg,El,topk,K,N", [(1, 32, 32, 8, 2048, 768), (700, 32, 16, 4, 2048, 768),
                                              (1500, 8, 8, 2, 1152, 640)])
def test_layer_of_real_width(M, Eg, El, topk, K, N):
    """As test_layer_forward_backward, on the widths of a layer in use; through autograd."""
    announce("layer", M, Eg, El, topk, K, N)
    layer = make_layer(M + 1, Eg, El, K, N)
    layer.w13.div_(4), layer.w2.div_(2)   # activations of order one
    x, ids, tw, dout = batch(M + 2, M, K, Eg, topk)
    ref = layer_ref_by_expert(layer, x, ids, tw, dout)
    x.requires_grad_(), tw.requires_grad_()
    out, _ = layer.forward(x, ids, tw)
    out.backward(dout)
    for got, want, what in zip((out.detach(), x.grad, tw.grad, layer.grad_w13, layer.grad_w2), ref,
                               ("out", "dx", "dtw", "dw13", "dw2")):
        assert rel(got, want) <= 6 * 2.0 ** -8, (what, rel(got, want))


# ---- offsets past 32 bits, tensors that start inside a line, nothing at all -------------------
def at_16_bytes(t):
    """A copy that starts 16 bytes past a 256-byte boundary."""
    buf = torch.empty(t.numel() + 8, dtype=t.dtype, device=DEV)[8 if t.dtype == BF else 4:]
    return buf[:t.numel()].view(t.shape).copy_(t)


@pytest.mark.parametrize("hint", [1, 1 << 20])
def test_products_past_32_bits(hint):
    """Rows, weights and gradients whose offsets pass 2^31 elements and 2^32 bytes: segments at a buffer's two ends."""
    announce("products past 32 bits", hint)
    E, n, k, cap = 140, 4096, 4096, 600_000
    cs = [0] * E
    cs[0], cs[70], cs[E - 1] = 5, 3, 260
    off = [0] + [16] * 69 + [cap - 400] + [cap - 384] * 69 + [cap]
    assert len(off) == E + 1 and (cap - 384) * k > 2 ** 31 and (E - 1) * n * k > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(hint)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device=DEV, dtype=torch.int8).to(BF)
    rows = {e: slice(off[e], off[e] + cs[e]) for e in (0, 70, E - 1)}
    a, dy, out, dx = (torch.empty((cap, 4096), dtype=BF, device=DEV) for _ in range(4))
    w, dw = torch.empty((E, n, k), dtype=BF, device=DEV), torch.empty((E, n, k), device=DEV)
    for e, r in rows.items():
        a[r], dy[r], w[e] = ints(cs[e], k), ints(cs[e], n), ints(n, k)
    out[cap - 124:], dx[cap - 124:] = 77, 77
    O, Cn = i32(off), i32(cs)
    moe.moe_grouped_gemm_bf16(a, w, O, Cn, out, hint)
    moe.moe_grouped_gemm_bf16_dgrad(dy, w, O, Cn, dx, hint)
    moe.moe_grouped_gemm_bf16_wgrad(dy, a, O, Cn, dw)
    for e, r in rows.items():
        ae, de, we = a[r].double(), dy[r].double(), w[e].double()
        assert torch.equal(out[r], (ae @ we.T.contiguous()).to(BF)) and torch.equal(dx[r], (de @ we).to(BF))
        assert torch.equal(dw[e], (de.T.contiguous() @ ae).float())
    assert not dw[1].any() and not dw[E - 2].any()
    assert (out[cap - 124:] == 77).all() and (dx[cap - 124:] == 77).all()


def test_row_operators_past_32_bits():
    announce("row operators past 32 bits")
    # SiLU-mul: the valid rows at the end of a buffer of 4.9 G elements
    rows, n = 600_000, 4096
    h, d, act = (torch.empty((rows, w), dtype=BF, device=DEV) for w in (2 * n, n, n))
    g = torch.Generator(device=DEV).manual_seed(1)
    h[-50:], d[-50:] = torch.randn((50, 2 * n), generator=g, device=DEV), torch.randn((50, n), generator=g, device=DEV)
    small = [t[-50:].clone() for t in (h, d)]
    O, Cn = i32([rows - 50, rows]), i32([50])
    moe.moe_silu_mul(h, n, act, O, Cn, 1)
    moe.moe_silu_mul_bwd(h, d, n, h, O, Cn, 1)
    want_act, want_dh = torch.empty_like(small[1]), torch.empty_like(small[0])
    moe.moe_silu_mul(small[0], n, want_act)
    moe.moe_silu_mul_bwd(*small, n, want_dh)
    assert torch.equal(act[-50:], want_act) and torch.equal(h[-50:], want_dh)
    del h, d, act
    # the weighted unpermute's gradient: rows at both ends
    y, dy = torch.empty((rows, 4096), dtype=BF, device=DEV), torch.empty((rows, 4096), dtype=BF, device=DEV)
    inv = i32([[0, rows - 1], [rows - 2, -1]])
    named = [0, rows - 1, rows - 2]
    y[named] = torch.randint(-2, 3, (3, 4096), generator=g, device=DEV, dtype=torch.int32).to(BF)
    dout = torch.randint(-2, 3, (2, 4096), generator=g, device=DEV, dtype=torch.int32).to(BF)
    tw, dtw = torch.tensor([[2.0, 3.0], [-1.0, 5.0]], device=DEV), torch.empty((2, 2), device=DEV)
    moe.moe_unpermute_weight_reduce_bwd(dout, y, inv, tw, dy, dtw)
    assert torch.equal(dy[named].float(), torch.stack([dout[0] * 2.0, dout[0] * 3.0, -dout[1]]).float())
    want = torch.stack([(y[r].double() * dout[t].double()).sum() for r, t in ((0, 0), (rows - 1, 0), (rows - 2, 1))])
    assert torch.equal(dtw.reshape(-1)[:3].double(), want) and dtw[1, 1] == 0
    del y, dy
    # the permute: 800000 rows of 4096 out of 100000 tokens, checked through its own indices
    M, topk, K, El = 100_000, 8, 4096, 16
    x = torch.randint(-2 ** 15, 2 ** 15, (M, K), generator=g, device=DEV, dtype=torch.int32).to(torch.int16)
    ids = torch.randint(0, El, (M, topk), generator=g, device=DEV, dtype=I32)
    cap = moe.moe_max_rows(M, topk, El, 16)
    a = torch.empty((cap, K), dtype=torch.int16, device=DEV)
    counts, off, inv, src = (torch.empty(s, dtype=I32, device=DEV) for s in ((El,), (El + 1,), (M, topk), (cap,)))
    ws = torch.empty(moe.moe_permute_workspace_size(M, topk, El), dtype=torch.uint8, device=DEV)
    moe.moe_permute_bf16(x, ids, None, El, El, 16, cap, a, counts, off, inv, src, ws)
    assert torch.equal(counts.long(), torch.bincount(ids.reshape(-1).long(), minlength=El))
    assert int(inv.max()) * K > 2 ** 31 and inv.unique().numel() == M * topk
    for k in range(topk):
        for lo in range(0, M, 20_000):
            assert torch.equal(a[inv[lo:lo + 20_000, k].long()], x[lo:lo + 20_000])


def test_clip_past_32_bits():
    """One gradient of 2^32 and some elements."""
    announce("clip past 32 bits")
    m = 2 ** 32 + 13
    t = torch.ones(m, dtype=BF, device=DEV)
    t[-1] = 2.0
    s, nrm = clip([t], None, 2.0 ** 8)
    assert s == m + 3 and abs(nrm - (m + 3) ** 0.5) <= 2.0 ** -24 * nrm
    # the factor, 2^8 / sqrt(2^32 + 16), is 2^-8 but for less than 2^-28 of it
    assert t[-1] == 2.0 ** -7 and t[0] == 2.0 ** -8
    assert int((t[:-1] == 2.0 ** -8).sum()) == m - 1


@pytest.mark.parametrize("hint", [1, 1 << 20])
def test_tensors_that_start_inside_a_line(hint):
    """The least alignment that the entry points take, 16 bytes, gives the bits of aligned tensors."""
    g = gen(61)
    cs, n, k = [70, 0, 3, 300], 264, 136
    off, cap = segments(cs, 16)
    mask = valid_mask(cs, off, cap)
    a, dy, w, h = (bf(s, g).to(DEV) for s in ((cap, k), (cap, n), (4, n, k), (cap, 2 * n)))
    tw, inv = torch.rand((cap, 1), generator=g).to(DEV), torch.randperm(cap, generator=g).to(I32)[:, None].to(DEV)
    x, dout = bf((cap, 256), g).to(DEV), bf((cap, 256), g).to(DEV)

    def run(c):
        O, Cn = c(i32(off)), c(i32(cs))
        out, dx, act, dh = (c(sentinel(s)) for s in ((cap, n), (cap, k), (cap, n), (cap, 2 * n)))
        dwf, dwb = c(torch.ones((4, n, k), device=DEV)), c(torch.ones((4, n, k), dtype=BF, device=DEV))
        moe.moe_grouped_gemm_bf16(c(a), c(w), O, Cn, out, hint)
        moe.moe_grouped_gemm_bf16_dgrad(c(dy), c(w), O, Cn, dx, hint)
        moe.moe_grouped_gemm_bf16_wgrad(c(dy), c(a), O, Cn, dwf, 1)
        moe.moe_grouped_gemm_bf16_wgrad(c(dy), c(a), O, Cn, dwb)
        moe.moe_silu_mul(c(h), n, act, O, Cn, 4)
        moe.moe_silu_mul_bwd(c(h), c(dy), n, dh, O, Cn, 4)
        du, dtw = c(sentinel((cap, 256))), c(torch.ones((cap, 1), device=DEV))
        moe.moe_unpermute_weight_reduce_bwd(c(dout), c(x), c(inv), c(tw), du, dtw)
        return out, dx, act, dh, dwf, dwb, du, dtw

    for p, q in zip(run(at_16_bytes), run(lambda t: t)):
        assert p.data_ptr() % 256 == 16 and torch.equal(p.view(torch.int16), q.view(torch.int16))
    assert mask.any()


def test_products_of_nothing():
    """No rows at all: an overwritten gradient is zeros, an accumulated one stays."""
    O, Cn = i32([0, 0, 0]), i32([0, 0])
    empty = torch.empty((0, 72), dtype=BF, device=DEV)
    a = torch.empty((0, 520), dtype=BF, device=DEV)
    for dt in (F32, BF):
        dw = torch.full((2, 72, 520), 3.0, dtype=dt, device=DEV)
        moe.moe_grouped_gemm_bf16_wgrad(empty, a, O, Cn, dw)
        assert not dw.any()
    dw = torch.full((2, 72, 520), 3.0, device=DEV)
    moe.moe_grouped_gemm_bf16_wgrad(empty, a, O, Cn, dw, 1)
    assert (dw == 3.0).all()
    w = torch.empty((2, 72, 520), dtype=BF, device=DEV)
    moe.moe_grouped_gemm_bf16(a, w, O, Cn, empty)
    moe.moe_grouped_gemm_bf16_dgrad(empty, w, O, Cn, a)
    moe.moe_silu_mul(torch.empty((0, 144), dtype=BF, device=DEV), 72, empty, O, Cn, 2)
