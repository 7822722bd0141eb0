"""The gated experts' fused operators and 8-bit checkpoints on the GPU against
plain 64-bit implementations.

Tolerances, derived before the first run.  A sum of C products of bf16 values
accumulated in fp32 in any order is off by at most e = C * 2^-23 * T, T the sum
of the products' magnitudes.  silu(g) u moves with its sums by at most
1.1 e_g |u| + |silu(g)| e_u + 1.1 e_g e_u (|silu'| < 1.1), and the fp32 formula
by 2^-22 (4 + |g|) relative: e^-g from the hardware exp2 of -g log2(e) rounded
in fp32 is off by at most 2^-22 (2 + |g|), each of at most six operations
after it by 2^-24, and 1 - s by 2^-24 absolute, which in g's gradient counts
(1 + |g|) times the other factors.  Rounding to bf16 adds 2^-8 relative, e4m3
2^-4 relative or, for small values, 2^-10 of the block's scale.
"""
import pytest
import torch

import unpermute_count_expert_amd as moe
from tests import test_gpu_bf16_experts as base
from tests.gpu_helpers import announce
from tests.test_gpu_bf16_experts import (BF, COUNTS, DEV, F32, F64, I32, TINY, bf, gen, i32, poison, segments, sentinel,
                                         untouched, valid_mask)

U8 = torch.uint8
F8 = torch.float8_e4m3fn
SLACK = 1 + 2.0 ** -7


def within(got, ref, tol, what):
    err = (got.double().cpu() - ref).abs()
    bad = ~(err <= tol * SLACK)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst " \
                          f"{float((err / tol).nan_to_num(1e30).max()):.3g} tolerances"


def silu(g):
    return g / (1 + torch.exp(-g))


def slope(g):
    s = 1 / (1 + torch.exp(-g))
    return s * (1 + g * (1 - s))


# ---- 8-bit blocks: the definition, in exact arithmetic ------------------------------
def scale_bytes(x):
    """Of float64 x [..., 32 * blocks]: the byte of the least power of two >= amax / 448, at least 2^-117; 255 where
    a value is not finite."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = b.abs().amax(-1)
    m, e = torch.frexp(torch.where(torch.isfinite(top), top, 1.0))   # top = m 2^e, 1/2 <= m < 1; 448 = 7/8 2^9
    k = (e - 9 + (m > 0.875).int()).clamp(min=-117)
    k = torch.where(top == 0, -117, k)
    return torch.where(torch.isfinite(top), k + 127, 255).to(U8)


def nearest_codes(v):
    """Codes of float64 v, |v| <= 448: the nearest e4m3 value, ties to the even code (by a table of all values)."""
    table = torch.arange(127, dtype=torch.int16).to(U8).view(F8).double()   # 0 .. 448, ascending
    a = v.abs().reshape(-1)
    hi = torch.searchsorted(table, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = table[hi] - a, a - table[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    pick = torch.where(table[hi] == a, hi, pick)
    return (pick + 128 * torch.signbit(v.reshape(-1))).to(U8).reshape(v.shape)


def encode(x):
    s = scale_bytes(x)
    wide = s.repeat_interleave(32, -1)
    fine = wide != 255
    c = nearest_codes(torch.where(fine, x, 0.0) / torch.exp2(wide.double() - 127))
    return c, s, fine


def decode(q, s):
    return q.view(F8).double() * torch.where(s == 255, float("nan"), torch.exp2(s.double() - 127)).repeat_interleave(32, -1)


def check_codes(q, s, x, what):
    c, want_s, fine = encode(x)
    q, s = q.cpu(), s.cpu()
    assert torch.equal(s, want_s), what
    assert torch.equal(q[fine], c[fine]), what
    assert torch.isnan(q[~fine].view(F8).float()).all(), what


def test_reference_codes_are_nearest():
    values = torch.arange(256, dtype=torch.int16).to(U8)
    values = values[(values & 127) != 127]
    assert torch.equal(nearest_codes(values.view(F8).double()), values)
    v = torch.linspace(-448, 448, 10001, dtype=F64)
    assert torch.equal(nearest_codes(v).view(F8).float(), v.float().to(F8).float())


def run_checkpoint(x, slot=None):
    rows, width = x.shape
    q = torch.full((rows, width), 0x5a, dtype=U8, device=DEV)
    s = torch.full((rows, width // 32), 0x5a, dtype=U8, device=DEV)
    moe.moe_checkpoint(x.to(DEV), q, s)
    torch.cuda.synchronize()
    return q, s


@pytest.mark.parametrize("rows,width", [(1, 32), (3, 96), (130, 2048), (7, 65536), (1000, 160), (0, 64)])
def test_checkpoint(rows, width):
    announce("checkpoint", rows, width)
    x = bf((rows, width), gen(rows + width)) * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=gen(1)).float()).to(BF)
    q, s = run_checkpoint(x)
    check_codes(q, s, x.double(), "checkpoint")
    out = sentinel((rows, width))
    moe.moe_checkpoint_restore(q, s, out)
    assert torch.equal(out.cpu().double(), decode(q.cpu(), s.cpu()))   # exact in bf16
    err = (out.cpu().double() - x.double()).abs()
    scale = torch.exp2(s.cpu().double() - 127).repeat_interleave(32, -1)
    assert (err <= torch.maximum(2.0 ** -4 * x.double().abs(), 2.0 ** -10 * scale)).all()


def test_checkpoint_every_bf16():
    """Every bf16 value as the largest of its block and every value below a largest one, ties among them; infinities
    and NaN (signalling ones too) take their block along and no other."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF)
    x = torch.zeros(65536, 32, dtype=BF)
    x[:, 7] = bits
    x[:, 20] = bits
    x[::3, 31] = bits[::3] / 3
    q, s = run_checkpoint(x)
    check_codes(q, s, x.double(), "alone")
    finite = bits[torch.isfinite(bits.float())]
    y = torch.zeros(len(finite) + -len(finite) % 31, dtype=BF)
    y[:len(finite)] = finite
    for largest in (448.0, 1.0, 2.0 ** -120, 2.0 ** -110, 3.0e38):
        z = torch.cat([torch.full((y.numel() // 31, 1), largest, dtype=BF), y.reshape(-1, 31)], 1)
        z = torch.where(z.double().abs() > z[:, :1].double().abs(), torch.zeros((), dtype=BF), z)
        q, s = run_checkpoint(z)
        check_codes(q, s, z.double(), largest)


def test_checkpoint_flags_non_finite_blocks():
    x = torch.ones(4, 128, dtype=BF)
    x[0, 3], x[1, 40], x[2, 127] = float("inf"), float("-inf"), float("nan")
    x[3] = 0
    q, s = run_checkpoint(x)
    assert s.cpu().tolist() == [[255, 119, 119, 119], [119, 255, 119, 119], [119, 119, 119, 255], [10] * 4]
    out = sentinel((4, 128))
    moe.moe_checkpoint_restore(q, s, out)
    nan = torch.isnan(out.cpu().float()).reshape(4, 4, 32)
    assert torch.equal(nan.all(-1), s.cpu() == 255) and torch.equal(nan.any(-1), s.cpu() == 255)


# ---- rows in expert order -----------------------------------------------------------
def places(M, topk, rows, g):
    p = torch.randperm(max(rows, M * topk), generator=g)[:M * topk].reshape(M, topk).to(I32)   # some >= rows
    p[torch.rand((M, topk), generator=g) < 0.3] = -1
    if M:
        p[-1] = -1   # a token without rows
    return p


@pytest.mark.parametrize("M,topk,width,rows", [(1, 1, 32, 4), (5, 8, 640, 60), (130, 3, 2176, 500), (3000, 2, 96, 7000),
                                               (2, 256, 256, 600), (4, 2, 128, 0), (0, 2, 64, 8), (9, 5, 65536, 50),
                                               (6000, 8, 64, 48000)])
def test_rows_in_expert_order(M, topk, width, rows):
    announce("rows", M, topk, width, rows)
    g = gen(M + width)
    x, tw = bf((M, width), g), torch.rand((M, topk), generator=g)
    inv = places(M, topk, rows, g)
    t, k = ((inv >= 0) & (inv < rows)).nonzero(as_tuple=True)
    r = inv[t, k].long()
    named = torch.zeros(rows, dtype=torch.bool)
    named[r] = True
    out, rw = sentinel((rows, width)), torch.full((rows,), 7.0, device=DEV)
    moe.moe_permute_rows(x.to(DEV), inv.to(DEV), out, tw.to(DEV), rw)
    plain = sentinel((rows, width))
    moe.moe_permute_rows(x.to(DEV), inv.to(DEV), plain)
    q, s = run_checkpoint(x)
    back = sentinel((rows, width))
    moe.moe_checkpoint_restore(q, s, back, inv.to(DEV))
    torch.cuda.synchronize()
    for o in (out, plain, back):
        assert untouched(o, named)
    assert torch.equal(out.cpu()[r], x[t]) and torch.equal(plain.cpu()[r], x[t])
    assert torch.equal(rw.cpu()[r], tw[t, k]) and (rw.cpu()[~named] == 7).all()
    assert torch.equal(back.cpu()[r].double(), decode(q.cpu(), s.cpu())[t])


@pytest.mark.parametrize("K", [8, 24, 2184])
def test_permute_rows_odd_widths(K):
    g = gen(K)
    x, inv = bf((37, K), g), torch.randperm(111, generator=g).reshape(37, 3).to(I32)
    out = sentinel((111, K))
    moe.moe_permute_rows(x.to(DEV), inv.to(DEV), out)
    assert torch.equal(out.cpu()[inv.long()], x[:, None].expand(-1, 3, -1))


@pytest.mark.parametrize("M,topk,nd,rows", [(1, 1, 1, 3), (130, 8, 12, 1040), (7, 3, 17, 30), (40, 2, 1024, 90), (3, 2, 5, 0),
                                            (0, 2, 5, 4)])
def test_topk_weights_bwd(M, topk, nd, rows):
    g = gen(nd + M)
    dots, inv = torch.randn((rows, nd), generator=g), places(M, topk, rows, g)
    dw = torch.full((M, topk), 7.0, device=DEV)
    moe.moe_topk_weights_bwd(dots.to(DEV), inv.to(DEV), dw)
    ok = (inv >= 0) & (inv < rows)
    r = inv[ok].long()
    ref = dots.double()[r]
    within(dw.cpu()[ok], ref.sum(1), nd * 2.0 ** -24 * ref.abs().sum(1) + TINY, "dweights")
    assert (dw.cpu()[~ok] == 0).all()


# ---- gate and up products with SiLU-mul ----------------------------------------------
def new_h(cap, n, keep):
    if keep == "none":
        return None, None
    if keep == "bf16":
        return sentinel((cap, 2 * n)), None
    return torch.full((cap, 2 * n), 0x5a, dtype=U8, device=DEV), torch.full((cap, n // 16), 0x5a, dtype=U8, device=DEV)


def rows_untouched(h, h_s, mask):
    if h is None:
        return True
    if h_s is None:
        return untouched(h, mask)
    return bool((h.cpu()[~mask] == 0x5a).all() and (h_s.cpu()[~mask] == 0x5a).all())


def run_fwd(a, w13, off, cs, keep, hint):
    cap, n = a.shape[0], w13.shape[1] // 2
    act = sentinel((cap, n))
    h, h_s = new_h(cap, n, keep)
    moe.moe_grouped_gemm_bf16_silu_mul(a.to(DEV), w13.to(DEV), i32(off), i32(cs), act, h, h_s, hint)
    torch.cuda.synchronize()
    return act, h, h_s


NK = [(8, 8), (64, 128), (40, 136), (264, 1000), (520, 72), (136, 2056)]
NK32 = [(32, 8), (64, 128), (96, 136), (288, 1000), (544, 72), (160, 2056)]


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("keep", ["none", "bf16", "e4m3"])
@pytest.mark.parametrize("hint", [1, 0, 1 << 20])
@pytest.mark.parametrize("size", range(len(NK)))
def test_gated_forward(counts, keep, hint, size):
    n, k = (NK32 if keep == "e4m3" else NK)[size]
    announce("gated", counts, n, k, keep, hint)
    cs = COUNTS[counts]
    E = len(cs)
    off, cap = segments(cs, 16)
    mask = valid_mask(cs, off, cap)
    g = gen(n * 7 + k + E)
    a, w13 = bf((cap, k), g), bf((E, 2 * n, k), g, 4 * k ** -0.5)
    act, h, h_s = run_fwd(poison(a, mask), w13, off, cs, keep, hint)
    assert untouched(act, mask) and rows_untouched(h, h_s, mask)
    for e, c in enumerate(cs):
        r = slice(off[e], off[e] + c)
        ae, we = a[r].double(), w13[e].double()
        ref, err = ae @ we.T, k * 2.0 ** -23 * (ae.abs() @ we.abs().T)
        gr, ur, ge, ue = ref[:, :n], ref[:, n:], err[:, :n], err[:, n:]
        want = silu(gr) * ur
        tol = 1.1 * ge * ur.abs() + silu(gr).abs() * ue + 1.1 * ge * ue
        within(act[r], want, tol + (2.0 ** -8 + 2.0 ** -22 * (4 + gr.abs())) * (want.abs() + tol) + TINY, "act")
        if keep == "bf16":
            within(h[r], ref, err + 2.0 ** -8 * (ref.abs() + err) + TINY, "h")
        if keep == "e4m3" and c:
            got = decode(h[r].cpu(), h_s[r].cpu())
            # the scale is below 2 amax / 448 (or the least one)
            scale = ((ref.abs() + err).reshape(c, -1, 32).amax(-1) / 224).clamp(min=2.0 ** -117).repeat_interleave(32, -1)
            within(got, ref, err + torch.maximum(2.0 ** -4 * (ref.abs() + err), 2.0 ** -10 * scale), "h in 8 bits")


@pytest.mark.parametrize("n,k", [(32, 64), (160, 256), (288, 2048)])
@pytest.mark.parametrize("hint", [1, 300, 1 << 20])
def test_gated_forward_codes_are_exact(n, k, hint):
    """Sums of small integers are exact in fp32: codes and scales of every kernel are the definition's."""
    announce("gated codes", n, k, hint)
    cs = [63, 0, 65, 1, 130]
    off, cap = segments(cs, 16)
    mask = valid_mask(cs, off, cap)
    g = gen(n + k)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g).to(BF)
    a, w13 = ints(cap, k), ints(5, 2 * n, k)
    a[off[2] + 5] = 0            # a row of zeros
    w13[4, 7] = 0
    _, h, h_s = run_fwd(a, w13, off, cs, "e4m3", hint)
    ref = torch.zeros(cap, 2 * n, dtype=F64)
    for e, c in enumerate(cs):
        ref[off[e]:off[e] + c] = a[off[e]:off[e] + c].double() @ w13[e].double().T
    check_codes(h[mask.to(DEV)], h_s[mask.to(DEV)], ref[mask], "codes")
    assert rows_untouched(h, h_s, mask)
    _, hb, _ = run_fwd(a, w13, off, cs, "bf16", hint)
    assert torch.equal(hb.cpu()[mask], ref[mask].float().to(BF))


# ---- the backward pass ----------------------------------------------------------------
def kept_rows(cap, n, keep, g, mask):
    """(h and h_s on the GPU with rubbish in invalid rows, the values they stand for)"""
    if keep == "bf16":
        h = bf((cap, 2 * n), g, 3.0)
        return poison(h, mask).to(DEV), None, h.double()
    q, s, _ = encode(bf((cap, 2 * n), g, 3.0).double())
    v = decode(q, s)
    q[~mask], s[~mask] = 0x7f, 255
    return q.to(DEV), s.to(DEV), v


def bwd_reference(h, d, derr, w, n):
    """(value, tolerance) of act, dg, du and the products that dots sums, from the kept h and d with its error."""
    g, u, w = h[:, :n], h[:, n:], w[:, None]
    rel = 2.0 ** -22 * (5 + g.abs())
    a, m = silu(g) * u, (slope(g) * u).abs()
    out = {"act": (w * a, rel * (w * a).abs()),
           "dg": (w * d * u * slope(g), (w * derr).abs() * m + (w * (d.abs() + derr) * u).abs() * (1 + g.abs()) * rel),
           "du": (w * d * silu(g), (w * derr * silu(g)).abs() + rel * (w * (d.abs() + derr) * silu(g)).abs()),
           "dot": (a * d, (a * derr).abs() + rel * (a * (d.abs() + derr)).abs())}
    # Where the sigmoid s = 1 / (1 + e^-g) is below 2^-126, the least normal fp32 number (g < -87.3), it counts as 0,
    # as documented: each value has s as a factor, so it loses at most 2^-126 times its other factors.
    lost = torch.where(g < -87.3, 2.0 ** -126, 0.0) * g.abs()
    for name, others in (("act", w * u), ("dg", w * (d.abs() + derr) * u * 2), ("du", w * (d.abs() + derr)),
                         ("dot", (d.abs() + derr) * u)):
        out[name] = out[name][0], out[name][1] + lost * others.abs()
    return out


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("hint", [1, 0, 1 << 20])
@pytest.mark.parametrize("size", range(len(NK)))
def test_gated_backward(counts, keep, hint, size):
    n, k = (NK32 if keep == "e4m3" else NK)[size]
    announce("gated_bwd", counts, n, k, keep, hint)
    cs = COUNTS[counts]
    E = len(cs)
    off, cap = segments(cs, 16)
    mask = valid_mask(cs, off, cap)
    g = gen(n * 5 + k + E)
    dy, w2 = bf((cap, k), g, 0.5), bf((E, k, n), g, k ** -0.5)
    H, HS, h = kept_rows(cap, n, keep, g, mask)
    w = torch.rand(cap, generator=g) * 2 - 0.5
    W = w.clone()
    W[~mask] = float("nan")
    D, w2d, O, Cn = poison(dy, mask).to(DEV), w2.to(DEV), i32(off), i32(cs)
    nd = (n + 63) // 64
    dh, act = sentinel((cap, 2 * n)), sentinel((cap, n))
    dots = torch.full((cap, nd), 7.25, device=DEV)
    moe.moe_grouped_gemm_bf16_dgrad_silu_mul(D, w2d, O, Cn, H, dh, act, HS, W.to(DEV), dots, hint)
    torch.cuda.synchronize()
    assert untouched(dh, mask) and untouched(act, mask) and (dots.cpu()[~mask] == 7.25).all()
    for e, c in enumerate(cs):
        r = slice(off[e], off[e] + c)
        de, we = dy[r].double(), w2[e].double()
        ref = bwd_reference(h[r], de @ we, k * 2.0 ** -23 * (de.abs() @ we.abs()), w[r].double(), n)
        for name, got in (("act", act[r]), ("dg", dh[r, :n]), ("du", dh[r, n:])):
            v, tol = ref[name]
            within(got, v, tol + 2.0 ** -8 * (v.abs() + tol) + TINY, name)
        v, tol = ref["dot"]
        pad = lambda t: torch.nn.functional.pad(t, (0, nd * 64 - n)).reshape(c, nd, 64)
        within(dots[r], pad(v).sum(-1), pad(tol).sum(-1) + 64 * 2.0 ** -23 * pad(v.abs() + tol).sum(-1) + TINY, "dots")
    # without weights and further outputs: the same as with weights of 1
    ones, plain = torch.ones(cap, device=DEV), sentinel((cap, 2 * n))
    moe.moe_grouped_gemm_bf16_dgrad_silu_mul(D, w2d, O, Cn, H, dh, None, HS, ones, None, hint)
    moe.moe_grouped_gemm_bf16_dgrad_silu_mul(D, w2d, O, Cn, H, plain, h_s=HS, rows_hint=hint)
    assert torch.equal(plain.view(torch.int16)[mask.to(DEV)], dh.view(torch.int16)[mask.to(DEV)])
    assert untouched(plain, mask)
    if keep == "bf16":   # in place
        before = H.view(torch.int16).cpu()
        moe.moe_grouped_gemm_bf16_dgrad_silu_mul(D, w2d, O, Cn, H, H, rows_hint=hint)
        got = H.view(torch.int16).cpu()
        assert torch.equal(got[mask], plain.view(torch.int16).cpu()[mask]) and torch.equal(got[~mask], before[~mask])


def test_gated_reference_matches_differences():
    g = gen(3)
    h = torch.randn(5, 12, generator=g, dtype=F64) * 3
    d, w = torch.randn(5, 6, generator=g, dtype=F64), torch.rand(5, generator=g, dtype=F64)
    ref = bwd_reference(h, d, torch.zeros_like(d), w, 6)
    f = lambda x: (w[:, None] * silu(x[:, :6]) * x[:, 6:] * d).sum(1)
    for c in range(12):
        hp, hm = h.clone(), h.clone()
        hp[:, c] += 1e-6
        hm[:, c] -= 1e-6
        want = ref["dg"][0][:, c] if c < 6 else ref["du"][0][:, c - 6]
        assert torch.allclose((f(hp) - f(hm)) / 2e-6, want, rtol=1e-7, atol=1e-7)


@pytest.mark.parametrize("hint", [1, 1 << 20])
def test_gated_inconsistent_segments_are_cut(hint):
    """A count past its slot is cut at the next segment and at the buffer; a negative one is empty; offsets past the
    buffer or out of order stay in bounds."""
    off, cap, n, k = [0, 16, 32, 40], 44, 64, 72
    g = gen(5)
    a, w13, dy, w2 = bf((cap, k), g), bf((3, 2 * n, k), g), bf((cap, k), g), bf((3, k, n), g)
    H, HS, _ = kept_rows(cap, n, "e4m3", g, torch.ones(cap, dtype=torch.bool))

    def run(o, c):
        act, h, h_s = run_fwd(a, w13, o, c, "e4m3", hint)
        dh, act2, dots = sentinel((cap, 2 * n)), sentinel((cap, n)), torch.full((cap, 1), 7.0, device=DEV)
        moe.moe_grouped_gemm_bf16_dgrad_silu_mul(dy.to(DEV), w2.to(DEV), i32(o), i32(c), H, dh, act2, HS, None, dots, hint)
        torch.cuda.synchronize()
        return [t.cpu().view(torch.int16 if t.dtype == BF else t.dtype) for t in (act, h, h_s, dh, act2, dots)]

    for x, y in zip(run(off, [100, -3, 900]), run(off, [16, 0, 8])):
        assert torch.equal(x, y)
    run([0, 500, 20, 44], [4, 9, 30])
    run([-7, 44, 44, 10], [50, 9, 30])


@pytest.mark.parametrize("hint", [1, 1 << 20])
def test_gated_non_finite_values_stay_in_their_rows(hint):
    cs, n, k = [20, 3, 40], 96, 104
    off, cap = segments(cs, 16)
    g = gen(6)
    a, w13, dy, w2 = bf((cap, k), g), bf((3, 2 * n, k), g), bf((cap, k), g), bf((3, k, n), g)
    mask = valid_mask(cs, off, cap)
    H, HS, _ = kept_rows(cap, n, "e4m3", g, mask)

    def run(aa, dd, hs):
        act, h, h_s = run_fwd(aa, w13, off, cs, "e4m3", hint)
        dh, act2, dots = sentinel((cap, 2 * n)), sentinel((cap, n)), torch.full((cap, 2), 7.0, device=DEV)
        moe.moe_grouped_gemm_bf16_dgrad_silu_mul(dd.to(DEV), w2.to(DEV), i32(off), i32(cs), H, dh, act2, hs, None, dots, hint)
        torch.cuda.synchronize()
        return [t.cpu() for t in (act, h, h_s, dh, act2, dots)]

    base = run(a, dy, HS)
    a2, dy2, hs2 = a.clone(), dy.clone(), HS.clone()
    bad_a, bad_d, bad_h = off[1] + 1, off[2] + 5, off[2] + 30
    a2[bad_a, 5] = float("inf")
    dy2[bad_d, 7] = float("nan")
    hs2[bad_h, 1] = 255
    got = run(a2, dy2, hs2)
    for j, bad in enumerate([(bad_a,), (bad_a,), (bad_a,), (bad_d, bad_h), (bad_h,), (bad_d, bad_h)]):
        rows = torch.ones(cap, dtype=torch.bool)
        rows[list(bad)] = False
        assert torch.equal(got[j].view(U8)[rows], base[j].view(U8)[rows]), j
    assert (got[2][bad_a] == 255).all() and torch.isnan(got[3][bad_d].float()).all() and torch.isnan(got[5][bad_d]).all()
    nan = torch.isnan(got[4][bad_h].float())   # gate columns 32 to 63 are NaN
    assert nan[32:64].all() and not nan[:32].any() and not nan[64:].any()


def test_gated_many_experts():
    """1024 experts, most without rows."""
    g = gen(7)
    cs = [0] * 1024
    for e, c in ((0, 2), (1, 1), (511, 40), (777, 5), (1023, 3)):
        cs[e] = c
    off, cap = segments(cs, 16, 0)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g).to(BF)
    n, k = 32, 16
    a, w13, w2 = ints(cap, k), ints(1024, 2 * n, k), ints(1024, k, n)
    mask = valid_mask(cs, off, cap)
    for hint in (1, 1 << 24):
        act, h, _ = run_fwd(a, w13, off, cs, "bf16", hint)
        dh = sentinel((cap, 2 * n))
        moe.moe_grouped_gemm_bf16_dgrad_silu_mul(a.to(DEV), w2.to(DEV), i32(off), i32(cs), h, dh, rows_hint=hint)
        torch.cuda.synchronize()
        assert untouched(dh, mask)
        for e in (0, 1, 2, 511, 777, 1023):
            r = slice(off[e], off[e] + cs[e])
            ref = a[r].double() @ w13[e].double().T
            assert torch.equal(h[r].cpu().double(), ref)
            v, tol = bwd_reference(ref, a[r].double() @ w2[e].double(), torch.zeros(cs[e], n, dtype=F64),
                                   torch.ones(cs[e], dtype=F64), n)["dg"]
            within(dh[r, :n], v, tol + 2.0 ** -8 * (v.abs() + tol) + TINY, "dg")


def test_restore_every_code_and_scale():
    """Every code with every scale byte, subnormal values among them, restored dense."""
    q = torch.arange(256, dtype=torch.int16).to(U8).repeat(256, 1)
    s = torch.arange(256, dtype=torch.int16).to(U8)[:, None].repeat(1, 8)
    out = sentinel((256, 256))
    moe.moe_checkpoint_restore(q.to(DEV), s.to(DEV), out)
    want = decode(q, s)
    within(out.cpu().double().nan_to_num(12345.0), want.float().to(BF).double().nan_to_num(12345.0), torch.zeros(()), "restored")
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(want))


# ---- longer walks, other layouts, side by side, large offsets ---------------------------
def gated_on_gpu(cs, n, k, off, cap, hints, seed, keeps=("none", "bf16", "e4m3")):
    """Both products against 64-bit ones on the GPU, every expert; the tolerances of the small tests."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    a, dy = rn(cap, k).to(BF), (rn(cap, k) * 0.5).to(BF)
    w13, w2 = (rn(len(cs), 2 * n, k) * (4 * k ** -0.5)).to(BF), (rn(len(cs), k, n) * k ** -0.5).to(BF)
    O, Cn, mask, w = i32(off), i32(cs), valid_mask(cs, off, cap), torch.rand(cap, generator=g, device=DEV) + 0.1
    nd = (n + 63) // 64
    for hint in hints:
        for keep in keeps:
            act = sentinel((cap, n))
            h, h_s = new_h(cap, n, keep)
            moe.moe_grouped_gemm_bf16_silu_mul(a, w13, O, Cn, act, h, h_s, hint)
            assert untouched(act, mask) and rows_untouched(h, h_s, mask)
            if keep != "none":
                dh, act2, dots = sentinel((cap, 2 * n)), sentinel((cap, n)), torch.full((cap, nd), 7.0, device=DEV)
                moe.moe_grouped_gemm_bf16_dgrad_silu_mul(dy, w2, O, Cn, h, dh, act2, h_s, w, dots, hint)
                assert untouched(dh, mask) and untouched(act2, mask) and (dots.cpu()[~mask] == 7).all()
            for e, c in enumerate(cs):
                if c == 0:
                    continue
                r = slice(off[e], off[e] + c)
                ae, we = a[r].double(), w13[e].double().T.contiguous()
                ref, err = ae @ we, k * 2.0 ** -23 * (ae.abs() @ we.abs())
                gr, ur, ge, ue = ref[:, :n], ref[:, n:], err[:, :n], err[:, n:]
                want = silu(gr) * ur
                tol = 1.1 * ge * ur.abs() + silu(gr).abs() * ue + 1.1 * ge * ue
                within(act[r], want.cpu(), (tol + (2.0 ** -8 + 2.0 ** -22 * (4 + gr.abs())) * (want.abs() + tol) + TINY).cpu(), "act")
                if keep == "none":
                    continue
                hv = h[r].double() if keep == "bf16" else \
                    h[r].view(F8).double() * torch.exp2(h_s[r].double() - 127).repeat_interleave(32, -1)
                step = 2.0 ** -8 * (ref.abs() + err)
                if keep == "e4m3":
                    scale = ((ref.abs() + err).reshape(c, -1, 32).amax(-1) / 224).repeat_interleave(32, -1)
                    step = torch.maximum(2.0 ** -4 * (ref.abs() + err), 2.0 ** -10 * scale)
                within(hv.cpu(), ref.cpu(), (err + step + TINY).cpu(), "h")
                de, we = dy[r].double(), w2[e].double()
                b = bwd_reference(hv, de @ we, k * 2.0 ** -23 * (de.abs() @ we.abs()), w[r].double(), n)
                for name, got in (("act", act2[r]), ("dg", dh[r, :n]), ("du", dh[r, n:])):
                    v, tol = b[name]
                    within(got, v.cpu(), (tol + 2.0 ** -8 * (v.abs() + tol) + TINY).cpu(), name)
                v, tol = b["dot"]
                pad = lambda t: torch.nn.functional.pad(t, (0, nd * 64 - n)).reshape(c, nd, 64)
                within(dots[r], pad(v).sum(-1).cpu(),
                       (pad(tol).sum(-1) + 64 * 2.0 ** -23 * pad(v.abs() + tol).sum(-1) + TINY).cpu(), "dots")


@pytest.mark.parametrize("cs,n,k", [([1100 + 7 * e for e in range(24)], 768, 512), ([40 + 3 * e for e in range(100)], 416, 264),
                                    ([9000, 1], 160, 2048), ([3] * 300, 96, 136)])
def test_gated_long_walks(cs, n, k):
    """More tiles than blocks, so that blocks go on from one tile, expert and wave group to the next."""
    announce("gated long", len(cs), n, k)
    off, cap = segments(cs, 16)
    gated_on_gpu(cs, n, k, off, cap, (1, sum(cs), 1 << 24), len(cs))


@pytest.mark.parametrize("E,n,k,rows", [(128, 768, 2048, (1, 16, 64, 160, 300, 1024)), (60, 416, 264, (1, 20, 100, 700, 5000)),
                                        (513, 64, 264, (1, 20, 160, 2000)), (512, 32, 136, (1, 40, 3000))])
def test_gated_every_kernel(E, n, k, rows):
    """Experts and row counts given that pick each kernel in turn (a few rows; 64-, 128- and 256-row tiles, the
    forward ones with staggered and with common starts of the contraction; no 64-row tiles past 512 experts)."""
    announce("gated every kernel", E, n, k)
    g = torch.Generator().manual_seed(n + k)
    cs = torch.randint(0, 30, (E,), generator=g).tolist()
    cs[3], cs[E // 2], cs[E - 1] = 0, 150, 290
    off, cap = segments(cs, 16)
    gated_on_gpu(cs, n, k, off, cap, [1] + [r * E for r in rows], n + k, ("bf16", "e4m3"))


@pytest.mark.parametrize("n,k", [(32768, 8), (32, 65536), (96, 30000)])
def test_gated_widest(n, k):
    announce("gated widest", n, k)
    cs = [3, 0, 20]
    off, cap = segments(cs, 16)
    gated_on_gpu(cs, n, k, off, cap, (1, 1 << 20), 5)


def test_gated_on_slots():
    """Slots of a fixed size, most of each unused (a batched, masked layout)."""
    gated_on_gpu([0, 7, 300, 1, 64], 160, 200, [i * 320 for i in range(6)], 1600, (1, 1 << 20), 6)


def all_ops(c, hint, g):
    """Every entry point once, tensors through c; what they wrote."""
    cs, n, k, M = [70, 0, 3, 300], 288, 136, 97
    off, cap = segments(cs, 16)
    O, Cn = c(i32(off)), c(i32(cs))
    new = lambda *s: c(bf(s, g).to(DEV))
    a, w13, dy, w2 = new(cap, k), new(4, 2 * n, k), new(cap, k), new(4, k, n)
    x, inv, tw = new(M, 256), c(torch.randperm(400, generator=g)[:3 * M].reshape(M, 3).to(I32).to(DEV)), \
        c(torch.rand((M, 3), generator=g).to(DEV))
    z8 = lambda *s: c(torch.zeros(s, dtype=U8, device=DEV))
    z16 = lambda *s: c(sentinel(s))
    z32 = lambda *s: c(torch.ones(s, device=DEV))
    act, h, q, s = z16(cap, n), z16(cap, 2 * n), z8(cap, 2 * n), z8(cap, n // 16)
    moe.moe_grouped_gemm_bf16_silu_mul(a, w13, O, Cn, act, h, None, hint)
    moe.moe_grouped_gemm_bf16_silu_mul(a, w13, O, Cn, act, q, s, hint)
    dh, dh8, act2, dots, rw = z16(cap, 2 * n), z16(cap, 2 * n), z16(cap, n), z32(cap, 5), z32(cap)
    moe.moe_grouped_gemm_bf16_dgrad_silu_mul(dy, w2, O, Cn, h, dh, act2, None, rw, dots, hint)
    moe.moe_grouped_gemm_bf16_dgrad_silu_mul(dy, w2, O, Cn, q, dh8, None, s, None, None, hint)
    xq, xs, rows, back, roww, dtw = z8(M, 256), z8(M, 8), z16(400, 256), z16(400, 256), z32(400), z32(M, 3)
    moe.moe_checkpoint(x, xq, xs)
    moe.moe_checkpoint_restore(xq, xs, back, inv)
    moe.moe_permute_rows(x, inv, rows, tw, roww)
    moe.moe_topk_weights_bwd(c(torch.randn((400, 5), generator=g).to(DEV)), inv, dtw)
    return act, h, q, s, dh, dh8, act2, dots, xq, xs, rows, back, roww, dtw


def bits(t):
    return t.contiguous().view(U8)


def at_16_bytes(t):
    """A copy that starts 16 bytes past a 256-byte boundary."""
    skip = 16 // t.element_size()
    return torch.empty(t.numel() + skip, dtype=t.dtype, device=DEV)[skip:].view(t.shape).copy_(t)


@pytest.mark.parametrize("hint", [1, 1 << 20])
def test_gated_tensors_that_start_inside_a_line(hint):
    """The least alignment that the entry points take, 16 bytes, gives the bits of aligned tensors."""
    for p, q in zip(all_ops(at_16_bytes, hint, gen(61)), all_ops(lambda t: t, hint, gen(61))):
        assert p.data_ptr() % 256 == 16 and torch.equal(bits(p), bits(q))


def test_gated_side_by_side():
    """Every entry point on two streams at once, each with its own tensors."""
    want = [[all_ops(lambda t: t, h, gen(seed)) for h in (1, 1 << 20)] for seed in (62, 63)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in want]
    for _ in range(4):
        got = []
        for seed, st in zip((62, 63), streams):
            with torch.cuda.stream(st):
                got.append([all_ops(lambda t: t, h, gen(seed)) for h in (1, 1 << 20)])
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            for p, q in zip(x, y):
                assert all(torch.equal(bits(a), bits(b)) for a, b in zip(p, q))


@pytest.mark.parametrize("hint", [1, 1 << 20])
def test_gated_past_32_bits(hint):
    """Rows, codes, scales and weights whose offsets pass 2^31 elements and 2^32 bytes: segments at a buffer's ends."""
    announce("gated past 32 bits", hint)
    E, n, k, cap = 140, 2048, 4096, 1_100_000
    cs = [0] * E
    cs[0], cs[70], cs[E - 1] = 5, 3, 260
    off = [0] + [16] * 69 + [cap - 400] + [cap - 384] * 69 + [cap]
    assert len(off) == E + 1 and (cap - 400) * 2 * n > 2 ** 32 and (E - 1) * 2 * n * k > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(hint)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device=DEV, dtype=torch.int8).to(BF)
    a, dy, act, act2 = (torch.empty((cap, w), dtype=BF, device=DEV) for w in (k, k, n, n))
    h, dh = (torch.empty((cap, 2 * n), dtype=BF, device=DEV) for _ in range(2))
    q, s = torch.empty((cap, 2 * n), dtype=U8, device=DEV), torch.empty((cap, n // 16), dtype=U8, device=DEV)
    w13, w2 = torch.empty((E, 2 * n, k), dtype=BF, device=DEV), torch.empty((E, k, n), dtype=BF, device=DEV)
    rw, dots = torch.ones(cap, device=DEV), torch.empty((cap, n // 64), device=DEV)
    rows = {e: slice(off[e], off[e] + cs[e]) for e in (0, 70, E - 1)}
    for e, r in rows.items():
        a[r], dy[r], w13[e], w2[e] = ints(cs[e], k), ints(cs[e], k), ints(2 * n, k), ints(k, n)
        rw[r] = 0.5
    tail = slice(cap - 124, cap)
    act[tail], h[tail], q[tail], s[tail], dh[tail], dots[tail] = 77, 77, 77, 77, 77, 77
    O, Cn = i32(off), i32(cs)
    moe.moe_grouped_gemm_bf16_silu_mul(a, w13, O, Cn, act, q, s, hint)
    moe.moe_grouped_gemm_bf16_silu_mul(a, w13, O, Cn, act, h, None, hint)
    for e, r in rows.items():
        ref = (a[r].double() @ w13[e].double().T.contiguous()).cpu()
        assert torch.equal(h[r].cpu(), ref.to(BF))
        check_codes(q[r], s[r], ref, e)
    for keep in ("bf16", "e4m3"):
        moe.moe_grouped_gemm_bf16_dgrad_silu_mul(dy, w2, O, Cn, h if keep == "bf16" else q, dh, act2,
                                                 None if keep == "bf16" else s, rw, dots, hint)
        for e, r in rows.items():
            hv = h[r].cpu().double() if keep == "bf16" else decode(q[r].cpu(), s[r].cpu())
            d = (dy[r].double() @ w2[e].double()).cpu()
            b = bwd_reference(hv, d, torch.zeros_like(d), torch.full((cs[e],), 0.5, dtype=F64), n)
            for name, got in (("act", act2[r]), ("dg", dh[r, :n]), ("du", dh[r, n:])):
                v, tol = b[name]
                within(got, v, tol + 2.0 ** -8 * (v.abs() + tol) + TINY, name)
            v, tol = (t.reshape(cs[e], -1, 64) for t in b["dot"])
            within(dots[r], v.sum(-1), tol.sum(-1) + 64 * 2.0 ** -23 * (v.abs() + tol).sum(-1) + TINY, "dots")
    for t in (act, h, q, s, dh, dots):
        assert (t[tail] == 77).all()


def test_rows_past_32_bits():
    """Tokens and rows past 2^32 elements, and more tokens than one launch has waves for."""
    M, K, g = 4_400_000, 1024, torch.Generator(device=DEV).manual_seed(3)
    x = torch.randint(-8, 9, (M, K), generator=g, device=DEV, dtype=torch.int8).to(BF)
    inv = torch.randperm(M, generator=g, device=DEV).to(I32)[:, None]
    out, q, s = torch.empty_like(x), torch.empty((M, K), dtype=U8, device=DEV), torch.empty((M, K // 32), dtype=U8, device=DEV)
    tw, rw = torch.rand((M, 1), generator=g, device=DEV), torch.empty(M, device=DEV)
    moe.moe_permute_rows(x, inv, out, tw, rw)
    at = inv[:, 0].long()
    assert torch.equal(rw[at], tw[:, 0])
    for lo in range(0, M, 400_000):
        assert torch.equal(out[at[lo:lo + 400_000]], x[lo:lo + 400_000])
    moe.moe_checkpoint(x, q, s)   # integers up to 8: exact in e4m3
    out.zero_()
    moe.moe_checkpoint_restore(q, s, out, inv)
    for lo in range(0, M, 400_000):
        assert torch.equal(out[at[lo:lo + 400_000]], x[lo:lo + 400_000])
    dots, dw = torch.randint(-8, 9, (M, 3), generator=g, device=DEV).float(), torch.empty((M, 1), device=DEV)
    moe.moe_topk_weights_bwd(dots, inv, dw)
    assert torch.equal(dw[:, 0], dots.sum(1)[at])


def test_gated_products_of_nothing():
    O, Cn = i32([0, 0, 0]), i32([0, 0])
    e = lambda *s, dt=BF: torch.empty(s, dtype=dt, device=DEV)
    moe.moe_grouped_gemm_bf16_silu_mul(e(0, 72), e(2, 64, 72), O, Cn, e(0, 32), e(0, 64))
    moe.moe_grouped_gemm_bf16_silu_mul(e(0, 72), e(2, 64, 72), O, Cn, e(0, 32), e(0, 64, dt=U8), e(0, 2, dt=U8))
    moe.moe_grouped_gemm_bf16_dgrad_silu_mul(e(0, 72), e(2, 72, 32), O, Cn, e(0, 64), e(0, 64), e(0, 32), None,
                                             e(0, dt=F32), e(0, 1, dt=F32))


# ---- the layer --------------------------------------------------------------------------
def make_layer(seed, keep, Eg=8, El=8, K=256, N=128):
    plain = base.make_layer(seed, Eg, El, K, N)
    return moe.MoeTrainLayer(plain.w13, plain.w2, Eg, plain.expert_map, plain.align, keep)


def restored(t, s):
    return t.detach().cpu().double() if s is None else decode(t.cpu(), s.cpu())


def grads_at(layer, saved, tw, dout):
    """The layer's gradients in 64 bits at the kept values, pair by pair."""
    d = lambda t: t.detach().cpu().double()
    w13, w2, TW, G, N = d(layer.w13), d(layer.w2), d(tw), d(dout), layer.N
    x, h = restored(saved.x, saved.x_s), restored(saved.h, saved.h_s)
    off, inv = saved.expert_offsets.tolist(), saved.inv_perm.cpu()
    dx, dtw, dw13, dw2 = torch.zeros_like(G), torch.zeros_like(TW), torch.zeros_like(w13), torch.zeros_like(w2)
    for e in range(layer.El):
        t, k = ((inv >= off[e]) & (inv < off[e + 1])).nonzero(as_tuple=True)
        r = inv[t, k].long()
        g, u, w = h[r, :N], h[r, N:], TW[t, k, None]
        da = G[t] @ w2[e]
        dh = w * torch.cat([da * u * slope(g), da * silu(g)], 1)
        dtw[t, k] = (silu(g) * u * da).sum(1)
        dw2[e] = (w * G[t]).T @ (silu(g) * u)
        dw13[e] = dh.T @ x[t]
        dx.index_add_(0, t, dh @ w13[e])
    return dx, dtw, dw13, dw2


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,Eg,El,topk,K,N", [(1, 8, 8, 2, 256, 128), (37, 8, 8, 2, 256, 128), (64, 8, 4, 3, 256, 128),
                                              (300, 8, 8, 1, 256, 128), (0, 8, 8, 2, 256, 128), (1, 32, 32, 8, 2048, 768),
                                              (500, 32, 16, 4, 2048, 768)])
def test_layer_with_a_checkpoint(keep, M, Eg, El, topk, K, N):
    """The output against the whole layer in 64 bits, the gradients against their formulas in 64 bits at the kept
    values: at most six bf16 roundings lie between, each linear, so 6 * 2^-8 in the 2-norm."""
    announce("layer with a checkpoint", keep, M, Eg, El, topk, K, N)
    layer = make_layer(M + 1, keep, Eg, El, K, N)
    if K == 2048:
        layer.w13.div_(4), layer.w2.div_(2)   # activations of order one
    x, ids, tw, dout = base.batch(M + 2, M, K, Eg, topk)
    out, saved = layer.forward(x, ids, tw)
    dx, dtw = layer.backward(dout, saved)
    torch.cuda.synchronize()
    full = base.layer_ref_by_expert(layer, x, ids, tw, dout) if M else [torch.zeros_like(t.cpu().double()) for t in
                                                                       (out, dx, dtw, layer.grad_w13, layer.grad_w2)]
    assert base.rel(out, full[0]) <= 6 * 2.0 ** -8
    for got, want, what in zip((dx, dtw, layer.grad_w13, layer.grad_w2), grads_at(layer, saved, tw, dout),
                               ("dx", "dtw", "dw13", "dw2")):
        assert got.shape == want.shape and base.rel(got, want) <= 6 * 2.0 ** -8, (what, base.rel(got, want))
    if keep == "e4m3":
        c, s, _ = encode(x.cpu().double())
        assert torch.equal(saved.x.cpu(), c) and torch.equal(saved.x_s.cpu(), s)
    else:   # nothing but roundings to bf16 lies between these gradients and the layer's own
        for got, want, what in zip((dx, dtw, layer.grad_w13, layer.grad_w2), full[1:], ("dx", "dtw", "dw13", "dw2")):
            assert base.rel(got, want) <= 6 * 2.0 ** -8, (what, base.rel(got, want))
    # what is kept makes no difference to the output, nor does keeping nothing
    other = make_layer(M + 1, "bf16" if keep == "e4m3" else "e4m3", Eg, El, K, N)
    other.w13.copy_(layer.w13), other.w2.copy_(layer.w2)
    assert torch.equal(out, other.forward(x, ids, tw)[0]) and torch.equal(out, layer.infer(x, ids, tw))


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
def test_layer_checkpoint_interleaved_and_repeated(keep):
    """Two forwards before their backwards equal one after the other, bit for bit; a backward run twice adds twice."""
    b1, b2 = base.batch(1, 40), base.batch(2, 23)
    l1, l2 = make_layer(9, keep), make_layer(9, keep)
    o1, s1 = l1.forward(*b1[:3])
    o2, s2 = l1.forward(*b2[:3])
    g1, g2 = l1.backward(b1[3], s1), l1.backward(b2[3], s2)
    p1, t1 = l2.forward(*b1[:3])
    q1 = l2.backward(b1[3], t1)
    p2, t2 = l2.forward(*b2[:3])
    q2 = l2.backward(b2[3], t2)
    for a, b in ((o1, p1), (o2, p2), *zip(g1, q1), *zip(g2, q2), (l1.grad_w13, l2.grad_w13), (l1.grad_w2, l2.grad_w2)):
        assert torch.equal(a, b)
    again = l1.backward(b2[3], s2)
    assert all(torch.equal(a, b) for a, b in zip(again, g2))


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
def test_layer_checkpoint_on_another_stream(keep):
    layer = make_layer(3, keep)
    x, ids, tw, dout = base.batch(4, 50)
    want = base.explicit(layer, x, ids, tw, dout)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = base.explicit(layer, x, ids, tw, dout)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("leaves", ["x", "tw", "w13", "w2", "x tw w13 w2"])
def test_layer_checkpoint_through_autograd(keep, leaves):
    layer = make_layer(31, keep)
    x, ids, tw, dout = base.batch(32, 45)
    want = base.explicit(layer, x, ids, tw, dout)
    names = leaves.split()
    x, tw = (t.clone().requires_grad_(n in names) for t, n in ((x, "x"), (tw, "tw")))
    for n in ("w13", "w2"):
        getattr(layer, n).requires_grad_(n in names)
    out, rows = layer.forward(x * 1, ids, tw * 1)
    assert out.requires_grad and torch.equal(out, want[0])
    (out.t() * 1).backward(dout.t().contiguous())
    got = (out, x.grad, tw.grad, layer.grad_w13, layer.grad_w2)
    for a, b, n in zip(got, want, ("out", "x", "tw", "w13", "w2")):
        assert torch.equal(a, b) if a is not None else n not in names, n
    assert not layer.infer(x, ids, tw).requires_grad
    dx, dtw = layer.backward(dout, rows)
    assert torch.equal(dx, want[1]) and torch.equal(dtw, want[2])


@pytest.mark.parametrize("keep,what", [("bf16", "x"), ("bf16", "tw"), ("bf16", "w13"), ("e4m3", "w2"), ("e4m3", "tw")])
def test_layer_checkpoint_refuses_what_changed_before_the_backward(keep, what):
    layer = make_layer(38, keep)
    x, ids, tw, dout = base.batch(39, 9)
    layer.w2.requires_grad_()
    out, _ = layer.forward(x, ids, tw)
    with torch.no_grad():
        {"x": x, "tw": tw, "w13": layer.w13, "w2": layer.w2}[what].mul_(0.5)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.backward(dout)


def test_layer_8_bit_checkpoint_is_the_layers_own():
    """The caller may overwrite its tokens after the forward: the codes are the layer's."""
    layer = make_layer(48, "e4m3")
    x, ids, tw, dout = base.batch(49, 30)
    want = base.explicit(layer, x, ids, tw, dout)
    layer.w2.requires_grad_()
    out, _ = layer.forward(x, ids, tw)
    x.zero_()
    out.backward(dout)
    assert torch.equal(layer.grad_w13, want[3]) and torch.equal(layer.grad_w2, want[4])


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
def test_layer_checkpoint_in_a_graph(keep):
    """Forward, backward, clip and the forward alone captured while an eager graph of the same layer lives, replayed
    on new inputs with eager work between the replays."""
    layer, eager = make_layer(5, keep), make_layer(5, keep)
    layer.w13.requires_grad_()
    x, ids, tw, dout = base.batch(6, 48)
    alive = layer.forward(x, ids, tw)

    def step(l, *b):
        l.zero_grad()
        out, s = l._forward(*b[:3])
        dx, dt = l.backward(b[3], s)
        n = l.clip_gradients(0.5)
        return out, dx, dt, n, l.grad_w13, l.grad_w2, l.infer(*b[:3])

    def auto():
        layer.zero_grad()
        out, _ = layer.forward(x, ids, tw)
        out.backward(dout)
        return out.detach()

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step(layer, x, ids, tw, dout)
        auto()
    torch.cuda.current_stream().wait_stream(st)
    graphs = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graphs[0]):
        got = step(layer, x, ids, tw, dout)
    with torch.cuda.graph(graphs[1]):
        got_auto = auto()
    for seed in (6, 7, 8, 9):
        new = base.batch(seed, 48)
        for dst, src in zip((x, ids, tw, dout), new):
            dst.copy_(src)
        graphs[0].replay()
        torch.cuda.synchronize()
        want = step(eager, *new)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), seed
        graphs[1].replay()
        torch.cuda.synchronize()
        want = base.explicit(eager, *new)
        for a, b in zip((got_auto, layer.grad_w13, layer.grad_w2), (want[0], want[3], want[4])):
            assert torch.equal(a, b), seed
    assert alive[0].requires_grad


def test_layer_checkpoint_keeps_less():
    """Bytes kept of a forward call, by the formulas of the layer's documentation."""
    M, topk, K, N = 64, 8, 256, 128
    x, ids, tw, _ = base.batch(3, M, K, 8, topk)
    kept = {}
    for keep in (None, "bf16", "e4m3"):
        layer = make_layer(4, keep, K=K, N=N)
        _, s = layer.forward(x, ids, tw)
        cap = moe.moe_max_rows(M, topk, 8, layer.align)
        parts = (s.a_perm, s.h, s.act, s.y) if keep is None else (s.h, s.h_s, s.x_s) + ((s.x,) if keep == "e4m3" else ())
        kept[keep] = sum(t.numel() * t.element_size() for t in parts if t is not None)
        want = {None: cap * (4 * K + 6 * N), "bf16": cap * 4 * N, "e4m3": (cap * 2 * N + M * K) * 33 // 32}[keep]
        assert kept[keep] == want
    assert kept["e4m3"] < kept["bf16"] < kept[None]
