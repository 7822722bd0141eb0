"""The gated experts' operators at the border of their ranges, on each of their
kernels and side by side, on the GPU against plain 64-bit implementations.
Tolerances: as derived in test_gpu_gated_experts.py."""
import pytest
import torch

import unpermute_count_expert_amd as moe
from tests import test_gpu_bf16_experts as base
from tests import test_gpu_gated_experts as whole
from tests.gpu_helpers import announce
from tests.test_gpu_bf16_experts import (BF, DEV, F64, I32, TINY, bf, gen, i32, poison, segments, sentinel, valid_mask)
from tests.test_gpu_gated_experts import (F8, at_16_bytes, bwd_reference, check_codes, decode, encode, kept_rows,
                                          nearest_codes, rows_untouched, run_checkpoint, run_fwd, scale_bytes, silu,
                                          within)

BORDER = 248 * 2.0 ** 120   # halfway between the last code that is finite at the largest scale and 2^128

# Rows of 40 experts, with which every kernel is reached by the rows given, at widths that end inside a tile and inside
# its parts of 64 and 32 columns
ROWS = [0, 1, 63, 64, 65, 16, 0, 128, 130, 3, 257, 2, 0, 300, 17] + [0, 5] * 12 + [31]
KERNELS = {"forward": ["16", "64 staggered", "128 staggered", "256 staggered", "256"], "backward": ["16", "64", "128", "256"]}
CASES = [(op, kernel) for op in KERNELS for kernel in KERNELS[op]]
N_OF, K_ODD = {"none": 1000, "bf16": 1000, "e4m3": 992}, 520


def hint_of(op, kernel, n, k, E=len(ROWS)):
    """The least power of 2^(1/8) rows for which the call takes the kernel."""
    at = (moe.MOE_GEMM_BF16_SILU_MUL, E, n, k) if op == "forward" else (moe.MOE_GEMM_BF16_DGRAD_SILU_MUL, E, k, n)
    for i in range(31 * 8):
        p = moe.moe_grouped_gemm_bf16_plan_info(*at, int(2 ** (i / 8)))
        if f"{p['tile_rows']}{' staggered' if p['staggered'] else ''}" == kernel:
            return int(2 ** (i / 8))
    raise AssertionError(f"no rows give {kernel} for {op} of {at}")


# ---- 8 bits at the end of the range -----------------------------------------------------
@pytest.mark.parametrize("beside", [0, 1, 31])
def test_checkpoint_bound_for_every_finite_bf16(beside):
    """Every finite bf16 value, alone in its block, next to another one or among 31 others, comes back within the
    documented bound; from the border on as an infinity of its sign, which leaves the rest of its block finite."""
    announce("checkpoint bound", beside)
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF)
    v = bits[torch.isfinite(bits.float())]
    x = torch.zeros(len(v), 32, dtype=BF)
    x[:, 9] = v
    g = gen(beside)
    for j in range(beside):
        x[:, j if j < 9 else j + 1] = v[torch.randperm(len(v), generator=g)]
    q, s = run_checkpoint(x)
    out = sentinel(x.shape)
    moe.moe_checkpoint_restore(q, s, out)
    out, x64 = out.cpu().double(), x.double()
    past = x64.abs() >= BORDER
    assert past.any() and torch.equal(out[past], float("inf") * x64[past].sign())
    scale = torch.exp2(s.cpu().double() - 127).expand(-1, 32)
    assert (s.cpu() != 255).all() and torch.isfinite(out[~past]).all()
    err = (out - x64).abs()
    assert (err[~past] <= torch.maximum(2.0 ** -4 * x64.abs(), 2.0 ** -10 * scale)[~past]).all()


@pytest.mark.parametrize("hint", [1, 300, 5000, 1 << 20])
def test_gated_codes_at_the_border(hint):
    """Gate and up sums about the border, and past bf16's range in fp32: the definition's codes from every kernel."""
    announce("codes at the border", hint)
    cs, n, k = [70, 3, 300], 64, 72
    off, cap = segments(cs, 16)
    mask = valid_mask(cs, off, cap)
    g = gen(hint)
    a, w13 = torch.zeros(cap, k, dtype=BF), torch.zeros(3, 2 * n, k, dtype=BF)
    a[:, 5] = 1
    a[::2, 40] = 1
    top = torch.tensor([0, 1, 100, 240, 247, 248, 249, 255], dtype=F64) * 2.0 ** 120
    w13[:, :, 5] = (top[torch.randint(0, 8, (3, 2 * n), generator=g)] *
                    (2.0 * torch.randint(0, 2, (3, 2 * n), generator=g) - 1)).to(BF)
    w13[:, :32, 5] = 2.0 ** 100   # blocks without large ones
    w13[:, :, 40] = (w13[:, :, 5].double().sign() * 0.875 * 2.0 ** 120).to(BF)
    w13[:, :32, 40] = 0
    ref = torch.zeros(cap, 2 * n, dtype=F64)   # two terms at most, whose sum fp32 holds exactly
    for e, c in enumerate(cs):
        r = slice(off[e], off[e] + c)
        ref[r] = a[r].double() @ w13[e].double().T
    assert float(ref.abs().max()) == 255.875 * 2.0 ** 120
    _, h, h_s = run_fwd(a, w13, off, cs, "e4m3", hint)
    assert rows_untouched(h, h_s, mask)
    check_codes(h[mask.to(DEV)], h_s[mask.to(DEV)], ref[mask], "codes")
    q, s, _ = encode(ref[mask])
    out = sentinel((int(mask.sum()), 2 * n))
    moe.moe_checkpoint_restore(h[mask.to(DEV)], h_s[mask.to(DEV)], out)
    assert torch.equal(out.cpu().double(), torch.where(ref[mask].abs() >= BORDER, float("inf") * ref[mask].sign(),
                                                       decode(q, s)))


@pytest.mark.parametrize("hint", [1, 300, 5000, 1 << 20])
@pytest.mark.parametrize("n,k", [(32, 72), (160, 136), (288, 1032)])
def test_gated_codes_differ_only_at_borders(n, k, hint):
    """The code of a sum is the nearest one of a value within the sum's fp32 error, under the scale of a largest
    magnitude within it, and the same in every run."""
    announce("codes at borders", n, k, hint)
    cs = [63, 0, 65, 1, 130, 290]
    off, cap = segments(cs, 16)
    mask = valid_mask(cs, off, cap)
    g = gen(n + k)
    a, w13 = bf((cap, k), g), bf((len(cs), 2 * n, k), g, 4 * k ** -0.5)
    _, h, h_s = run_fwd(a, w13, off, cs, "e4m3", hint)
    _, h2, h_s2 = run_fwd(a, w13, off, cs, "e4m3", hint)
    assert torch.equal(h, h2) and torch.equal(h_s, h_s2)
    ref, err = torch.zeros(cap, 2 * n, dtype=F64), torch.zeros(cap, 2 * n, dtype=F64)
    for e, c in enumerate(cs):
        r = slice(off[e], off[e] + c)
        ae, we = a[r].double(), w13[e].double()
        ref[r], err[r] = ae @ we.T, k * 2.0 ** -23 * (ae.abs() @ we.abs().T)
    ref, err, q, s = ref[mask], err[mask], h.cpu()[mask], h_s.cpu()[mask].int()
    low = (ref.abs() - err).clamp(min=0)
    assert (scale_bytes(low).int() <= s).all() and (s <= scale_bytes(ref.abs() + err).int()).all()
    scale = torch.exp2(s.double() - 127).repeat_interleave(32, -1)
    nearest = lambda v: nearest_codes((v / scale).clamp(-448, 448)).view(F8).double()
    got = q.view(F8).double()
    assert (nearest(ref - err) <= got).all() and (got <= nearest(ref + err)).all()


# ---- side by side -----------------------------------------------------------------------
class Calls:
    """Every entry point and each of its kernels, with inputs and outputs made beforehand: the steps call the library
    alone."""

    def __init__(self, seed):
        g = gen(seed)
        cs, n, k, M, T, W = ROWS, 992, 520, 700, 3, 2048
        off, cap = segments(cs, 16)
        E, out = len(cs), []

        def dev(t):
            return t.to(DEV)

        def result(*shape, dtype=BF):
            out.append(torch.zeros(shape, dtype=dtype, device=DEV))
            return out[-1]
        U, F = torch.uint8, torch.float32
        O, Cn = i32(off), i32(cs)
        a, w13, dy, w2 = (dev(bf(s, g)) for s in ((cap, k), (E, 2 * n, k), (cap, k), (E, k, n)))
        rw, x, tw = dev(torch.rand(cap, generator=g)), dev(bf((M, W), g)), dev(torch.rand((M, T), generator=g))
        inv = dev(torch.randperm(cap, generator=g)[torch.arange(M * T) % cap].reshape(M, T).to(I32))
        inv[M // 2:] = -1   # a row belongs to one pair
        assert M // 2 * T <= cap
        table = dev(torch.randn((cap, 16), generator=g))
        self.out, self.steps = out, []
        add = lambda f, *args: self.steps.append(lambda: f(*args))
        up, down = ([hint_of(op, kernel, n, k) for kernel in KERNELS[op]] for op in ("forward", "backward"))
        for i, hint in enumerate(up):
            back = down[i % len(down)]
            h, q, s = result(cap, 2 * n), result(cap, 2 * n, dtype=U), result(cap, n // 16, dtype=U)
            add(moe.moe_grouped_gemm_bf16_silu_mul, a, w13, O, Cn, result(cap, n), None, None, hint)
            add(moe.moe_grouped_gemm_bf16_silu_mul, a, w13, O, Cn, result(cap, n), h, None, hint)
            add(moe.moe_grouped_gemm_bf16_silu_mul, a, w13, O, Cn, result(cap, n), q, s, hint)
            add(moe.moe_grouped_gemm_bf16_dgrad_silu_mul, dy, w2, O, Cn, q, result(cap, 2 * n), result(cap, n), s, rw,
                result(cap, -(-n // 64), dtype=F), back)
            add(moe.moe_grouped_gemm_bf16_dgrad_silu_mul, dy, w2, O, Cn, h, h, None, None, rw, None, back)
        xq, xs = result(M, W, dtype=U), result(M, W // 32, dtype=U)
        add(moe.moe_checkpoint, x, xq, xs)
        add(moe.moe_checkpoint_restore, xq, xs, result(cap, W), inv)
        add(moe.moe_permute_rows, x, inv, result(cap, W), tw, result(cap, dtype=F))
        add(moe.moe_topk_weights_bwd, table, inv, result(M, T, dtype=F))

    def clear(self):
        for t in self.out:
            t.zero_()


def test_gated_entry_points_of_two_streams_in_flight_together():
    """Two streams held back until both are filled: their kernels run beside each other and give the bits of each
    alone."""
    work = [Calls(71), Calls(72)]
    want = []
    for w in work:
        for step in w.steps:
            step()
        torch.cuda.synchronize()
        want.append([t.clone() for t in w.out])
    streams = [torch.cuda.Stream() for _ in work]
    big = torch.ones(1 << 28, device=DEV)
    for turn in range(4):
        for w in work:
            w.clear()
        torch.cuda.synchronize()
        for _ in range(40):   # some milliseconds, in which the host fills both streams
            big.mul_(1.0)
        held = torch.cuda.Event()
        held.record()
        span = [[torch.cuda.Event(enable_timing=True) for _ in range(2)] for _ in work]
        for st, ev in zip(streams, span):
            st.wait_event(held)
            ev[0].record(st)
        order = range(len(work[0].steps))
        for j in order:   # in step, or two kernels (five calls each) apart, so that different kernels meet
            for w, st, at in zip(work, streams, (j, j if turn % 2 else (j + 10) % len(order))):
                with torch.cuda.stream(st):
                    w.steps[at]()
        filled_early = not held.query()
        for st, ev in zip(streams, span):
            ev[1].record(st)
        torch.cuda.synchronize()
        assert filled_early, "the streams ran while they were filled"
        assert span[0][0].elapsed_time(span[1][1]) > 0 and span[1][0].elapsed_time(span[0][1]) > 0
        for w, ref in zip(work, want):
            for i, (t, r) in enumerate(zip(w.out, ref)):
                assert torch.equal(t.view(torch.uint8), r.view(torch.uint8)), (turn, i)


# ---- each kernel -------------------------------------------------------------------------
class Guarded:
    """Tensors inside larger ones, whose margins (4 KB on either side) nothing writes."""

    def __init__(self):
        self.all = []

    def __call__(self, *shape, dtype=BF):
        size = torch.empty(0, dtype=dtype).element_size()
        whole = torch.full((torch.Size(shape).numel() * size + 8192,), 0x7b, dtype=torch.uint8, device=DEV)
        self.all.append(whole)
        return whole[4096:-4096].view(dtype).view(shape)

    def intact(self):
        return all(bool((w[:4096] == 0x7b).all() and (w[-4096:] == 0x7b).all()) for w in self.all)


def outputs(op, keep, cap, n, new):
    U, F = torch.uint8, torch.float32
    if op == "backward":
        return [new(cap, 2 * n), new(cap, n), new(cap, -(-n // 64), dtype=F)]
    kept = {"none": [], "bf16": [new(cap, 2 * n)], "e4m3": [new(cap, 2 * n, dtype=U), new(cap, n // 16, dtype=U)]}[keep]
    return [new(cap, n)] + kept


def call(op, rows, w, off, cs, out, hint, kept=(None, None), weights=None):
    if op == "forward":
        moe.moe_grouped_gemm_bf16_silu_mul(rows, w, off, cs, *out, rows_hint=hint)
    else:
        moe.moe_grouped_gemm_bf16_dgrad_silu_mul(rows, w, off, cs, kept[0], out[0], out[1], kept[1], weights, out[2], hint)


def inputs(op, keep, cap, n, g, E=len(ROWS)):
    """(rows, weights of the experts, kept gate and up rows with scales, router weights) on the GPU; small integers in
    the products, whose sums fp32 holds exactly, so that every kernel gives the same bits."""
    ints = lambda *s: torch.randint(-2, 3, s, generator=g).to(BF)
    rows = ints(cap, K_ODD).to(DEV)
    if op == "forward":
        return rows, ints(E, 2 * n, K_ODD).to(DEV), (None, None), None
    h = bf((cap, 2 * n), g, 3.0)
    if keep == "e4m3":
        q, s, _ = encode(h.double())
        kept = q.to(DEV), s.to(DEV)
    else:
        kept = h.to(DEV), None
    return rows, ints(E, K_ODD, n).to(DEV), kept, (torch.rand(cap, generator=g) + 0.5).to(DEV)


def equal_rows(x, y, mask):
    m = mask.to(DEV)
    return all(torch.equal(a[m].view(torch.uint8), b[m].view(torch.uint8)) for a, b in zip(x, y))


KEEPS = {"forward": ("none", "bf16", "e4m3"), "backward": ("bf16", "e4m3")}


@pytest.mark.parametrize("op,kernel,keep", [(*c, keep) for c in CASES for keep in KEEPS[c[0]]])
def test_each_kernel_at_odd_widths(op, kernel, keep):
    """Random rows at widths that end inside a tile, NaN in the rows of no expert, against 64 bits; margins intact."""
    announce("each kernel", op, kernel, keep)
    n, k, new, cs = N_OF[keep], K_ODD, Guarded(), ROWS
    hint = hint_of(op, kernel, n, k)
    off, cap = segments(cs, 16)
    mask = valid_mask(cs, off, cap)
    g = gen(int(kernel.split()[0]) + n)
    out = outputs(op, keep, cap, n, new)
    O, Cn, E = i32(off), i32(cs), len(cs)
    if op == "forward":
        a, w = bf((cap, k), g), bf((E, 2 * n, k), g, 4 * k ** -0.5)
        call(op, poison(a, mask).to(DEV), w.to(DEV), O, Cn, out, hint)
    else:
        a, w = bf((cap, k), g, 0.5), bf((E, k, n), g, k ** -0.5)
        H, HS, h = kept_rows(cap, n, keep, g, mask)
        rw = torch.rand(cap, generator=g) * 2 - 0.5
        RW = torch.where(mask, rw, float("nan"))
        call(op, poison(a, mask).to(DEV), w.to(DEV), O, Cn, out, hint, (H, HS), RW.to(DEV))
    torch.cuda.synchronize()
    assert new.intact()
    for t in out:
        assert (t.cpu()[~mask].view(torch.uint8) == 0x7b).all()
    nd = -(-n // 64)
    for e, c in enumerate(cs):
        if c == 0:
            continue
        r = slice(off[e], off[e] + c)
        ae, we = a[r].double(), w[e].double().T if op == "forward" else w[e].double()
        ref, err = ae @ we, k * 2.0 ** -23 * (ae.abs() @ we.abs())
        if op == "backward":
            b = bwd_reference(h[r], ref, err, rw[r].double(), n)
            for name, got in (("act", out[1][r]), ("dg", out[0][r, :n]), ("du", out[0][r, n:])):
                v, tol = b[name]
                within(got, v, tol + 2.0 ** -8 * (v.abs() + tol) + TINY, name)
            v, tol = b["dot"]
            pad = lambda t: torch.nn.functional.pad(t, (0, nd * 64 - n)).reshape(c, nd, 64)
            within(out[2][r], pad(v).sum(-1), pad(tol).sum(-1) + 64 * 2.0 ** -23 * pad(v.abs() + tol).sum(-1) + TINY, "dots")
            continue
        gr, ur, ge, ue = ref[:, :n], ref[:, n:], err[:, :n], err[:, n:]
        want = silu(gr) * ur
        tol = 1.1 * ge * ur.abs() + silu(gr).abs() * ue + 1.1 * ge * ue
        within(out[0][r], want, tol + (2.0 ** -8 + 2.0 ** -22 * (4 + gr.abs())) * (want.abs() + tol) + TINY, "act")
        if keep == "bf16":
            within(out[1][r], ref, err + 2.0 ** -8 * (ref.abs() + err) + TINY, "h")
        if keep == "e4m3":
            scale = ((ref.abs() + err).reshape(c, -1, 32).amax(-1) / 224).repeat_interleave(32, -1)
            within(decode(out[1][r].cpu(), out[2][r].cpu()), ref,
                   err + torch.maximum(2.0 ** -4 * (ref.abs() + err), 2.0 ** -10 * scale), "h in 8 bits")


@pytest.mark.parametrize("op,keep", [(op, keep) for op in KERNELS for keep in KEEPS[op]])
def test_kernels_agree_where_sums_are_exact(op, keep):
    """Sums that fp32 holds exactly: the same bits from every kernel, from calls with other rows given that take the
    same one, and from tensors that start 16 bytes into a line."""
    announce("kernels agree", op, keep)
    n = N_OF[keep]
    off, cap = segments(ROWS, 16)
    mask = valid_mask(ROWS, off, cap)
    rows, w, kept, weights = inputs(op, keep, cap, n, gen(n))
    O, Cn, first = i32(off), i32(ROWS), None
    for kernel in KERNELS[op]:
        hint, new = hint_of(op, kernel, n, K_ODD), Guarded()
        out = outputs(op, keep, cap, n, new)
        call(op, rows, w, O, Cn, out, hint, kept, weights)
        first = first or out
        if op == "backward":   # the sums of 64 columns' products are rounded: in each kernel's order
            assert equal_rows(out[:2], first[:2], mask)
        else:
            assert equal_rows(out, first, mask)
        moved = [t if t is None else at_16_bytes(t) for t in (rows, w, O, Cn, *kept, weights)]
        there = [at_16_bytes(t) for t in outputs(op, keep, cap, n, new)]
        call(op, *moved[:4], there, hint, tuple(moved[4:6]), moved[6])
        assert all(t.data_ptr() % 256 == 16 for t in there) and equal_rows(out, there, mask) and new.intact()


def cut_rows(off, cs, cap):
    """The rows of each expert as documented: its segment cut at the next one's start and at the buffer."""
    rows = []
    for e, c in enumerate(cs):
        end = min(max(off[e + 1], 0), cap)
        lo = min(max(off[e], 0), end)
        rows.append(range(lo, min(lo + max(c, 0), end)))
    return rows


@pytest.mark.parametrize("op,kernel,keep", [(*c, keep) for c in CASES for keep in ("bf16", "e4m3")])
def test_each_kernel_cuts_inconsistent_segments(op, kernel, keep):
    """Counts past their slot, negative counts and offsets out of order or past the buffer: rows outside every segment
    and the memory around the outputs stay as they are, and segments that do not overlap have their values."""
    announce("cut segments", op, kernel, keep)
    n, E = N_OF[keep], len(ROWS)
    hint = hint_of(op, kernel, n, K_ODD)
    off, cap = segments(ROWS, 16)
    rows, w, kept, weights = inputs(op, keep, cap, n, gen(n + 1))

    def run(o, c):
        new = Guarded()
        out = outputs(op, keep, cap, n, new)
        call(op, rows, w, i32(o), i32(c), out, hint, kept, weights)
        torch.cuda.synchronize()
        assert new.intact()
        named = torch.zeros(cap, dtype=torch.bool)
        for r in cut_rows(o, c, cap):
            named[r.start:r.stop] = True
        for t in out:
            assert (t.cpu()[~named].view(torch.uint8) == 0x7b).all()
        return out, named

    long = [c if e % 3 else 1 << 20 for e, c in enumerate(ROWS)]
    long[4], long[8] = -3, -(1 << 31)
    got, named = run(off, long)
    plain, same = run(off, [len(r) for r in cut_rows(off, long, cap)])
    assert torch.equal(named, same) and equal_rows(got, plain, named)
    run([-7] + [cap + 5] * 20 + [40] * 20, [200] * E)
    run([500 * (e % 3) - 9 * e for e in range(E + 1)], ROWS)
    run([cap - 3 + e // 20 for e in range(E + 1)], [1 << 30] * E)


@pytest.mark.parametrize("op,kernel,keep", [(*c, keep) for c in CASES for keep in ("bf16", "e4m3")])
def test_each_kernel_keeps_non_finite_values_in_their_rows(op, kernel, keep):
    announce("non-finite", op, kernel, keep)
    n = N_OF[keep]
    hint = hint_of(op, kernel, n, K_ODD)
    off, cap = segments(ROWS, 16)
    mask = valid_mask(ROWS, off, cap)
    rows, w, kept, weights = inputs(op, keep, cap, n, gen(n + 2))
    bad = [off[3] + 40, off[10] + 256, off[13] + 128, off[1]]   # inside a tile, an expert's last row, its only one
    out = outputs(op, keep, cap, n, Guarded())
    call(op, rows, w, i32(off), i32(ROWS), out, hint, kept, weights)
    planted = rows.clone()
    for i, b in enumerate(bad):
        planted[b, (5, 519, 100, 0)[i]] = float("inf") if i % 2 else float("nan")
    planted[~mask.to(DEV)] = float("nan")
    if op == "backward":   # the kept rows of no expert as well
        h, h_s = kept[0].clone(), kept[1]
        if keep == "bf16":
            h[~mask.to(DEV)] = float("nan")
        else:
            h_s = h_s.clone()
            h_s[~mask.to(DEV)] = 255
        kept = h, h_s
    got = outputs(op, keep, cap, n, Guarded())
    call(op, planted, w, i32(off), i32(ROWS), got, hint, kept, weights)
    clean = mask.clone()
    clean[bad] = False
    assert equal_rows(got, out, clean)
    what = got[0] if op == "backward" else got[2] if keep == "e4m3" else got[1]
    marked = what.cpu()[bad] == 255 if what.dtype == torch.uint8 else ~torch.isfinite(what.cpu()[bad].float())
    assert marked.any(1).all()


@pytest.mark.parametrize("up,down", [("64 staggered", "64"), ("128 staggered", "128"), ("256 staggered", "128")])
def test_each_kernel_past_32_bits(up, down):
    """test_gated_past_32_bits with rows given that take these kernels (its own take the others)."""
    at = 140, 2048, 4096
    rows = {hint_of("forward", up, *at[1:], at[0]), hint_of("backward", down, *at[1:], at[0])}
    name = lambda p: f"{p['tile_rows']}{' staggered' if p['staggered'] else ''}"
    hint = max(rows)   # both kernels' ranges have begun: the first one's has not ended
    assert name(moe.moe_grouped_gemm_bf16_plan_info(moe.MOE_GEMM_BF16_SILU_MUL, *at, hint)) == up
    assert name(moe.moe_grouped_gemm_bf16_plan_info(moe.MOE_GEMM_BF16_DGRAD_SILU_MUL, 140, 4096, 2048, hint)) == down
    whole.test_gated_past_32_bits(hint)


@pytest.mark.parametrize("kernel", KERNELS["backward"])
def test_each_kernel_in_place_with_every_output(kernel):
    """dh in h's place beside act, dots and router weights: the bits of the call that keeps h."""
    n = N_OF["bf16"]
    off, cap = segments(ROWS, 16)
    mask = valid_mask(ROWS, off, cap)
    g = gen(n + 3)
    rows, w = bf((cap, K_ODD), g).to(DEV), bf((len(ROWS), K_ODD, n), g, K_ODD ** -0.5).to(DEV)
    h, weights = bf((cap, 2 * n), g, 3.0).to(DEV), torch.rand(cap, generator=g).to(DEV)
    hint, new = hint_of("backward", kernel, n, K_ODD), Guarded()
    want, got = outputs("backward", "bf16", cap, n, new), outputs("backward", "bf16", cap, n, new)
    call("backward", rows, w, i32(off), i32(ROWS), want, hint, (h, None), weights)
    got[0].copy_(h)
    call("backward", rows, w, i32(off), i32(ROWS), got, hint, (got[0], None), weights)
    assert equal_rows(got, want, mask) and new.intact()
    assert torch.equal(got[0][~mask.to(DEV)], h[~mask.to(DEV)])


# ---- the layer ----------------------------------------------------------------------------
@pytest.mark.parametrize("keep", [None, "bf16", "e4m3"])
def test_layer_from_buffers_of_nan(keep):
    """Every buffer that the layer takes starts as NaN (codes and scales as 255): the same bits."""
    x, ids, tw, dout = base.batch(52, 37, topk=3)
    want = base.explicit(whole.make_layer(51, keep, El=5), x, ids, tw, dout)
    before = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)   # fills what torch.empty gives
    try:
        assert torch.isnan(torch.empty(5, device=DEV)).all()
        layer = whole.make_layer(51, keep, El=5)
        got = base.explicit(layer, x, ids, tw, dout)
        alone = layer.infer(x, ids, tw)
    finally:
        torch.use_deterministic_algorithms(before)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    if keep is not None:
        assert torch.equal(alone, want[0])


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
def test_layer_without_rows_of_its_own(keep):
    """Every token goes to experts elsewhere: zeros, and the weights' gradients stay."""
    layer = whole.make_layer(53, keep, El=4)
    x, ids, tw, dout = base.batch(54, 20)
    ids = ids % 4   # the last four of eight are here
    layer.grad_w13.fill_(2), layer.grad_w2.fill_(3)
    out, saved = layer.forward(x, ids, tw)
    for t in (out, *layer.backward(dout, saved), layer.infer(x, ids, tw)):
        assert not t.any()
    assert (layer.grad_w13 == 2).all() and (layer.grad_w2 == 3).all()


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
def test_layer_with_an_expert_picked_twice(keep):
    """A token that picks one expert twice has two rows there, and pairs without an expert (-1) none: the output
    against 64 bits, the gradients against their formulas at the kept values (six bf16 roundings, as in
    test_layer_with_a_checkpoint)."""
    layer = whole.make_layer(55, keep)
    x, ids, tw, dout = base.batch(56, 60, topk=4)
    ids[::2, 1] = ids[::2, 0]
    ids[::3, 2] = ids[::3, 0]
    ids[::5, 3] = -1
    out, saved = layer.forward(x, ids, tw)
    dx, dtw = layer.backward(dout, saved)
    assert (dtw[::5, 3] == 0).all()
    d = lambda t: t.cpu().double()
    want = torch.zeros(x.shape, dtype=F64)
    for t, picks in enumerate(ids.tolist()):
        for j, e in enumerate(picks):
            if e >= 0:
                h = d(layer.w13[e]) @ d(x[t])
                want[t] += d(tw[t, j]) * (d(layer.w2[e]) @ (silu(h[:layer.N]) * h[layer.N:]))
    assert base.rel(out, want) <= 6 * 2.0 ** -8
    for got, ref, what in zip((dx, dtw, layer.grad_w13, layer.grad_w2), whole.grads_at(layer, saved, tw, dout),
                              ("dx", "dtw", "dw13", "dw2")):
        assert base.rel(got, ref) <= 6 * 2.0 ** -8, (what, base.rel(got, ref))
