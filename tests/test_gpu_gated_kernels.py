"""The gated experts' operators at the border of their ranges, on each of their
kernels and side by side, on the GPU against plain 64-bit implementations.
Tolerances: as derived in test_gpu_gated_experts.py."""
import pytest
import torch

import unpermute_count_expert_amd as moe
from tests.gpu_helpers import announce
from tests.test_gpu_bf16_experts import BF, DEV, F64, I32, bf, gen, i32, segments, sentinel, valid_mask
from tests.test_gpu_gated_experts import (F8, check_codes, decode, encode, nearest_codes, rows_untouched, run_checkpoint,
                                          run_fwd, scale_bytes)

BORDER = 248 * 2.0 ** 120   # halfway between the last code that is finite at the largest scale and 2^128


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
    """Every entry point over every kernel's hints, with inputs and outputs of its own made beforehand: enqueue()
    calls the library alone."""

    def __init__(self, seed):
        g = gen(seed)
        cs, n, k, M, T, W = [170, 0, 3, 600, 65, 1000], 544, 1032, 700, 3, 2048
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
        assert (M // 2) * T <= cap
        table = dev(torch.randn((cap, 9), generator=g))
        self.out, self.steps = out, []
        add = lambda f, *args: self.steps.append(lambda: f(*args))
        for hint in (1, 300, 3000, 30000, 1 << 20):
            h, q, s = result(cap, 2 * n), result(cap, 2 * n, dtype=U), result(cap, n // 16, dtype=U)
            add(moe.moe_grouped_gemm_bf16_silu_mul, a, w13, O, Cn, result(cap, n), None, None, hint)
            add(moe.moe_grouped_gemm_bf16_silu_mul, a, w13, O, Cn, result(cap, n), h, None, hint)
            add(moe.moe_grouped_gemm_bf16_silu_mul, a, w13, O, Cn, result(cap, n), q, s, hint)
            add(moe.moe_grouped_gemm_bf16_dgrad_silu_mul, dy, w2, O, Cn, q, result(cap, 2 * n), result(cap, n), s, rw,
                result(cap, -(-n // 64), dtype=F), hint)
            add(moe.moe_grouped_gemm_bf16_dgrad_silu_mul, dy, w2, O, Cn, h, h, None, None, rw, None, hint)
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
        for j in order:   # in step, or two hints (five calls each) apart, so that different kernels meet
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
