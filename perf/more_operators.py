"""The gated experts' fused operators and their 8-bit activation checkpoints as
measured work: the gate and up products with SiLU-mul in one kernel, the same
in training with what the backward pass needs (bf16, or 8 bits with a
power-of-two scale for every 32 values), the backward pass from it with the
router weights' gradient, and tokens kept in 8 bits and restored in expert
order.

`own` False: the plain form, elementary torch operations in 32 bits, rounded
once at the end.  `own` True: the calls of unpermute_count_expert_amd.  Shapes
are those of the layer configurations in generators.py (hidden 2048, expert
intermediate 768, 128 experts, top-8) and of the tests' odd layers (hidden
2176, 300 tokens, 130 tokens, align 16).
"""
import math

import torch

own = False
DEV = "cuda"
BF = torch.bfloat16
F8 = torch.float8_e4m3fn
BLOCK = 32   # values that share a scale


def listed():
    return [
        # one decoding step of one sequence: 8 routed rows, weight bandwidth and latency
        dict(name="gated_1_token", op="gated", tokens=1, topk=8, experts=128, local=128, routing="uniform", n=768,
             k=2048, align=16, keep="none"),
        # a short fine-tuning batch on one of two expert-parallel ranks, skewed routing, odd widths, gate and up kept
        dict(name="gated_300_tokens", op="gated", tokens=300, topk=8, experts=128, local=64, routing="zipf", n=1000,
             k=2176, align=16, keep="bf16"),
        # a large prefill: nothing is kept
        dict(name="gated_16384_tokens", op="gated", tokens=16384, topk=8, experts=128, local=128, routing="uniform",
             n=768, k=2048, align=128, keep="none"),
        # forward and backward of a ragged chunk through an 8-bit checkpoint
        dict(name="train_130_tokens", op="train", tokens=130, topk=8, experts=128, local=64, routing="zipf", n=672,
             k=2176, align=128, keep="e4m3"),
        # a training batch with hot experts, gate and up kept in bf16
        dict(name="train_4096_tokens", op="train", tokens=4096, topk=8, experts=128, local=128, routing="hot", n=768,
             k=2048, align=128, keep="bf16"),
        # a large training batch, 8-bit checkpoint
        dict(name="train_16384_tokens", op="train", tokens=16384, topk=8, experts=128, local=128, routing="uniform",
             n=768, k=2048, align=128, keep="e4m3"),
        # the backward pass from the layer's output gradient to the gate's and the router weights', ragged, odd widths
        dict(name="gated_bwd_130_tokens", op="gated_bwd", tokens=130, topk=8, experts=128, local=64, routing="zipf",
             n=1000, k=2176, align=16, keep="bf16"),
        # and of a large batch from its 8-bit checkpoint
        dict(name="gated_bwd_16384_tokens", op="gated_bwd", tokens=16384, topk=8, experts=128, local=128,
             routing="uniform", n=768, k=2048, align=128, keep="e4m3"),
        # a ragged chunk's tokens into 8 bits and back, into expert order
        dict(name="checkpoint_130_tokens", op="checkpoint", tokens=130, topk=8, experts=128, local=64, routing="zipf",
             k=2176, align=128),
        # and a large batch's
        dict(name="checkpoint_16384_tokens", op="checkpoint", tokens=16384, topk=8, experts=128, local=128,
             routing="uniform", k=2048, align=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "train", "gated_bwd", "checkpoint"])
    experts = rng.choice([8, 32, 60, 128])
    c = dict(op=op, tokens=_log(rng, 1, 12000), topk=rng.choice([1, 2, 4, 6, 8]), experts=experts,
             local=rng.choice([experts, experts // 2]), routing=rng.choice(["uniform", "zipf", "hot"]),
             align=rng.choice([16, 32, 64, 128]))
    if c["routing"] == "zipf":
        c["tokens"] = min(c["tokens"], 4096)   # one expert takes a large share; its plain form is padded to it
    c["k"] = 128 * _log(rng, 1, 16)
    if op != "checkpoint":
        c["keep"] = rng.choice(["none", "bf16"] if op == "gated" else ["bf16", "e4m3"])
        c["n"] = 32 * _log(rng, 2, 32) if c["keep"] == "e4m3" else 8 * _log(rng, 8, 128)
    return c


# ---- inputs ---------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1_000_003 * int(seed) + 17)
    return g


def _route(c, g):
    """Router picks: distinct experts per token, weights renormalised over the picks."""
    E, M, T = c["experts"], c["tokens"], c["topk"]
    logit = torch.randn(M, E, device=DEV, generator=g)
    rank = torch.randperm(E, device=DEV, generator=g).float()
    if c["routing"] == "zipf":
        logit = logit * 1.28 - 1.2 * torch.log1p(rank)
    elif c["routing"] == "hot":
        logit = logit + 1.6 * (rank < max(1, E // 10))
    top, ids = torch.topk(logit, T, dim=1)
    return ids.to(torch.int32), torch.softmax(top, dim=1).contiguous()


def _max_rows(c):
    pairs = c["tokens"] * c["topk"]
    return pairs + min(c["local"], pairs) * (c["align"] - 1)


def _rows(c, g):
    """Routing of one batch and its expert segments, as the permute lays them out: stable, padded to align."""
    ids, tw = _route(c, g)
    E, L, T, A, cap = c["experts"], c["local"], c["topk"], c["align"], _max_rows(c)
    key = (ids.long() - (E - L)).reshape(-1)   # the last L experts are here
    key = torch.where(key < 0, L, key)
    order = torch.sort(key, stable=True).indices
    hist = torch.zeros(L + 1, dtype=torch.int64, device=DEV).scatter_add_(0, key, torch.ones_like(key))
    counts = hist[:L]
    offsets = torch.zeros(L + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum((counts + A - 1) // A * A, 0)
    first = torch.cumsum(hist, 0) - hist
    ks = key[order]
    row = torch.where(ks < L, offsets[ks.clamp(max=L - 1)] + torch.arange(key.numel(), device=DEV) - first[ks], -1)
    inv = torch.empty_like(key).scatter_(0, order, row)
    src = torch.full((cap + 1,), -1, dtype=torch.int64, device=DEV)
    src.scatter_(0, torch.where(row < 0, cap, row), torch.where(row < 0, -1, order // T))
    i32 = torch.int32
    return dict(tw=tw, counts=counts.to(i32), offsets=offsets.to(i32), inv=inv.view(-1, T).to(i32),
                src=src[:cap].to(i32), longest=max(1, int(counts.max())), cap=cap)


def _randn(shape, g, scale=1.0, dtype=BF):
    return torch.randn(shape, device=DEV, generator=g).mul_(scale).to(dtype)


def _padding(t, src, value=float("nan")):
    """Rows that belong to no expert hold whatever was there: NaN here."""
    t.masked_fill_((src < 0)[:, None], value)
    return t


def _zeros(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype, device=DEV)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=dict(c))
    r = _rows(c, g)
    s.update(r)
    cap, M, L, T, k = r["cap"], c["tokens"], c["local"], c["topk"], c["k"]
    if c["op"] == "checkpoint":
        s["x"] = _randn((M, k), g) * torch.exp(_randn((M, 1), g, 0.5, torch.float32)).to(BF)   # tokens differ in size
        s["q"], s["q_s"] = _zeros(M, k, dtype=torch.uint8), _zeros(M, k // BLOCK, dtype=torch.uint8)
        s["a"] = _zeros(cap, k)
        return s
    n, e4m3 = c["n"], c["keep"] == "e4m3"
    if c["op"] in ("gated", "train"):
        s["w13"] = _randn((L, 2 * n, k), g, 0.02)
        s["a"] = _padding(_randn((cap, k), g), r["src"])
        s["act"] = _zeros(cap, n)
        if c["keep"] != "none":
            s["h"] = _zeros(cap, 2 * n, dtype=torch.uint8 if e4m3 else BF)
            s["h_s"] = _zeros(cap, 2 * n // BLOCK, dtype=torch.uint8) if e4m3 else None
    if c["op"] == "train":
        s["dy"] = _padding(_randn((cap, k), g, 0.1), r["src"])
    if c["op"] == "gated_bwd":
        s["dout"] = _randn((M, k), g, 0.1)
        if e4m3:   # codes of both signs and all exponents but NaN's, scales about those of values near 1
            code = _randn((cap, 2 * n), g, 100.0, torch.float32).clamp_(-448, 448).to(F8)
            s["h"] = _padding(code.view(torch.uint8), r["src"], 0x7f)
            s["h_s"] = _padding(torch.randint(118, 122, (cap, 2 * n // BLOCK), device=DEV, generator=g,
                                              dtype=torch.uint8), r["src"], 255)
        else:
            s["h"], s["h_s"] = _padding(_randn((cap, 2 * n), g, 1.5), r["src"]), None
        s["d"], s["row_w"] = _zeros(cap, k), _zeros(cap, dtype=torch.float32)
        s["dots"] = _zeros(cap, -(-n // 64), dtype=torch.float32)
        s["dtw"] = _zeros(M, T, dtype=torch.float32)
    if c["op"] != "gated":
        s["w2"] = _randn((L, k, n), g, 0.02)
        s["dh"], s["act2"] = _zeros(cap, 2 * n), _zeros(cap, n)
    return s


# ---- one pass -------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    return _PLAIN[c["op"]](s, c)


def _run_own(s, c):
    import unpermute_count_expert_amd as moe
    if c["op"] == "checkpoint":
        moe.moe_checkpoint(s["x"], s["q"], s["q_s"])
        moe.moe_checkpoint_restore(s["q"], s["q_s"], s["a"], inv_perm=s["inv"])
        return s["a"]
    off, cnt = s["offsets"], s["counts"]
    hint = max(1, c["tokens"] * c["topk"] * c["local"] // c["experts"])   # the rows this rank expects
    if c["op"] == "gated":
        moe.moe_grouped_gemm_bf16_silu_mul(s["a"], s["w13"], off, cnt, s["act"], h=s.get("h"), rows_hint=hint)
        return (s["act"], s["h"]) if c["keep"] == "bf16" else s["act"]
    if c["op"] == "train":
        moe.moe_grouped_gemm_bf16_silu_mul(s["a"], s["w13"], off, cnt, s["act"], h=s["h"], h_s=s["h_s"],
                                           rows_hint=hint)
        moe.moe_grouped_gemm_bf16_dgrad_silu_mul(s["dy"], s["w2"], off, cnt, s["h"], s["dh"], act=s["act2"],
                                                 h_s=s["h_s"], rows_hint=hint)
        return s["act"], s["act2"], s["dh"]
    moe.moe_permute_rows(s["dout"], s["inv"], s["d"], topk_weights=s["tw"], row_weights=s["row_w"])
    moe.moe_grouped_gemm_bf16_dgrad_silu_mul(s["d"], s["w2"], off, cnt, s["h"], s["dh"], act=s["act2"], h_s=s["h_s"],
                                             row_weights=s["row_w"], dots=s["dots"], rows_hint=hint)
    moe.moe_topk_weights_bwd(s["dots"], s["inv"], s["dtw"])
    return s["d"], s["act2"], s["dh"], s["dtw"]


def _by_expert(t, s):
    """fp32 [experts, longest, width]: each expert's rows, zeros past its count."""
    i = torch.arange(s["longest"], device=DEV)
    at = (s["offsets"][:-1, None].long() + i).clamp_(max=t.shape[0] - 1)
    return torch.where((i < s["counts"][:, None])[:, :, None], t[at].float(), 0.0)


def _place(s):
    """Of each row, its expert and its place in it, clamped on rows of no expert; and whether it belongs to one."""
    r = torch.arange(s["cap"], device=DEV)
    e = (torch.searchsorted(s["offsets"].long(), r, right=True) - 1).clamp_(max=s["counts"].numel() - 1)
    return e, (r - s["offsets"][e]).clamp_(max=s["longest"] - 1), s["src"] >= 0


def _to_rows(t, s):
    """[cap, width] of [experts, longest, width], zeros on rows of no expert."""
    e, i, valid = _place(s)
    return torch.where(valid[:, None], t[e, i], 0.0)


def _blocks8(x):
    """fp32 x as 8-bit blocks give it back: 32 values share the least power of two that brings them to 448 or below."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    scale = torch.exp2((e - 9 + (m > 0.875)).clamp(min=-117).float())
    return ((b / scale).to(F8).float() * scale).reshape(x.shape)


def _silu_parts(g):
    s = 1.0 / (1.0 + torch.exp(-g))
    return g * s, s * (1.0 + g * (1.0 - s))   # silu and its derivative


def _gate_up(s, c):
    """fp32 gate and up products, [experts, longest, 2 n]."""
    return torch.bmm(_by_expert(s["a"], s), s["w13"].float().transpose(1, 2))


def _act(h, n):
    return _silu_parts(h[..., :n])[0] * h[..., n:]


def _gated(s, c):
    h = _gate_up(s, c)
    act = _to_rows(_act(h, c["n"]), s).to(BF)
    return (act, _to_rows(h, s).to(BF)) if c["keep"] == "bf16" else act


def _act_bwd(h, d, n):
    """act and the gradient of h from kept fp32 h and the gradient d of act."""
    silu, slope = _silu_parts(h[..., :n])
    return silu * h[..., n:], torch.cat([d * h[..., n:] * slope, d * silu], dim=-1)


def _train(s, c):
    h = _gate_up(s, c)
    kept = _blocks8(h) if c["keep"] == "e4m3" else h.to(BF).float()
    act2, dh = _act_bwd(kept, torch.bmm(_by_expert(s["dy"], s), s["w2"].float()), c["n"])
    return _to_rows(_act(h, c["n"]), s).to(BF), _to_rows(act2, s).to(BF), _to_rows(dh, s).to(BF)


def _gated_bwd(s, c):
    cap, n, inv, src = s["cap"], c["n"], s["inv"].long(), s["src"].long()
    valid = (src >= 0)[:, None]
    w = torch.zeros(cap + 1, device=DEV)
    w = w.scatter_(0, torch.where(inv >= 0, inv, cap).reshape(-1), s["tw"].reshape(-1))[:cap, None]
    d = torch.where(valid, s["dout"][src.clamp(min=0)], 0.0)
    g = _to_rows(torch.bmm(_by_expert(d, s), s["w2"].float()), s)   # the gradient of act before the router weight
    if c["keep"] == "e4m3":
        h = s["h"].view(F8).float() * torch.exp2(s["h_s"].float() - 127).repeat_interleave(BLOCK, dim=1)
    else:
        h = s["h"].float()
    h = torch.where(valid, h, 0.0)
    act, dh = _act_bwd(h, w * g, n)
    dots = (act * g).sum(1)
    return d, (w * act).to(BF), dh.to(BF), torch.where(inv >= 0, dots[inv.clamp(min=0)], 0.0)


def _checkpoint(s, c):
    x = _blocks8(s["x"].float())
    src = s["src"].long()
    return torch.where((src >= 0)[:, None], x[src.clamp(min=0)], 0.0).to(BF)


_PLAIN = dict(gated=_gated, train=_train, gated_bwd=_gated_bwd, checkpoint=_checkpoint)


# ---- what a pass cannot do without -------------------------------------------------
def work(case):
    c = case
    M, k = c["tokens"], c["k"]
    P = max(1.0, M * c["topk"] * c["local"] / c["experts"])   # rows expected on this rank
    eight = 1 + 1 / BLOCK
    if c["op"] == "checkpoint":   # tokens read, kept, read again and written in expert order
        return {"bytes": M * k * (2 + 2 * eight) + 2 * P * k + 4 * M * c["topk"], "flops": 0}
    n = c["n"]
    touched = c["local"] * (1 - (1 - 1 / c["experts"]) ** (M * c["topk"]))
    kept = {"none": 0, "bf16": 2, "e4m3": eight}[c["keep"]] * 2 * P * n
    fwd = {"bytes": 2 * P * (k + n) + 4 * touched * n * k + kept, "flops": 4 * P * n * k + 8 * P * n}
    bwd = {"bytes": 2 * P * (k + 3 * n) + 2 * touched * n * k + kept, "flops": 2 * P * n * k + 16 * P * n}
    if c["op"] == "gated":
        return fwd
    if c["op"] == "train":
        return {x: fwd[x] + bwd[x] for x in fwd}
    return {"bytes": bwd["bytes"] + 2 * M * k + 12 * M * c["topk"], "flops": bwd["flops"] + 2 * P * n}


# ---- the definitions in 64 bits ---------------------------------------------------
def _nearest8(x):
    """float64 x [rows, width] in 8-bit blocks: e4m3 has 3 fraction bits down to 2^-6 and steps of 2^-9 below."""
    b = x.reshape(x.shape[0], x.shape[1] // BLOCK, BLOCK)
    top = b.abs().amax(2, keepdim=True).clamp(min=2.0 ** -200)
    scale = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(min=-117))
    scale = torch.where(top > 448 * scale, 2 * scale, scale)   # the logarithm may have come out just below
    scale = torch.where((top <= 224 * scale) & (scale > 2.0 ** -117), scale / 2, scale)   # or above
    v = b / scale
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step * scale).reshape(x.shape)


def exact(case, seed):
    s, c = prepare(case, seed), case
    f64 = torch.float64
    cap, M, T, k = s["cap"], c["tokens"], c["topk"], c["k"]
    zeros = lambda *shape: torch.zeros(shape, dtype=f64, device=DEV)   # noqa: E731
    if c["op"] == "checkpoint":
        x, out = _nearest8(s["x"].to(f64)), zeros(cap, k)
        for j in range(T):
            t = torch.nonzero(s["inv"][:, j] >= 0).flatten()
            out[s["inv"][t, j].long()] = x[t]
        return out
    n = c["n"]
    lo = s["offsets"].tolist()
    hi = [a + b for a, b in zip(lo, s["counts"].tolist())]
    h, act, act2, dh = zeros(cap, 2 * n), zeros(cap, n), zeros(cap, n), zeros(cap, 2 * n)
    if c["op"] == "gated_bwd":
        d, w, dots, dtw = zeros(cap, k), zeros(cap), zeros(cap), zeros(M, T)
        for j in range(T):
            t = torch.nonzero(s["inv"][:, j] >= 0).flatten()
            d[s["inv"][t, j].long()] = s["dout"][t].to(f64)
            w[s["inv"][t, j].long()] = s["tw"][t, j].to(f64)
    for e in range(c["local"]):
        r = slice(lo[e], hi[e])
        if c["op"] in ("gated", "train"):
            h[r] = s["a"][r].to(f64) @ s["w13"][e].to(f64).T.contiguous()
            act[r] = h[r, :n] * h[r, n:] / (1 + torch.exp(-h[r, :n]))
        if c["op"] == "gated":
            continue
        if c["op"] == "train":
            kept = _nearest8(h[r]) if c["keep"] == "e4m3" else h[r].to(torch.float32).to(BF).to(f64)
            grad, wr = s["dy"][r].to(f64) @ s["w2"][e].to(f64), 1.0
        else:
            kept = s["h"][r].to(f64)
            if c["keep"] == "e4m3":
                kept = s["h"][r].view(F8).to(f64) * torch.exp2(s["h_s"][r].to(f64) - 127).repeat_interleave(BLOCK, 1)
            grad, wr = d[r] @ s["w2"][e].to(f64), w[r, None]
        g, u = kept[:, :n], kept[:, n:]
        q = 1 + torch.exp(-g)
        act2[r] = wr * g * u / q
        dh[r, :n] = wr * grad * u * (1 / q + g * torch.exp(-g) / q ** 2)
        dh[r, n:] = wr * grad * g / q
        if c["op"] == "gated_bwd":
            dots[r] = (grad * g * u / q).sum(1)
    if c["op"] == "gated":
        return (act, h) if c["keep"] == "bf16" else act
    if c["op"] == "train":
        return act, act2, dh
    for j in range(T):
        t = torch.nonzero(s["inv"][:, j] >= 0).flatten()
        dtw[t, j] = dots[s["inv"][t, j].long()]
    return d, act2, dh, dtw
