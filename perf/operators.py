"""The bf16 expert operators as measured work: the grouped products and their
gradients, the permute of bf16 rows, SiLU-mul with its gradient, the weighted
unpermute's gradient, and the global gradient norm with clipping.

`own` False: the plain form, elementary torch operations in 32 bits (64 for
the long sum of squares), rounded once at the end.  `own` True: the calls of
unpermute_count_expert_amd.  Shapes are those of the layer configurations in
generators.py (hidden 2048, expert intermediate 768, 128 experts, top-8) and
of the tests' odd layers (hidden 2176, 300 tokens, 130 tokens, align 16).
"""
import math

import torch

own = False
DEV = "cuda"
BF = torch.bfloat16


def listed():
    return [
        # one decoding step of one sequence: 8 routed rows, weight bandwidth and latency
        dict(name="forward_1_token", op="forward", tokens=1, topk=8, experts=128, local=128, routing="uniform",
             n=1536, k=2048, align=16),
        # the gate/up product of a large prefill or training batch
        dict(name="forward_16384_tokens", op="forward", tokens=16384, topk=8, experts=128, local=128,
             routing="uniform", n=1536, k=2048, align=128),
        # a short fine-tuning batch on one of two expert-parallel ranks, skewed routing, odd widths, fp32 gradients
        dict(name="backward_300_tokens", op="backward", tokens=300, topk=8, experts=128, local=64, routing="zipf",
             n=1000, k=2176, align=16, dw="f32"),
        # the down product's gradients of a training batch with hot experts, bf16 weight gradients
        dict(name="backward_4096_tokens", op="backward", tokens=4096, topk=8, experts=128, local=128, routing="hot",
             n=2048, k=768, align=128, dw="bf16"),
        # rows of a decoding batch into expert order, half the experts on this rank
        dict(name="permute_64_tokens", op="permute", tokens=64, topk=4, experts=128, local=64, routing="uniform",
             k=2048, align=128),
        # the same for a large batch
        dict(name="permute_16384_tokens", op="permute", tokens=16384, topk=8, experts=128, local=128,
             routing="uniform", k=2048, align=128),
        # activation and its gradient on a ragged chunk, odd width
        dict(name="silu_130_tokens", op="silu", tokens=130, topk=8, experts=128, local=64, routing="zipf", n=1000,
             align=16),
        # and on a large batch
        dict(name="silu_16384_tokens", op="silu", tokens=16384, topk=8, experts=128, local=128, routing="uniform",
             n=768, align=128),
        # gradient of the weighted combine, short ragged chunk
        dict(name="combine_bwd_130_tokens", op="combine_bwd", tokens=130, topk=8, experts=128, local=64,
             routing="zipf", k=2048, align=128),
        # and a large batch
        dict(name="combine_bwd_16384_tokens", op="combine_bwd", tokens=16384, topk=8, experts=128, local=128,
             routing="uniform", k=2048, align=128),
        # many small gradients (norm scales, biases, a tiny layer), bf16 and fp32
        dict(name="clip_97_small", op="clip", tensors=97, total=300_000, dw="mixed"),
        # the weight gradients of the large layer: 128 experts' gate/up and down matrices in fp32
        dict(name="clip_experts", op="clip", tensors=2, total=128 * 3 * 768 * 2048, dw="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "backward", "forward", "backward", "permute", "silu", "combine_bwd", "clip"])
    if op == "clip":
        return dict(op=op, tensors=_log(rng, 1, 400), total=_log(rng, 2000, 300_000_000),
                    dw=rng.choice(["f32", "bf16", "mixed"]))
    experts = rng.choice([8, 32, 60, 128])
    c = dict(op=op, tokens=_log(rng, 1, 12000), topk=rng.choice([1, 2, 4, 6, 8]), experts=experts,
             local=rng.choice([experts, experts // 2]), routing=rng.choice(["uniform", "zipf", "hot"]),
             align=rng.choice([16, 32, 64, 128]))
    if c["routing"] == "zipf":
        c["tokens"] = min(c["tokens"], 4096)   # one expert takes a large share; its plain form is padded to it
    if op in ("forward", "backward"):
        c["n"] = 8 * _log(rng, 16, 256)
        c["k"] = 8 * _log(rng, 16, 256)
        if op == "backward":
            c["dw"] = rng.choice(["f32", "bf16"])
    elif op == "silu":
        c["n"] = 8 * _log(rng, 16, 192)
    else:
        c["k"] = 128 * _log(rng, 1, 17)
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


def _local(c):
    """expert_map of the second of two ranks (None where every expert is local)."""
    E, L = c["experts"], c["local"]
    if L == E:
        return None
    m = torch.full((E,), -1, dtype=torch.int32, device=DEV)
    m[E - L:] = torch.arange(L, dtype=torch.int32, device=DEV)
    return m


def _max_rows(c):
    pairs = c["tokens"] * c["topk"]
    return pairs + min(c["local"], pairs) * (c["align"] - 1)


def _rows(c, g):
    """Routing of one batch and its expert segments, as the permute lays them out."""
    ids, tw = _route(c, g)
    emap = _local(c)
    local = ids.long() if emap is None else emap.long()[ids.long()]
    counts, offsets, inv, src = _layout(c, local)
    return dict(ids=ids, tw=tw, emap=emap, counts=counts, offsets=offsets, inv=inv, src=src,
                longest=max(1, int(counts.max())), cap=_max_rows(c))


def _layout(c, local):
    """counts, offsets, inverse indices and row sources of stable expert segments padded to align."""
    L, T, A, cap = c["local"], c["topk"], c["align"], _max_rows(c)
    key = torch.where(local < 0, L, local).reshape(-1)
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
    return counts.to(i32), offsets.to(i32), inv.view(-1, T).to(i32), src[:cap].to(i32)


def _randn(shape, g, scale=1.0, dtype=BF):
    return torch.randn(shape, device=DEV, generator=g).mul_(scale).to(dtype)


def _padding(t, src):
    """Rows that belong to no expert hold whatever was there: NaN here."""
    t.masked_fill_((src < 0)[:, None], float("nan"))
    return t


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=dict(c))
    if c["op"] == "clip":
        n, total = c["tensors"], c["total"]
        cut = [total // (2 * n)] * n if n > 2 else [2 * total // 3, total - 2 * total // 3][:n]
        if n > 2:   # half the total spread evenly, half by a falling share, so that sizes are odd and unlike
            share = [1.0 / (i + 1) for i in range(n)]
            cut = [max(1, a + int(total / 2 * b / sum(share))) for a, b in zip(cut, share)]
        kinds = [torch.float32 if c["dw"] == "f32" or (c["dw"] == "mixed" and i % 3 == 0) else BF for i in range(n)]
        # the gradients lie end to end in one buffer for each type, as buckets of a training program do
        size = {d: sum(m for m, q in zip(cut, kinds) if q == d) for d in (torch.float32, BF)}
        flat = {d: _randn((m,), g, 0.02, d) for d, m in size.items()}
        s["flat_out"] = {d: torch.empty_like(t) for d, t in flat.items()}
        s["grads"], s["outs"], at = [], [], dict.fromkeys(size, 0)
        for m, d in zip(cut, kinds):
            s["grads"].append(flat[d][at[d]:at[d] + m])
            s["outs"].append(s["flat_out"][d][at[d]:at[d] + m])
            at[d] += m
        s["max_norm"] = 1.0
        s["sumsq"] = torch.zeros(1, dtype=torch.float64, device=DEV)
        s["norm"] = torch.zeros(1, dtype=torch.float32, device=DEV)
        s["ws"] = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
        return s
    r = _rows(c, g)
    s.update(r)
    cap, M, L = r["cap"], c["tokens"], c["local"]
    if c["op"] in ("forward", "backward"):
        s["w"] = _randn((L, c["n"], c["k"]), g, 0.02)
        s["a"] = _padding(_randn((cap, c["k"]), g), r["src"])
        if c["op"] == "forward":
            s["out"] = torch.zeros(cap, c["n"], dtype=BF, device=DEV)
        else:
            s["dy"] = _padding(_randn((cap, c["n"]), g, 0.1), r["src"])
            s["dx"] = torch.zeros(cap, c["k"], dtype=BF, device=DEV)
            s["dw"] = torch.empty(L, c["n"], c["k"], dtype=torch.float32 if c["dw"] == "f32" else BF, device=DEV)
    elif c["op"] == "permute":
        s["x"] = _randn((M, c["k"]), g)
        s["a"] = torch.zeros(cap, c["k"], dtype=BF, device=DEV)
        s["out_counts"], s["out_offsets"] = torch.empty_like(r["counts"]), torch.empty_like(r["offsets"])
        s["out_inv"], s["out_src"] = torch.empty_like(r["inv"]), torch.empty_like(r["src"])
        blocks = -(-M // max(1, 256 // c["topk"]))
        s["ws"] = torch.empty(4 * blocks * L + 4096, dtype=torch.uint8, device=DEV)
    elif c["op"] == "silu":
        s["h"] = _padding(_randn((cap, 2 * c["n"]), g, 1.5), r["src"])
        s["dact"] = _padding(_randn((cap, c["n"]), g, 0.1), r["src"])
        s["act"] = torch.zeros(cap, c["n"], dtype=BF, device=DEV)
        s["dh"] = torch.zeros(cap, 2 * c["n"], dtype=BF, device=DEV)
    else:
        s["dout"] = _randn((M, c["k"]), g, 0.1)
        s["y"] = _padding(_randn((cap, c["k"]), g), r["src"])
        s["dy"] = torch.zeros(cap, c["k"], dtype=BF, device=DEV)
        s["dtw"] = torch.empty(M, c["topk"], dtype=torch.float32, device=DEV)
    return s


# ---- one pass -------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    return _PLAIN[c["op"]](s, c)


def _run_own(s, c):
    import unpermute_count_expert_amd as moe
    op = c["op"]
    if op == "clip":
        moe.moe_grad_sumsq(s["grads"], s["sumsq"], s["ws"])
        moe.moe_grad_clip(s["grads"], s["outs"], s["sumsq"], s["max_norm"], s["norm"])
        return [s["norm"]] + list(s["flat_out"].values())
    off, cnt = s["offsets"], s["counts"]
    hint = c["tokens"] * c["topk"] * c["local"] // c["experts"]   # the rows this rank expects
    if op == "forward":
        moe.moe_grouped_gemm_bf16(s["a"], s["w"], off, cnt, s["out"], rows_hint=hint)
        return s["out"]
    if op == "backward":
        moe.moe_grouped_gemm_bf16_dgrad(s["dy"], s["w"], off, cnt, s["dx"], rows_hint=hint)
        moe.moe_grouped_gemm_bf16_wgrad(s["dy"], s["a"], off, cnt, s["dw"], rows_hint=hint)
        return s["dx"], s["dw"]
    if op == "permute":
        moe.moe_permute_bf16(s["x"], s["ids"], s["emap"], c["experts"], c["local"], c["align"], s["cap"], s["a"],
                             s["out_counts"], s["out_offsets"], s["out_inv"], s["out_src"], s["ws"])
        return s["a"], s["out_counts"], s["out_offsets"], s["out_inv"], s["out_src"]
    if op == "silu":
        moe.moe_silu_mul(s["h"], c["n"], s["act"], off, cnt, c["local"])
        moe.moe_silu_mul_bwd(s["h"], s["dact"], c["n"], s["dh"], off, cnt, c["local"])
        return s["act"], s["dh"]
    moe.moe_unpermute_weight_reduce_bwd(s["dout"], s["y"], s["inv"], s["tw"], s["dy"], s["dtw"])
    return s["dy"], s["dtw"]


def _packed(tensors):
    """The fp32 tensors end to end, and the bf16 ones, by the gradients' types."""
    empty = torch.empty(0, device=DEV)
    return [torch.cat([empty.to(d)] + [t for t in tensors if t.dtype == d]) for d in (torch.float32, BF)]


def _by_expert(t, s):
    """fp32 [experts, longest, width]: each expert's rows, zeros past its count."""
    i = torch.arange(s["longest"], device=DEV)
    at = (s["offsets"][:-1, None].long() + i).clamp_(max=t.shape[0] - 1)
    return torch.where((i < s["counts"][:, None])[:, :, None], t[at].float(), 0.0)


def _to_rows(t, s):
    """bf16 [cap, width] of [experts, longest, width], zeros on rows of no expert."""
    r = torch.arange(s["cap"], device=DEV)
    e = (torch.searchsorted(s["offsets"].long(), r, right=True) - 1).clamp_(max=t.shape[0] - 1)
    i = (r - s["offsets"][e]).clamp_(max=s["longest"] - 1)
    return torch.where((s["src"] >= 0)[:, None], t[e, i], 0.0).to(BF)


def _forward(s, c):
    return _to_rows(torch.bmm(_by_expert(s["a"], s), s["w"].float().transpose(1, 2)), s)


def _backward(s, c):
    dy, a = _by_expert(s["dy"], s), _by_expert(s["a"], s)
    dx = _to_rows(torch.bmm(dy, s["w"].float()), s)
    return dx, torch.bmm(dy.transpose(1, 2), a).to(s["dw"].dtype)


def _permute(s, c):
    local = s["ids"].long() if s["emap"] is None else s["emap"].long()[s["ids"].long()]
    counts, offsets, inv, src = _layout(c, local)
    rows = torch.where((src >= 0)[:, None], s["x"][src.clamp(min=0).long()], 0.0)
    return rows, counts, offsets, inv, src


def _silu(s, c):
    keep = (s["src"] >= 0)[:, None]
    g, u, d = s["h"][:, :c["n"]].float(), s["h"][:, c["n"]:].float(), s["dact"].float()
    sg = 1.0 / (1.0 + torch.exp(-g))
    act = torch.where(keep, g * sg * u, 0.0).to(BF)
    dh = torch.cat([d * u * sg * (1.0 + g * (1.0 - sg)), d * g * sg], dim=1)
    return act, torch.where(keep, dh, 0.0).to(BF)


def _combine_bwd(s, c):
    inv, cap = s["inv"].long(), s["cap"]
    here = inv >= 0
    d = s["dout"].float()
    dtw = torch.where(here, (s["y"][inv.clamp(min=0)].float() * d[:, None, :]).sum(-1), 0.0)
    w = torch.zeros(cap + 1, device=DEV).scatter_(0, torch.where(here, inv, cap).reshape(-1), s["tw"].reshape(-1))
    src = s["src"].long()
    dy = torch.where((src >= 0)[:, None], w[:cap, None] * d[src.clamp(min=0)], 0.0)
    return dy.to(BF), dtw


def _clip(s, c):
    sumsq = torch.stack([t.double().square().sum() for t in s["grads"]]).sum()
    norm = sumsq.sqrt().float().reshape(1)
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return [norm] + _packed([(t.float() * coef).to(t.dtype) for t in s["grads"]])


_PLAIN = dict(forward=_forward, backward=_backward, permute=_permute, silu=_silu, combine_bwd=_combine_bwd, clip=_clip)


# ---- what a pass cannot do without -------------------------------------------------
def work(case):
    c = case
    if c["op"] == "clip":
        per = 4 if c["dw"] == "f32" else 2 if c["dw"] == "bf16" else 8 / 3
        return {"bytes": 2 * per * c["total"], "flops": 3 * c["total"]}
    share = c["local"] / c["experts"]
    P = max(1.0, c["tokens"] * c["topk"] * share)   # rows expected on this rank
    M = c["tokens"]
    if c["op"] in ("forward", "backward"):
        n, k = c["n"], c["k"]
        touched = c["local"] * (1 - (1 - 1 / c["experts"]) ** (c["tokens"] * c["topk"]))
        fwd = {"bytes": 2 * P * (n + k) + 2 * touched * n * k, "flops": 2 * P * n * k}
        if c["op"] == "forward":
            return fwd
        dw = (4 if c["dw"] == "f32" else 2) * c["local"] * n * k
        return {"bytes": fwd["bytes"] + 2 * P * k + dw, "flops": 2 * fwd["flops"]}
    if c["op"] == "permute":
        return {"bytes": 2 * (M + P) * c["k"] + 8 * M * c["topk"] + 4 * _max_rows(c), "flops": 0}
    if c["op"] == "silu":
        return {"bytes": 2 * P * c["n"] * (2 + 1 + 1 + 2), "flops": 20 * P * c["n"]}
    return {"bytes": 2 * (M + 2 * P) * c["k"] + 12 * M * c["topk"], "flops": 3 * P * c["k"]}


# ---- the definitions in 64 bits ---------------------------------------------------
def exact(case, seed):
    s, c = prepare(case, seed), case
    f64 = torch.float64
    if c["op"] == "clip":
        norm = math.sqrt(sum(float((t.to(f64) ** 2).sum()) for t in s["grads"]))
        coef = min(1.0, s["max_norm"] / (norm + 1e-6))
        outs = [torch.cat([t.to(f64) * coef for t in s["grads"] if t.dtype == d] + [torch.empty(0, dtype=f64, device=DEV)])
                for d in (torch.float32, BF)]
        return [torch.tensor([norm], dtype=f64, device=DEV)] + outs
    lo = s["offsets"].tolist()
    hi = [a + b for a, b in zip(lo, s["counts"].tolist())]
    if c["op"] == "forward":
        out = torch.zeros(s["cap"], c["n"], dtype=f64, device=DEV)
        for e in range(c["local"]):
            out[lo[e]:hi[e]] = s["a"][lo[e]:hi[e]].to(f64) @ s["w"][e].to(f64).T.contiguous()
        return out
    if c["op"] == "backward":
        dx = torch.zeros(s["cap"], c["k"], dtype=f64, device=DEV)
        dw = torch.zeros(c["local"], c["n"], c["k"], dtype=f64, device=DEV)
        for e in range(c["local"]):
            d, a = s["dy"][lo[e]:hi[e]].to(f64), s["a"][lo[e]:hi[e]].to(f64)
            dx[lo[e]:hi[e]] = d @ s["w"][e].to(f64)
            dw[e] = d.T.contiguous() @ a
        return dx, dw
    if c["op"] == "permute":
        rows = torch.zeros(s["cap"], c["k"], dtype=f64, device=DEV)
        for k in range(c["topk"]):
            t = torch.nonzero(s["inv"][:, k] >= 0).flatten()
            rows[s["inv"][t, k].long()] = s["x"][t].to(f64)
        return rows, None, None, None, None
    if c["op"] == "silu":
        n = c["n"]
        act = torch.zeros(s["cap"], n, dtype=f64, device=DEV)
        dh = torch.zeros(s["cap"], 2 * n, dtype=f64, device=DEV)
        for e in range(c["local"]):
            r = slice(lo[e], hi[e])
            g, u, d = s["h"][r, :n].to(f64), s["h"][r, n:].to(f64), s["dact"][r].to(f64)
            up = 1 + torch.exp(-g)
            act[r] = g * u / up
            dh[r, :n] = d * u * (1 / up + g * torch.exp(-g) / up ** 2)
            dh[r, n:] = d * g / up
        return act, dh
    dy = torch.zeros(s["cap"], c["k"], dtype=f64, device=DEV)
    dtw = torch.zeros(c["tokens"], c["topk"], dtype=f64, device=DEV)
    d = s["dout"].to(f64)
    for k in range(c["topk"]):
        t = torch.nonzero(s["inv"][:, k] >= 0).flatten()
        row = s["inv"][t, k].long()
        dy[row] = s["tw"][t, k, None].to(f64) * d[t]
        dtw[t, k] = (s["y"][row].to(f64) * d[t]).sum(1)
    return dy, dtw
