"""Timed cases of the operators around the expert products of a Mixture-of-Experts layer.

Three kinds of case, each a call or a few calls that a program makes in one go:

  route   softmax top-k routing with per-expert counts and the balance loss; with "train" its gradient too
  rows    the plan that sorts (token, choice) slots by expert, rows dispatched by it and combined back with
          the routing weights; with "train" both gradients too
  fp8     the grouped product of bf16 rows with e4m3 expert weights (a power-of-two scale for each block of
          128); "serve": the weights are there; "train": they are quantised in the call, fwd and dgrad follow

run() computes the plain forms below (elementary torch operations in fp32, rounded once at the end) or, where
`own` is true, calls the package.  exact() is the same mathematics in fp64, written apart.
"""
import math

import numpy as np
import torch

own = False

NEG_INF = float("-inf")
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # one token of a serving loop through a 256-expert router: latency
        {"name": "route_token", "kind": "route", "tokens": 1, "experts": 256, "top_k": 8, "dtype": "bf16",
         "normalize": True, "masked": False, "train": False},
        # a batch of the 8-expert top-2 layer, fp32 router, 8192 tokens, forward and gradient
        {"name": "route_e8_train", "kind": "route", "tokens": 8192, "experts": 8, "top_k": 2, "dtype": "fp32",
         "normalize": True, "masked": False, "train": True},
        # the 256-expert layer: an odd number of tokens, padding tokens masked, experts switched off in some rows
        {"name": "route_e256_masked", "kind": "route", "tokens": 8191, "experts": 256, "top_k": 8, "dtype": "bf16",
         "normalize": False, "masked": True, "train": True},
        # a long batch through a 128-expert router, fp32 logits
        {"name": "route_long", "kind": "route", "tokens": 65536, "experts": 128, "top_k": 4, "dtype": "fp32",
         "normalize": True, "masked": False, "train": True},
        # three tokens of a serving loop, hidden size 4096, top-2 of 8
        {"name": "rows_tokens", "kind": "rows", "tokens": 3, "experts": 8, "top_k": 2, "hidden": 4096,
         "dtype": "bf16", "masked": False, "train": False},
        # the fine-grained 64-expert layer: 4096 tokens, 8 choices, hidden 2048, forward and gradients
        {"name": "rows_fine_train", "kind": "rows", "tokens": 4096, "experts": 64, "top_k": 8, "hidden": 2048,
         "dtype": "bf16", "masked": False, "train": True},
        # hidden size 7168 over 128 experts, an odd number of tokens, some choices without an expert
        {"name": "rows_wide_train", "kind": "rows", "tokens": 4095, "experts": 128, "top_k": 8, "hidden": 7168,
         "dtype": "bf16", "masked": True, "train": True},
        # one token of a serving loop through the 8-expert top-2 layer (K=4096, N=14336): the weights' bytes
        {"name": "fp8_token", "kind": "fp8", "rows": 2, "experts": 8, "n": 14336, "k": 4096, "mode": "serve"},
        # a decode batch of 61 tokens, 8 choices, over the fine-grained layer's 64 experts
        {"name": "fp8_decode", "kind": "fp8", "rows": 488, "experts": 64, "n": 1536, "k": 2048, "mode": "serve"},
        # odd sizes: a K that ends inside a block of 128, an N that ends inside a tile
        {"name": "fp8_ragged", "kind": "fp8", "rows": 3001, "experts": 16, "n": 1000, "k": 2000, "mode": "serve"},
        # a prompt batch of the 8-expert layer: 8192 tokens, top-2
        {"name": "fp8_prompt", "kind": "fp8", "rows": 16384, "experts": 8, "n": 14336, "k": 4096, "mode": "serve"},
        # a training step's products of the fine-grained layer, weights quantised in the step
        {"name": "fp8_fine_train", "kind": "fp8", "rows": 32768, "experts": 64, "n": 1536, "k": 2048, "mode": "train"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["route", "rows", "fp8"])
    if kind == "route":
        experts = _log_int(rng, 4, 500)
        return {"kind": kind, "tokens": min(_log_int(rng, 1, 65536), 65536 * 128 // experts), "experts": experts,
                "top_k": rng.randint(1, min(8, experts)), "dtype": rng.choice(["bf16", "fp32"]),
                "normalize": rng.random() < 0.5, "masked": rng.random() < 0.5, "train": rng.random() < 0.7}
    if kind == "rows":
        experts, top_k, hidden = _log_int(rng, 4, 256), rng.randint(1, 8), 8 * _log_int(rng, 32, 896)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        most = 4095 * 8 * 7168 * 2 // (top_k * hidden * BYTES[dtype])
        return {"kind": kind, "tokens": min(_log_int(rng, 1, 8192), most), "experts": max(experts, top_k),
                "top_k": top_k, "hidden": hidden, "dtype": dtype, "masked": rng.random() < 0.5,
                "train": rng.random() < 0.7}
    while True:
        c = {"kind": kind, "rows": _log_int(rng, 1, 32768), "experts": _log_int(rng, 1, 64),
             "n": 8 * _log_int(rng, 16, 1792), "k": 16 * _log_int(rng, 8, 448),
             "mode": rng.choice(["serve", "serve", "train"])}
        flops = 2 * c["rows"] * c["n"] * c["k"] * (2 if c["mode"] == "train" else 1)
        if flops <= 9e11 and c["experts"] * c["n"] * c["k"] <= 4.7e8:
            return c


def work(case):
    c = case
    if c["kind"] == "route":
        t, e, k, s = c["tokens"], c["experts"], c["top_k"], BYTES[c["dtype"]]
        passes = 3 if c["train"] else 1                       # logits read, read again, gradient written
        return {"bytes": t * e * s * passes + t * k * (20 if c["train"] else 8) + 8 * e,
                "flops": t * e * (18 if c["train"] else 10)}
    if c["kind"] == "rows":
        t, r, row = c["tokens"], c["tokens"] * c["top_k"], c["hidden"] * BYTES[c["dtype"]]
        moved = 2 * (t + r) + ((t + r) + (t + 2 * r) if c["train"] else 0)
        return {"bytes": moved * row + r * 20, "flops": 2 * r * c["hidden"] * (4 if c["train"] else 1)}
    m, e, n, k = c["rows"], c["experts"], c["n"], c["k"]
    used = e * (1 - (1 - 1 / e) ** m)                         # experts with rows, expected
    if c["mode"] == "serve":
        return {"bytes": m * k * 2 + m * n * 2 + int(used * n * k), "flops": 2 * m * n * k}
    return {"bytes": m * (n + k) * 4 + e * n * k * (2 + 2) + 2 * int(used * n * k), "flops": 4 * m * n * k}


# ----------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, gen, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale)


def _rand(shape, gen):
    return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32)


def _sizes(rows, experts, seed):
    rng = np.random.default_rng(seed)
    return rng.multinomial(rows, rng.dirichlet(np.full(experts, 4.0)))


def prepare(case, seed):
    c, gen = case, _gen(seed)
    s = dict(case)
    if c["kind"] == "route":
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        logits = _randn((t, e), gen, 1.5) + _randn((1, e), gen, 0.7)   # some experts are liked more than others
        s["mask"] = None
        if c["masked"]:
            off = (_rand((t, 1), gen) < 0.125) & (_rand((t, e), gen) < 0.6)
            off |= _rand((t, 1), gen) < 0.02                            # rows with no expert at all
            logits = logits.masked_fill(off, NEG_INF)
            s["mask"] = _rand((t,), gen) >= 0.0625                      # padding tokens
        s["logits"] = logits.to(DTYPES[c["dtype"]])
        if c["train"]:
            s["dweight"] = _randn((t, k), gen)
            s["dloss"] = torch.full((), 0.01, device="cuda")
    elif c["kind"] == "rows":
        t, e, k, h, dt = c["tokens"], c["experts"], c["top_k"], c["hidden"], DTYPES[c["dtype"]]
        score = _rand((t, e), gen) * (0.3 + _rand((1, e), gen))         # k different experts of each token
        idx = torch.sort(score, dim=1, descending=True).indices[:, :k].to(torch.int32)
        weight = _rand((t, k), gen) + 0.05
        if c["masked"]:
            none = (_rand((t, 1), gen) < 0.0625) | (_rand((t, k), gen) < 0.03)
            idx = idx.masked_fill(none, -1)
            weight = weight.masked_fill(none, 0.0)
        s["idx"], s["weight"] = idx.contiguous(), weight
        s["x"] = _randn((t, h), gen).to(dt)
        s["y"] = _randn((t * k, h), gen).to(dt)                         # the experts' outputs
        if c["train"]:
            s["dout"] = _randn((t, h), gen).to(dt)
            s["dxp"] = _randn((t * k, h), gen).to(dt)
    else:
        m, e, n, k = c["rows"], c["experts"], c["n"], c["k"]
        sizes = _sizes(m, e, seed)
        s["most"] = int(sizes.max())                                    # rows of the largest group
        s["offs"] = torch.from_numpy(np.cumsum(sizes).astype(np.int32)).cuda()
        loud = 1.0 + 7.0 * (_rand((1, k), gen) < 0.01)                  # a few channels are louder
        s["x"] = (_randn((m, k), gen) * loud).to(torch.bfloat16)
        w = torch.empty((e, n, k), dtype=torch.bfloat16, device="cuda")
        for i in range(e):
            w[i] = _randn((n, k), gen, 1.0 / math.sqrt(k))
        if c["mode"] == "serve":
            wq, ws = _quantize_weight(w)
            s["wq"], s["ws"] = wq, ws.view(torch.float8_e8m0fnu)
        else:
            s["w"] = w
            s["g"] = _randn((m, n), gen).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------------------------ plain forms
def _route(s):
    logits, mask, k = s["logits"].float(), s["mask"], s["top_k"]
    t, e = logits.shape
    if mask is not None:
        logits = torch.where(mask[:, None], logits, NEG_INF)
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)  # ties: the lowest index first
    top, idx = top[:, :k], idx[:, :k]
    there = top != NEG_INF
    big = logits.max(dim=1).values
    live = big != NEG_INF
    ex = torch.where(live[:, None], torch.exp(logits - torch.where(live, big, 0.0)[:, None]), 0.0)
    total = ex.sum(dim=1)
    p = ex / torch.where(live, total, 1.0)[:, None]
    chosen = torch.where(there, torch.gather(ex, 1, idx), 0.0)
    by = chosen.sum(dim=1) if s["normalize"] else total
    weight = chosen / torch.where(live, by, 1.0)[:, None]
    ids = torch.where(there, idx, -1).to(torch.int32)
    slot = torch.where(there, idx, e).reshape(-1)
    counts = torch.zeros(e + 1, dtype=torch.int32, device=logits.device)
    counts = counts.index_add(0, slot, torch.ones_like(slot, dtype=torch.int32))[:e]
    routed = live.sum().float()
    a = e * counts.float() / (k * torch.clamp(routed * routed, min=1.0))
    loss = (a * p.sum(dim=0)).sum()
    out = {"weight": weight, "idx": ids, "counts": counts, "loss": loss}
    if s["train"]:
        dw = torch.where(there, s["dweight"], 0.0)
        inner = (weight * dw).sum(dim=1, keepdim=True)
        d = s["dloss"] * (p * a).sum(dim=1, keepdim=True)
        dl = p * (s["dloss"] * a - (d if s["normalize"] else d + inner))
        own_part = weight * (dw - inner) if s["normalize"] else weight * dw
        dl = dl.scatter_add(1, idx, torch.where(there, own_part, 0.0))
        out["dlogits"] = dl.to(s["logits"].dtype)
    return out


def _rows(s):
    idx, weight, x, y, k = s["idx"], s["weight"], s["x"], s["y"], s["top_k"]
    t, h = x.shape
    e, r = s["experts"], t * k
    flat = idx.reshape(-1).long()
    key = torch.where(flat >= 0, flat, e)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(r, device=order.device)
    dest = torch.where(flat >= 0, place, -1)
    counts = torch.zeros(e + 1, dtype=torch.int64, device=x.device).index_add(0, key, torch.ones_like(key))
    offs = torch.cumsum(counts[:e], 0).to(torch.int32)
    there = (dest >= 0).reshape(t, k, 1)
    to = torch.where(dest >= 0, dest, r)                                # slots without a row: one past the end
    at = dest.clamp(min=0)
    xp = torch.zeros((r + 1, h), dtype=x.dtype, device=x.device)
    xp[to] = x[:, None, :].expand(t, k, h).reshape(r, h)
    got = torch.where(there, y[at].reshape(t, k, h).float(), 0.0)
    out = {"offs": offs, "dest": dest.reshape(t, k).to(torch.int32), "xp": xp[:r],
           "out": (got * weight[:, :, None]).sum(dim=1).to(x.dtype)}
    if s["train"]:
        dout = s["dout"].float()
        dy = torch.zeros((r + 1, h), dtype=x.dtype, device=x.device)
        dy[to] = (weight[:, :, None] * dout[:, None, :]).reshape(r, h).to(x.dtype)
        out["dy"] = dy[:r]
        out["dweight"] = (got * dout[:, None, :]).sum(dim=2)
        dx = torch.where(there, s["dxp"][at].reshape(t, k, h).float(), 0.0)
        out["dx"] = dx.sum(dim=1).to(x.dtype)
    return out


def _scale_code(amax):
    """e8m0 code of the smallest power of two 2^e with amax <= 448 * 2^e (448 = 1.75 * 2^8)."""
    bits = amax.contiguous().view(torch.int32)
    code = (bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    return torch.where((bits >> 23) == 255, 255, code.clamp(min=0))


def _pow2(code):
    """2^(code - 127) in fp32 (a subnormal at code 0, NaN at 255)."""
    bits = torch.where(code == 0, 0x00400000, torch.where(code == 255, 0x7FC00000, code << 23))
    return bits.to(torch.int32).view(torch.float32)


def _pad_to_128(x, dim):
    short = -x.shape[dim] % 128
    if not short:
        return x
    pad = [0, 0] * (x.dim() - dim if dim >= 0 else -dim)
    pad[-1] = short
    return torch.nn.functional.pad(x, pad)


def _quantize_rows(x):
    m, k = x.shape
    b = _pad_to_128(x.float(), -1).reshape(m, -1, 128)
    code = _scale_code(b.abs().amax(dim=2))
    q = (b * _pow2(254 - code)[:, :, None]).to(torch.float8_e4m3fn).reshape(m, -1)
    return q, code.to(torch.uint8)


def _quantize_weight(w):
    e, n, k = w.shape
    b = _pad_to_128(_pad_to_128(w.float(), -1), -2)
    b = b.reshape(e, b.shape[1] // 128, 128, b.shape[2] // 128, 128)
    code = _scale_code(b.abs().amax(dim=4).amax(dim=2))
    q = (b * _pow2(254 - code)[:, :, None, :, None]).to(torch.float8_e4m3fn)
    q = q.reshape(e, q.shape[1] * 128, q.shape[3] * 128)[:, :n, :k].contiguous()
    return q, code.to(torch.uint8)


def _weight_values(wq, ws):
    e, n, k = wq.shape
    b = _pow2(ws.int()).repeat_interleave(128, dim=1, output_size=ws.shape[1] * 128)[:, :n]
    b = b.repeat_interleave(128, dim=2, output_size=ws.shape[2] * 128)[:, :, :k]
    return wq.float() * b


def _product(x, wt, offs, most):
    """Rows of x (bf16) in 8 bits times wt [E, K, N] (fp32) of their group: rows padded to [E, most, K]."""
    m, k = x.shape
    e = wt.shape[0]
    q, code = _quantize_rows(x)
    v = (q.float().reshape(m, -1, 128) * _pow2(code.int())[:, :, None]).reshape(m, -1)[:, :k]
    row = torch.arange(m, device=x.device, dtype=torch.int32)
    group = torch.bucketize(row, offs, right=True)
    start = torch.cat([torch.zeros_like(offs[:1]), offs[:-1]])
    at = group * most + (row - start[group])
    padded = torch.zeros((e * most, k), device=x.device)
    padded[at] = v
    y = torch.bmm(padded.reshape(e, most, k), wt)
    return y.reshape(e * most, -1)[at].to(torch.bfloat16)


def _fp8(s):
    if s["mode"] == "serve":
        wt = _weight_values(s["wq"], s["ws"].view(torch.uint8)).transpose(1, 2).contiguous()
        return {"y": _product(s["x"], wt, s["offs"], s["most"])}
    wv = _weight_values(*_quantize_weight(s["w"]))
    y = _product(s["x"], wv.transpose(1, 2).contiguous(), s["offs"], s["most"])
    return {"y": y, "dx": _product(s["g"], wv, s["offs"], s["most"])}


# -------------------------------------------------------------------------------------- one pass
def run(state):
    s = state
    if not own:
        return {"route": _route, "rows": _rows, "fp8": _fp8}[s["kind"]](s)
    import moe_ragged_bf16_amd as mdg
    if s["kind"] == "route":
        r = mdg.moe_route_fwd(s["logits"], s["top_k"], normalize=s["normalize"], token_mask=s["mask"])
        out = {"weight": r.weight, "idx": r.idx, "counts": r.counts, "loss": r.loss}
        if s["train"]:
            out["dlogits"] = mdg.moe_route_bwd(s["dweight"], s["dloss"], s["logits"], r, normalize=s["normalize"])
        return out
    if s["kind"] == "rows":
        plan = mdg.moe_plan(s["idx"], s["experts"])
        out = {"offs": plan.offs, "dest": plan.dest, "xp": mdg.moe_dispatch_fwd(s["x"], plan),
               "out": mdg.moe_combine_fwd(s["y"], s["weight"], plan)}
        if s["train"]:
            out["dy"], out["dweight"] = mdg.moe_combine_bwd(s["dout"], s["y"], s["weight"], plan)
            out["dx"] = mdg.moe_dispatch_bwd(s["dxp"], plan)
        return out
    if s["mode"] == "serve":
        return {"y": mdg.grouped_fp8_gemm_fwd(s["x"], s["wq"], s["ws"], s["offs"])}
    w8 = mdg.quantize_fp8_weight(s["w"], transpose=True)
    return {"y": mdg.grouped_fp8_gemm_fwd(s["x"], w8.q, w8.scale, s["offs"]),
            "dx": mdg.grouped_fp8_gemm_dgrad(s["g"], w8.qt, w8.scale_t, s["offs"])}


# ------------------------------------------------------------------------------ the same in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "rows": _exact_rows, "fp8": _exact_fp8}[case["kind"]](s)


def _exact_route(s):
    l = s["logits"].double()
    if s["mask"] is not None:
        l = l.masked_fill(~s["mask"][:, None], NEG_INF)
    t, e = l.shape
    k = s["top_k"]
    lse = torch.logsumexp(l, dim=1, keepdim=True)
    live = torch.isfinite(lse)
    p = torch.where(live, torch.exp(l - torch.where(live, lse, torch.zeros_like(lse))), torch.zeros_like(l))
    left, hit, w = l.clone(), torch.zeros_like(l), []
    cols = torch.arange(e, device=l.device)
    picks = []
    for _ in range(k):                                                  # the largest left, lowest index first
        best = left.max(dim=1, keepdim=True).values
        i = torch.where(left == best, cols, e).min(dim=1, keepdim=True).values
        ok = best != NEG_INF
        w.append(torch.where(ok, p.gather(1, i), torch.zeros_like(best)))
        hit.scatter_add_(1, i, ok.double())
        left.scatter_(1, i, NEG_INF)
        picks.append((i, ok))
    w = torch.cat(w, dim=1)
    norm = w.sum(dim=1, keepdim=True)
    if s["normalize"]:
        w = w / torch.where(norm > 0, norm, torch.ones_like(norm))
    routed = max(1, int(live.sum()))
    a = e * hit.sum(dim=0) / (k * float(routed) ** 2)
    out = {"weight": w, "idx": None, "counts": None, "loss": (a * p.sum(dim=0)).sum()}
    if s["train"]:
        dp = s["dloss"].double() * a.expand(t, e).clone()               # d/dp of loss and weights
        dw = s["dweight"].double()
        for j, (i, ok) in enumerate(picks):
            if s["normalize"]:
                v = (dw[:, j:j + 1] - (w * dw).sum(dim=1, keepdim=True)) / torch.where(norm > 0, norm, torch.ones_like(norm))
            else:
                v = dw[:, j:j + 1]
            dp.scatter_add_(1, i, torch.where(ok, v, torch.zeros_like(v)))
        out["dlogits"] = p * (dp - (p * dp).sum(dim=1, keepdim=True))
    return out


def _exact_rows(s):
    idx, (t, h), k = s["idx"].cpu().numpy().reshape(-1), s["x"].shape, s["top_k"]
    slots = np.argsort(np.where(idx < 0, s["experts"], idx), kind="stable")[:int((idx >= 0).sum())]
    slots = torch.from_numpy(slots).cuda()                              # slots[row]: the slot that row holds
    n, tok = slots.shape[0], slots // k
    w = s["weight"].double().reshape(-1)[slots][:, None]
    out = {"offs": None, "dest": None, "xp": torch.zeros((t * k, h), dtype=torch.float64, device="cuda")}
    out["xp"][:n] = s["x"].double()[tok]
    y = s["y"][:n].double()
    out["out"] = torch.zeros((t, h), dtype=torch.float64, device="cuda").index_add_(0, tok, w * y)
    if s["train"]:
        g = s["dout"].double()[tok]
        out["dy"] = torch.zeros_like(out["xp"])
        out["dy"][:n] = w * g
        dw = torch.zeros(t * k, dtype=torch.float64, device="cuda")
        dw[slots] = (g * y).sum(dim=1)
        out["dweight"] = dw.reshape(t, k)
        out["dx"] = torch.zeros((t, h), dtype=torch.float64, device="cuda").index_add_(0, tok, s["dxp"][:n].double())
    return out


def _two(e):
    """2^e in fp64, exactly (built from its bits)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_block(v):
    """fp64 values of blocks (last dimension) after rounding to e4m3 under their power-of-two scale."""
    amax = v.abs().amax(dim=-1, keepdim=True)
    f, e = torch.frexp(amax / 448.0)                                    # amax / 448 = f 2^e, 0.5 <= f < 1
    e = torch.where(f == 0.5, e - 1, e)
    e = torch.where(amax == 0, torch.full_like(e, -127), e.clamp(min=-127))
    two = _two(e)
    u = v / two
    g = torch.frexp(u).exponent.clamp(min=-5) - 4                       # 4 significant bits, subnormals of 2^-9
    step = _two(g)
    return torch.round(u / step) * step * two                           # (round: half to even)


def _exact_rows8(x):
    m, k = x.shape
    cols = [_exact_block(x[:, c:c + 128].double()) for c in range(0, k, 128)]
    return torch.cat(cols, dim=1)


def _exact_fp8(s):
    ends = s["offs"].tolist()
    x, y = _exact_rows8(s["x"]), []
    g, dx = (_exact_rows8(s["g"]), []) if s["mode"] == "train" else (None, None)
    for i, end in enumerate(ends):
        rows = slice(ends[i - 1] if i else 0, end)
        if s["mode"] == "serve":
            n, k = s["wq"].shape[1:]
            two = _two(s["ws"].view(torch.uint8)[i].int() - 127)
            w = s["wq"][i].double() * torch.kron(two, torch.ones((128, 128), device="cuda", dtype=torch.float64))[:n, :k]
        else:
            n, k = s["w"].shape[1:]
            w = torch.empty((n, k), dtype=torch.float64, device="cuda")
            for a in range(0, n, 128):
                strip = s["w"][i, a:a + 128].double()
                for b in range(0, k, 128):
                    blk = strip[:, b:b + 128]
                    w[a:a + 128, b:b + 128] = _exact_block(blk.reshape(1, -1)).reshape(blk.shape)
        y.append(x[rows] @ w.t())
        if g is not None:
            dx.append(g[rows] @ w)
    out = {"y": torch.cat(y)}
    if g is not None:
        out["dx"] = torch.cat(dx)
    return out
