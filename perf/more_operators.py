"""Timed cases of what a Mixture-of-Experts block needs around its routing and its products.

Three kinds of case, each a call or a few calls that a program makes in one go:

  gated   the gated feed-forward of the experts: both projections, the activation and their product; "serve":
          the hidden rows; "train": with the projections kept and the gradient through the down product and the
          activation; "block": y = down(act(gate) * up) and the gradients of x and of both weights
  norm    the norms before and after a block with its gate and residual scale; "train": with the gradients
  clip    the norm of all gradients and the clipped gradients

run() computes the plain forms below (elementary torch operations in fp32, in fp64 for the long sum of squares) or,
where `own` is true, calls the package.  Tensors that one operator writes and the next one reads (the kept
projections, the hidden rows and the projections' gradient; the residual stream) are in the inputs' type, in every form.
exact() is the same mathematics in fp64, written apart.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}
EPS = 1e-6


def listed():
    return [
        # one token of a serving loop through the 8-expert top-2 layer (K=4096, F=14336): the weights' bytes
        {"name": "gated_token", "kind": "gated", "rows": 2, "experts": 8, "ffn": 14336, "hidden": 4096,
         "act": "silu", "mode": "serve"},
        # a decode batch of 61 tokens, 8 choices, over the fine-grained layer's 64 experts
        {"name": "gated_decode", "kind": "gated", "rows": 488, "experts": 64, "ffn": 1536, "hidden": 2048,
         "act": "silu", "mode": "serve"},
        # odd sizes: widths that end inside tiles, groups of any size, the other activation, with its gradient
        {"name": "gated_ragged", "kind": "gated", "rows": 3001, "experts": 16, "ffn": 1000, "hidden": 2000,
         "act": "gelu_tanh", "mode": "train"},
        # a prompt batch of the 8-expert layer: 8192 tokens, top-2
        {"name": "gated_prompt", "kind": "gated", "rows": 16384, "experts": 8, "ffn": 14336, "hidden": 4096,
         "act": "silu", "mode": "serve"},
        # a training step of the gate_up / down layer of 16 experts: the whole block and all its gradients
        {"name": "gated_block", "kind": "gated", "rows": 16384, "experts": 16, "ffn": 2048, "hidden": 6144,
         "act": "silu", "mode": "block"},
        # one token of a serving loop: the norm after a block, gate, residual and the norm before the next
        {"name": "norm_token", "kind": "norm", "tokens": 1, "hidden": 4096, "dtype": "bf16", "post": True,
         "gate": True, "scale": 1.0, "train": False},
        # the fine-grained layer's training batch: plain residual and the norm before the block, fp32 stream
        {"name": "norm_fine_train", "kind": "norm", "tokens": 4096, "hidden": 2048, "dtype": "fp32", "post": False,
         "gate": False, "scale": 0.25, "train": True},
        # a long batch of wide rows, an odd number of tokens, everything fused
        {"name": "norm_wide_train", "kind": "norm", "tokens": 16383, "hidden": 7168, "dtype": "bf16", "post": True,
         "gate": True, "scale": 0.5, "train": True},
        # a prompt's rows, no gradients, both norms without a gate
        {"name": "norm_prompt", "kind": "norm", "tokens": 8192, "hidden": 4096, "dtype": "bf16", "post": True,
         "gate": False, "scale": 1.0, "train": False},
        # the small parameters of a layer: router and norm weights: latency
        {"name": "clip_small", "kind": "clip", "fp32": 7, "bf16": 2, "elements": 300_000, "clipped": True},
        # many tensors of odd sizes, two types, starting anywhere in two flat buffers
        {"name": "clip_many", "kind": "clip", "fp32": 200, "bf16": 101, "elements": 60_000_000, "clipped": True},
        # the main_grads of the fine-grained layer's experts: [64, 2 * 1536, 2048] and [64, 2048, 1536] in fp32
        {"name": "clip_experts", "kind": "clip", "fp32": 2, "bf16": 0, "elements": 64 * 3 * 1536 * 2048,
         "clipped": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


#: products of one pass, as multiples of rows * ffn * hidden
PRODUCTS = {"serve": 2, "train": 3, "block": 9}


def draw(rng):
    kind = rng.choice(["gated", "gated", "norm", "clip"])
    if kind == "gated":
        while True:
            c = {"kind": kind, "rows": _log_int(rng, 1, 16384), "experts": _log_int(rng, 1, 64),
                 "ffn": 8 * _log_int(rng, 16, 1792), "hidden": 8 * _log_int(rng, 16, 896),
                 "act": rng.choice(["silu", "gelu_tanh"]), "mode": rng.choice(["serve", "train", "block"])}
            size = c["ffn"] * c["hidden"]
            if 2 * PRODUCTS[c["mode"]] * c["rows"] * size <= 3.7e12 and c["experts"] * size <= 2.1e8:
                return c
    if kind == "norm":
        hidden = 8 * _log_int(rng, 8, 1024)
        return {"kind": kind, "tokens": min(_log_int(rng, 1, 32768), 16383 * 7168 // (2 * hidden)), "hidden": hidden,
                "dtype": rng.choice(["bf16", "bf16", "fp32"]), "post": rng.random() < 0.5, "gate": rng.random() < 0.5,
                "scale": rng.choice([1.0, 0.5, 0.22]), "train": rng.random() < 0.7}
    return {"kind": kind, "fp32": rng.randint(1, 300), "bf16": rng.randint(0, 300),
            "elements": _log_int(rng, 10_000, 300_000_000), "clipped": rng.random() < 0.8}


def work(case):
    c = case
    if c["kind"] == "gated":
        m, e, f, k = c["rows"], c["experts"], c["ffn"], c["hidden"]
        used = e * (1 - (1 - 1 / e) ** m)                         # experts with rows, expected
        flops = 2 * PRODUCTS[c["mode"]] * m * f * k
        if c["mode"] == "serve":
            return {"bytes": 2 * m * (k + f) + int(4 * used * f * k), "flops": flops}
        if c["mode"] == "train":                                  # x, dy, both weights; h, gate_up, its gradient
            return {"bytes": 2 * m * (2 * k + 5 * f) + int(6 * used * f * k), "flops": flops}
        return {"bytes": 2 * m * 4 * k + int(6 * used * f * k) + 6 * e * f * k, "flops": flops}
    if c["kind"] == "norm":
        rows = 4 + (4 if c["train"] else 0)                       # residual, y, out, normed; dout, dnormed, dresidual, dy
        return {"bytes": rows * c["tokens"] * c["hidden"] * BYTES[c["dtype"]],
                "flops": c["tokens"] * c["hidden"] * (30 if c["train"] else 10)}
    b = _clip_bytes(c)
    return {"bytes": 2 * b, "flops": 3 * c["elements"]}


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


def _weight(e, n, k, gen):
    w = torch.empty((e, n, k), dtype=torch.bfloat16, device="cuda")
    for i in range(e):
        w[i] = _randn((n, k), gen, 1.0 / math.sqrt(k))
    return w


def _clip_counts(c):
    """Elements of the fp32 and of the bf16 tensors."""
    n = c["fp32"] + c["bf16"]
    to32 = c["elements"] * c["fp32"] // n
    return max(to32, c["fp32"]), max(c["elements"] - to32, c["bf16"]) if c["bf16"] else 0


def _clip_bytes(c):
    a, b = _clip_counts(c)
    return 4 * a + 2 * b


def _split(total, parts, seed):
    """Lengths of `parts` consecutive tensors that fill `total` elements, one at least each, of any size."""
    if parts == 2 and total % 3 == 0:                             # a gated block's two weights
        return [total // 3 * 2, total // 3]
    rng = np.random.default_rng(seed)
    n = 1 + np.floor(rng.dirichlet(np.full(parts, 0.7)) * (total - parts)).astype(np.int64)
    n[-1] += total - n.sum()
    return [int(x) for x in n]


def prepare(case, seed):
    c, gen = case, _gen(seed)
    s = dict(case)
    if c["kind"] == "gated":
        m, e, f, k = c["rows"], c["experts"], c["ffn"], c["hidden"]
        sizes = _sizes(m, e, seed)
        s["most"] = int(sizes.max())                              # rows of the largest group
        s["offs"] = torch.from_numpy(np.cumsum(sizes).astype(np.int32)).cuda()
        loud = 1.0 + 7.0 * (_rand((1, k), gen) < 0.01)            # a few channels are louder
        s["x"] = (_randn((m, k), gen) * loud).to(torch.bfloat16)
        s["w"] = _weight(e, 2 * f, k, gen)
        if c["mode"] != "serve":
            s["w_down"] = _weight(e, k, f, gen)
            s["dy"] = _randn((m, k), gen).to(torch.bfloat16)
        if c["mode"] == "block":
            for name in ("x", "w", "w_down"):
                s[name].requires_grad_()
    elif c["kind"] == "norm":
        t, h, dt = c["tokens"], c["hidden"], DTYPES[c["dtype"]]
        s["residual"] = _randn((t, h), gen, 2.0).to(dt)
        s["y"] = (_randn((t, h), gen) * (0.5 + _rand((t, 1), gen))).to(dt)
        s["weight"] = (1.0 + _randn((h,), gen, 0.2)).to(dt)
        s["post_weight"] = (1.0 + _randn((h,), gen, 0.2)).to(dt) if c["post"] else None
        s["gate_of"] = torch.sigmoid(_randn((t,), gen)) if c["gate"] else None
        if c["train"]:
            s["dout"] = _randn((t, h), gen).to(dt)
            s["dnormed"] = _randn((t, h), gen).to(dt)
    else:
        a, b = _clip_counts(c)
        s["flat"], s["out"], s["grads"], s["outs"] = [], [], [], []
        for n, parts, dt in ((a, c["fp32"], torch.float32), (b, c["bf16"], torch.bfloat16)):
            if not parts:
                continue
            flat = (_randn((n,), gen) * 0.01).to(dt)              # (gradients of a loss that is a mean over tokens)
            lengths = _split(n, parts, seed + parts)
            s["flat"].append(flat)
            s["out"].append(torch.empty_like(flat))
            s["grads"] += list(torch.split(flat, lengths))
            s["outs"] += list(torch.split(s["out"][-1], lengths))
        s["max_norm"] = 1.0 if c["clipped"] else 1e6              # the norm is about 0.01 sqrt(elements)
        if c["clipped"] and c["elements"] < 20_000:
            s["max_norm"] = 0.1
    return s


# ------------------------------------------------------------------------------------ plain forms
def _padded(rows, s):
    """Rows in fp32 as [E, most, columns], zeros behind each group's, and the place of each row."""
    m, e, most, offs = rows.shape[0], s["experts"], s["most"], s["offs"]
    row = torch.arange(m, device=rows.device, dtype=torch.int32)
    group = torch.bucketize(row, offs, right=True)
    start = torch.cat([torch.zeros_like(offs[:1]), offs[:-1]])
    at = group * most + (row - start[group])
    out = torch.zeros((e * most, rows.shape[1]), device=rows.device)
    out[at] = rows.float()
    return out.reshape(e, most, -1), at


def _logistic(a, act):
    """(s, q'): the logistic function of q(a) and q's derivative."""
    if act == "silu":
        return torch.sigmoid(a), 1.0
    c = 2.0 * math.sqrt(2.0 / math.pi)
    return torch.sigmoid(c * (a + 0.044715 * a * a * a)), c * (1.0 + 0.134145 * a * a)


def _times_t(rows, w):
    """rows [E, most, K] by w [E, N, K] transposed."""
    return torch.bmm(rows, w.float().transpose(1, 2).contiguous())


def _gated(s):
    with torch.no_grad():
        f, act, mode = s["ffn"], s["act"], s["mode"]
        x, at = _padded(s["x"], s)
        ab = _times_t(x, s["w"])
        flat = ab.reshape(-1, 2 * f)[at]
        a, b = flat[:, :f], flat[:, f:]
        h = (a * _logistic(a, act)[0] * b).to(torch.bfloat16)
        if mode == "serve":
            return {"h": h}
        gate_up = flat.to(torch.bfloat16)
        del ab, flat, a, b
        dy, _ = _padded(s["dy"], s)
        dh = torch.bmm(dy, s["w_down"].float()).reshape(-1, f)[at]
        a, b = gate_up[:, :f].float(), gate_up[:, f:].float()
        sg, dq = _logistic(a, act)
        dgate_up = torch.cat([dh * b * (sg + a * sg * (1.0 - sg) * dq), dh * a * sg], dim=1).to(torch.bfloat16)
        if mode == "train":
            return {"h": h, "gate_up": gate_up, "dgate_up": dgate_up}
        del dh, a, b, sg, dq
        hp, _ = _padded(h, s)
        y = _times_t(hp, s["w_down"]).reshape(-1, s["hidden"])[at].to(torch.bfloat16)
        dw_down = torch.bmm(dy.transpose(1, 2).contiguous(), hp).to(torch.bfloat16)
        del hp, dy
        dp, _ = _padded(dgate_up, s)
        dx = torch.bmm(dp, s["w"].float()).reshape(-1, s["hidden"])[at].to(torch.bfloat16)
        dw = torch.bmm(dp.transpose(1, 2).contiguous(), x).to(torch.bfloat16)
        return {"y": y, "dx": dx, "dw": dw, "dw_down": dw_down}


def _norm(s):
    r, y, dt = s["residual"].float(), s["y"].float(), s["residual"].dtype
    w, scale = s["weight"].float(), s["scale"]
    z, post = y, s["post_weight"]
    if post is not None:
        ry = torch.rsqrt((y * y).mean(dim=1, keepdim=True) + EPS)
        z = y * ry * post.float()
    g = scale if s["gate_of"] is None else scale * s["gate_of"][:, None]
    out = (r + g * z).to(dt)
    o = out.float()
    ro = torch.rsqrt((o * o).mean(dim=1, keepdim=True) + EPS)
    got = {"out": out, "normed": (o * ro * w).to(dt)}
    if s["train"]:
        dn, xh = s["dnormed"].float(), o * ro
        dw = dn * w
        do = s["dout"].float() + ro * (dw - xh * (dw * xh).mean(dim=1, keepdim=True))
        got["dresidual"], got["dweight"] = do.to(dt), (dn * xh).sum(dim=0).to(dt)
        dz = g * do
        if s["gate_of"] is not None:
            got["dgate"] = scale * (do * z).sum(dim=1)
        if post is not None:
            yh, dp = y * ry, dz * post.float()
            got["dpost_weight"] = (dz * yh).sum(dim=0).to(dt)
            dz = ry * (dp - yh * (dp * yh).mean(dim=1, keepdim=True))
        got["dy"] = dz.to(dt)
    return got


def _clip(s):
    # (the flat buffers hold nothing but the tensors: one operation over each does for all of its tensors)
    norm = torch.sqrt(sum(f.double().square().sum() for f in s["flat"]))
    by = torch.clamp(s["max_norm"] / (norm + EPS), max=1.0).float()
    return {"norm": norm.float(), "grads": [(f.float() * by).to(f.dtype) for f in s["flat"]]}


# -------------------------------------------------------------------------------------- one pass
def run(state):
    s = state
    if not own:
        return {"gated": _gated, "norm": _norm, "clip": _clip}[s["kind"]](s)
    import moe_ragged_bf16_amd as mdg
    if s["kind"] == "gated":
        if s["mode"] == "block":
            y = mdg.grouped_gated_ffn(s["x"], s["w"], s["w_down"], s["offs"], activation=s["act"])
            dx, dw, dw_down = torch.autograd.grad(y, (s["x"], s["w"], s["w_down"]), s["dy"])
            return {"y": y, "dx": dx, "dw": dw, "dw_down": dw_down}
        train = s["mode"] == "train"
        r = mdg.grouped_gated_gemm_fwd(s["x"], s["w"], s["offs"], activation=s["act"], keep=train)
        if not train:
            return {"h": r.h}
        d = mdg.grouped_gated_gemm_dgrad(s["dy"], s["w_down"], r.gate_up, s["offs"], activation=s["act"])
        return {"h": r.h, "gate_up": r.gate_up, "dgate_up": d}
    if s["kind"] == "norm":
        how = {"weight": s["weight"], "post_weight": s["post_weight"], "gate": s["gate_of"], "scale": s["scale"]}
        r = mdg.block_norm_fwd(s["residual"], s["y"], eps=EPS, **how)
        got = {"out": r.out, "normed": r.normed}
        if s["train"]:
            d = mdg.block_norm_bwd(s["dout"], s["dnormed"], r, s["y"], **how)
            got |= {k: v for k, v in d._asdict().items() if v is not None}
        return got
    norm = mdg.clip_grads(s["grads"], s["max_norm"], out=s["outs"])
    return {"norm": norm, "grads": s["out"]}


# ------------------------------------------------------------------------------ the same in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"gated": _exact_gated, "norm": _exact_norm, "clip": _exact_clip}[case["kind"]](s)


def _bf16(v):
    return v.to(torch.bfloat16).double()


def _exact_act(a, act):
    """act(a) and its derivative in fp64."""
    if act == "silu":
        v = 1.0 / (1.0 + torch.exp(-a))
        return a * v, v * (1.0 + a * (1.0 - v))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (a + 0.044715 * a ** 3))
    return 0.5 * a * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * a * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * a * a)


def _exact_gated(s):
    ends, f, act, mode = s["offs"].tolist(), s["ffn"], s["act"], s["mode"]
    got = {}
    with torch.no_grad():
        for i, end in enumerate(ends):
            rows = slice(ends[i - 1] if i else 0, end)
            x, w = s["x"][rows].double(), s["w"][i].double()
            a, b = x @ w[:f].t(), x @ w[f:].t()
            one = {"h": _exact_act(a, act)[0] * b}
            if mode != "serve":
                dy, wd = s["dy"][rows].double(), s["w_down"][i].double()
                dh = dy @ wd
                one["gate_up"] = torch.cat([a, b], dim=1)
                a, b = _bf16(a), _bf16(b)
                v, d = _exact_act(a, act)
                one["dgate_up"] = torch.cat([dh * b * d, dh * v], dim=1)
            if mode == "block":
                h, dgu = _bf16(one["h"]), _bf16(one["dgate_up"])
                one = {"y": h @ wd.t(), "dx": dgu @ w, "dw": (dgu.t() @ x)[None], "dw_down": (dy.t() @ h)[None]}
            for k, v in one.items():
                got.setdefault(k, []).append(v)
            del one
        return {k: torch.cat(v) for k, v in got.items()}


def _exact_norm(s):
    r, y, w = s["residual"].double(), s["y"].double(), s["weight"].double()
    t, h = y.shape
    gate = torch.full((t, 1), s["scale"], dtype=torch.float64, device=y.device)
    if s["gate_of"] is not None:
        gate = gate * s["gate_of"].double()[:, None]
    post = None if s["post_weight"] is None else s["post_weight"].double()
    sy = torch.sqrt(y.square().sum(dim=1, keepdim=True) / h + EPS)
    z = y if post is None else y / sy * post
    out = r + gate * z
    o = out.to(s["residual"].dtype).double()                      # the stream is stored in its type
    so = torch.sqrt(o.square().sum(dim=1, keepdim=True) / h + EPS)
    got = {"out": out, "normed": o / so * w}
    if s["train"]:
        dn = s["dnormed"].double()
        u = dn * w
        do = s["dout"].double() + u / so - o * (u * o).sum(dim=1, keepdim=True) / (h * so ** 3)
        got["dresidual"], got["dweight"] = do, (dn * o / so).sum(dim=0)
        if s["gate_of"] is not None:
            got["dgate"] = s["scale"] * (do * z).sum(dim=1)
        dz = gate * do
        if post is not None:
            got["dpost_weight"] = (dz * y / sy).sum(dim=0)
            v = dz * post
            dz = v / sy - y * (v * y).sum(dim=1, keepdim=True) / (h * sy ** 3)
        got["dy"] = dz
    return got


def _exact_clip(s):
    total = math.fsum(float(torch.linalg.vector_norm(f.double())) ** 2 for f in s["flat"])
    norm = math.sqrt(total)
    by = min(1.0, s["max_norm"] / (norm + EPS))
    return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": [f.double() * by for f in s["flat"]]}
