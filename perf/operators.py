"""The expert path's operators, measured: the router, the experts' products
over ragged segments and their gradients, and the 4-bit products of decoding.

Every case is one call of one operator (``op``) on synthetic inputs of the
shapes that a Mixture-of-Experts layer gives it.  Rows of one expert lie
together, as ``dispatch_rows`` leaves them: expert e owns the rows from
``expert_offsets[e]``, ``problem_sizes[e][0]`` of them, and the rows up to the
next offset are padding, whose contents nobody wrote (NaN here).

``run`` computes the plain form (elementary torch operations in float32, or
float64 where a selection depends on it) or, with ``own``, makes the library's
calls.  ``exact`` computes the same from the definitions in float64.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # Router of a decode batch of 32 tokens over 256 experts: latency.
        {"name": "gating_decode_T32", "op": "gating", "tokens": 32, "experts": 256, "topk": 8,
         "dtype": "bf16", "scoring": "softmax", "bias": False, "off": 0},
        # Router of a long prefill over 288 expert slots, some switched off
        # (masked with -inf), sigmoid scores with a selection bias.
        {"name": "gating_prefill_T65536", "op": "gating", "tokens": 65536, "experts": 288,
         "topk": 8, "dtype": "f32", "scoring": "sigmoid", "bias": True, "off": 3},
        # The router's gradient in training.
        {"name": "gating_backward_T16384", "op": "gating_backward", "tokens": 16384,
         "experts": 128, "topk": 8, "dtype": "bf16", "scoring": "softmax", "off": 0},
        # Gate and up projection of 32 tokens x 8 picks over 256 experts, with
        # the gated activation: each expert sees about one row, the weights
        # are the traffic.
        {"name": "gated_decode_rows256", "op": "gemm", "rows": 256, "experts": 256,
         "n": 2048, "k": 4096, "dtype": "bf16", "out": "bf16", "gated": True, "align": 1,
         "skew": 0.0},
        # The same projection of 4096 picks on one rank of 32 experts, hidden
        # 7168, segments padded to 128 rows: between the two bounds.
        {"name": "gated_prefill_rows4096", "op": "gemm", "rows": 4096, "experts": 32,
         "n": 2048, "k": 7168, "dtype": "bf16", "out": "bf16", "gated": True, "align": 128,
         "skew": 0.0},
        # Down projection of 32768 picks: bound by the matrix cores.
        {"name": "down_prefill_rows32768", "op": "gemm", "rows": 32768, "experts": 32,
         "n": 7168, "k": 2048, "dtype": "bf16", "out": "bf16", "gated": False, "align": 1,
         "skew": 0.5},
        # Training: gradient of the rows through the transposed weights.
        {"name": "dgrad_rows16384", "op": "dgrad", "rows": 16384, "experts": 16, "n": 4096,
         "k": 4096, "dtype": "f16", "out": "f16", "align": 1, "skew": 1.0},
        # Training: gradient of the weights in float32, ragged sums over rows.
        {"name": "wgrad_rows16384", "op": "wgrad", "rows": 16384, "experts": 16, "n": 4096,
         "k": 4096, "dtype": "bf16", "out": "f32", "align": 128, "skew": 0.5},
        # Training: gradient of the gated activation between the two products.
        {"name": "silu_backward_rows16384", "op": "silu_backward", "rows": 16384, "experts": 16,
         "n": 2048, "dtype": "bf16", "align": 128, "skew": 0.5},
        # FP8 serving: block-scaled e4m3 rows (as dispatch_rows_fp8 writes
        # them) and weights, 16384 picks over 128 experts, skewed routing.
        {"name": "fp8_prefill_rows16384", "op": "fp8", "rows": 16384, "experts": 128,
         "n": 4096, "k": 4096, "out": "bf16", "gated": False, "align": 128, "skew": 0.7},
        # 4-bit serving of a single token: 8 picks of 256 experts.
        {"name": "w4_token_rows8", "op": "w4", "rows": 8, "experts": 256, "n": 2048, "k": 4096,
         "group": 128, "dtype": "bf16", "gated": True, "zeros": False, "skew": 0.0},
        # 4-bit serving of a batch of 32 tokens on one rank of 64 experts, with
        # zero points.
        {"name": "w4_batch_rows256", "op": "w4", "rows": 256, "experts": 64, "n": 7168,
         "k": 2048, "group": 64, "dtype": "f16", "gated": False, "zeros": True, "skew": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gating", "gating_backward", "gemm", "gemm", "gemm", "dgrad", "wgrad",
                     "silu_backward", "fp8", "w4", "w4"))
    dtype = rng.choice(("bf16", "f16"))
    skew = rng.choice((0.0, 0.5, 1.0))
    align = rng.choice((1, 1, 16, 128))
    if op in ("gating", "gating_backward"):
        c = {"op": op, "tokens": _log(rng, 1, 32768), "experts": rng.randint(16, 512),
             "topk": rng.randint(1, 10), "dtype": rng.choice(("bf16", "f16", "f32")),
             "scoring": rng.choice(("softmax", "sigmoid")), "off": rng.choice((0, 0, 5))}
        if op == "gating":
            c["bias"] = c["scoring"] == "sigmoid" and rng.random() < 0.7
        return c
    if op == "silu_backward":
        return {"op": op, "rows": _log(rng, 1, 16384), "experts": rng.randint(1, 64),
                "n": rng.randint(64, 3000), "dtype": dtype, "align": align, "skew": skew}
    if op == "fp8":
        return {"op": op, "rows": _log(rng, 1, 16384), "experts": rng.randint(1, 48),
                "n": 16 * rng.randint(16, 256), "k": 128 * rng.randint(2, 40),
                "out": dtype, "gated": rng.random() < 0.5,
                "align": align, "skew": skew}
    if op == "w4":
        group = rng.choice((32, 64, 128))
        return {"op": op, "rows": _log(rng, 1, 512), "experts": rng.randint(1, 48),
                "n": rng.randint(200, 3000), "k": 128 * rng.randint(2, 40), "group": group,
                "dtype": dtype, "gated": rng.random() < 0.5, "zeros": rng.random() < 0.5,
                "skew": skew}
    # 8 elements are 16 bytes: the usual widths; now and then an odd one
    k = 8 * rng.randint(32, 640) - (rng.randint(1, 7) if rng.random() < 0.1 else 0)
    c = {"op": op, "rows": _log(rng, 1, 16384), "experts": rng.randint(1, 32),
         "n": rng.randint(100, 2500) if rng.random() < 0.3 else 8 * rng.randint(16, 320), "k": k,
         "dtype": dtype, "out": rng.choice((dtype, "f32")), "align": align, "skew": skew}
    if op == "gemm":
        c["gated"] = rng.random() < 0.5
    return c


def _active(c):
    """Experts with a row, on average (all of them but in small batches)."""
    return min(c["rows"], c["experts"]) if c["rows"] < c["experts"] else c["experts"]


def work(c):
    op = c["op"]
    if op in ("gating", "gating_backward"):
        t, e, k, b = c["tokens"], c["experts"], c["topk"], BYTES[c["dtype"]]
        if op == "gating":
            return {"bytes": t * e * b + t * k * 8 + (4 * e if c["bias"] else 0),
                    "flops": 4 * t * e}
        return {"bytes": 2 * t * e * b + t * k * 8, "flops": 8 * t * e}
    r, n = c["rows"], c["n"]
    if op == "silu_backward":
        return {"bytes": 5 * r * n * BYTES[c["dtype"]], "flops": 12 * r * n}
    k, e = c["k"], _active(c)
    wide = 2 * n if c.get("gated") else n
    flops = 2 * r * wide * k
    if op == "fp8":
        by = r * k * (1 + 4 / 128) + e * wide * k * (1 + 4 / 16384) + r * n * BYTES[c["out"]]
    elif op == "w4":
        b = BYTES[c["dtype"]]
        by = r * k * b + e * wide * (k / 2 + k // c["group"] * (b + c["zeros"])) + r * n * b
    elif op == "wgrad":
        b = BYTES[c["dtype"]]
        by = r * (n + k) * b + c["experts"] * n * k * BYTES[c["out"]]
    elif op == "dgrad":
        by = (r * n + e * n * k) * BYTES[c["dtype"]] + r * k * BYTES[c["out"]]
    else:
        by = (r * k + e * wide * k) * BYTES[c["dtype"]] + r * n * BYTES[c["out"]]
    return {"bytes": by, "flops": flops}


# ---- inputs ------------------------------------------------------------------

def _normal(g, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale).to(dtype)


def _weights(g, e, rows, k, dtype):
    """[e, rows, k] from N(0, 1/k), an expert at a time (float32 of all of them
    would be twice the tensor)."""
    w = torch.empty(e, rows, k, device=DEV, dtype=dtype)
    for i in range(e):
        w[i] = torch.randn(rows, k, generator=g, device=DEV).mul_(k ** -0.5)
    return w


def _segments(c, seed):
    """Routing of ``rows`` picks: expert popularity ~ rank^-skew, the ranks
    shuffled; few rows go to distinct experts, as one token's picks do."""
    r, e = c["rows"], c["experts"]
    g = torch.Generator().manual_seed(seed * 31 + 7)
    if r < e and not c["skew"]:
        counts = torch.zeros(e, dtype=torch.int64)
        counts[torch.randperm(e, generator=g)[:r]] = 1
    else:
        p = (torch.randperm(e, generator=g).double() + 1) ** -c["skew"]
        counts = torch.bincount(torch.multinomial(p, r, replacement=True, generator=g),
                                minlength=e)
    a = c.get("align", 1)
    offsets = torch.zeros(e + 1, dtype=torch.int64)
    offsets[1:] = torch.cumsum((counts + a - 1) // a * a, 0)
    sizes = torch.stack((counts, torch.zeros_like(counts), torch.zeros_like(counts)), 1)
    capacity = r + e * (a - 1)
    return {"offsets": offsets.to(torch.int32).to(DEV), "sizes": sizes.to(torch.int32).to(DEV),
            "cap": int(counts.max()), "capacity": capacity}


def _padding(s):
    """[capacity] truth values: rows that belong to no expert."""
    o, n = s["offsets"].long(), s["sizes"][:, 0].long()
    r = torch.arange(s["capacity"], device=DEV)[:, None]
    return ~((r >= o[:-1]) & (r < o[:-1] + n)).any(1)


def prepare(case, seed):
    c, op = case, case["op"]
    g = torch.Generator(device=DEV).manual_seed(seed)
    if op in ("gating", "gating_backward"):
        t, e, k = c["tokens"], c["experts"], c["topk"]
        logits = _normal(g, (t, e), TYPES[c["dtype"]], 1.5)
        if c["off"]:
            logits[:, torch.randperm(e, generator=g, device=DEV)[:c["off"]]] = -math.inf
        s = {"logits": logits, "bias": None}
        if c.get("bias"):
            s["bias"] = _normal(g, (e,), torch.float32, 0.05)
        if op == "gating":
            s["ids"] = torch.empty(t, k, dtype=torch.int32, device=DEV)
            s["weights"] = torch.empty(t, k, dtype=torch.float32, device=DEV)
        else:
            s["ids"] = torch.sort(logits.float(), dim=1, descending=True, stable=True)[1][:, :k].int().contiguous()
            s["grad"] = _normal(g, (t, k), torch.float32)
            s["grad_logits"] = torch.empty_like(logits)
        return {"case": dict(c), **s}
    s = _segments(c, seed)
    cap, e, n = s["capacity"], c["experts"], c["n"]
    pad = _padding(s)
    if op == "silu_backward":
        dt = TYPES[c["dtype"]]
        s["gate_up"] = _normal(g, (cap, 2 * n), dt)
        s["grad"] = _normal(g, (cap, n), dt)
        s["gate_up"][pad] = math.nan
        s["grad"][pad] = math.nan
        s["result"] = torch.zeros(cap, 2 * n, dtype=dt, device=DEV)
        return {"case": dict(c), **s}
    k = c["k"]
    wide = 2 * n if c.get("gated") else n
    if op == "fp8":
        x = _normal(g, (cap, k), torch.float32).view(cap, k // 128, 128)
        sc = x.abs().amax(2) / 448
        s["x"] = (x / sc[..., None]).view(cap, k).to(torch.float8_e4m3fn)
        s["x_scales"] = sc.contiguous()
        s["x"].view(torch.uint8)[pad] = 0x7f                       # NaN
        s["x_scales"][pad] = math.nan
        nb = (wide + 127) // 128
        s["w"] = torch.empty(e, wide, k, dtype=torch.float8_e4m3fn, device=DEV)
        s["w_scales"] = torch.empty(e, nb, k // 128, device=DEV)
        for i in range(e):
            w = torch.zeros(nb * 128, k, device=DEV)
            w[:wide] = torch.randn(wide, k, generator=g, device=DEV) * k ** -0.5
            b = w.view(nb, 128, k // 128, 128)
            ws = b.abs().amax((1, 3)) / 448
            s["w_scales"][i] = ws
            s["w"][i] = (b / ws[:, None, :, None]).view(nb * 128, k)[:wide].to(torch.float8_e4m3fn)
        s["result"] = torch.zeros(cap, n, dtype=TYPES[c["out"]], device=DEV)
        return {"case": dict(c), **s}
    dt = TYPES[c["dtype"]]
    if op == "w4":
        s["x"] = _normal(g, (cap, k), dt)
        s["w"] = torch.randint(0, 256, (e, wide, k // 2), generator=g, device=DEV,
                               dtype=torch.uint8)
        u = torch.rand(e, wide, k // c["group"], generator=g, device=DEV)
        s["w_scales"] = ((0.5 + u) * (k ** -0.5 / 4.6)).to(dt)
        s["zeros"] = torch.randint(5, 11, (e, wide, k // c["group"]), generator=g, device=DEV,
                                   dtype=torch.uint8) if c["zeros"] else None
        s["result"] = torch.zeros(cap, n, dtype=dt, device=DEV)
        return {"case": dict(c), **s}
    if op == "wgrad":
        s["grad"] = _normal(g, (cap, n), dt)
        s["x"] = _normal(g, (cap, k), dt)
        s["grad"][pad] = math.nan
        s["x"][pad] = math.nan
        s["result"] = torch.zeros(e, n, k, dtype=TYPES[c["out"]], device=DEV)
        return {"case": dict(c), **s}
    s["w"] = _weights(g, e, wide, k, dt)
    s["x"] = _normal(g, (cap, n if op == "dgrad" else k), dt, n ** -0.5 if op == "dgrad" else 1.0)
    s["x"][pad] = math.nan
    s["result"] = torch.zeros(cap, k if op == "dgrad" else n, dtype=TYPES[c["out"]], device=DEV)
    return {"case": dict(c), **s}


# ---- the plain form ----------------------------------------------------------

def _rows_by_expert(s):
    """Row indices [E, cap] and which of them are an expert's rows."""
    o, n = s["offsets"].long(), s["sizes"][:, 0].long()
    i = torch.arange(s["cap"], device=DEV)
    idx = o[:-1, None] + i
    live = i < n[:, None]
    return torch.where(live, idx, s["capacity"]), live


def _gather(x, idx, live):
    """[E, cap, width] float32, zeros where an expert has fewer rows."""
    last = max(x.shape[0] - 1, 0)
    return torch.where(live[..., None], x[idx.clamp(max=last)].float(), 0.0)


def _scatter(y, idx, rows, dtype):
    """Rows back in their places, zeros elsewhere."""
    out = torch.zeros(rows + 1, y.shape[-1], dtype=dtype, device=DEV)
    out[idx.reshape(-1)] = y.reshape(-1, y.shape[-1]).to(dtype)
    return out[:rows]


def _expert_of_row(s):
    """[rows] of a batch without padding."""
    r = torch.arange(s["capacity"], device=DEV)
    return (r[:, None] >= s["offsets"][1:].long()).sum(1)


def _silu_mul(y, n):
    g, u = y[..., :n], y[..., n:]
    return g / (1 + torch.exp(-g)) * u


def _products(s, x, w, gated, dtype):
    """x [rows, K] float32 rows by expert times w [E, N, K]: w is a function of
    expert indices, or None for all of them, that gives float32 weights."""
    c = s["case"]
    if c["rows"] < c["experts"] and c.get("align", 1) == 1:      # each row with its own weights
        y = (x.float()[:, None] @ w(_expert_of_row(s)).transpose(1, 2))[:, 0]
        return (_silu_mul(y, c["n"]) if gated else y).to(dtype)
    idx, live = _rows_by_expert(s)
    y = torch.bmm(_gather(x, idx, live), w(None).transpose(1, 2))
    return _scatter(_silu_mul(y, c["n"]) if gated else y, idx, s["capacity"], dtype)


def _blocks(scales, rows, block):
    return scales.repeat_interleave(block, 1)[:, :rows].repeat_interleave(128, 2)


def _plain_gating(s):
    c, x = s["case"], s["logits"].double()
    x = torch.where(torch.isnan(x), -math.inf, x)
    key = x
    if s["bias"] is not None:
        key = torch.where(x > -math.inf, 1 / (1 + torch.exp(-x)) + s["bias"].double(), -math.inf)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    ids = ids[:, :c["topk"]]
    live = top[:, :c["topk"]] > -math.inf
    chosen = torch.where(live, torch.gather(x, 1, ids), -math.inf).float()
    if c["scoring"] == "softmax":
        m = chosen.amax(1, keepdim=True)
        p = torch.where(live, torch.where(chosen == m, 1.0, torch.exp(chosen - m)), 0.0)
    else:
        p = torch.where(live, 1 / (1 + torch.exp(-chosen)), 0.0)
    total = p.sum(1, keepdim=True)
    return torch.where(live, ids, -1).int(), torch.where(total > 0, p / total, 0.0)


def _plain_gating_backward(s):
    c, x = s["case"], s["logits"].float()
    ids, g = s["ids"].long(), s["grad"]
    chosen = torch.gather(x, 1, ids)
    if c["scoring"] == "softmax":
        w = torch.exp(chosen - chosen.amax(1, keepdim=True))
        w = w / w.sum(1, keepdim=True)
        d = w * (g - (w * g).sum(1, keepdim=True))
    else:
        p = 1 / (1 + torch.exp(-chosen))
        total = p.sum(1, keepdim=True)
        w = p / total
        d = (g - (w * g).sum(1, keepdim=True)) / total * p * (1 - p)
    d = torch.where(chosen > -math.inf, d, 0.0)
    return torch.zeros_like(x).scatter_(1, ids, d).to(s["logits"].dtype)


def _plain_silu_backward(s):
    n = s["case"]["n"]
    idx, live = _rows_by_expert(s)
    gu, d = _gather(s["gate_up"], idx, live), _gather(s["grad"], idx, live)
    g, u = gu[..., :n], gu[..., n:]
    p = 1 / (1 + torch.exp(-g))
    y = torch.cat((d * u * p * (1 + g * (1 - p)), d * g * p), -1)
    return _scatter(y, idx, s["capacity"], s["result"].dtype)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "gating":
        return _plain_gating(s)
    if op == "gating_backward":
        return _plain_gating_backward(s)
    if op == "silu_backward":
        return _plain_silu_backward(s)
    gated, dtype = c.get("gated", False), s["result"].dtype
    if op == "gemm":
        return _products(s, s["x"], lambda i: (s["w"] if i is None else s["w"][i]).float(),
                         gated, dtype)
    if op == "dgrad":
        return _products(s, s["x"], lambda i: (s["w"] if i is None else s["w"][i]).float()
                         .transpose(1, 2).contiguous(), False, dtype)
    if op == "wgrad":
        idx, live = _rows_by_expert(s)
        d = _gather(s["grad"], idx, live).transpose(1, 2).contiguous()
        return torch.bmm(d, _gather(s["x"], idx, live)).to(dtype)
    if op == "fp8":
        def weights(i):
            w, sc = (s["w"], s["w_scales"]) if i is None else \
                (s["w"].view(torch.uint8)[i].view(torch.float8_e4m3fn), s["w_scales"][i])
            return w.float() * _blocks(sc, w.shape[1], 128)
        x = s["x"].float() * s["x_scales"].repeat_interleave(128, 1)
        return _products(s, x, weights, gated, dtype)

    def weights(i):                                              # 4 bits, low nibble first
        w, sc, z = (t if t is None or i is None else t[i]
                    for t in (s["w"], s["w_scales"], s["zeros"]))
        q = torch.stack((w & 15, w >> 4), -1).view(*sc.shape, c["group"]).float()
        q = (q - (8.0 if z is None else z.float()[..., None])) * sc.float()[..., None]
        return q.view(w.shape[0], w.shape[1], -1)
    return _products(s, s["x"], weights, gated, dtype)


# ---- the library's calls -----------------------------------------------------

def _own(s):
    import combine_topk_ids_expert_amd as mx
    c = s["case"]
    op = c["op"]
    if op == "gating":
        mx.topk_gating(s["logits"], s["ids"], s["weights"], scoring=c["scoring"], bias=s["bias"])
        return s["ids"], s["weights"]
    if op == "gating_backward":
        mx.topk_gating_backward(s["logits"], s["ids"], s["grad"], s["grad_logits"],
                                scoring=c["scoring"])
        return s["grad_logits"]
    o, z, out = s["offsets"], s["sizes"], s["result"]
    if op == "silu_backward":
        mx.silu_mul_backward(s["grad"], s["gate_up"], o, out, z)
    elif op == "gemm":
        mx.grouped_gemm(s["x"], s["w"], o, out, z, silu_mul=c["gated"])
    elif op == "dgrad":
        mx.grouped_gemm(s["x"], s["w"], o, out, z, transpose_weight=True)
    elif op == "wgrad":
        mx.grouped_gemm_wgrad(s["grad"], s["x"], o, out, z)
    elif op == "fp8":
        mx.grouped_gemm_fp8(s["x"], s["x_scales"], s["w"], s["w_scales"], o, out, z,
                            silu_mul=c["gated"])
    else:
        mx.grouped_gemm_w4(s["x"], s["w"], s["w_scales"], o, out, z, zeros=s["zeros"],
                           silu_mul=c["gated"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definitions in 64 bits ----------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op in ("gating", "gating_backward"):
        x = s["logits"].double()
        soft = c["scoring"] == "softmax"
        score = torch.exp(x) if soft else torch.sigmoid(x)
        if op == "gating":
            key = (x if s["bias"] is None else score + s["bias"].double()).masked_fill(
                x == -math.inf, -math.inf)
            ids = key.argsort(dim=1, descending=True, stable=True)[:, :c["topk"]]
            on = torch.gather(x, 1, ids) > -math.inf
            w = torch.gather(score, 1, ids) * on
            return torch.where(on, ids, -1).int(), w / w.sum(1, True).clamp_min(1e-300)
        x = x.requires_grad_()
        score = torch.exp(x) if soft else torch.sigmoid(x)
        w = torch.gather(score, 1, s["ids"].long())
        ((w / w.sum(1, True)) * s["grad"].double()).sum().backward()
        return torch.nan_to_num(x.grad, nan=0.0)
    starts, counts = s["offsets"].tolist(), s["sizes"][:, 0].tolist()
    out = torch.zeros(s["result"].shape, dtype=torch.float64, device=DEV)
    n = c["n"]
    for e, (b, m) in enumerate(zip(starts, counts)):
        at = slice(b, b + m)
        if not m:
            continue
        if op == "silu_backward":
            gu = s["gate_up"][at].double().requires_grad_()
            h = torch.nn.functional.silu(gu[:, :n]) * gu[:, n:]
            h.backward(s["grad"][at].double())
            out[at] = gu.grad
            continue
        if op == "wgrad":
            out[e] = s["grad"][at].double().t() @ s["x"][at].double()
            continue
        x, w = s["x"][at].double(), s["w"][e]
        if op == "dgrad":
            out[at] = x @ w.double()
            continue
        if op == "fp8":
            x = (x.view(m, -1, 128) * s["x_scales"][at].double()[..., None]).view(m, -1)
            wide, k = w.shape
            full = torch.zeros((wide + 127) // 128 * 128, k, dtype=torch.float64, device=DEV)
            full[:wide] = w.double()
            w = (full.view(-1, 128, k // 128, 128)
                 * s["w_scales"][e].double()[:, None, :, None]).view(-1, k)[:wide]
        elif op == "w4":
            q = torch.empty(w.shape[0], 2 * w.shape[1], dtype=torch.float64, device=DEV)
            q[:, 0::2], q[:, 1::2] = (w % 16).double(), (w // 16).double()
            zero = 8.0 if s["zeros"] is None else \
                s["zeros"][e].double().repeat_interleave(c["group"], 1)
            w = (q - zero) * s["w_scales"][e].double().repeat_interleave(c["group"], 1)
        y = x @ w.double().t()
        out[at] = torch.nn.functional.silu(y[:, :n]) * y[:, n:] if c.get("gated") else y
    return out
