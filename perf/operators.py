"""Cases of the operators around the quantized matmul: norm and quantize, the
matmul with an epilogue, the product grouped by expert, its router and its
combination.

`run` computes an operator in plain torch operations where `own` is false and
calls the framework's entry points where it is true; both on what `prepare`
makes from the seed.  `exact` is the same from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda:0"
FLT_MAX = torch.finfo(torch.float32).max
ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ------------------------------------------------------------------- cases
def listed():
    return [
        # A decode step of one sequence: the attention output joins the
        # residual stream, and the FFN's input is normed and quantized.
        dict(name="norm decode step", op="norm", n=1, k=4096, y="f32", post=False, gate="none", alpha=1.0, codes=True),
        # Prefill with norms on both sides of the block and a learned gate per
        # channel; the next reader takes float32 (a router, an output head).
        dict(name="norm prefill gated", op="norm", n=8192, k=4096, y="f16", post=True, gate="channel", alpha=0.75,
             codes=False),
        # Attention output projection in prefill: bias, and the residual added.
        dict(name="epilogue q-proj prefill", op="epilogue", fmt="q4k", m=4096, k=4096, n=2630, bias=True, act="none",
             residual="f32", f16=False),
        # Wide gate projection at a few decoding sequences.
        dict(name="epilogue wide decode", op="epilogue", fmt="q4k", m=28672, k=8192, n=7, bias=True, act="silu",
             residual="none", f16=False),
        # Down projection in the 6-bit format for a small batch, half output.
        dict(name="epilogue q6k down", op="epilogue", fmt="q6k", m=4096, k=11008, n=33, bias=True, act="gelu",
             residual="f16", f16=True),
        # Two decoding sequences over eight experts, two each: gate projection
        # with the tokens gathered by slot.
        dict(name="grouped decode", op="grouped", fmt="q4k", experts=8, m=14336, k=4096, tokens=2, top=2, skew=1.0,
             drop=0.0, gather=True, bias=False, act="none", f16=False),
        # The same projection in prefill, uneven loads.
        dict(name="grouped prefill gate", op="grouped", fmt="q4k", experts=8, m=14336, k=4096, tokens=2048, top=2,
             skew=1.0, drop=0.0, gather=True, bias=False, act="silu", f16=False),
        # Many small experts, down projection in the 6-bit format, some slots unused.
        dict(name="grouped many q6k", op="grouped", fmt="q6k", experts=64, m=4096, k=1536, tokens=512, top=8, skew=0.6,
             drop=0.05, gather=False, bias=True, act="none", f16=True),
        # The router of a small decode batch, and of a prefill with padding rows.
        dict(name="route decode", op="route", n=16, experts=64, top=8, normalize=True, pad=0.0),
        dict(name="route prefill", op="route", n=8192, experts=128, top=8, normalize=False, pad=0.05),
        # The experts' outputs back in token order.
        dict(name="combine decode", op="combine", n=16, m=4096, top=8, f16=False, residual=False, drop=0.0),
        dict(name="combine prefill", op="combine", n=8192, m=4096, top=4, f16=True, residual=True, drop=0.05),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "epilogue", "epilogue", "grouped", "grouped", "route", "combine"])
    if op == "norm":
        k = 32 * _log(rng, 1, 896)
        n = _log(rng, 1, max(1, min(8192, 8192 * 4096 // k)))
        return dict(op=op, n=n, k=k, y=rng.choice(["f32", "f16", "none"]), post=rng.random() < 0.5,
                    gate=rng.choice(["none", "channel", "token"]), alpha=rng.choice([1.0, 0.5, 0.8125]),
                    codes=rng.random() < 0.5)
    if op == "epilogue":
        k = 256 * _log(rng, 1, 112)
        m = _log(rng, 1, min(28672, 28672 * 8192 // k))
        n = _log(rng, 1, max(1, min(4096, 2630 * 4096 * 4096 // (m * k))))
        return dict(op=op, fmt=rng.choice(["q4k", "q6k"]), m=m, k=k, n=n, bias=rng.random() < 0.7,
                    act=rng.choice(ACTIVATIONS), residual=rng.choice(["none", "f32", "f16"]), f16=rng.random() < 0.5)
    if op == "grouped":
        experts = _log(rng, 2, 128)
        k = 256 * _log(rng, 1, 28)
        m = 8 * _log(rng, 1, min(1792, max(8, 8 * 14336 * 4096 // (8 * experts * k))))
        top = rng.randint(1, min(8, experts))
        tokens = _log(rng, 1, min(2048, max(1, 4096 // top)))
        return dict(op=op, fmt=rng.choice(["q4k", "q6k"]), experts=experts, m=m, k=k, tokens=tokens, top=top,
                    skew=rng.choice([0.0, 0.6, 1.5]), drop=rng.choice([0.0, 0.0, 0.1]), gather=rng.random() < 0.5,
                    bias=rng.random() < 0.5, act=rng.choice(ACTIVATIONS), f16=rng.random() < 0.5)
    if op == "route":
        experts = _log(rng, 2, 256)
        return dict(op=op, n=_log(rng, 1, 8192), experts=experts, top=rng.randint(1, min(8, experts)),
                    normalize=rng.random() < 0.5, pad=rng.choice([0.0, 0.05]))
    m = _log(rng, 1, 8192)
    top = rng.randint(1, 8)
    return dict(op=op, n=_log(rng, 1, max(1, min(8192, 8192 * 4096 * 4 // (m * top)))), m=m, top=top,
                f16=rng.random() < 0.5, residual=rng.random() < 0.5, drop=rng.choice([0.0, 0.1]))


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _q4k(g, rows, k):
    """Random q4_K super-blocks (144 bytes per 256 weights) of `rows` rows."""
    w = torch.randint(0, 256, (rows * (k // 256), 144), generator=g, device=DEV, dtype=torch.uint8)
    d = (_randn(g, w.shape[0], 2).abs() * 1e-2).to(torch.float16)
    w[:, :4] = d.view(torch.uint8)
    return w.view(-1)


def _q6k(g, rows, k):
    """Random q6_K super-blocks (210 bytes per 256 weights) of `rows` rows."""
    w = torch.randint(0, 256, (rows * (k // 256), 210), generator=g, device=DEV, dtype=torch.uint8)
    d = (_randn(g, w.shape[0], 1).abs() * 1e-2).to(torch.float16)
    w[:, 208:] = d.view(torch.uint8)
    return w.view(-1)


def _codes(x):
    """q8 codes and scale words of the rows of x."""
    n, k = x.shape
    b = x.view(n, k // 32, 32)
    da = b.abs().amax(-1) / 127
    q = torch.clamp(torch.round(b / da.unsqueeze(-1)), -127, 127)
    low = da.to(torch.float16).view(torch.int16).to(torch.int32) & 0xFFFF
    return q.to(torch.int8).view(n, k), low | (q.sum(-1).to(torch.int32) << 16)


def _slot_plan(case, g):
    """Slots per token of a skewed routing: expert ids [n, top] (-1: dropped),
    and from them offsets, the token of each slot and the slot of each token."""
    n, top, experts = case["tokens"], case["top"], case["experts"]
    pop = -case["skew"] * torch.log1p(torch.arange(experts, device=DEV, dtype=torch.float32))
    u = torch.rand(n, experts, generator=g, device=DEV).clamp_min(1e-9)
    ids = (pop - torch.log(-torch.log(u).clamp_min(1e-9))).argsort(dim=1, descending=True)[:, :top]
    ids[torch.rand(n, top, generator=g, device=DEV) < case["drop"]] = experts
    key, order = ids.reshape(-1).sort(stable=True)
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device=DEV)).to(torch.int32)
    return offsets, (order // top).to(torch.int32)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = {"case": case}
    if op == "norm":
        n, k = case["n"], case["k"]
        s["x"] = _randn(g, n, k) * 2
        s["y"] = None if case["y"] == "none" else _randn(g, n, k).to(torch.float16 if case["y"] == "f16" else torch.float32)
        s["weight"] = 1 + 0.2 * _randn(g, k)
        s["y_weight"] = 1 + 0.2 * _randn(g, k) if case["post"] and s["y"] is not None else None
        s["gate"] = None
        if s["y"] is not None and case["gate"] != "none":
            s["gate"] = 0.5 * _randn(g, k) if case["gate"] == "channel" else 0.5 * _randn(g, n, k)
        s["alpha"] = case["alpha"] if s["y"] is not None else 1.0
    elif op == "epilogue":
        m, k, n = case["m"], case["k"], case["n"]
        s["w"] = _q4k(g, m, k) if case["fmt"] == "q4k" else _q6k(g, m, k)
        s["q"], s["ds"] = _codes(_randn(g, n, k) / math.sqrt(k))
        s["bias"] = _randn(g, m) if case["bias"] else None
        s["residual"] = None
        if case["residual"] != "none":
            s["residual"] = _randn(g, n, m).to(torch.float16 if case["residual"] == "f16" else torch.float32)
    elif op == "grouped":
        m, k, experts = case["m"], case["k"], case["experts"]
        slots = case["tokens"] * case["top"]
        s["w"] = _q4k(g, experts * m, k) if case["fmt"] == "q4k" else _q6k(g, experts * m, k)
        s["offsets"], rows = _slot_plan(case, g)
        s["rows"] = rows if case["gather"] else None
        s["q"], s["ds"] = _codes(_randn(g, case["tokens"] if case["gather"] else slots, k) / math.sqrt(k))
        s["bias"] = _randn(g, experts, m) if case["bias"] else None
        s["slots"] = slots
        # the user's output buffer: rows past the last slot keep what they hold
        s["out"] = torch.zeros(slots, m, device=DEV, dtype=torch.float16 if case["f16"] else torch.float32)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    elif op == "route":
        # scores as a half-precision router matrix gives them: ties occur
        l = (_randn(g, case["n"], case["experts"]) * 2).to(torch.bfloat16).float()
        l[torch.rand(case["n"], generator=g, device=DEV) < case["pad"]] = -math.inf
        s["logits"] = l
    else:
        n, m, top = case["n"], case["m"], case["top"]
        s["y"] = _randn(g, n * top, m).to(torch.float16 if case["f16"] else torch.float32)
        slot = torch.randperm(n * top, generator=g, device=DEV).to(torch.int32).view(n, top)
        slot[torch.rand(n, top, generator=g, device=DEV) < case["drop"]] = -1
        s["slot"] = slot
        s["weights"] = torch.softmax(_randn(g, n, top), dim=1)
        s["residual"] = _randn(g, n, m) if case["residual"] else None
    return s


# ------------------------------------------------------------- plain forms
def _unpack_q4k(w, rows, k):
    """float32 [rows, k] of q4_K super-blocks: d * sc * code - dmin * min."""
    b = w.view(-1, 144)
    d = b[:, :4].contiguous().view(torch.float16).float()
    a, c, e = b[:, 4:8], b[:, 8:12], b[:, 12:16]
    sc = torch.cat((a & 63, (e & 15) | ((a >> 6) << 4)), 1).float() * d[:, :1]
    mn = torch.cat((c & 63, (e >> 4) | ((c >> 6) << 4)), 1).float() * d[:, 1:]
    qs = b[:, 16:].reshape(-1, 4, 1, 32)
    code = torch.cat((qs & 15, qs >> 4), 2).reshape(-1, 8, 32)
    return (code * sc.unsqueeze(-1) - mn.unsqueeze(-1)).view(rows, k)


def _unpack_q6k(w, rows, k):
    """float32 [rows, k] of q6_K super-blocks: d * sc * (code - 32)."""
    b = w.view(-1, 210)
    d = b[:, 208:].contiguous().view(torch.float16).float()
    ql = b[:, :128].reshape(-1, 2, 1, 2, 32)
    qh = b[:, 128:192].reshape(-1, 2, 1, 32)
    lo = torch.cat((ql & 15, ql >> 4), 2).reshape(-1, 2, 4, 32)
    hi = torch.cat((qh & 3, (qh >> 2) & 3, (qh >> 4) & 3, qh >> 6), 2)
    code = (lo | (hi << 4)).to(torch.int8).reshape(-1, 16, 16) - 32
    sc = b[:, 192:208].contiguous().view(torch.int8).float() * d
    return (code * sc.unsqueeze(-1)).view(rows, k)


def _unpack(fmt, w, rows, k):
    return _unpack_q4k(w, rows, k) if fmt == "q4k" else _unpack_q6k(w, rows, k)


def _da(ds):
    """The binary16 scales of the scale words, a view of their low halves."""
    return ds.view(torch.float16)[:, ::2]


def _values(q, ds):
    """What q8 codes stand for, code * scale, rounded to binary16."""
    n, k = q.shape
    return (q.view(n, k // 32, 32) * _da(ds).unsqueeze(-1)).view(n, k)


def _activations(q, ds):
    n, k = q.shape
    return (q.view(n, k // 32, 32) * _da(ds).float().unsqueeze(-1)).view(n, k)


def _activate(v, act):
    if act == "relu":
        return v.clamp_min(0)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * torch.erfc(-v * math.sqrt(0.5))
    if act == "gelu_tanh":
        # 0.5 v (1 + tanh(u)) = v / (1 + exp(-2 u))
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_norm(s, eps=1e-5):
    # in 64 bits: a code next to a rounding border must not depend on the
    # order of a sum
    r = s["x"]
    if s["y"] is not None:
        z = s["y"].double()
        if s["y_weight"] is not None:
            z = z * s["y_weight"].double() / torch.sqrt((z * z).mean(-1, keepdim=True) + eps)
        if s["gate"] is not None:
            z = z * s["gate"].double()
        r = (s["alpha"] * r.double() + z).float()
    rd = r.double()
    h = (rd * s["weight"].double() / torch.sqrt((rd * rd).mean(-1, keepdim=True) + eps)).float()
    if not s["case"]["codes"]:
        return {"r": r, "h": h}
    n, k = h.shape
    b = h.view(n, k // 32, 32)
    da = b.abs().amax(-1) / 127
    t = (b / da.unsqueeze(-1)).double()
    q = torch.where(da.unsqueeze(-1) > 0, (t.abs() + 0.5).floor().clamp_max(127) * t.sign(), 0.0)
    return {"r": r, "values": (q * da.to(torch.float16).unsqueeze(-1)).to(torch.float16).view(n, k)}


def _plain_epilogue(s):
    c = s["case"]
    v = _activations(s["q"], s["ds"]) @ _unpack(c["fmt"], s["w"], c["m"], c["k"]).t()
    if s["bias"] is not None:
        v = v + s["bias"]
    v = _activate(v, c["act"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(torch.float16) if c["f16"] else v


def _expert_of_slot(s):
    c = s["case"]
    at = torch.arange(s["slots"], device=DEV, dtype=torch.int32)
    return at, torch.bucketize(at, s["offsets"][1:], right=True)


def _plain_grouped(s):
    c = s["case"]
    experts, m, k = c["experts"], c["m"], c["k"]
    w = _unpack(c["fmt"], s["w"], experts * m, k).view(experts, m, k)
    x = _activations(s["q"], s["ds"])
    if s["rows"] is not None:
        x = x[s["rows"].long()]
    at, e = _expert_of_slot(s)
    used = e < experts
    e = e.clamp_max(experts - 1)
    place = (at - s["offsets"][e]).clamp(0, s["most"] - 1)
    # slots padded to the largest group; unused ones go to a spare row
    batch = torch.zeros(experts, s["most"] + 1, k, device=DEV)
    batch[e, torch.where(used, place, s["most"])] = x
    v = torch.bmm(w, batch.transpose(1, 2).contiguous())[e, :, place]
    if s["bias"] is not None:
        v = v + s["bias"][e]
    v = _activate(v, c["act"])
    return torch.where(used.unsqueeze(1), v.to(s["out"].dtype), s["out"])


def _plain_route(s):
    c = s["case"]
    n, experts, top = c["n"], c["experts"], c["top"]
    l = s["logits"]
    l = torch.where(l.isnan(), -math.inf, l).clamp_max(FLT_MAX)
    v, ids = l.sort(dim=1, descending=True, stable=True)   # ties to the lowest index
    live = v > -math.inf
    ex = torch.where(live, torch.exp(v - v[:, :1]), 0.0)
    v, ids, live = v[:, :top], ids[:, :top], live[:, :top]
    total = ex[:, :top].sum(1, keepdim=True) if c["normalize"] else ex.sum(1, keepdim=True)
    weights = torch.where(live, ex[:, :top] / total, 0.0)
    key, order = torch.where(live, ids, experts).reshape(-1).sort(stable=True)
    at = torch.arange(n * top, device=DEV, dtype=torch.int32)
    slot = torch.empty_like(at)
    slot[order] = torch.where(key < experts, at, -1)
    return {"ids": torch.where(live, ids, -1).to(torch.int32), "weights": weights, "slot": slot.view(n, top),
            "rows": torch.where(key < experts, order // top, -1).to(torch.int32),
            "offsets": torch.searchsorted(key, torch.arange(experts + 1, device=DEV)).to(torch.int32)}


def _plain_combine(s):
    live = (s["slot"] >= 0).unsqueeze(-1)
    y = s["y"][s["slot"].clamp_min(0).long()].float()
    v = torch.where(live, y * s["weights"].unsqueeze(-1), 0.0).sum(1)
    return v if s["residual"] is None else s["residual"] + v


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from q4_q8_integer_amd import binding as b
        if op == "norm":
            if c["codes"]:
                q, ds, r = b.quantize_norm(s["x"], s["weight"], 1e-5, s["y"], s["y_weight"], s["gate"], s["alpha"])
                return {"r": r, "values": _values(q, ds)}
            h, r = b.norm(s["x"], s["weight"], 1e-5, s["y"], s["y_weight"], s["gate"], s["alpha"])
            return {"r": r, "h": h}
        act = ACTIVATIONS.index(c.get("act", "none"))
        fmt = b.FORMAT_Q4K if c.get("fmt") == "q4k" else b.FORMAT_Q6K
        if op == "epilogue":
            return b.fold_epilogue(fmt, s["w"], c["m"], c["k"], s["q"], s["ds"], s["bias"], act, s["residual"],
                                   f16=c["f16"])
        if op == "grouped":
            return b.fold_grouped(fmt, s["w"], c["experts"], c["m"], c["k"], s["q"], s["ds"], s["offsets"], s["rows"],
                                  s["bias"], act, out=s["out"], f16=c["f16"])
        if op == "route":
            return b.route(s["logits"], c["top"], c["normalize"])._asdict()
        return b.combine(s["y"], s["slot"], s["weights"], s["residual"])
    return {"norm": _plain_norm, "epilogue": _plain_epilogue, "grouped": _plain_grouped, "route": _plain_route,
            "combine": _plain_combine}[op](s)


# -------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "norm":
        n, k = case["n"], case["k"]
        per = 4 + {"f32": 8, "f16": 6, "none": 0}[case["y"]]              # x; y read and r written
        per += 4 if case["gate"] == "token" and case["y"] != "none" else 0
        per += 1 + 4 / 32 if case["codes"] else 4
        return {"bytes": n * k * per, "flops": 12 * n * k}
    if op == "epilogue":
        m, k, n = case["m"], case["k"], case["n"]
        wb = 144 if case["fmt"] == "q4k" else 210
        out = (2 if case["f16"] else 4) + {"none": 0, "f16": 2, "f32": 4}[case["residual"]]
        return {"bytes": m * (k // 256) * wb + n * k * 1.125 + n * m * out, "flops": 2 * m * k * n}
    if op == "grouped":
        m, k, slots = case["m"], case["k"], case["tokens"] * case["top"]
        wb = 144 if case["fmt"] == "q4k" else 210
        # experts that some token needs, for an even routing
        active = case["experts"] * (1 - (1 - case["top"] / case["experts"]) ** case["tokens"])
        x = case["tokens"] if case["gather"] else slots
        return {"bytes": active * m * (k // 256) * wb + x * k * 1.125 + slots * m * (2 if case["f16"] else 4),
                "flops": 2 * m * k * slots * (1 - case["drop"])}
    if op == "route":
        n, experts, top = case["n"], case["experts"], case["top"]
        return {"bytes": 4 * n * experts + 16 * n * top + 4 * experts, "flops": 4 * n * experts}
    n, m, top = case["n"], case["m"], case["top"]
    return {"bytes": n * m * (top * (2 if case["f16"] else 4) * (1 - case["drop"]) + 4 + (4 if case["residual"] else 0)),
            "flops": 2 * n * m * top}


# ------------------------------------------------------- 64-bit definitions
def _weights64(fmt, w, rows, k):
    """float64 [rows, k] from the bytes, one sub-block (or scale group) at a time."""
    out = torch.empty(rows * (k // 256), 256, device=DEV, dtype=torch.float64)
    if fmt == "q4k":
        b = w.view(-1, 144).to(torch.int32)
        half = w.view(-1, 144)[:, :4].contiguous().view(torch.float16).double()
        for j in range(8):
            if j < 4:
                sc, mn = b[:, 4 + j] % 64, b[:, 8 + j] % 64
            else:
                sc = b[:, 8 + j] % 16 + 16 * (b[:, j] // 64)
                mn = b[:, 8 + j] // 16 + 16 * (b[:, 4 + j] // 64)
            run32 = b[:, 16 + 32 * (j // 2):48 + 32 * (j // 2)]
            code = run32 // 16 if j % 2 else run32 % 16
            out[:, 32 * j:32 * j + 32] = (half[:, 0] * sc)[:, None] * code - (half[:, 1] * mn)[:, None]
    else:
        b = w.view(-1, 210).to(torch.int32)
        d = w.view(-1, 210)[:, 208:].contiguous().view(torch.float16).double()[:, 0]
        for j in range(16):                      # weights 16 j .. 16 j + 15
            h, g, l = j // 8, (j % 8) // 2, 16 * (j % 2)
            lo = b[:, 64 * h + 32 * (g % 2) + l:][:, :16] // (16 if g > 1 else 1) % 16
            hi = b[:, 128 + 32 * h + l:][:, :16] // 4 ** g % 4
            sc = b[:, 192 + j]
            sc = torch.where(sc > 127, sc - 256, sc)
            out[:, 16 * j:16 * j + 16] = (d * sc)[:, None] * (lo + 16 * hi - 32)
    return out.view(rows, k)


def _x64(q, ds):
    da = (ds & 0xFFFF).to(torch.int16).view(torch.float16).double()
    return q.double() * da.repeat_interleave(32, dim=1)


def _act64(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * (0.5 * torch.erfc(-v / math.sqrt(2.0)))
    if act == "gelu_tanh":
        return v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        r = s["x"].double()
        if s["y"] is not None:
            z = s["y"].double()
            if s["y_weight"] is not None:
                z = z * torch.rsqrt(z.pow(2).mean(1) + 1e-5)[:, None] * s["y_weight"].double()
            r = s["alpha"] * r + (z if s["gate"] is None else s["gate"].double() * z)
        # the stream is stored in float32, and the second norm reads it as stored
        rf = r.to(torch.float32).double()
        h = rf * torch.rsqrt(rf.pow(2).mean(1) + 1e-5)[:, None] * s["weight"].double()
        if not case["codes"]:
            return {"r": r, "h": h}
        h32 = h.to(torch.float32)
        n, k = h32.shape
        da = h32.view(n, -1, 32).abs().max(2).values / 127.0
        wide = da.repeat_interleave(32, dim=1)
        t = torch.where(wide > 0, h32 / wide, torch.zeros_like(h32)).double()
        q = torch.trunc(t + torch.copysign(torch.full_like(t, 0.5), t)).clamp(-127, 127)
        return {"r": r, "values": q * wide.to(torch.float16).double()}
    if op == "epilogue":
        v = _x64(s["q"], s["ds"]) @ _weights64(case["fmt"], s["w"], case["m"], case["k"]).T
        if s["bias"] is not None:
            v += s["bias"].double()
        v = _act64(v, case["act"])
        return v if s["residual"] is None else v + s["residual"].double()
    if op == "grouped":
        x, m, k = _x64(s["q"], s["ds"]), case["m"], case["k"]
        out, off = s["out"].double(), s["offsets"].tolist()
        per = s["w"].numel() // case["experts"]
        for e in range(case["experts"]):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            xe = x[a:b] if s["rows"] is None else x[s["rows"][a:b].long()]
            v = xe @ _weights64(case["fmt"], s["w"][e * per:(e + 1) * per], m, k).T
            if s["bias"] is not None:
                v += s["bias"][e].double()
            out[a:b] = _act64(v, case["act"])
        return out
    if op == "route":
        l = s["logits"].double().cpu()
        n, experts, top = case["n"], case["experts"], case["top"]
        ids = torch.full((n, top), -1, dtype=torch.int32)
        weights = torch.zeros(n, top, dtype=torch.float64)
        left = l.clone()
        ex = torch.exp(l - l.max(1, keepdim=True).values).nan_to_num(0.0)
        for j in range(top):
            v, i = left.max(1, keepdim=True)
            i = (left == v).to(torch.int8).argmax(1, keepdim=True)      # the first of equals
            live = (v > -math.inf)[:, 0]
            ids[live, j] = i[live, 0].to(torch.int32)
            weights[live, j] = ex.gather(1, i)[live, 0]
            left.scatter_(1, i, -math.inf)
        total = weights.sum(1, keepdim=True) if case["normalize"] else ex.sum(1, keepdim=True)
        weights = weights / torch.where(total > 0, total, 1.0)
        flat = ids.view(-1).tolist()
        groups = [[] for _ in range(experts)]
        for p, e in enumerate(flat):
            if e >= 0:
                groups[e].append(p)
        order = [p for group in groups for p in group]
        slot = torch.full((n * top,), -1, dtype=torch.int32)
        slot[torch.tensor(order, dtype=torch.long)] = torch.arange(len(order), dtype=torch.int32)
        offsets = [0]
        for group in groups:
            offsets.append(offsets[-1] + len(group))
        rows = [p // top for p in order] + [-1] * (n * top - len(order))
        return {"ids": ids, "weights": weights, "slot": slot.view(n, top),
                "rows": torch.tensor(rows, dtype=torch.int32), "offsets": torch.tensor(offsets, dtype=torch.int32)}
    out = torch.zeros(case["n"], case["m"], device=DEV, dtype=torch.float64)
    if s["residual"] is not None:
        out += s["residual"].double()
    for j in range(case["top"]):
        live = (s["slot"][:, j] >= 0).nonzero()[:, 0]
        out[live] += s["weights"][live, j].double()[:, None] * s["y"][s["slot"][live, j].long()].double()
    return out
