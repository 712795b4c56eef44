"""Cases that measure the operators of a MoE block in bf16: the experts' products in both directions, the combine's
gradient, and the norm before the experts.

Six kinds of pass:

  product   rows of a dispatched layout times their expert's weights
  swiglu    the gate and up products with SwiGLU, for training with the gate and up values kept
  rows      the experts' gradient with respect to their rows: the down product's gradient through SwiGLU, then through
            the gate and up products
  weights   the gradients of the experts' weights: sums over each expert's rows
  combine   the gradient of the weighted sum back to token order: of the experts' outputs and of the weights
  norm      root-mean-square norm of x + residual, in bf16 and in FP8 with a scale for each 128 values; for training
            with its gradient

A pass that writes into a layout's buffer leaves the rows that no token maps to as prepare() made them: zero.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # the down product of a decode batch in the masked layout: about 4 rows an expert, weights dominate
        dict(name="product decode", op="product", layout="masked", tokens=128, cols=7168, inner=1024, experts=256, topk=8,
             capacity=128, align=1, routing="uniform", invalid=0.0),
        # one sequence being decoded: eight experts with a row each, latency
        dict(name="swiglu one token", op="swiglu", keep=False, layout="normal", tokens=1, hidden=4096, inter=768,
             experts=128, topk=8, capacity=0, align=1, routing="uniform", invalid=0.0),
        # the largest: a full batch through the gate and up products of all experts, their values kept for the gradient
        dict(name="swiglu prefill", op="swiglu", keep=True, layout="normal", tokens=8192, hidden=7168, inter=1024,
             experts=256, topk=8, capacity=0, align=128, routing="uniform", invalid=0.0),
        # a training step's batch, backwards through all experts
        dict(name="rows' gradient batch", op="rows", layout="normal", tokens=8192, hidden=4096, inter=768, experts=128,
             topk=8, capacity=0, align=128, routing="uniform", invalid=0.0),
        # one partition of 16 experts, segments without padding, dropped slots, an odd number of tokens
        dict(name="rows' gradient ragged", op="rows", layout="normal", tokens=1501, hidden=2112, inter=704, experts=16,
             topk=4, capacity=0, align=1, routing="uniform", invalid=0.05),
        # the weights' gradients of the same training step, in fp32
        dict(name="weights' gradient batch", op="weights", out="float32", layout="normal", tokens=8192, hidden=4096,
             inter=768, experts=128, topk=8, capacity=0, align=128, routing="uniform", invalid=0.0),
        # a few popular experts and some without a row, sizes that fill no tile, bf16 gradients
        dict(name="weights' gradient skewed", op="weights", out="bfloat16", layout="normal", tokens=777, hidden=1544,
             inter=520, experts=32, topk=4, capacity=0, align=1, routing="zipf", invalid=0.05),
        # a training step's batch in the contiguous layout
        dict(name="combine's gradient batch", op="combine", layout="normal", tokens=16384, hidden=4096, experts=128, topk=8,
             capacity=0, align=1, routing="uniform", invalid=0.05),
        # a small batch in the masked layout, odd sizes
        dict(name="combine's gradient masked", op="combine", layout="masked", tokens=301, hidden=2120, experts=16, topk=3,
             capacity=128, align=1, routing="uniform", invalid=0.1),
        # the rows of a decode batch on their way into the dispatch: latency
        dict(name="norm decode", op="norm", train=False, quant="fp8g128", residual=True, tokens=128, hidden=7168),
        # a training step's batch
        dict(name="norm training", op="norm", train=True, quant="none", residual=True, tokens=16384, hidden=4096),
        # both forms of the output, a hidden size that is no power of two, an odd number of tokens
        dict(name="norm training ragged", op="norm", train=True, quant="fp8g128", residual=True, tokens=1003, hidden=2176),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["product", "swiglu", "rows", "weights", "combine", "norm"])
    if op == "norm":
        quant = rng.choice(["none", "fp8g128", "fp8g128"])
        hidden = 8 * log(16, 1024) if quant == "none" else 128 * log(1, 64)
        return dict(op=op, train=rng.choice([True, False]), quant=quant, residual=rng.choice([True, True, False]),
                    tokens=log(1, min(16384, (1 << 26) // hidden)), hidden=hidden)
    hidden, inter = 8 * log(32, 1024), 8 * log(16, 256)
    experts = min(log(4, 256), max(4, int(1.0e9) // (3 * hidden * inter)))
    topk = min(rng.randint(1, 8), experts)
    layout = rng.choice(["masked", "normal"])
    most = 512 if layout == "masked" else max(64, min(6000, int(1.2e12 / (6 * hidden * inter * topk))))
    tokens = log(1, most)
    # a few popular experts have all tokens: padding every expert to their rows has a limit
    routing = rng.choice(["uniform", "zipf"]) if experts * tokens <= 1 << 17 else "uniform"
    c = dict(op=op, layout=layout, tokens=tokens, experts=experts, topk=topk,
             capacity=-(-tokens // 16) * 16 if layout == "masked" else 0,
             align=rng.choice([1, 16, 128]) if layout == "normal" else 1, routing=routing,
             invalid=rng.choice([0.0, 0.0, 0.05, 0.3]))
    if op == "product":
        return dict(c, cols=hidden, inner=inter)
    if op == "combine":
        return dict(c, hidden=hidden)
    c = dict(c, hidden=hidden, inter=inter)
    if op == "swiglu":
        return dict(c, keep=rng.choice([True, False]))
    if op == "weights":
        return dict(c, out=rng.choice(["float32", "bfloat16"]))
    return c


def work(case):
    c = dict(case)
    if c["op"] == "norm":
        each = 2 + 2 * c["residual"]                             # x, residual
        each += 2 * c["residual"]                                # their sum
        each += (1 + 4 / 128) if c["quant"] != "none" else 0     # codes and scales
        if c["train"] or c["quant"] == "none":
            each += 2                                            # bf16 rows
        if c["train"]:
            each += 2 + 2 * c["residual"] + 2                    # both gradients in, one out
        return {"bytes": c["tokens"] * c["hidden"] * each, "flops": 0}
    rows = c["tokens"] * c["topk"] * (1 - c["invalid"])
    if c["op"] == "combine":
        return {"bytes": c["tokens"] * c["hidden"] * 2 + rows * c["hidden"] * 4 + c["tokens"] * c["topk"] * 16, "flops": 0}
    active = c["experts"] * (1 - (1 - c["topk"] * (1 - c["invalid"]) / c["experts"]) ** c["tokens"])  # of uniform routing
    if c["op"] == "product":
        n, k = c["cols"], c["inner"]
        return {"bytes": 2 * (active * n * k + rows * (k + n)), "flops": 2 * rows * n * k}
    h, i = c["hidden"], c["inter"]
    if c["op"] == "swiglu":
        return {"bytes": 2 * (active * 2 * i * h + rows * (h + i + (2 * i if c["keep"] else 0))), "flops": 4 * rows * h * i}
    if c["op"] == "rows":
        # the gradient of gate and up is an output: it is written, and read back by nobody who keeps it
        return {"bytes": 2 * (active * 3 * h * i + rows * (2 * h + 4 * i)), "flops": 6 * rows * h * i}
    each = 4 if c["out"] == "float32" else 2
    return {"bytes": c["experts"] * 3 * h * i * each + 2 * rows * (2 * h + 3 * i), "flops": 6 * rows * h * i}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _route(gen, c):
    """Expert ids [T, K] int32, distinct in a token, some of them -1."""
    t, e, k = c["tokens"], c["experts"], c["topk"]
    if c["routing"] == "zipf":
        p = (torch.randperm(e, device=DEV, generator=gen) + 1.0) ** -1.2
    else:
        p = torch.ones(e, device=DEV)
    ids = torch.multinomial(p.expand(t, e), k, generator=gen).int()
    if c["invalid"]:
        ids[torch.rand(t, k, device=DEV, generator=gen) < c["invalid"]] = -1
    return ids


def _layout(s, c, ids):
    """Where the pairs of ids lie in a dispatched layout, into s: counts [E], seg [E + 1], src2dst [T * K], the number of
    rows, the row, token and slot of each valid pair, and each expert's rows as index [E, most], absent ones = rows."""
    e, k = c["experts"], c["topk"]
    flat = ids.flatten().long()
    pair = torch.nonzero(flat >= 0).flatten()
    pair = pair[torch.sort(flat[pair], stable=True).indices]
    exp = flat[pair]
    counts = torch.bincount(exp, minlength=e)
    start = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    rank = torch.arange(len(pair), device=DEV) - start[exp]
    if c["layout"] == "masked":
        seg, base, rows = start, torch.arange(e, device=DEV) * c["capacity"], e * c["capacity"]
    else:
        a = c["align"]
        seg = torch.cat((counts.new_zeros(1), ((counts + a - 1) // a * a).cumsum(0)))
        base, rows = seg[:-1], ids.numel() + e * (a - 1)
    most = max(1, int(counts.max()))
    j = torch.arange(most, device=DEV)
    s["counts"], s["seg"], s["rows"] = counts.int(), seg, rows
    s["src2dst"] = torch.full((ids.numel(),), -1, dtype=torch.int32, device=DEV)
    s["src2dst"][pair] = (seg[exp] + rank).int()
    s["at"], s["token"], s["slot"] = base[exp] + rank, pair // k, pair % k
    s["index"] = torch.where(j < counts[:, None], base[:, None] + j, rows)


def _normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, device=DEV, generator=gen) * std).bfloat16()


def _weights(gen, experts, rows, inner):
    w = torch.empty(experts, rows, inner, dtype=torch.bfloat16, device=DEV)
    for e in range(experts):
        w[e] = torch.randn(rows, inner, device=DEV, generator=gen) * inner ** -0.5
    return w


def _rows_of(s, gen, c, width, std=1.0):
    """bf16 values in the rows that pairs map to, zeros in the others."""
    out = torch.zeros(s["rows"], width, dtype=torch.bfloat16, device=DEV)
    out[s["at"]] = _normal(gen, len(s["at"]), width, std=std)
    return out


def _tokens_of(s, gen, c, width):
    """The same, each pair's row its token's."""
    out = torch.zeros(s["rows"], width, dtype=torch.bfloat16, device=DEV)
    out[s["at"]] = _normal(gen, c["tokens"], width)[s["token"]]
    return out


def _empty_rows(s, width):
    return torch.zeros(s["rows"], width, dtype=torch.bfloat16, device=DEV)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c, "status": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if c["op"] == "norm":
        t, h = c["tokens"], c["hidden"]
        # a few channels are much larger than the others, as they are in trained models
        channel = 1 + 9 * (torch.rand(h, device=DEV, generator=gen) < 0.01)
        s["x"] = (torch.randn(t, h, device=DEV, generator=gen) * channel).bfloat16()
        s["residual"] = (torch.randn(t, h, device=DEV, generator=gen) * 3 * channel).bfloat16() if c["residual"] else None
        s["weight"] = (1 + 0.1 * torch.randn(h, device=DEV, generator=gen)).bfloat16()
        if c["train"]:
            s["grad"] = _normal(gen, t, h)
            s["grad_residual"] = _normal(gen, t, h) if c["residual"] else None
        return s
    ids = _route(gen, c)
    _layout(s, c, ids)
    if c["op"] == "combine":
        s["ids"], s["w"] = ids, torch.randn(c["tokens"], c["topk"], device=DEV, generator=gen).softmax(-1)
        s["grad"] = _normal(gen, c["tokens"], c["hidden"])
        s["expert_out"] = _rows_of(s, gen, c, c["hidden"])
        s["grad_rows"] = _empty_rows(s, c["hidden"])
        s["grad_w"] = torch.empty(c["tokens"], c["topk"], device=DEV)
        return s
    if c["op"] == "product":
        s["a"] = _rows_of(s, gen, c, c["inner"])
        s["w"] = _weights(gen, c["experts"], c["cols"], c["inner"])
        s["out"] = _empty_rows(s, c["cols"])
        return s
    h, i, e = c["hidden"], c["inter"], c["experts"]
    if c["op"] == "swiglu":
        s["a"], s["w13"] = _tokens_of(s, gen, c, h), _weights(gen, e, 2 * i, h)
        s["h"] = _empty_rows(s, i)
        s["gate_up"] = _empty_rows(s, 2 * i) if c["keep"] else None
    elif c["op"] == "rows":
        s["grad"], s["gate_up"] = _rows_of(s, gen, c, h), _rows_of(s, gen, c, 2 * i)
        s["w13"], s["w2"] = _weights(gen, e, 2 * i, h), _weights(gen, e, h, i)
        s["grad_gate_up"], s["grad_rows"] = _empty_rows(s, 2 * i), _empty_rows(s, h)
    else:
        s["a"], s["grad"] = _tokens_of(s, gen, c, h), _rows_of(s, gen, c, h)
        s["h"], s["grad_gate_up"] = _rows_of(s, gen, c, i, 0.4), _rows_of(s, gen, c, 2 * i, 0.5)
        dtype = torch.float32 if c["out"] == "float32" else torch.bfloat16
        s["grad_w13"] = torch.empty(e, 2 * i, h, dtype=dtype, device=DEV)
        s["grad_w2"] = torch.empty(e, h, i, dtype=dtype, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    return {"product": _run_product, "swiglu": _run_swiglu, "rows": _run_rows, "weights": _run_weights,
            "combine": _run_combine, "norm": _run_norm}[c["op"]](s, c)


def _where(s, c):
    """Where the rows of a layout's experts lie, as the entry points take it."""
    return dict(seg_indptr=s["seg"] if c["layout"] == "normal" else None, max_tokens_per_expert=c["capacity"])


def _of_layout(s, t):
    """Rows of a layout as [E, most, ..] in fp32, zeros in the absent ones."""
    return torch.cat((t, torch.zeros_like(t[:1])))[s["index"]].float()


def _to_layout(s, y):
    """[E, most, N] back to the layout's rows, as bf16."""
    out = torch.zeros(s["rows"] + 1, y.shape[-1], dtype=torch.bfloat16, device=DEV)
    out[s["index"].flatten()] = y.flatten(0, 1).bfloat16()
    out[s["rows"]] = 0
    return out[:s["rows"]]


def _run_product(s, c):
    if own:
        import combine_moe_route_meta_gb300 as moe
        moe.moe_expert_gemm_bf16(c["layout"], s["a"], s["counts"], s["w"], s["out"], s["status"], **_where(s, c))
        return s["out"]
    return _to_layout(s, torch.bmm(_of_layout(s, s["a"]), s["w"].float().transpose(1, 2)))


def _run_swiglu(s, c):
    if own:
        import combine_moe_route_meta_gb300 as moe
        moe.moe_expert_gemm_swiglu_bf16(c["layout"], s["a"], s["counts"], s["w13"], s["h"], s["status"],
                                        gate_up=s["gate_up"], **_where(s, c))
        return {"h": s["h"], "gate_up": s["gate_up"]}
    y = torch.bmm(_of_layout(s, s["a"]), s["w13"].float().transpose(1, 2))
    gate, up = y.chunk(2, dim=-1)
    return {"h": _to_layout(s, up * (gate / (1 + torch.exp(-gate)))), "gate_up": _to_layout(s, y) if c["keep"] else None}


def _run_rows(s, c):
    if own:
        import combine_moe_route_meta_gb300 as moe
        moe.moe_expert_gemm_dswiglu_bf16(c["layout"], s["grad"], s["counts"], s["w2"], s["gate_up"], s["grad_gate_up"],
                                         s["status"], **_where(s, c))
        moe.moe_expert_gemm_bf16(c["layout"], s["grad_gate_up"], s["counts"], s["w13"], s["grad_rows"], s["status"],
                                 transposed=True, **_where(s, c))
        return {"grad_gate_up": s["grad_gate_up"], "grad_rows": s["grad_rows"]}
    dh = torch.bmm(_of_layout(s, s["grad"]), s["w2"].float())
    gate, up = _of_layout(s, s["gate_up"]).chunk(2, dim=-1)
    p = 1 / (1 + torch.exp(-gate))
    d = torch.cat((dh * up * (p * (1 + gate * (1 - p))), dh * (gate * p)), dim=-1)
    return {"grad_gate_up": _to_layout(s, d), "grad_rows": _to_layout(s, torch.bmm(d, s["w13"].float()))}


def _run_weights(s, c):
    if own:
        import combine_moe_route_meta_gb300 as moe
        moe.moe_expert_wgrad_bf16(c["layout"], s["grad"], s["h"], s["counts"], s["grad_w2"], s["status"], **_where(s, c))
        moe.moe_expert_wgrad_bf16(c["layout"], s["grad_gate_up"], s["a"], s["counts"], s["grad_w13"], s["status"],
                                  **_where(s, c))
        return {"grad_w2": s["grad_w2"], "grad_w13": s["grad_w13"]}
    dtype = s["grad_w2"].dtype
    return {"grad_w2": torch.bmm(_of_layout(s, s["grad"]).transpose(1, 2), _of_layout(s, s["h"])).to(dtype),
            "grad_w13": torch.bmm(_of_layout(s, s["grad_gate_up"]).transpose(1, 2), _of_layout(s, s["a"])).to(dtype)}


def _run_combine(s, c):
    if own:
        import combine_moe_route_meta_gb300 as moe
        moe.moe_combine_backward(c["layout"], s["grad"], s["expert_out"], s["ids"], s["w"], c["experts"], s["src2dst"],
                                 s["seg"], s["grad_rows"], s["grad_w"], s["status"],
                                 max_tokens_per_expert=c["capacity"], expert_out_rows=s["rows"])
        return {"grad_rows": s["grad_rows"], "grad_w": s["grad_w"]}
    g = s["grad"].float()[s["token"]]
    rows = torch.zeros(s["rows"], c["hidden"], dtype=torch.bfloat16, device=DEV)
    rows[s["at"]] = (g * s["w"][s["token"], s["slot"]][:, None]).bfloat16()
    w = torch.zeros(c["tokens"], c["topk"], device=DEV)
    w[s["token"], s["slot"]] = (g * s["expert_out"][s["at"]].float()).sum(-1)
    return {"grad_rows": rows, "grad_w": w}


def _run_norm(s, c):
    if own:
        import combine_moe_route_meta_gb300 as moe
        y = moe.rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], quant=c["quant"],
                        bf16=c["train"] or c["quant"] == "none", keep=c["train"])
        out = {"rows": y.out, "codes": None, "scales": y.scales, "sum": y.sum if c["residual"] else None, "rstd": y.rstd}
        if c["quant"] != "none":
            out["codes"] = y.codes.view(torch.float8_e4m3fn)
        if c["train"]:
            out["grad_x"], out["grad_weight"] = moe.rmsnorm_backward(s["grad"], y.sum, s["weight"], y.rstd,
                                                                     grad_residual=s["grad_residual"])
        return out
    h = s["x"]
    if c["residual"]:
        h = (h.float() + s["residual"].float()).bfloat16()
    f, w = h.float(), s["weight"].float()
    r = 1 / torch.sqrt((f * f).mean(-1) + EPS)
    hat = f * r[:, None]
    y = hat * w
    out = {"rows": y.bfloat16() if c["train"] or c["quant"] == "none" else None, "codes": None, "scales": None,
           "sum": h if c["residual"] else None, "rstd": r if c["train"] else None}
    if c["quant"] != "none":
        b = y.unflatten(-1, (-1, 128))
        out["scales"] = b.abs().amax(-1).clamp(min=1e-10) / 448.0
        out["codes"] = (b / out["scales"][..., None]).to(torch.float8_e4m3fn).flatten(-2)
    if c["train"]:
        g = s["grad"].float()
        d = r[:, None] * (g * w - hat * (g * w * hat).mean(-1, keepdim=True))
        out["grad_x"] = (d + s["grad_residual"].float() if c["residual"] else d).bfloat16()
        out["grad_weight"] = (g * hat).sum(0)
    return out


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _e4m3_nearest(v):
    """The e4m3 values nearest to v, |v| <= 448 and a little, in 64 bits (ties to the even code)."""
    _, e = torch.frexp(v.abs().clamp(min=2.0 ** -7))          # |v| in [2^(e-1), 2^e): steps of 2^(e-4), at least 2^-9
    step = torch.ldexp(torch.ones_like(v), (e - 4).clamp(min=-9))
    return (torch.round(v / step) * step).clamp(-448, 448)


def _experts64(s):
    """(expert, its rows as a slice) of every expert with rows."""
    for e, (n, first) in enumerate(zip(s["counts"].tolist(), s["index"][:, 0].tolist())):
        if n:
            yield e, slice(first, first + n)


def _zeros64(s, width):
    return torch.zeros(s["rows"], width, dtype=torch.float64, device=DEV)


def exact(case, seed):
    c = dict(case)
    if work(c)["flops"] > 1e13:
        return None
    s = prepare(case, seed)
    if c["op"] == "norm":
        x = s["x"].double()
        if c["residual"]:
            x = (x + s["residual"].double()).to(torch.bfloat16).double()
        w = s["weight"].double()
        r = (x.square().mean(-1) + EPS).rsqrt()
        y = x * r[:, None] * w
        out = {"rows": y if c["train"] or c["quant"] == "none" else None, "codes": None, "scales": None,
               "sum": x if c["residual"] else None, "rstd": r if c["train"] else None}
        if c["quant"] != "none":
            amax = y.view(c["tokens"], -1, 128).abs().max(-1).values
            out["scales"] = torch.maximum(amax, torch.full_like(amax, 1e-10)) / 448
            out["codes"] = _e4m3_nearest(y / out["scales"].repeat_interleave(128, dim=1))
        if c["train"]:
            g = s["grad"].double()
            dot = torch.einsum("th,th,h,th->t", g, x, w, r[:, None].expand_as(x)) / c["hidden"]
            out["grad_x"] = r[:, None] * (g * w) - (r * r * dot)[:, None] * x
            if c["residual"]:
                out["grad_x"] = out["grad_x"] + s["grad_residual"].double()
            out["grad_weight"] = torch.einsum("th,th,t->h", g, x, r)
        return out
    if c["op"] == "combine":
        rows = _zeros64(s, c["hidden"])
        w = torch.zeros(c["tokens"], c["topk"], dtype=torch.float64, device=DEV)
        for k in range(c["topk"]):
            m = s["slot"] == k
            t, at = s["token"][m], s["at"][m]
            g = s["grad"][t].double()
            rows[at] = s["w"][t, k].double()[:, None] * g
            w[t, k] = torch.einsum("rh,rh->r", g, s["expert_out"][at].double())
        return {"grad_rows": rows, "grad_w": w}
    if c["op"] == "product":
        out = _zeros64(s, c["cols"])
        for e, at in _experts64(s):
            out[at] = s["a"][at].double() @ s["w"][e].double().T
        return out
    h, i = c["hidden"], c["inter"]
    if c["op"] == "swiglu":
        out, gu = _zeros64(s, i), _zeros64(s, 2 * i)
        for e, at in _experts64(s):
            gu[at] = s["a"][at].double() @ s["w13"][e].double().T
            out[at] = gu[at, i:] * gu[at, :i] * torch.sigmoid(gu[at, :i])
        return {"h": out, "gate_up": gu if c["keep"] else None}
    if c["op"] == "rows":
        d, dx = _zeros64(s, 2 * i), _zeros64(s, h)
        for e, at in _experts64(s):
            dh = s["grad"][at].double() @ s["w2"][e].double()
            g, u = s["gate_up"][at, :i].double(), s["gate_up"][at, i:].double()
            p = torch.sigmoid(g)
            d[at, :i], d[at, i:] = dh * u * (p + g * p * (1 - p)), dh * g * p
            dx[at] = d[at] @ s["w13"][e].double()
        return {"grad_gate_up": d, "grad_rows": dx}
    w13 = torch.zeros(c["experts"], 2 * i, h, dtype=torch.float64, device=DEV)
    w2 = torch.zeros(c["experts"], h, i, dtype=torch.float64, device=DEV)
    for e, at in _experts64(s):
        w2[e] = s["grad"][at].double().T @ s["h"][at].double()
        w13[e] = s["grad_gate_up"][at].double().T @ s["a"][at].double()
    return {"grad_w2": w2, "grad_w13": w13}
