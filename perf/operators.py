"""Cases that measure the expert operators between dispatch and combine.

Four kinds of pass, all on the NVFP4 form that the dispatch writes (e2m1 codes, two a byte, and an e4m3
scale for each 16 values) or, for the few-token layer, on bf16 weights too:

  quantise   bf16 rows -> codes and scales -> bf16 rows read back from them
  product    rows of a dispatched layout times their expert's weights, bf16 out
  experts    gate and up products, SwiGLU, requantisation, down product: a dispatched layout in, bf16 out
  layer      a whole layer for a few tokens: routed experts and their weighted sum in token order

A pass that writes into a layout's buffer leaves the rows that no token maps to as prepare() made them: zero.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
H_SCALE = 168.0  # global scale of the SwiGLU outputs: 448 * 6 over an expected maximum of 16


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # the rows of a decode batch on their way into an expert: latency
        dict(name="quantise 128 rows", op="quantise", groups=1, rows=128, hidden=7168, scales="swizzled"),
        # ragged: rows that fill no tile, a hidden size that is no power of two, scales row by row
        dict(name="quantise ragged rows", op="quantise", groups=3, rows=1001, hidden=4160, scales="row"),
        # gate and up weights of one partition's 32 experts, quantised when a checkpoint is loaded
        dict(name="quantise weights", op="quantise", groups=32, rows=2048, hidden=7168, scales="swizzled"),
        # the down product of a decode batch in the masked layout: about 4 rows an expert, weights dominate
        dict(name="product decode", op="product", layout="masked", tokens=128, cols=7168, inner=1024, experts=256,
             topk=8, capacity=128, align=1, scales="row", routing="uniform", invalid=0.0),
        # a prefill batch with a few popular experts, segments aligned to 128 rows
        dict(name="product skewed prefill", op="product", layout="normal", tokens=2048, cols=4096, inner=768,
             experts=128, topk=8, capacity=0, align=128, scales="swizzled", routing="zipf", invalid=0.0),
        # all experts' MLPs of a decode batch
        dict(name="experts decode", op="experts", layout="masked", tokens=128, hidden=7168, inter=1024, experts=256,
             topk=8, capacity=128, align=1, scales="swizzled", routing="uniform", invalid=0.0),
        # one partition of 16 experts, segments without padding, dropped slots, an odd number of tokens
        dict(name="experts ragged", op="experts", layout="normal", tokens=1501, hidden=4096, inter=704, experts=16,
             topk=4, capacity=0, align=1, scales="row", routing="uniform", invalid=0.05),
        # the largest: a full prefill batch over all experts
        dict(name="experts prefill", op="experts", layout="normal", tokens=8192, hidden=7168, inter=1024, experts=256,
             topk=8, capacity=0, align=128, scales="swizzled", routing="uniform", invalid=0.0),
        # one sequence being decoded
        dict(name="layer 1 token", op="layer", weights="nvfp4", tokens=1, hidden=7168, inter=1024, experts=256,
             topk=8, invalid=0.0),
        # a handful of sequences on a model kept in bf16
        dict(name="layer 5 tokens bf16", op="layer", weights="bf16", tokens=5, hidden=4096, inter=768, experts=128,
             topk=8, invalid=0.0),
        # a small serving batch
        dict(name="layer 32 tokens", op="layer", weights="nvfp4", tokens=32, hidden=7168, inter=1024, experts=256,
             topk=8, invalid=0.0),
        # few experts that many tokens share, dropped slots, odd sizes
        dict(name="layer 61 tokens bf16", op="layer", weights="bf16", tokens=61, hidden=2112, inter=704, experts=16,
             topk=3, invalid=0.1),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    def size(a, b):  # a multiple of 64
        while True:
            n = 64 * log(a // 64, b // 64)
            if n != 3072 and 2 * n != 3072:
                return n

    op = rng.choice(["quantise", "product", "experts", "layer"])
    if op == "quantise":
        hidden, groups = size(256, 8192), log(1, 32)
        rows = log(1, max(2, min(65536, (1 << 28) // (hidden * groups))))
        return dict(op=op, groups=groups, rows=rows + (rows == 3072), hidden=hidden,
                    scales=rng.choice(["row", "swizzled"]))
    hidden, inter = size(512, 8192), size(128, 2048)
    experts = min(log(4, 256), max(4, int(1.5e9) // (3 * hidden * inter)))
    topk = min(rng.randint(1, 8), experts)
    invalid = rng.choice([0.0, 0.0, 0.05, 0.3])
    if op == "layer":
        return dict(op=op, weights=rng.choice(["nvfp4", "bf16"]), tokens=log(1, 64), hidden=hidden, inter=inter,
                    experts=experts, topk=topk, invalid=invalid)
    layout = rng.choice(["masked", "normal"])
    tokens = log(1, 512) if layout == "masked" else log(64, 4000)
    shape = dict(cols=hidden, inner=inter) if op == "product" else dict(hidden=hidden, inter=inter)
    return dict(op=op, layout=layout, tokens=tokens, experts=experts, topk=topk,
                capacity=-(-tokens // 16) * 16 if layout == "masked" else 0,
                align=rng.choice([1, 16, 128]) if layout == "normal" else 1,
                scales=rng.choice(["row", "swizzled"]), routing=rng.choice(["uniform", "zipf"]),
                invalid=invalid, **shape)


def work(case):
    c = dict(case)
    if c["op"] == "quantise":
        # values in, codes and scales out; codes and scales in, values out
        return {"bytes": c["groups"] * c["rows"] * c["hidden"] * (2 + 2 * 0.5625 + 2), "flops": 0}
    keep = 1 - c["invalid"]
    rows = c["tokens"] * c["topk"] * keep
    active = c["experts"] * (1 - (1 - c["topk"] * keep / c["experts"]) ** c["tokens"])  # of uniform routing
    if c["op"] == "product":
        n, k = c["cols"], c["inner"]
        return {"bytes": active * n * k * 0.5625 + rows * (k * 0.5625 + n * 2), "flops": 2 * rows * n * k}
    h, i = c["hidden"], c["inter"]
    if c["op"] == "experts":
        return {"bytes": active * 3 * h * i * 0.5625 + rows * h * (0.5625 + 2), "flops": 6 * rows * h * i}
    each = 0.5625 if c["weights"] == "nvfp4" else 2
    return {"bytes": active * 3 * h * i * each + c["tokens"] * h * 4, "flops": 6 * rows * h * i}


# ---------------------------------------------------------------------------------------------
# the formats, in elementary operations
# ---------------------------------------------------------------------------------------------

def _pairs():
    """[256, 2]: the two values that a byte of codes stands for."""
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV)
    b = torch.arange(256, device=DEV)
    return torch.stack((v[b & 15], v[b >> 4]), dim=1)


def _quantise(x, g):
    """Codes [.., K/2] and scales [.., K/16] (bytes) of x [.., K], in binary32 steps; g broadcasts against [.., K/16]."""
    b = x.float().unflatten(-1, (-1, 16))
    sf = ((b.abs().amax(-1) / 6.0) * g).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = sf.float()
    r = torch.where(s > 0, g / s, torch.zeros_like(s)).unsqueeze(-1)
    y = b * r
    m = y.abs()
    code = ((m > 0.25).byte() + (m >= 0.75).byte() + (m > 1.25).byte() + (m >= 1.75).byte() + (m > 2.5).byte()
            + (m >= 3.5).byte() + (m > 5.0).byte())
    code = torch.where(r > 0, code + 8 * torch.signbit(y).byte(), torch.zeros_like(code)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), sf.view(torch.uint8)


def _swizzle(sf):
    """Scales [.., R, C] as the bytes of 128 x 4 tiles, rows padded with zeros: [.., roundup(R, 128) * C]."""
    r, c = sf.shape[-2:]
    pad = -r % 128
    if pad:
        sf = torch.cat((sf, sf.new_zeros(*sf.shape[:-2], pad, c)), dim=-2)
    t = sf.unflatten(-1, (c // 4, 4)).unflatten(-3, ((r + pad) // 128, 4, 32))  # [.., block, r/32, r%32, c/4, c%4]
    n = t.dim()
    return t.permute(*range(n - 5), n - 5, n - 2, n - 3, n - 4, n - 1).reshape(*sf.shape[:-2], -1)


def _unswizzle(b, r, c):
    """The scales [.., R, C] of the bytes of _swizzle()."""
    t = b.reshape(*b.shape[:-1], -1, c // 4, 32, 4, 4)
    n = t.dim()
    return t.permute(*range(n - 5), n - 5, n - 2, n - 3, n - 4, n - 1).reshape(*b.shape[:-1], -1, c)[..., :r, :]


def _values(codes, sf):
    """The float32 values of codes [.., K/2] and scale bytes [.., K/16]."""
    v = _pairs()[codes.int()].flatten(-2).unflatten(-1, (-1, 16))
    return (v * sf.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _row_scales(s, r, c, layout):
    return s.reshape(*s.shape[:-1], r, c) if layout == "row" else _unswizzle(s, r, c)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _weights(gen, experts, halves, rows, inner):
    """NVFP4 weights of N(0, 1/inner): codes [E, halves*rows, inner/2], tiled scales [E, halves, ..], global scales [E]."""
    codes = torch.empty(experts, halves * rows, inner // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(experts, halves, -(-rows // 128) * 128 * (inner // 16), dtype=torch.uint8, device=DEV)
    g = torch.empty(experts, device=DEV)
    for e in range(experts):
        w = (torch.randn(halves, rows, inner, device=DEV, generator=gen) * inner ** -0.5).bfloat16()
        g[e] = 2688.0 / w.abs().amax().float()
        q, s = _quantise(w, g[e])
        codes[e] = q.flatten(0, 1)
        scales[e] = _swizzle(s)
    return codes, scales, g


def _route(gen, c):
    """Expert ids [T, K] int32, distinct in a token, some of them -1."""
    t, e, k = c["tokens"], c["experts"], c["topk"]
    if c.get("routing") == "zipf":
        p = (torch.randperm(e, device=DEV, generator=gen) + 1.0) ** -1.2
    else:
        p = torch.ones(e, device=DEV)
    ids = torch.multinomial(p.expand(t, e), k, generator=gen).int()
    if c["invalid"]:
        ids[torch.rand(t, k, device=DEV, generator=gen) < c["invalid"]] = -1
    return ids


def _layout(c, ids):
    """Where the pairs of ids lie in a dispatched layout: counts [E], first rows [E+1], the number of rows, the
    row of each valid pair, its token, and the rows of each expert as [E, most], absent ones = the number of rows."""
    e = c["experts"]
    flat = ids.flatten().long()
    pair = torch.nonzero(flat >= 0).flatten()
    exp = flat[pair]
    order = torch.sort(exp, stable=True).indices
    pair, exp = pair[order], exp[order]
    counts = torch.bincount(exp, minlength=e)
    start = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    rank = torch.arange(len(pair), device=DEV) - start[exp]
    if c["layout"] == "masked":
        base, rows = torch.arange(e + 1, device=DEV) * c["capacity"], e * c["capacity"]
    else:
        a = c["align"]
        base = torch.cat((counts.new_zeros(1), ((counts + a - 1) // a * a).cumsum(0)))
        rows = ids.numel() + e * (a - 1)
    most = max(1, int(counts.max()))
    j = torch.arange(most, device=DEV)
    index = torch.where(j < counts[:, None], base[:-1, None] + j, rows)
    return counts.int(), base, rows, base[exp] + rank, pair // c["topk"], index


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "quantise":
        x = torch.empty(c["groups"], c["rows"], c["hidden"], dtype=torch.bfloat16, device=DEV)
        for g in range(c["groups"]):
            x[g] = torch.randn(c["rows"], c["hidden"], device=DEV, generator=gen)
        s["x"], s["g"] = x, 2688.0 / x.abs().amax(dim=(1, 2)).float()
        return s
    ids = _route(gen, c)
    if c["op"] == "layer":
        t, h, i, e = c["tokens"], c["hidden"], c["inter"], c["experts"]
        s["x"] = torch.randn(t, h, device=DEV, generator=gen).bfloat16()
        s["ids"], s["w"] = ids, torch.randn(t, c["topk"], device=DEV, generator=gen).softmax(-1)
        if c["weights"] == "nvfp4":
            s["w13"], s["w13_s"], g = _weights(gen, e, 2, i, h)
            s["a13"] = 1 / g
            s["w2"], s["w2_s"], g = _weights(gen, e, 1, h, i)
            s["a2"] = 1 / g
        else:
            s["w13"] = torch.empty(e, 2 * i, h, dtype=torch.bfloat16, device=DEV)
            s["w2"] = torch.empty(e, h, i, dtype=torch.bfloat16, device=DEV)
            for j in range(e):
                s["w13"][j] = torch.randn(2 * i, h, device=DEV, generator=gen) * h ** -0.5
                s["w2"][j] = torch.randn(h, i, device=DEV, generator=gen) * i ** -0.5
            s["w13_s"] = s["w2_s"] = s["a13"] = s["a2"] = None
        s["out"] = torch.empty(t, h, dtype=torch.bfloat16, device=DEV)
    else:
        inner, cols = (c["inner"], c["cols"]) if c["op"] == "product" else (c["hidden"], c["hidden"])
        s["counts"], s["seg"], rows, at, token, s["index"] = _layout(c, ids)
        x = torch.randn(c["tokens"], inner, device=DEV, generator=gen).bfloat16()
        g = 2688.0 / x.abs().amax().float()
        q, sf = _quantise(x, g)
        codes = torch.zeros(rows, inner // 2, dtype=torch.uint8, device=DEV)
        scales = torch.zeros(rows, inner // 16, dtype=torch.uint8, device=DEV)
        codes[at], scales[at] = q[token], sf[token]
        s["a"], s["a_s"] = codes, (_swizzle(scales) if c["scales"] == "swizzled" else scales.flatten())
        if c["op"] == "product":
            s["w"], s["w_s"], gw = _weights(gen, c["experts"], 1, cols, inner)
            s["alpha"] = 1 / (g * gw)
        else:
            i = c["inter"]
            s["w13"], s["w13_s"], gw = _weights(gen, c["experts"], 2, i, inner)
            s["a13"] = 1 / (g * gw)
            s["w2"], s["w2_s"], gw = _weights(gen, c["experts"], 1, cols, i)
            s["a2"] = 1 / (H_SCALE * gw)
            s["h"] = torch.zeros(rows, i // 2, dtype=torch.uint8, device=DEV)
            s["h_s"] = torch.zeros(-(-rows // 128) * 128 * (i // 16), dtype=torch.uint8, device=DEV)
        s["out"] = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    return {"quantise": _run_quantise, "product": _run_product, "experts": _run_experts, "layer": _run_layer}[c["op"]](s, c)


def _run_quantise(s, c):
    if own:
        import combine_moe_route_meta_gb300 as moe
        q = moe.quantize_nvfp4(s["x"], s["g"], scale_layout=c["scales"])
        return {"values": moe.dequantize_nvfp4(q, s["g"]), "scales": q.scales.view(torch.float8_e4m3fn)}
    g = s["g"][:, None, None]
    codes, sf = _quantise(s["x"], g)
    values = (_values(codes, sf) / g).bfloat16()
    sf = _swizzle(sf) if c["scales"] == "swizzled" else sf
    return {"values": values, "scales": sf.view(torch.float8_e4m3fn)}


def _of_layout(s, t):
    """Rows of a layout as [E, most, ..], zeros in the absent ones."""
    return torch.cat((t, torch.zeros_like(t[:1])))[s["index"]]


def _to_layout(s, y, rows):
    """[E, most, N] back to the layout's rows, as bf16."""
    out = torch.zeros(rows + 1, y.shape[-1], dtype=torch.bfloat16, device=DEV)
    out[s["index"].flatten()] = y.flatten(0, 1).bfloat16()
    return out[:rows]


def _rows_in(s, c, inner):
    rows = s["a"].shape[0]
    return _values(_of_layout(s, s["a"]), _of_layout(s, _row_scales(s["a_s"], rows, inner // 16, c["scales"])))


def _run_product(s, c):
    if own:
        import combine_moe_route_meta_gb300 as moe
        moe.moe_expert_gemm(c["layout"], s["a"], s["a_s"], s["counts"], s["w"], s["w_s"], s["out"], s["status"],
                            alpha=s["alpha"], seg_indptr=s["seg"], max_tokens_per_expert=c["capacity"],
                            scale_layout=c["scales"])
        return s["out"]
    w = _values(s["w"], _unswizzle(s["w_s"], c["cols"], c["inner"] // 16).flatten(1, 2))
    y = torch.bmm(_rows_in(s, c, c["inner"]), w.transpose(1, 2)) * s["alpha"][:, None, None]
    return _to_layout(s, y, s["a"].shape[0])


def _swiglu(y):
    gate, up = y.chunk(2, dim=-1)
    return up * (gate / (1 + torch.exp(-gate)))


def _run_experts(s, c):
    if own:
        import combine_moe_route_meta_gb300 as moe
        moe.moe_expert_gemm_swiglu(c["layout"], s["a"], s["a_s"], s["counts"], s["w13"], s["w13_s"], s["h"], s["h_s"],
                                   s["status"], out_global_scale=H_SCALE, alpha=s["a13"], seg_indptr=s["seg"],
                                   max_tokens_per_expert=c["capacity"], scale_layout=c["scales"])
        moe.moe_expert_gemm(c["layout"], s["h"], s["h_s"], s["counts"], s["w2"], s["w2_s"], s["out"], s["status"],
                            alpha=s["a2"], seg_indptr=s["seg"], max_tokens_per_expert=c["capacity"],
                            scale_layout=c["scales"])
        return s["out"]
    h, i = c["hidden"], c["inter"]
    w = _values(s["w13"], _unswizzle(s["w13_s"], i, h // 16).flatten(1, 2))
    y = _swiglu(torch.bmm(_rows_in(s, c, h), w.transpose(1, 2)) * s["a13"][:, None, None])
    w = _values(s["w2"], _unswizzle(s["w2_s"], h, i // 16).flatten(1, 2))
    y = torch.bmm(_values(*_quantise(y, H_SCALE)), w.transpose(1, 2)) * s["a2"][:, None, None]
    return _to_layout(s, y, s["a"].shape[0])


def _run_layer(s, c):
    if own:
        import combine_moe_route_meta_gb300 as moe
        if "workspace" not in s:  # kept, as a program keeps it
            s["workspace"] = moe.new_layer_workspace(c["tokens"], c["topk"], c["hidden"], c["inter"], c["experts"])
        moe.moe_layer_few_tokens(s["x"], s["ids"], s["w"], s["w13"], s["w2"], s["out"], s["workspace"], s["status"],
                                 w13_scales=s["w13_s"], w2_scales=s["w2_s"], alpha13=s["a13"], alpha2=s["a2"])
        return s["out"]
    t, k, h, i = c["tokens"], c["topk"], c["hidden"], c["inter"]
    e = s["ids"].flatten().clamp(min=0).long()
    used = (s["w"] * (s["ids"] >= 0)).flatten()[:, None]
    if c["weights"] == "nvfp4":
        w13 = _values(s["w13"][e], _unswizzle(s["w13_s"][e], i, h // 16).flatten(1, 2)) * s["a13"][e][:, None, None]
        w2 = _values(s["w2"][e], _unswizzle(s["w2_s"][e], h, i // 16).flatten(1, 2)) * s["a2"][e][:, None, None]
    else:
        w13, w2 = s["w13"][e].float(), s["w2"][e].float()
    x = s["x"].float().repeat_interleave(k, 0)
    y = _swiglu(torch.bmm(w13, x[:, :, None])[:, :, 0])
    y = torch.bmm(w2, y[:, :, None])[:, :, 0] * used
    return y.view(t, k, h).sum(1).bfloat16()


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _e4m3_table():
    """The finite values of the non-negative codes 0..126."""
    return torch.tensor([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                         for e in range(16) for m in range(8)][:127], dtype=torch.float64, device=DEV)


def _nearest(v, table):
    """Index of the entry nearest to v >= 0 (ties: the even index), the last one beyond the table."""
    mid = (table[1:] + table[:-1]) / 2
    low = torch.bucketize(v, mid)  # entries below v's interval; v equal to a middle stays at the lower one
    tie = (low < len(mid)) & (v == mid[low.clamp(max=len(mid) - 1)]) & (low % 2 == 1)
    return low + tie


def _r32(v):
    return v.float().double()


def _quantised64(x, g):
    """The values and scales [.., K/16] that x [.., K] in 64 bits is quantised to."""
    table, e2m1 = _e4m3_table(), torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    b = x.unflatten(-1, (-1, 16))
    s = table[_nearest(_r32(_r32(b.abs().amax(-1) / 6) * g), table)]
    r = torch.where(s > 0, _r32(g / s.clamp(min=2.0 ** -9)), torch.zeros_like(s))
    v = e2m1[_nearest(_r32(b * r[..., None]).abs(), e2m1)] * torch.where(b < 0, -1.0, 1.0).double()
    return (v * s[..., None]).flatten(-2), s


def _tiles64(b, rows, cols):
    """Scales [rows, cols] in 64 bits of one matrix's 128 x 4 tiles, entry by entry."""
    r, c = torch.arange(rows, device=DEV)[:, None], torch.arange(cols, device=DEV)
    at = ((r // 128) * (cols // 4) + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4
    return torch.cat((_e4m3_table(), _e4m3_table()[:1]))[b.long()][at]


def _codes64(q):
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device=DEV)
    return torch.stack((v[(q & 15).long()], v[(q >> 4).long()]), dim=-1).flatten(-2)


def _matrix64(codes, scales, halves, rows, inner):
    sf = torch.cat([_tiles64(scales[j], rows, inner // 16) for j in range(halves)])
    return _codes64(codes) * sf.repeat_interleave(16, dim=1)


def exact(case, seed):
    c = dict(case)
    if work(c)["flops"] > 1e13:  # minutes in 64 bits
        return None
    s = prepare(case, seed)
    if c["op"] == "quantise":
        values = torch.empty(s["x"].shape, dtype=torch.float64, device=DEV)
        scales = []
        for j in range(c["groups"]):
            g = s["g"][j].double()
            v, f = _quantised64(s["x"][j].double(), g)
            values[j] = v / g
            if c["scales"] == "swizzled":
                r, n = torch.arange(f.shape[0], device=DEV)[:, None], f.shape[1]
                k = torch.arange(n, device=DEV)
                at = ((r // 128) * (n // 4) + k // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + k % 4
                t = f.new_zeros(-(-f.shape[0] // 128) * 128 * n)
                t[at.flatten()] = f.flatten()
                f = t
            scales.append(f)
        return {"values": values, "scales": torch.stack(scales)}
    if c["op"] == "layer":
        h, i = c["hidden"], c["inter"]
        out = torch.zeros(c["tokens"], h, dtype=torch.float64, device=DEV)
        for e in torch.unique(s["ids"]).tolist():
            if e < 0:
                continue
            t, k = torch.nonzero(s["ids"] == e, as_tuple=True)
            if c["weights"] == "nvfp4":
                w13 = _matrix64(s["w13"][e], s["w13_s"][e], 2, i, h) * s["a13"][e].double()
                w2 = _matrix64(s["w2"][e], s["w2_s"][e], 1, h, i) * s["a2"][e].double()
            else:
                w13, w2 = s["w13"][e].double(), s["w2"][e].double()
            y = s["x"][t].double() @ w13.T
            y = y[:, i:] * y[:, :i] * torch.sigmoid(y[:, :i])
            out.index_add_(0, t, (y @ w2.T) * s["w"][t, k].double()[:, None])
        return out
    inner = c["inner"] if c["op"] == "product" else c["hidden"]
    rows = s["a"].shape[0]
    sf = _tiles64(s["a_s"], rows, inner // 16) if c["scales"] == "swizzled" else \
        torch.cat((_e4m3_table(), _e4m3_table()[:1]))[s["a_s"].long()].view(rows, -1)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for e, (n, first) in enumerate(zip(s["counts"].tolist(), s["seg"].tolist())):
        if not n:
            continue
        at = slice(first, first + n)
        a = _codes64(s["a"][at]) * sf[at].repeat_interleave(16, dim=1)
        if c["op"] == "product":
            out[at] = a @ _matrix64(s["w"][e], s["w_s"][e], 1, c["cols"], inner).T * s["alpha"][e].double()
            continue
        i = c["inter"]
        y = a @ _matrix64(s["w13"][e], s["w13_s"][e], 2, i, inner).T * s["a13"][e].double()
        y, _ = _quantised64(y[:, i:] * y[:, :i] * torch.sigmoid(y[:, :i]), H_SCALE)
        out[at] = y @ _matrix64(s["w2"][e], s["w2_s"][e], 1, inner, i).T * s["a2"][e].double()
    return out
