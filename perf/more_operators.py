"""Cases that measure the operators of 4-bit microscaled values (MXFP4: E2M1
codes with one power-of-two scale per 32 values) and of expert layers for a
few tokens:

  quantize  rows quantised to MXFP4 and read back
  route     tokens sorted by expert into the products' rows, quantised on the way
  glu       the gated activation between two products, quantised
  gemm      the MXFP4 x MXFP4 products, dense and grouped
  experts   a whole expert layer (both products, the activation, the weighted
            sum) for a few tokens, with FP8 or MXFP4 weights

`run` computes a case either in elementary torch operations in 32 bits
(`own` false; the activation's values, which are rounded to four bits, in 64)
or through the package's entry points (`own` true). Quantised results are
returned as the values that they stand for.
"""

import math

import torch

own = False

LAYOUTS = ("contiguous", "nopad", "masked")
BLOCK = 128       # rows of a segment, values of an FP8 scale
MX = 32           # values of an MXFP4 scale
FP8_MAX = 448.0


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # A decode batch's activations on their way into a dense product: an odd count of rows.
        {"name": "quantize_rows", "op": "quantize", "groups": 1, "rows": 67, "k": 7168, "wide": False},
        # Eight experts' weights quantised once from a float32 master copy.
        {"name": "quantize_weights", "op": "quantize", "groups": 8, "rows": 4096, "k": 7168, "wide": True},
        # A decode step of a few requests: five tokens to the rows of sixteen local experts.
        {"name": "route_decode", "op": "route", "layout": "nopad", "tokens": 5, "top_k": 8, "groups": 16,
         "hidden": 7168, "skew": 0.0, "drop": 0.0},
        # A long prompt: 65536 rows over 32 experts by a Zipf law, in 128-row segments.
        {"name": "route_prefill", "op": "route", "layout": "contiguous", "tokens": 8192, "top_k": 8, "groups": 32,
         "hidden": 7168, "skew": 1.2, "drop": 0.0},
        # The activation of a decode step: masked receive rows, half of them empty.
        {"name": "glu_decode", "op": "glu", "layout": "masked", "groups": 16, "rows": 256, "inner": 2048},
        # The activation of a prompt: eight experts of 3000 to 5000 rows, 128-row segments.
        {"name": "glu_prefill", "op": "glu", "layout": "contiguous", "groups": 8, "rows": 4000, "inner": 2048},
        # The second product of a decode step, bound by the weights that it reads.
        {"name": "gemm_decode", "op": "gemm", "layout": "masked", "groups": 16, "rows": 256, "n": 7168, "k": 2048},
        # A dense product of a prompt.
        {"name": "gemm_dense", "op": "gemm", "layout": "dense", "groups": 1, "rows": 4096, "n": 7168, "k": 2048},
        # The first product of a prompt: eight experts, 128-row segments, ragged.
        {"name": "gemm_prefill", "op": "gemm", "layout": "contiguous", "groups": 8, "rows": 3677, "n": 4096,
         "k": 7168},
        # One token through eight of sixteen experts held in four bits.
        {"name": "experts_one", "op": "experts", "fp4": True, "tokens": 1, "top_k": 8, "groups": 16, "hidden": 7168,
         "inner": 2048, "drop": 0.0},
        # Three tokens through a small layer: latency is all.
        {"name": "experts_small", "op": "experts", "fp4": False, "tokens": 3, "top_k": 2, "groups": 8, "hidden": 2048,
         "inner": 512, "drop": 0.0},
        # A decode batch through 32 experts in FP8: every expert has a few tokens.
        {"name": "experts_batch", "op": "experts", "fp4": False, "tokens": 61, "top_k": 8, "groups": 32,
         "hidden": 7168, "inner": 2048, "drop": 0.0},
    ]


def draw(rng):
    def log_size(low, high, step=1):
        v = int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)) * step
        return min(max(v, low), high)

    op = rng.choice(("quantize", "route", "glu", "gemm", "gemm", "experts", "experts"))
    if op == "quantize":
        return {"op": op, "groups": rng.choice((1, 1, 2, 5, 8)), "rows": log_size(1, 4096),
                "k": log_size(128, 7168, 128), "wide": rng.random() < 0.4}
    if op == "route":
        top_k = rng.randint(1, 8)
        return {"op": op, "layout": rng.choice(LAYOUTS), "tokens": log_size(1, 8192), "top_k": top_k,
                "groups": log_size(max(2, top_k), 256), "hidden": log_size(256, 7168, 128),
                "skew": rng.choice((0.0, 0.6, 1.2)), "drop": rng.choice((0.0, 0.1, 0.5))}
    groups = log_size(1, 32)
    if op == "glu":
        return {"op": op, "layout": rng.choice(LAYOUTS), "groups": groups, "rows": log_size(1, max(2, 29000 // groups)),
                "inner": log_size(128, 2048, 128)}
    if op == "gemm":
        layout = rng.choice(("dense", *LAYOUTS))
        groups = 1 if layout == "dense" else groups
        k = log_size(128, 7168, 128)
        n = min(log_size(128, 7168, 128), max(128, 8 * 4096 * 7168 // (groups * k) // 128 * 128))
        most = max(2, min(29000, 8 * 3677 * 4096 * 7168 // (n * k)) // groups)
        return {"op": op, "layout": layout, "groups": groups, "rows": log_size(1, most), "n": n, "k": k}
    top_k = rng.randint(1, 8)
    hidden, inner = log_size(256, 7168, 128), log_size(128, 2048, 128)
    groups = log_size(max(2, top_k), max(32, min(128, 32 * 7168 * 2048 // (hidden * inner))))
    return {"op": op, "fp4": rng.random() < 0.5, "tokens": log_size(1, 64), "top_k": top_k, "groups": groups,
            "hidden": hidden, "inner": inner, "drop": rng.choice((0.0, 0.1, 0.5))}


def work(case):
    op = case["op"]
    mx = 0.5 + 1 / MX          # bytes of an MXFP4 value
    if op == "quantize":       # read, and the values written
        values = case["groups"] * case["rows"] * case["k"]
        return {"bytes": values * ((4 if case["wide"] else 2) + 2), "flops": 4.0 * values}
    if op == "route":
        slots = case["tokens"] * case["top_k"]
        rows = slots * (1.0 - case["drop"])
        layout = 4 * capacity(case) if case["layout"] == "contiguous" else 0
        return {"bytes": 2 * case["tokens"] * case["hidden"] + 2 * rows * case["hidden"] + 8 * slots
                + 4 * case["groups"] + layout, "flops": 4.0 * case["tokens"] * case["hidden"]}
    if op in ("glu", "gemm"):
        # masked counts are uniform in [0, rows]: half of the rows on average
        m = case["groups"] * case["rows"] * (0.5 if case["layout"] == "masked" else 1.0)
    if op == "glu":
        return {"bytes": m * case["inner"] * (4 + 2), "flops": 8.0 * m * case["inner"]}
    if op == "gemm":
        n, k = case["n"], case["k"]
        return {"bytes": mx * (m + case["groups"] * n) * k + 2 * m * n, "flops": 2.0 * m * n * k}
    k = case["top_k"] * (1.0 - case["drop"])
    active = case["groups"] * (1.0 - (1.0 - k / case["groups"]) ** case["tokens"])
    weights = 3 * case["hidden"] * case["inner"]
    return {"bytes": active * weights * (mx if case["fp4"] else 1 + 4 / BLOCK ** 2) + 4 * case["tokens"] * case["hidden"]
            + 8 * case["tokens"] * case["top_k"], "flops": 2.0 * case["tokens"] * k * weights}


def capacity(case):
    """Rows of the permuted buffers of `route`: what a program that knows only
    the token count has to set aside (masked: rows of a group, the mean load
    with room above it, so that a few rows may overflow under a skewed draw)."""
    slots = case["tokens"] * case["top_k"]
    if case["layout"] == "masked":
        return min(max(8, -(-2 * slots // case["groups"])), 65536 // case["groups"])
    if case["layout"] == "nopad":
        return slots
    return up(slots + min(case["groups"], slots) * (BLOCK - 1), BLOCK)


def up(m, step):
    return (m + step - 1) // step * step


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _device():
    return torch.device("cuda:0" if torch.cuda.is_available() else "cpu")


def _to_codes(blocks, exponent):
    """E2M1 codes (sign bit 3) of blocks [..., 32] over 2^exponent, ties to the even code."""
    a = torch.ldexp(blocks.abs(), -exponent[..., None])
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code | torch.signbit(blocks).to(torch.uint8) << 3


def _mx_exponent(blocks):
    """Exponent of the smallest power of two that is not below amax / 6."""
    mantissa, exponent = torch.frexp(blocks.abs().amax(-1))
    exponent = exponent - 3 + (mantissa > 0.75).to(exponent.dtype)
    return torch.where(mantissa == 0, -127, exponent.clamp(-127, 127))


def _mx(x):
    """x [..., M, K] quantised as the products take it: codes packed two a byte
    [..., M, K/2] and scales [..., K/128, M up to a multiple of 4] int32, byte i
    of which is the E8M0 code of the i-th 32 values of the 128."""
    blocks = x.unflatten(-1, (-1, MX))
    exponent = _mx_exponent(blocks)
    code = _to_codes(blocks, exponent).flatten(-2)
    packed = code[..., 0::2] | code[..., 1::2] << 4
    words = (exponent + 127).to(torch.uint8).contiguous().view(torch.int32)
    *lead, m, blocks128 = words.shape
    sf = torch.zeros(*lead, blocks128, up(m, 4), dtype=torch.int32, device=x.device)
    sf[..., :m] = words.transpose(-1, -2)
    return packed.contiguous(), sf


def _inputs(case, seed):
    """Everything that comes from the seed, as tensors by name."""
    dev = _device()
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32) * scale).to(dtype)

    def hidden_states(*shape, dtype=torch.bfloat16):
        x = normal(*shape, dtype=dtype)
        x[..., :: shape[-1] // 4] *= 20.0  # a few channels far above the rest, as hidden states have them
        return x

    def experts_of(n, k, g, skew, drop):
        """Experts by a Zipf law of exponent `skew` over a shuffled order, the k
        of a token distinct (the largest of its perturbed log weights)."""
        logits = -skew * torch.log(torch.arange(1, g + 1, device=dev, dtype=torch.float32))
        logits = logits[torch.randperm(g, generator=gen, device=dev)]
        noise = -torch.log(-torch.log(torch.rand(n, g, generator=gen, device=dev).clamp(1e-6, 1 - 1e-6)))
        ids = torch.topk(logits + noise, k, dim=1).indices
        away = torch.rand(n, k, generator=gen, device=dev) < drop
        return torch.where(away, -1, ids).to(torch.int32).contiguous()

    def fp8_weights(g, n, k, scale):
        w = normal(g, n // BLOCK, BLOCK, k // BLOCK, BLOCK, scale=scale, dtype=torch.float32)
        sf = w.abs().amax(dim=(2, 4)) / FP8_MAX
        return (w / sf[:, :, None, :, None]).clamp(-FP8_MAX, FP8_MAX).view(g, n, k).to(torch.float8_e4m3fn), sf

    op = case["op"]
    t = {}
    if op == "quantize":
        if case["wide"]:
            t["x"] = normal(case["groups"], case["rows"], case["k"], scale=0.02, dtype=torch.float32)
        else:
            t["x"] = hidden_states(case["groups"], case["rows"], case["k"])
        return t
    if op == "route":
        t["ids"] = experts_of(case["tokens"], case["top_k"], case["groups"], case["skew"], case["drop"])
        t["x"] = hidden_states(case["tokens"], case["hidden"])
        return t
    if op == "experts":
        n, k, g, h, i = (case[name] for name in ("tokens", "top_k", "groups", "hidden", "inner"))
        t["ids"] = experts_of(n, k, g, 0.0, case["drop"])
        t["w"] = torch.softmax(torch.randn(n, k, generator=gen, device=dev), dim=1)
        t["x"] = normal(n, h)
        for name, rows, cols in (("1", 2 * i, h), ("2", h, i)):
            if case["fp4"]:
                t["b" + name], t["sfb" + name] = _mx(normal(g, rows, cols, scale=cols ** -0.5, dtype=torch.float32))
            else:
                t["b" + name], t["sfb" + name] = fp8_weights(g, rows, cols, cols ** -0.5)
        return t
    g, r = case["groups"], case["rows"]
    if case["layout"] == "dense":
        shape = (r,)
    elif case["layout"] == "masked":
        t["rows"] = torch.randint(0, r + 1, (g,), generator=gen, device=dev, dtype=torch.int32)
        shape = (g, r)
    else:
        # counts a quarter below to a quarter above the mean; the no-padding
        # buffer holds r rows a group, so the last groups may be cut off
        low, high = r - r // 4, r + r // 4
        counts = torch.randint(low, high + 1, (g,), generator=gen, device=dev)
        t["rows"] = counts.to(torch.int32)
        shape = (g * r,)
        if case["layout"] == "contiguous":
            padded = (counts + BLOCK - 1) // BLOCK * BLOCK
            m = g * up(high, BLOCK)
            row = torch.arange(m, device=dev)
            ends = padded.cumsum(0)
            group = torch.searchsorted(ends, row, right=True).clamp(max=g - 1)
            inside = row - (ends - padded)[group]
            t["rows"] = torch.where(inside < counts[group], group, -1).to(torch.int32)
            shape = (m,)
    if op == "glu":
        t["gu"] = normal(*shape, 2 * case["inner"], scale=1.5)
        return t
    t["a"], t["sfa"] = _mx(hidden_states(*shape, case["k"], dtype=torch.float32))
    lead = () if case["layout"] == "dense" else (g,)
    t["b"], t["sfb"] = _mx(normal(*lead, case["n"], case["k"], scale=case["k"] ** -0.5, dtype=torch.float32))
    return t


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    dev = _device()
    op = case["op"]

    def operand(*shape):
        """Empty rows of codes, their scales, and room for their values."""
        *lead, m, k = shape
        s["q"] = torch.zeros(*lead, m, k // 2, dtype=torch.uint8, device=dev)
        s["sf"] = torch.zeros(*lead, k // BLOCK, up(m, 4), dtype=torch.int32, device=dev)
        s["out"] = torch.zeros(*shape, dtype=torch.bfloat16, device=dev)

    if op == "quantize":
        operand(*s["x"].shape)
    elif op == "route":
        lead = (case["groups"],) if case["layout"] == "masked" else ()
        operand(*lead, capacity(case), case["hidden"])
    elif op == "glu":
        operand(*s["gu"].shape[:-1], case["inner"])
    elif op == "gemm":
        s["out"] = torch.zeros(*s["a"].shape[:-1], case["n"], dtype=torch.bfloat16, device=dev)
    else:
        s["out"] = torch.zeros(case["tokens"], case["hidden"], dtype=torch.bfloat16, device=dev)
    if own:
        # the plan and workspace that a program keeps from call to call
        from moe_grouped_gemm_amd import dg, moe
        s["dg"], s["moe"] = dg, moe
        if op == "route":
            s["plan"] = moe.Plan(case["tokens"], case["top_k"], case["groups"], case["layout"], capacity(case),
                                 case["hidden"], dev)
        if op == "experts":
            s["workspace"] = moe.experts_workspace(case["tokens"], case["top_k"], case["groups"], case["inner"], dev)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    case, dg, moe = s["case"], s["dg"], s["moe"]
    op = case["op"]
    if op == "quantize":
        dg.quantize_fp4(s["x"], s["q"], s["sf"])
        return {"x": dg.dequantize_fp4(s["q"], s["sf"], s["out"])}
    if op == "route":
        plan = s["plan"]
        moe.dispatch_fp4(plan, s["x"], s["q"], s["sf"], topk_ids=s["ids"])
        return {"row_of": plan.row_of, "group_rows": plan.group_rows, "grouped_layout": plan.grouped_layout,
                "xp": dg.dequantize_fp4(s["q"], s["sf"], s["out"])}
    if op == "glu":
        moe.swiglu_fp4(s["gu"], s["q"], s["sf"], rows=s["rows"], layout=case["layout"])
        return {"a": dg.dequantize_fp4(s["q"], s["sf"], s["out"])}
    if op == "gemm":
        operands = (s["a"], s["sfa"], s["b"], s["sfb"], s["out"])
        if case["layout"] == "dense":
            return {"d": dg.fp4_gemm_nt(*operands)}
        gemm = {"contiguous": dg.m_grouped_fp4_gemm_nt_contiguous, "nopad": dg.m_grouped_fp4_gemm_nt_nopad,
                "masked": dg.m_grouped_fp4_gemm_nt_masked}[case["layout"]]
        return {"d": gemm(*operands, s["rows"])}
    return {"y": moe.experts(s["x"], s["ids"], s["w"], s["b1"], s["sfb1"], s["b2"], s["sfb2"], s["out"],
                             s["workspace"])}


def _values(q, sf):
    """What packed codes [..., M, K/2] and scales [..., K/128, >= M] stand for, in float32."""
    m = q.shape[-2]
    nibbles = torch.stack([q & 15, q >> 4], -1).flatten(-2)
    size = (nibbles & 7).float()
    size = torch.where(size < 4, size / 2, torch.where(size < 6, size - 2, 2 * size - 8))
    word = sf[..., :m].transpose(-1, -2)[..., None]
    code = (word >> torch.arange(0, 32, 8, device=q.device, dtype=torch.int32) & 255).flatten(-2)
    scale = torch.ldexp(torch.ones((), device=q.device), code - 127)
    v = torch.where(nibbles < 8, size, -size).unflatten(-1, (-1, MX))
    return (v * scale[..., None]).flatten(-2)


def _rounded(x):
    """The MXFP4 values nearest to x."""
    blocks = x.unflatten(-1, (-1, MX))
    exponent = _mx_exponent(blocks)
    code = _to_codes(blocks, exponent)
    size = (code & 7).float()
    size = torch.where(size < 4, size / 2, torch.where(size < 6, size - 2, 2 * size - 8))
    return torch.ldexp(torch.where(code < 8, size, -size), exponent[..., None]).flatten(-2)


def _sorted(case, ids):
    """(row of each slot or -1, rows of each group, group of each row or None)."""
    g, m = case["groups"], capacity(case)
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < g), flat, g)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(g + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    before = counts.cumsum(0) - counts
    of = key[order]
    rank = torch.arange(flat.numel(), device=ids.device) - before[of]
    kept = counts[:g]
    if case["layout"] == "masked":
        start = torch.arange(g + 1, device=ids.device) * m
        fits = rank < m
        kept = kept.clamp(max=m)
    else:
        size = (counts + BLOCK - 1) // BLOCK * BLOCK if case["layout"] == "contiguous" else counts
        start = size.cumsum(0) - size
        fits = start[of] + rank < m
        kept = torch.minimum(kept, (m - start[:g]).clamp(min=0))
    row = torch.where(fits & (of < g), start[of] + rank, -1)
    row_of = torch.empty_like(row).scatter_(0, order, row).to(torch.int32).view(ids.shape)
    layout = None
    if case["layout"] == "contiguous":
        layout = torch.full((m + 1,), -1, dtype=torch.int64, device=ids.device)
        layout = layout.scatter_(0, torch.where(row >= 0, row, m), torch.where(row >= 0, of, -1))[:m].to(torch.int32)
    return row_of, kept.to(torch.int32), layout


def _held(case, rows, m):
    """Truth of each row of the buffer: does it hold a token?"""
    if case["layout"] == "masked":
        return torch.arange(m, device=rows.device)[None] < rows[:, None]
    if case["layout"] == "contiguous":
        return rows >= 0
    return torch.arange(m, device=rows.device) < rows.clamp(min=0).sum()


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        return {"x": _rounded(s["x"].float()).to(torch.bfloat16)}
    if op == "route":
        row_of, group_rows, layout = _sorted(case, s["ids"])
        total = s["out"].numel() // case["hidden"]
        at = torch.where(row_of >= 0, row_of, total).reshape(-1).long()
        token = torch.arange(at.numel(), device=at.device) // case["top_k"]
        xp = torch.zeros(total + 1, case["hidden"], device=at.device)
        xp = xp.index_copy_(0, at, _rounded(s["x"].float())[token])[:total].to(torch.bfloat16)
        return {"row_of": row_of, "group_rows": group_rows, "grouped_layout": layout, "xp": xp.view(s["out"].shape)}
    if op == "glu":
        # in 64 bits: a value next to a border between two codes goes by its last places
        g, u = s["gu"].double().chunk(2, -1)
        a = _rounded(g / (1.0 + torch.exp(-g)) * u)
        held = _held(case, s["rows"], s["gu"].shape[-2])
        return {"a": torch.where(held[..., None], a, 0.0).to(torch.bfloat16)}
    if op == "gemm":
        a, b = _values(s["a"], s["sfa"]), _values(s["b"], s["sfb"]).transpose(-1, -2)
        if case["layout"] == "dense":
            return {"d": (a @ b).to(torch.bfloat16)}
        m, dev = a.shape[-2], a.device
        held = _held(case, s["rows"], m)
        if case["layout"] == "masked":
            return {"d": torch.where(held[..., None], a @ b, 0.0).to(torch.bfloat16)}
        # the groups' rows side by side, each group's padded to the most that one has
        row = torch.arange(m, device=dev)
        if case["layout"] == "contiguous":
            group = s["rows"].long()
            counts = torch.zeros(case["groups"] + 1, dtype=torch.int64, device=dev)
            counts = counts.scatter_add_(0, torch.where(held, group, case["groups"]), torch.ones_like(group))[:-1]
            size = (counts + BLOCK - 1) // BLOCK * BLOCK
        else:
            size = s["rows"].long()
            group = torch.searchsorted(size.cumsum(0), row, right=True).clamp(max=case["groups"] - 1)
        most = case["rows"] + case["rows"] // 4
        inside = row - (size.cumsum(0) - size)[group]
        at = torch.where(held, group * most + inside, case["groups"] * most)
        wide = torch.zeros(case["groups"] * most + 1, case["k"], device=dev).index_copy_(0, at, a)[:-1]
        d = (wide.view(case["groups"], most, -1) @ b).flatten(0, 1)
        d = d[at.clamp(max=case["groups"] * most - 1)]
        return {"d": torch.where(held[:, None], d, 0.0).to(torch.bfloat16)}
    # every token through every expert, and the routed ones summed with their weights
    if case["fp4"]:
        b1, b2 = _values(s["b1"], s["sfb1"]), _values(s["b2"], s["sfb2"])
    else:
        b1, b2 = ((b.float().unflatten(2, (-1, BLOCK)).unflatten(1, (-1, BLOCK)) * sf[:, :, None, :, None]).view(b.shape)
                  for b, sf in ((s["b1"], s["sfb1"]), (s["b2"], s["sfb2"])))
    g = case["groups"]
    away = (s["ids"] < 0) | (s["ids"] >= g)
    share = torch.zeros(case["tokens"], g + 1, device=b1.device)
    share = share.scatter_add_(1, torch.where(away, g, s["ids"]).long(), s["w"])[:, :g]
    gate, up_ = (s["x"].float() @ b1.transpose(-1, -2)).chunk(2, -1)       # [G, T, I]
    act = gate / (1.0 + torch.exp(-gate)) * up_ * share.t()[..., None]
    return {"y": (act @ b2.transpose(-1, -2)).sum(0).to(torch.bfloat16)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    dev = _device()
    levels = torch.tensor(E2M1, dtype=torch.float64, device=dev)

    def nearest(x):
        """x's blocks of 32 over the power of two at or above their largest / 6,
        each to the nearest level, ties to the even one, times the scale."""
        b = x.double().reshape(-1, MX)
        top = b.abs().max(1, keepdim=True).values
        step = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -120) / 6)))
        a = b.abs() / step
        above = torch.searchsorted(levels, a).clamp(max=7)
        below = (above - 1).clamp(min=0)
        to_above, to_below = levels[above] - a, a - levels[below]
        take = (to_above < to_below) | ((to_above == to_below) & (above % 2 == 0))
        return (torch.where(take, levels[above], levels[below]) * step * torch.sign(b)).view(x.shape)

    def decode(q, sf):
        pair = torch.cat([levels, -levels])
        v = torch.empty(*q.shape[:-1], 2 * q.shape[-1], dtype=torch.float64, device=dev)
        v[..., 0::2], v[..., 1::2] = pair[(q % 16).long()], pair[(q // 16).long()]
        word = sf[..., : q.shape[-2]].long() & 0xFFFFFFFF
        for i in range(4):
            scale = torch.exp2(((word >> 8 * i) & 255).double() - 127).transpose(-1, -2)
            part = v.view(*v.shape[:-1], -1, 4, MX)[..., i, :]
            part *= scale[..., None]
        return v

    if op == "quantize":
        return {"x": nearest(s["x"])}
    if op == "route":
        g, k, m = case["groups"], case["top_k"], capacity(case)
        counts, slots = [0] * g, []
        for e in s["ids"].reshape(-1).tolist():
            slots.append((e, counts[e]) if 0 <= e < g else None)
            if slots[-1]:
                counts[e] += 1
        start, at = [], 0
        for e, c in enumerate(counts):
            start.append(e * m if case["layout"] == "masked" else at)
            at += up(c, BLOCK) if case["layout"] == "contiguous" else c
        rows = [-1 if p is None or (case["layout"] == "masked" and p[1] >= m) else start[p[0]] + p[1] for p in slots]
        total = m * (g if case["layout"] == "masked" else 1)
        kept = [(i // k, r) for i, r in enumerate(rows) if 0 <= r < total]
        pairs = torch.tensor(kept, dtype=torch.int64, device=dev).view(-1, 2)
        xp = torch.zeros(total, case["hidden"], dtype=torch.float64, device=dev)
        xp[pairs[:, 1]] = nearest(s["x"])[pairs[:, 0]]
        lead = (g,) if case["layout"] == "masked" else ()
        return {"row_of": None, "group_rows": None, "grouped_layout": None, "xp": xp.view(*lead, m, case["hidden"])}
    if op == "experts":
        y = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device=dev)
        x = s["x"].double()
        for e in range(case["groups"]):
            t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
            if not t.numel():
                continue
            w = []
            for b, sf in ((s["b1"][e], s["sfb1"][e]), (s["b2"][e], s["sfb2"][e])):
                w.append(decode(b, sf) if case["fp4"] else
                         b.double() * sf.double().repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1))
            gu = x[t] @ w[0].t()
            g, u = gu[:, : case["inner"]], gu[:, case["inner"]:]
            y.index_add_(0, t, s["w"][t, j].double()[:, None] * ((g * torch.sigmoid(g) * u) @ w[1].t()))
        return {"y": y}
    m = (s["gu"] if op == "glu" else s["a"]).shape[-2]
    if case["layout"] == "dense":
        groups = [(slice(None), ())]
    elif case["layout"] == "masked":
        groups = [((e, slice(0, c)), e) for e, c in enumerate(s["rows"].tolist())]
    elif case["layout"] == "contiguous":
        groups = [(torch.nonzero(s["rows"] == e)[:, 0], e) for e in range(case["groups"])]
    else:
        ends = [min(m, sum(s["rows"].tolist()[: e + 1])) for e in range(case["groups"])]
        groups = [(slice(a, b), e) for e, (a, b) in enumerate(zip([0] + ends, ends))]
    if op == "glu":
        a = torch.zeros(*s["gu"].shape[:-1], case["inner"], dtype=torch.float64, device=dev)
        for rows, _ in groups:
            gu = s["gu"][rows].double()
            g, u = gu[..., : case["inner"]], gu[..., case["inner"]:]
            a[rows] = nearest(g * torch.sigmoid(g) * u)
        return {"a": a}
    d = torch.zeros(*s["a"].shape[:-1], case["n"], dtype=torch.float64, device=dev)
    a = decode(s["a"], s["sfa"])
    for rows, e in groups:
        d[rows] = a[rows] @ decode(s["b"][e], s["sfb"][e]).t()
    return {"d": d}
