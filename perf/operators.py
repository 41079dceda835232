"""Cases that measure the operators around the grouped FP8 products: tokens
sorted into the products' row layouts and back (`route`, `combine`, `grad`),
the norms before and after the block with its gate and residual scale
(`norm`, `norm_grad`) and the gated activation between the two products
(`glu`, `glu_grad`).

`run` computes a case either in elementary torch operations in 32 bits
(`own` false) or through the package's entry points (`own` true).
"""

import math

import torch

own = False

LAYOUTS = ("contiguous", "nopad", "masked")
GATES = ("none", "channel", "token", "full")
BLOCK = 128
FP8_MAX = 448.0
AMAX_FLOOR = 1e-4
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # A decode step of a few requests: five tokens into the masked layout of
        # sixteen local experts with 256 receive rows each. Latency is all.
        {"name": "route_decode", "op": "route", "layout": "masked", "fp8": True, "ue8m0": False, "tokens": 5,
         "top_k": 8, "groups": 16, "max_m": 256, "hidden": 7168, "skew": 0.0, "drop": 0.0},
        # A long prompt (or a batch of them): 65536 rows over 32 experts by a
        # Zipf law, FP8 with power-of-two scales into 128-row segments.
        {"name": "route_prefill", "op": "route", "layout": "contiguous", "fp8": True, "ue8m0": True, "tokens": 8192,
         "top_k": 8, "groups": 32, "max_m": 0, "hidden": 7168, "skew": 1.2, "drop": 0.0},
        # A training micro-batch under expert parallelism: BF16 rows for eight
        # local experts, one slot in ten routed to an expert elsewhere.
        {"name": "route_train", "op": "route", "layout": "nopad", "fp8": False, "ue8m0": False, "tokens": 7354,
         "top_k": 4, "groups": 8, "max_m": 0, "hidden": 7168, "skew": 0.0, "drop": 0.1},
        # The way back in a decode step with a full batch, an odd token count.
        {"name": "combine_decode", "op": "combine", "layout": "masked", "weighted": True, "tokens": 259, "top_k": 8,
         "groups": 16, "max_m": 256, "hidden": 7168, "skew": 0.0, "drop": 0.0},
        # The way back of the long prompt.
        {"name": "combine_prefill", "op": "combine", "layout": "contiguous", "weighted": True, "tokens": 8192,
         "top_k": 8, "groups": 32, "max_m": 0, "hidden": 7168, "skew": 1.2, "drop": 0.0},
        # Both gradients of the training micro-batch: of the weighted way back
        # (rows and weights) and of the way in (tokens).
        {"name": "route_grad", "op": "grad", "layout": "nopad", "tokens": 7354, "top_k": 4, "groups": 8, "max_m": 0,
         "hidden": 7168, "skew": 0.0, "drop": 0.1},
        # The residual step between two blocks for a few decoded tokens.
        {"name": "norm_decode", "op": "norm", "tokens": 7, "hidden": 7168, "gate": "channel", "residual_scale": 1.0},
        # The same for a long prompt, with a scaled residual stream.
        {"name": "norm_prefill", "op": "norm", "tokens": 8192, "hidden": 7168, "gate": "channel",
         "residual_scale": 0.5},
        # Its gradient in training, an odd number of tokens.
        {"name": "norm_grad", "op": "norm_grad", "tokens": 4099, "hidden": 7168, "gate": "channel",
         "residual_scale": 0.5},
        # The activation of a decode step: masked receive rows, half of them empty.
        {"name": "glu_decode", "op": "glu", "layout": "masked", "groups": 16, "rows": 256,
         "inner": 2048},
        # The activation of a prompt: eight experts of 3000 to 5000 rows, 128-row segments.
        {"name": "glu_prefill", "op": "glu", "layout": "contiguous", "groups": 8, "rows": 4000,
         "inner": 2048},
        # Its gradient for the no-padding layout of a training step.
        {"name": "glu_grad", "op": "glu_grad", "layout": "nopad", "groups": 8, "rows": 3677, "inner": 2048},
    ]


def draw(rng):
    def log_size(low, high, step=1):
        while True:
            v = int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)) * step
            v = min(max(v, low), high)
            if v != 3072 and 2 * v != 3072:
                return v

    op = rng.choice(("route", "route", "combine", "grad", "norm", "norm_grad", "glu", "glu_grad"))
    if op in ("norm", "norm_grad"):
        return {"op": op, "tokens": log_size(1, 8192 if op == "norm" else 4099), "hidden": log_size(256, 7168, 128),
                "gate": rng.choice(GATES), "residual_scale": rng.choice((1.0, 0.5, 0.22))}
    layout = rng.choice(LAYOUTS)
    if op in ("glu", "glu_grad"):
        groups = log_size(1, 32)
        most = max(2, 29000 // groups)
        return {"op": op, "layout": layout, "groups": groups, "rows": log_size(1, most),
                "inner": log_size(128, 2048, 128)}
    top_k = rng.randint(1, 8)
    groups = log_size(max(2, top_k), 256)
    hidden = log_size(256, 7168, 128)
    most = 8192 if op in ("route", "combine") else 7354 * 4 // max(top_k, 4)
    tokens = log_size(1, most)
    # masked receive rows: the mean load with room above it, so a few rows may overflow under a skewed draw
    max_m = min(max(8, -(-2 * tokens * top_k // groups)), 65536 // groups) if layout == "masked" else 0
    c = {"op": op, "layout": layout, "tokens": tokens, "top_k": top_k, "groups": groups, "max_m": max_m,
         "hidden": hidden, "skew": rng.choice((0.0, 0.6, 1.2)), "drop": rng.choice((0.0, 0.1, 0.5))}
    if op == "route":
        c["fp8"] = rng.random() < 0.6
        c["ue8m0"] = c["fp8"] and rng.random() < 0.5
    if op == "combine":
        c["weighted"] = rng.random() < 0.7
    return c


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        values = case["tokens"] * case["hidden"]
        gate = {"none": 0, "channel": 4 * case["hidden"], "token": 4 * case["tokens"], "full": 2 * values}[case["gate"]]
        if op == "norm":
            return {"bytes": 2 * 4 * values + gate + 8 * case["hidden"] + 8 * case["tokens"], "flops": 12.0 * values}
        return {"bytes": 2 * 6 * values + 2 * gate + 16 * case["hidden"] + 8 * case["tokens"], "flops": 24.0 * values}
    if op in ("glu", "glu_grad"):
        # masked counts are uniform in [0, rows]: half of the rows on average
        m = case["groups"] * case["rows"] * (0.5 if case["layout"] == "masked" else 1.0)
        values = m * case["inner"]
        if op == "glu":
            return {"bytes": values * (4 + 1 + 4 / BLOCK), "flops": 8.0 * values}
        return {"bytes": 2 * 5 * values, "flops": 14.0 * values}
    slots = case["tokens"] * case["top_k"]
    rows = slots * (1.0 - case["drop"])
    token_values, row_values = case["tokens"] * case["hidden"], rows * case["hidden"]
    if op == "route":
        layout = 4 * capacity(case) if case["layout"] == "contiguous" else 0
        per = (1 + 4 / BLOCK) if case["fp8"] else 2
        return {"bytes": 2 * token_values + per * row_values + 8 * slots + 4 * case["groups"] + layout,
                "flops": (4.0 if case["fp8"] else 0.0) * token_values}
    if op == "combine":
        return {"bytes": 2 * row_values + 2 * token_values + 8 * slots, "flops": 2.0 * row_values}
    # dy and yp read, dyp and dw written; dxp read, dx written
    return {"bytes": 6 * row_values + 4 * token_values + 12 * slots, "flops": 4.0 * row_values}


def capacity(case):
    """Rows of the permuted buffers: what a program that knows only the token
    count has to set aside."""
    if case["layout"] == "masked":
        return case["groups"] * case["max_m"]
    slots = case["tokens"] * case["top_k"]
    if case["layout"] == "nopad":
        return slots
    return (slots + min(case["groups"], slots) * (BLOCK - 1) + BLOCK - 1) // BLOCK * BLOCK


def rows_shape(case):
    """Leading dimensions of the permuted buffers."""
    return (case["groups"], case["max_m"]) if case["layout"] == "masked" else (capacity(case),)


def aligned4(m):
    return (m + 3) // 4 * 4


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _device():
    return torch.device("cuda:0" if torch.cuda.is_available() else "cpu")


def _inputs(case, seed):
    """Everything that comes from the seed, as tensors by name."""
    dev = _device()
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32) * scale).to(dtype)

    op = case["op"]
    t = {}
    if op in ("norm", "norm_grad"):
        n, h = case["tokens"], case["hidden"]
        t["y"] = normal(n, h, scale=3.0)
        t["w_post"] = 1.0 + normal(h, scale=0.2, dtype=torch.float32)
        t["w_pre"] = 1.0 + normal(h, scale=0.2, dtype=torch.float32)
        t["gate"] = {"none": lambda: None,
                     "channel": lambda: normal(h, scale=0.5, dtype=torch.float32),
                     "token": lambda: torch.rand(n, 1, generator=gen, device=dev),
                     "full": lambda: normal(n, h, scale=0.5)}[case["gate"]]()
        if op == "norm":
            t["x"] = normal(n, h, scale=2.0)
        else:
            t["h"] = normal(n, h, scale=2.0)
            t["dh"] = normal(n, h, scale=0.1)
            t["dn"] = normal(n, h, scale=0.1)
            t["rstd_post"] = torch.rsqrt(t["y"].float().square().mean(1) + EPS)
            t["rstd_pre"] = torch.rsqrt(t["h"].float().square().mean(1) + EPS)
        return t
    if op in ("glu", "glu_grad"):
        g, r = case["groups"], case["rows"]
        if case["layout"] == "masked":
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
                m = g * ((high + BLOCK - 1) // BLOCK * BLOCK)
                row = torch.arange(m, device=dev)
                ends = padded.cumsum(0)
                group = torch.searchsorted(ends, row, right=True).clamp(max=g - 1)
                inside = row - (ends - padded)[group]
                t["rows"] = torch.where(inside < counts[group], group, -1).to(torch.int32)
                shape = (m,)
        t["gu"] = normal(*shape, 2 * case["inner"], scale=1.5)
        if op == "glu_grad":
            t["da"] = normal(*shape, case["inner"], scale=0.1)
        return t
    # Experts by a Zipf law of exponent `skew` over a shuffled order, the k of a
    # token distinct (the largest of its perturbed log weights).
    n, k, g = case["tokens"], case["top_k"], case["groups"]
    logits = -case["skew"] * torch.log(torch.arange(1, g + 1, device=dev, dtype=torch.float32))
    logits = logits[torch.randperm(g, generator=gen, device=dev)]
    noise = -torch.log(-torch.log(torch.rand(n, g, generator=gen, device=dev).clamp(1e-6, 1 - 1e-6)))
    ids = torch.topk(logits + noise, k, dim=1).indices.to(torch.int32)
    if case["drop"] > 0:
        ids = torch.where(torch.rand(n, k, generator=gen, device=dev) < case["drop"], -1, ids).to(torch.int32)
    t["ids"] = ids.contiguous()
    if op == "route":
        # a few channels far above the rest, as hidden states have them
        t["x"] = normal(n, case["hidden"])
        t["x"][:, :: case["hidden"] // 4] *= 20.0
        return t
    t["row_of"] = _sorted(case, t["ids"])[0]
    shape = rows_shape(case)
    t["w"] = torch.softmax(torch.randn(n, k, generator=gen, device=dev), dim=1)
    if op == "combine":
        t["w"] = t["w"] if case["weighted"] else None
        t["yp"] = normal(*shape, case["hidden"])
    else:
        t["yp"] = normal(*shape, case["hidden"])
        t["dxp"] = normal(*shape, case["hidden"], scale=0.1)
        t["dy"] = normal(n, case["hidden"], scale=0.1)
    return t


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    dev = _device()
    if case["op"] in ("norm", "norm_grad"):
        n, h = case["tokens"], case["hidden"]
        names = ("h", "n") if case["op"] == "norm" else ("dx", "dy")
        for name in names:
            s["out_" + name] = torch.zeros(n, h, dtype=torch.bfloat16, device=dev)
        if case["op"] == "norm":
            s["out_rstd"] = torch.zeros(2, n, dtype=torch.float32, device=dev)
        else:
            s["out_dw"] = torch.zeros(2, h, dtype=torch.float32, device=dev)
            s["out_dgate"] = None if s["gate"] is None else torch.zeros_like(s["gate"])
    elif case["op"] == "glu":
        lead, m = s["gu"].shape[:-2], s["gu"].shape[-2]
        s["q"] = torch.zeros(*s["gu"].shape[:-1], case["inner"], dtype=torch.float8_e4m3fn, device=dev)
        s["sfa"] = torch.zeros(*lead, case["inner"] // BLOCK, aligned4(m), dtype=torch.float32, device=dev)
    elif case["op"] == "glu_grad":
        s["dgu"] = torch.zeros_like(s["gu"])
    elif case["op"] == "route":
        *lead, m = rows_shape(case)
        h = case["hidden"]
        if case["fp8"]:
            s["q"] = torch.zeros(*lead, m, h, dtype=torch.float8_e4m3fn, device=dev)
            s["sfa"] = torch.zeros(*lead, h // BLOCK, aligned4(m), dtype=torch.float32, device=dev)
        else:
            s["xp"] = torch.zeros(*lead, m, h, dtype=torch.bfloat16, device=dev)
    else:
        s["out"] = torch.zeros(case["tokens"], case["hidden"], dtype=torch.bfloat16, device=dev)
        if case["op"] == "grad":
            s["dyp"] = torch.zeros_like(s["yp"])
            s["dw"] = torch.zeros(case["tokens"], case["top_k"], dtype=torch.float32, device=dev)
    if own:
        # the plan and workspaces that a program keeps from call to call
        from moe_grouped_gemm_amd import moe
        s["moe"] = moe
        if "ids" in s:
            rows = case["max_m"] if case["layout"] == "masked" else capacity(case)
            s["plan"] = moe.Plan(case["tokens"], case["top_k"], case["groups"], case["layout"], rows, case["hidden"],
                                 dev)
            if "row_of" in s:
                s["plan"].row_of.copy_(s["row_of"])
        if case["op"] == "norm_grad":
            s["workspace"] = moe.block_norm_workspace(case["tokens"], case["hidden"], dev)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    case, moe = s["case"], s["moe"]
    op = case["op"]
    if op == "route":
        plan = s["plan"]
        if case["fp8"]:
            moe.dispatch_fp8(plan, s["x"], s["q"], s["sfa"], topk_ids=s["ids"], ue8m0=case["ue8m0"])
            moved = {"q": s["q"], "sfa": s["sfa"]}
        else:
            moe.dispatch(plan, s["x"], s["xp"], topk_ids=s["ids"])
            moved = {"xp": s["xp"]}
        return {"row_of": plan.row_of, "group_rows": plan.group_rows, "grouped_layout": plan.grouped_layout, **moved}
    if op == "combine":
        return {"y": moe.combine(s["plan"], s["yp"], s["out"], weights=s["w"])}
    if op == "grad":
        moe.combine_bwd(s["plan"], s["dy"], s["yp"], s["w"], s["dyp"], s["dw"])
        moe.combine(s["plan"], s["dxp"], s["out"])
        return {"dyp": s["dyp"], "dw": s["dw"], "dx": s["out"]}
    if op == "norm":
        moe.block_norm(s["x"], s["y"], s["w_post"], s["gate"], s["w_pre"], s["out_h"], s["out_n"],
                       s["out_rstd"][0], s["out_rstd"][1], residual_scale=case["residual_scale"], eps=EPS)
        return {"h": s["out_h"], "n": s["out_n"], "rstd": s["out_rstd"]}
    if op == "norm_grad":
        moe.block_norm_bwd(s["dh"], s["dn"], s["h"], s["y"], s["w_post"], s["gate"], s["w_pre"], s["rstd_post"],
                           s["rstd_pre"], s["out_dx"], s["out_dy"], s["out_dw"][0], s["out_dgate"], s["out_dw"][1],
                           s["workspace"], residual_scale=case["residual_scale"])
        return {"dx": s["out_dx"], "dy": s["out_dy"], "dw": s["out_dw"], "dgate": s["out_dgate"]}
    if op == "glu":
        moe.swiglu_fp8(s["gu"], s["q"], s["sfa"], rows=s["rows"], layout=case["layout"])
        return {"q": s["q"], "sfa": s["sfa"]}
    moe.swiglu_bwd(s["da"], s["gu"], s["dgu"], rows=s["rows"], layout=case["layout"])
    return {"dgu": s["dgu"]}


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
        start = torch.arange(g + 1, device=ids.device) * case["max_m"]
        fits = rank < case["max_m"]
        kept = kept.clamp(max=case["max_m"])
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


def _fp8_scale(a, ue8m0):
    """Scales of 128-wide blocks of a [..., blocks, 128] float32."""
    scale = a.abs().amax(-1).clamp(min=AMAX_FLOOR) / FP8_MAX
    if ue8m0:
        mantissa, exponent = torch.frexp(scale)
        scale = torch.ldexp(torch.ones_like(scale), torch.where(mantissa == 0.5, exponent - 1, exponent))
    return scale


def _rms_norm(v, w):
    rstd = torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)
    return v * rstd * w, rstd


def _row_mask(case, rows, m):
    """Truth of each row of the buffer: does it hold a token?"""
    if case["layout"] == "masked":
        return torch.arange(m, device=rows.device)[None] < rows[:, None]
    if case["layout"] == "contiguous":
        return rows >= 0
    return torch.arange(m, device=rows.device) < rows.clamp(min=0).sum()


def _rows_by_slot(v, row_of):
    """v's row of each slot in float32, [T, k, H]; zero where there is none."""
    safe = row_of.long().clamp(min=0)
    return v.view(-1, v.shape[-1])[safe].float() * (row_of >= 0)[..., None]


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "route":
        row_of, group_rows, layout = _sorted(case, s["ids"])
        x, m = s["x"].float(), capacity(case)
        at = torch.where(row_of >= 0, row_of, m).reshape(-1).long()
        token = torch.arange(at.numel(), device=at.device) // case["top_k"]
        out = {"row_of": row_of, "group_rows": group_rows, "grouped_layout": layout}
        if not case["fp8"]:
            xp = torch.zeros(m + 1, case["hidden"], device=x.device)
            out["xp"] = xp.index_copy_(0, at, x[token])[:m].to(torch.bfloat16).view(s["xp"].shape)
            return out
        blocks = x.view(case["tokens"], -1, BLOCK)
        scale = _fp8_scale(blocks, case["ue8m0"])
        codes = (blocks / scale[..., None]).clamp(-FP8_MAX, FP8_MAX).view_as(x)
        q = torch.zeros(m + 1, case["hidden"], device=x.device).index_copy_(0, at, codes[token])[:m]
        rows = torch.zeros(m + 1, scale.shape[1], device=x.device).index_copy_(0, at, scale[token])[:m]
        like_q, like_sfa = s["q"], s["sfa"]
        per = like_q.shape[-2]
        sfa = torch.zeros_like(like_sfa)
        sfa[..., :per] = rows.view(*like_q.shape[:-1], -1).transpose(-1, -2)
        out["q"], out["sfa"] = q.view(like_q.shape).to(torch.float8_e4m3fn), sfa
        return out
    if op == "combine":
        v = _rows_by_slot(s["yp"], s["row_of"])
        return {"y": (v if s["w"] is None else v * s["w"][..., None]).sum(1).to(torch.bfloat16)}
    if op == "grad":
        m, row_of, dy = capacity(case), s["row_of"], s["dy"].float()
        dw = (_rows_by_slot(s["yp"], row_of) * dy[:, None]).sum(-1)
        at = torch.where(row_of >= 0, row_of, m).reshape(-1).long()
        dyp = torch.zeros(m + 1, case["hidden"], device=dy.device)
        dyp = dyp.index_copy_(0, at, (s["w"][..., None] * dy[:, None]).flatten(0, 1))[:m].to(torch.bfloat16)
        return {"dyp": dyp.view(s["dyp"].shape), "dw": dw, "dx": _rows_by_slot(s["dxp"], row_of).sum(1).to(torch.bfloat16)}
    if op in ("norm", "norm_grad"):
        gate = s["gate"]
        wide = 1.0 if gate is None else gate.float()
        rs = case["residual_scale"]
        if op == "norm":
            post, rstd_post = _rms_norm(s["y"].float(), s["w_post"])
            h = rs * s["x"].float() + wide * post
            n, rstd_pre = _rms_norm(h, s["w_pre"])
            return {"h": h.to(torch.bfloat16), "n": n.to(torch.bfloat16),
                    "rstd": torch.stack([rstd_post[:, 0], rstd_pre[:, 0]])}
        dn, hn = s["dn"].float(), s["h"].float() * s["rstd_pre"][:, None]
        a = dn * s["w_pre"]
        dres = s["dh"].float() + s["rstd_pre"][:, None] * (a - hn * (a * hn).mean(1, keepdim=True))
        yn = s["y"].float() * s["rstd_post"][:, None]
        dgate = dres * yn * s["w_post"]
        dpost = dres * wide
        b = dpost * s["w_post"]
        dy = s["rstd_post"][:, None] * (b - yn * (b * yn).mean(1, keepdim=True))
        dgate = {"none": lambda: None, "channel": lambda: dgate.sum(0), "token": lambda: dgate.sum(1, keepdim=True),
                 "full": lambda: dgate.to(torch.bfloat16)}[case["gate"]]()
        return {"dx": (rs * dres).to(torch.bfloat16), "dy": dy.to(torch.bfloat16),
                "dw": torch.stack([(dpost * yn).sum(0), (dn * hn).sum(0)]), "dgate": dgate}
    inner = case["inner"]
    g, u = s["gu"][..., :inner].float(), s["gu"][..., inner:].float()
    held = _row_mask(case, s["rows"], s["gu"].shape[-2])
    sig = 1.0 / (1.0 + torch.exp(-g))
    if op == "glu_grad":
        da = s["da"].float()
        dgu = torch.cat([da * u * sig * (1.0 + g * (1.0 - sig)), da * g * sig], -1)
        return {"dgu": torch.where(held[..., None], dgu, 0.0).to(torch.bfloat16)}
    blocks = (g * sig * u).unflatten(-1, (-1, BLOCK))
    scale = _fp8_scale(blocks, False)
    codes = (blocks / scale[..., None]).clamp(-FP8_MAX, FP8_MAX).flatten(-2)
    sfa = torch.zeros_like(s["sfa"])
    sfa[..., : codes.shape[-2]] = torch.where(held[..., None], scale, 0.0).transpose(-1, -2)
    return {"q": torch.where(held[..., None], codes, 0.0).to(torch.float8_e4m3fn), "sfa": sfa}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    def walk(ids):
        """Row of each slot, by going through the slots in order (host)."""
        counts = [0] * case["groups"]
        ranks = []
        for e in ids.reshape(-1).tolist():
            ok = 0 <= e < case["groups"]
            ranks.append((e, counts[e]) if ok else None)
            if ok:
                counts[e] += 1
        start, at = [], 0
        for g, c in enumerate(counts):
            start.append(g * case["max_m"] if case["layout"] == "masked" else at)
            at += -(-c // BLOCK) * BLOCK if case["layout"] == "contiguous" else c
        rows = []
        for r in ranks:
            if r is None or (case["layout"] == "masked" and r[1] >= case["max_m"]):
                rows.append(-1)
            else:
                row = start[r[0]] + r[1]
                rows.append(row if row < capacity(case) else -1)
        return rows

    s = _inputs(case, seed)
    op = case["op"]
    dev = _device()
    f64 = {"dtype": torch.float64, "device": dev}
    if op in ("route", "combine", "grad"):
        k, h, m = case["top_k"], case["hidden"], capacity(case)
        walked = walk(s["ids"])
        slots = [torch.tensor([(i // k, r) for i, r in enumerate(walked) if i % k == j and r >= 0],
                              dtype=torch.int64, device=dev).view(-1, 2).unbind(1) for j in range(k)]
    if op == "route":
        x = s["x"].double()
        none = {"row_of": None, "group_rows": None, "grouped_layout": None}
        if not case["fp8"]:
            xp = torch.zeros(m, h, **f64)
            for t, r in slots:
                xp[r] = x[t]
            return {**none, "xp": xp.view(*rows_shape(case), h)}
        # the value each code stands for before rounding: x over its block's scale
        step = torch.maximum(x.view(-1, h // BLOCK, BLOCK).abs().max(2).values,
                             torch.tensor(AMAX_FLOOR, **f64)) / FP8_MAX
        if case["ue8m0"]:
            step = torch.exp2(torch.ceil(torch.log2(step)))
        over = x / step.repeat_interleave(BLOCK, 1)
        q, rows = torch.zeros(m, h, **f64), torch.zeros(m, h // BLOCK, **f64)
        for t, r in slots:
            q[r], rows[r] = over[t], step[t]
        if case["layout"] == "masked":
            q, rows = q.view(case["groups"], -1, h), rows.view(case["groups"], -1, h // BLOCK)
        per = rows.shape[-2]
        sfa = torch.zeros(*rows.shape[:-2], h // BLOCK, aligned4(per), **f64)
        sfa[..., :per] = rows.transpose(-1, -2)
        return {**none, "q": q, "sfa": sfa}
    if op == "combine":
        y = torch.zeros(case["tokens"], h, **f64)
        for j, (t, r) in enumerate(slots):
            w = 1.0 if s["w"] is None else s["w"][t, j].double()[:, None]
            y[t] += w * s["yp"].view(m, h)[r].double()
        return {"y": y}
    if op == "grad":
        dy = s["dy"].double()
        dyp, dw = torch.zeros(m, h, **f64), torch.zeros(case["tokens"], k, **f64)
        dx = torch.zeros(case["tokens"], h, **f64)
        for j, (t, r) in enumerate(slots):
            dyp[r] = s["w"][t, j].double()[:, None] * dy[t]
            dw[t, j] = (dy[t] * s["yp"].view(m, h)[r].double()).sum(1)
            dx[t] += s["dxp"].view(m, h)[r].double()
        return {"dyp": dyp.view(s["yp"].shape), "dw": dw, "dx": dx}
    if op in ("norm", "norm_grad"):
        d = {name: v.double() for name, v in s.items() if v is not None}
        rs, hidden = case["residual_scale"], case["hidden"]
        gate = torch.ones(1, 1, **f64) if s["gate"] is None else d["gate"].view(
            {"channel": (1, -1), "token": (-1, 1), "full": (-1, hidden)}[case["gate"]])
        if op == "norm":
            r1 = ((d["y"] ** 2).sum(1) / hidden + EPS) ** -0.5
            h = rs * d["x"] + gate * (d["w_post"] * (d["y"] * r1[:, None]))
            r2 = ((h ** 2).sum(1) / hidden + EPS) ** -0.5
            return {"h": h, "n": d["w_pre"] * (h * r2[:, None]), "rstd": torch.stack([r1, r2])}
        r1, r2 = d["rstd_post"][:, None], d["rstd_pre"][:, None]
        inner = (d["dn"] * d["w_pre"] * d["h"]).sum(1, keepdim=True)
        total = d["dh"] + r2 * d["dn"] * d["w_pre"] - r2 ** 3 * d["h"] * inner / hidden
        up = total * gate * d["w_post"]
        inner = (up * d["y"]).sum(1, keepdim=True)
        dg = total * d["y"] * r1 * d["w_post"]
        return {"dx": rs * total, "dy": r1 * up - r1 ** 3 * d["y"] * inner / hidden,
                "dw": torch.stack([(total * gate * d["y"] * r1).sum(0), (d["dn"] * d["h"] * r2).sum(0)]),
                "dgate": None if s["gate"] is None else dg if case["gate"] == "full"
                else dg.sum(0) if case["gate"] == "channel" else dg.sum(1, keepdim=True)}
    inner = case["inner"]
    gate, up = s["gu"].double().split(inner, -1)
    m = s["gu"].shape[-2]
    if case["layout"] == "masked":
        held = torch.stack([torch.arange(m, device=dev) < c for c in s["rows"].tolist()])
    elif case["layout"] == "contiguous":
        held = s["rows"] != -1
    else:
        held = torch.arange(m, device=dev) < sum(s["rows"].tolist())
    if op == "glu_grad":
        da, sg = s["da"].double(), torch.sigmoid(gate)
        dgu = torch.cat([da * up * (sg + gate * sg * (1.0 - sg)), da * gate * sg], -1)
        return {"dgu": dgu * held[..., None]}
    act = gate * torch.sigmoid(gate) * up
    top = torch.maximum(act.unflatten(-1, (-1, BLOCK)).abs().max(-1).values, torch.tensor(AMAX_FLOOR, **f64))
    step = top / FP8_MAX
    q = act / step.repeat_interleave(BLOCK, -1) * held[..., None]
    sfa = torch.zeros(*s["gu"].shape[:-2], inner // BLOCK, aligned4(m), **f64)
    sfa[..., :m] = (step * held[..., None]).transpose(-1, -2)
    return {"q": q, "sfa": sfa}
