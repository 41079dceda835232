"""A mixture-of-experts block in FP8 from end to end on one GPU, forward in the
three row layouts and backward, with the package's own calls:

    h, n      = the previous block's output into the residual stream, normalised
    rows      = n sorted by expert and quantised                (moe.dispatch_fp8)
    gate | up = rows times the experts' first weights           (grouped FP8 GEMM)
    act       = silu(gate) * up, quantised                      (moe.swiglu_fp8)
    out rows  = act times the experts' second weights           (grouped FP8 GEMM)
    y         = a token's rows, summed with the router's weights   (moe.combine)
    h', n'    = y into the residual stream, normalised for what follows (moe.block_norm)

Run: python examples/moe_block.py [tokens] -- prints how far the block is from
the same mathematics in float32, and the time of a pass.
"""

from __future__ import annotations

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_grouped_gemm_amd import dg, moe, synth  # noqa: E402


class Block:
    """Weights, plan and buffers of one block: what a program keeps."""

    def __init__(self, tokens: int, top_k: int, groups: int, hidden: int, inner: int, layout: str, seed: int = 0,
                 device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.layout, self.top_k, self.groups, self.inner = layout, top_k, groups, inner
        rows = {"masked": tokens, "nopad": tokens * top_k,
                "contiguous": moe.contiguous_rows(tokens * top_k, groups)}[layout]
        self.plan = moe.Plan(tokens, top_k, groups, layout, rows, hidden, device)

        def weights(n, k):
            return torch.randn(groups, n, k, generator=gen, device=device) * k ** -0.5

        self.w1, self.w2 = weights(2 * inner, hidden), weights(hidden, inner)      # float32, for comparison
        self.b1, self.sfb1 = quantize_experts(self.w1)
        self.b2, self.sfb2 = quantize_experts(self.w2)
        self.post = 1 + 0.1 * torch.randn(hidden, generator=gen, device=device)
        self.pre = 1 + 0.1 * torch.randn(hidden, generator=gen, device=device)
        self.gate = 0.5 + 0.1 * torch.randn(hidden, generator=gen, device=device)
        lead = self.plan.rows_shape[:-1]
        self.q = torch.empty(self.plan.rows_shape, dtype=torch.float8_e4m3fn, device=device)
        self.sfa = torch.empty(self.plan.scale_shape, device=device)
        self.gu = torch.empty(*lead, 2 * inner, dtype=torch.bfloat16, device=device)
        self.aq = torch.empty(*lead, inner, dtype=torch.float8_e4m3fn, device=device)
        self.asf = torch.empty(*lead[:-1], inner // 128, self.plan.scale_shape[-1], device=device)
        self.yp = torch.empty(self.plan.rows_shape, dtype=torch.bfloat16, device=device)
        self.y, self.h, self.n = (torch.empty(tokens, hidden, dtype=torch.bfloat16, device=device) for _ in range(3))
        self.rstd_post, self.rstd_pre = torch.empty(tokens, device=device), torch.empty(tokens, device=device)

    def gemm(self, a, sfa, b, sfb, d):
        if self.layout == "masked":
            return dg.m_grouped_fp8_gemm_nt_masked(a, sfa, b, sfb, d, self.plan.group_rows)
        if self.layout == "nopad":
            return dg.m_grouped_fp8_gemm_nt_nopad(a, sfa, b, sfb, d, self.plan.group_rows)
        return dg.m_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, d, self.plan.grouped_layout)

    @property
    def held(self):
        """What says which rows hold tokens, as the GEMM of the layout takes it."""
        return self.plan.grouped_layout if self.layout == "contiguous" else self.plan.group_rows

    def forward(self, x, n, ids, weights):
        """x: the residual stream, n: its norm, both [tokens, hidden] bfloat16;
        ids, weights [tokens, top_k]: the router's choice. Returns (h', n')."""
        moe.dispatch_fp8(self.plan, n, self.q, self.sfa, topk_ids=ids)
        self.gemm(self.q, self.sfa, self.b1, self.sfb1, self.gu)
        moe.swiglu_fp8(self.gu, self.aq, self.asf, rows=self.held, layout=self.layout)
        self.gemm(self.aq, self.asf, self.b2, self.sfb2, self.yp)
        moe.combine(self.plan, self.yp, self.y, weights=weights)
        return moe.block_norm(x, self.y, self.post, self.gate, self.pre, self.h, self.n, self.rstd_post, self.rstd_pre)

    def backward(self, dh, dn, weights):
        """Gradients of a forward() in the no-padding layout, from those of h' and
        n': dict of x, n (through the experts), the router's weights, the
        norms' weights and the gate. The data gradients run through the FP8
        GEMM with the weights transposed and the gradients quantised by row."""
        plan, dev = self.plan, dh.device
        tokens, hidden = dh.shape
        g = {name: torch.empty(hidden, device=dev) for name in ("post", "gate", "pre")}
        dx, dy = torch.empty_like(dh), torch.empty_like(dh)
        moe.block_norm_bwd(dh, dn, self.h, self.y, self.post, self.gate, self.pre, self.rstd_post, self.rstd_pre,
                           dx, dy, g["post"], g["gate"], g["pre"],
                           moe.block_norm_workspace(tokens, hidden, dev))
        dyp, dw = torch.empty_like(self.yp), torch.empty_like(weights)
        moe.combine_bwd(plan, dy, self.yp, weights, dyp, dw)
        da = self._data_gradient(dyp, self.w2)
        dgu = torch.empty_like(self.gu)
        moe.swiglu_bwd(da, self.gu, dgu, rows=self.held, layout=self.layout)
        dxp = self._data_gradient(dgu, self.w1)
        d_n = torch.empty_like(dh)
        moe.combine(plan, dxp, d_n)
        return {"x": dx, "n": d_n, "weights": dw, **g}

    def _data_gradient(self, dout, w):
        """dout [rows, N] bfloat16 times the experts' weights [G, N, K]: [rows, K]."""
        rows, n = dout.shape
        # every row to itself, quantised: a dispatch of one slot a row into one group
        each = moe.Plan(rows, 1, 1, "nopad", rows, n, dout.device)
        q = torch.empty(rows, n, dtype=torch.float8_e4m3fn, device=dout.device)
        sf = torch.empty(each.scale_shape, device=dout.device)
        moe.dispatch_fp8(each, dout, q, sf, topk_ids=torch.zeros(rows, 1, dtype=torch.int32, device=dout.device))
        b, sfb = quantize_experts(w.transpose(1, 2).contiguous())
        out = torch.empty(rows, w.shape[2], dtype=torch.bfloat16, device=dout.device)
        return dg.m_grouped_fp8_gemm_nt_nopad(q, sf, b, sfb, out, self.plan.group_rows)


def quantize_experts(w):
    """[G, N, K] float32 to the grouped GEMMs' RHS operand."""
    parts = [synth.quantize_rhs(e) for e in w]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def plain_block(b: Block, x, n, ids, weights):
    """The block in float32 torch; every expert sees every token."""
    y = torch.zeros_like(n)
    for e in range(b.groups):
        gate, up = (n @ b.w1[e].T).chunk(2, dim=1)
        share = (weights * (ids == e)).sum(1, keepdim=True)
        y = y + share * ((torch.nn.functional.silu(gate) * up) @ b.w2[e].T)

    def norm(v, w):
        return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6) * w

    h = x + b.gate * norm(y, b.post)
    return h, norm(h, b.pre)


def inputs(tokens, top_k, groups, hidden, seed=1, device="cuda"):
    gen = torch.Generator(device=device).manual_seed(seed)
    x = torch.randn(tokens, hidden, generator=gen, device=device).bfloat16()
    n = torch.empty_like(x)
    moe.block_norm(x, None, None, None, torch.ones(hidden, device=device), None, n)
    logits = torch.randn(tokens, groups, generator=gen, device=device)
    weights, ids = torch.topk(logits.softmax(1), top_k, dim=1)
    return x, n, ids.int().contiguous(), (weights / weights.sum(1, keepdim=True)).contiguous()


def relative(got, want):
    return ((got.float() - want).norm() / want.norm()).item()


def compare(tokens=96, top_k=4, groups=8, hidden=512, inner=256):
    """{name: relative error against float32} of the block in each layout and of
    its gradients. The errors are those of FP8 operands, 2-3% a product."""
    x, n, ids, w = inputs(tokens, top_k, groups, hidden)
    errors = {}
    for layout in ("masked", "contiguous", "nopad"):
        b = Block(tokens, top_k, groups, hidden, inner, layout)
        h, m = b.forward(x, n, ids, w)
        want_h, want_n = plain_block(b, x.float(), n.float(), ids, w)
        errors[f"{layout} h"], errors[f"{layout} n"] = relative(h, want_h), relative(m, want_n)
    leaves = {"x": x.float(), "n": n.float(), "weights": w.clone(), "post": b.post, "gate": b.gate, "pre": b.pre}
    for v in leaves.values():
        v.requires_grad_()
    gen = torch.Generator(device=x.device).manual_seed(2)
    dh, dn = (torch.randn(tokens, hidden, generator=gen, device=x.device).bfloat16() for _ in range(2))
    want_h, want_n = plain_block(b, leaves["x"], leaves["n"], ids, leaves["weights"])
    ((want_h * dh).sum() + (want_n * dn).sum()).backward()
    with torch.no_grad():
        got = b.backward(dh, dn, w)
    for name, v in leaves.items():
        errors[f"gradient of {name}"] = relative(got[name], v.grad)
    return errors


def main():
    for name, e in compare().items():
        print(f"{name:20s} {100 * e:5.2f}% from float32")
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 64
    top_k, groups, hidden, inner = 8, 16, 7168, 2048
    x, n, ids, w = inputs(tokens, top_k, groups, hidden)
    b = Block(tokens, top_k, groups, hidden, inner, "masked" if tokens <= 256 else "contiguous")
    for _ in range(5):
        b.forward(x, n, ids, w)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(20):
        b.forward(x, n, ids, w)
    torch.cuda.synchronize()
    print(f"{tokens} tokens, {groups} experts of {inner}, top {top_k}, hidden {hidden} ({b.layout}): "
          f"{(time.perf_counter() - t) / 20 * 1e6:.1f} us a block")


if __name__ == "__main__":
    main()
