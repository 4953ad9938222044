"""A mixture-of-experts layer in block-scaled FP8 on the library's calls, forward and router gradient.

    python examples/moe_layer.py [tokens hidden inner experts top_k]

One pass, every step on the current stream and without the host waiting for the GPU:

    logits   = x router^T                       gemm_run (BF16 -> FP32)
    routing  = moe_route(logits)                experts, weights, rows, counts, balance loss
    a        = moe_dispatch(x)                  the experts' rows, e4m3 with a scale per 128
    inner    = relu(a up_e^T)                   gemm_grouped_run, the counts as group rows
    b        = moe_dispatch(inner)              the same rows, quantized in their order
    rows     = b down_e^T                       gemm_grouped_run
    out      = moe_combine(rows)                each token's rows, weighted

and for the router's training moe_combine_backward (the weights' gradient from out's) and
moe_route_backward (the logits' gradient from the weights' and the balance loss's).  The expert
weights are quantized once, in 128 x 128 blocks.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tile_scheduled_tensor_gb300 as tst  # noqa: E402

BLOCK = 128


def quantize_weight(w):
    """e4m3 values and scales of w (experts x N x K) in 128 x 128 blocks."""
    e, n, k = w.shape
    pad = torch.nn.functional.pad(w.float(), (0, -k % BLOCK, 0, -n % BLOCK))
    b = pad.reshape(e, pad.shape[1] // BLOCK, BLOCK, pad.shape[2] // BLOCK, BLOCK)
    scale = b.abs().amax(dim=(2, 4)).clamp(min=2.0 ** -96) / 448.0
    q = (b / scale[:, :, None, :, None]).reshape(pad.shape)[:, :n, :k]
    return q.to(torch.float8_e4m3fn).contiguous(), scale.contiguous()


class MoELayer:
    """Plans, quantized weights and buffers for up to max_tokens tokens."""

    def __init__(self, router, up, down, max_tokens, top_k, balance_coef=0.01):
        experts, inner, hidden = up.shape
        self.experts, self.inner, self.hidden, self.top_k, self.max_tokens = experts, inner, hidden, top_k, max_tokens
        self.router = router.to(torch.bfloat16).contiguous()
        (self.up, self.up_scales), (self.down, self.down_scales) = quantize_weight(up), quantize_weight(down)
        self.plan = tst.moe_plan_create(max_tokens, experts, top_k, normalize=True, balance_coef=balance_coef)
        rows = max_tokens * top_k
        grouped = dict(dtype="e4m3", out_dtype="bf16", ab_block=(1, BLOCK, BLOCK))
        self.up_plan = tst.gemm_grouped_plan_create(experts, rows, inner, hidden, relu=True, **grouped)
        self.down_plan = tst.gemm_grouped_plan_create(experts, rows, hidden, inner, **grouped)
        self.router_plans = {}
        new = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
        self.expert, self.row = (new(max_tokens, top_k, dt=torch.int32) for _ in range(2))
        self.weight, self.counts = new(max_tokens, top_k), new(experts, dt=torch.int32)
        self.totals, self.loss = new(2, dt=torch.int32), new(1)
        self.a, self.a_scales = new(rows, hidden, dt=torch.uint8), new(rows, -(-hidden // BLOCK))
        self.mid = new(rows, inner, dt=torch.bfloat16)
        self.b, self.b_scales = new(rows, inner, dt=torch.uint8), new(rows, -(-inner // BLOCK))
        self.rows = new(rows, hidden, dt=torch.bfloat16)

    def forward(self, x, mask=None):
        """(out, balance loss) of x (tokens x hidden, BF16); mask: one byte per token, 0 for padding."""
        t = x.shape[0]
        if t not in self.router_plans:   # the plan of a GEMM is for one shape
            self.router_plans[t] = tst.gemm_plan_create(t, self.experts, self.hidden, out_dtype="f32")
        self.x, self.mask, self.t = x, mask, t
        self.logits = torch.empty(t, self.experts, device="cuda")
        tst.gemm_run(self.router_plans[t], x, self.router, self.logits)
        tst.moe_route(self.plan, self.logits, self.expert[:t], self.weight[:t], self.row[:t], self.counts, self.totals,
                      self.loss, mask=mask)
        tst.moe_dispatch(self.plan, x, self.row[:t], self.a, scales=self.a_scales)
        tst.gemm_grouped_run(self.up_plan, self.counts, self.a, self.up, self.mid, a_block_scales=self.a_scales,
                             b_block_scales=self.up_scales)
        tst.moe_dispatch(self.plan, self.mid, None, self.b, scales=self.b_scales)
        tst.gemm_grouped_run(self.down_plan, self.counts, self.b, self.down, self.rows, a_block_scales=self.b_scales,
                             b_block_scales=self.down_scales)
        out = torch.empty_like(x)
        tst.moe_combine(self.plan, self.rows, self.row[:t], out, weight=self.weight[:t])
        return out, self.loss

    def router_gradient(self, d_out, d_loss):
        """d_logits of the last forward, from out's gradient and the loss's (a CUDA tensor of one element)."""
        d_rows, d_weight = torch.empty_like(self.rows), torch.empty_like(self.weight[:self.t])
        tst.moe_combine_backward(self.plan, self.rows, self.row[:self.t], self.weight[:self.t], d_out, d_rows, d_weight)
        d_logits = torch.empty_like(self.logits)
        tst.moe_route_backward(self.plan, self.logits, self.expert[:self.t], self.counts, self.totals, d_logits,
                               d_weight=d_weight, d_loss=d_loss, mask=self.mask)
        return d_logits


def plain_layer(logits, x, up, down, top_k, mask=None, balance_coef=0.01):
    """The same layer in FP32 torch from given logits: (out, loss)."""
    experts = up.shape[0]
    live = torch.ones(len(x), dtype=torch.bool, device=x.device) if mask is None else mask.bool()
    p = torch.softmax(logits, 1)
    w, expert = torch.topk(p, top_k, dim=1)
    w = w / w.sum(1, keepdim=True) * live[:, None]
    out = torch.zeros(x.shape, device=x.device)
    for e in range(experts):
        t, j = torch.nonzero((expert == e) & live[:, None], as_tuple=True)
        out = out.index_add(0, t, torch.relu(x[t].float() @ up[e].T) @ down[e].T * w[t, j, None])
    counts = torch.bincount(expert[live].reshape(-1), minlength=experts)
    loss = balance_coef * experts * (counts / counts.sum() * p[live].mean(0)).sum()
    return out, loss


def run(tokens=96, hidden=512, inner=768, experts=16, top_k=4, seed=0, padded=0):
    """The layer against plain FP32 torch: the relative 2-norm error of out, and the largest error of the
    loss and of the logits' gradient relative to their largest values."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    up, down = new(experts, inner, hidden) * hidden ** -0.5, new(experts, hidden, inner) * inner ** -0.5
    layer = MoELayer(new(experts, hidden) * hidden ** -0.5, up, down, tokens, top_k)
    x = new(tokens, hidden).bfloat16()
    mask = None
    if padded:
        mask = torch.ones(tokens, dtype=torch.uint8, device="cuda")
        mask[-padded:] = 0
    out, loss = layer.forward(x, mask)
    d_out, d_loss = new(tokens, hidden).bfloat16(), torch.ones(1, device="cuda")
    d_logits = layer.router_gradient(d_out, d_loss)
    for plan in (layer.up_plan, layer.down_plan):
        status, word = tst.gemm_status_query(plan)
        assert status == tst.TST_OK, (tst.gemm_status_string(status), hex(word))
    assert tst.moe_status_query(layer.plan) == tst.TST_OK
    want, want_loss = plain_layer(layer.logits, x, up, down, top_k, mask)
    # the router's gradient by autograd, through the weights alone (the library's rows, held fixed) and the loss
    logits = layer.logits.clone().requires_grad_(True)
    p = torch.softmax(logits, 1)
    live = layer.expert >= 0
    w = p.gather(1, layer.expert.clamp(min=0).long()) * live
    w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    rows = torch.where(live[:, :, None], layer.rows[layer.row.clamp(min=0).long()].float(), 0.0)
    n = layer.totals[1].float()
    share = layer.counts.float() / layer.totals[0].float()
    alive = live.any(1)
    again = 0.01 * experts * (share * (p * alive[:, None]).sum(0) / n).sum()
    (((w[:, :, None] * rows).sum(1) * d_out.float()).sum() + again).backward()
    return ((out.float() - want).norm() / want.norm()).item(), abs(loss.item() / want_loss.item() - 1), \
        ((d_logits - logits.grad).abs().max() / logits.grad.abs().max()).item()


if __name__ == "__main__":
    names = ("tokens", "hidden", "inner", "experts", "top_k")
    args = {n: int(v) for n, v in zip(names, sys.argv[1:])}
    error, loss_error, grad_error = run(**args)
    print(f"moe layer {args or 'default sizes'}: out off by {error:.4f} (two e4m3 roundings per product), "
          f"balance loss by {loss_error:.1e}, router gradient by {grad_error:.1e}")
