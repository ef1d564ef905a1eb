"""Training the experts of an MoE layer, one step after another.

    python examples/train_experts.py [--steps N] [--state-bits 8|32] [--batches N]

A student layer learns a teacher's outputs on synthetic tokens.  The router is
fixed (its top-k ids and weights are the layer's input); the gradient of its
weights, which a trainable router would go on from, comes with the others.
Every product, gather and update is one of libmoe's kernels; torch holds the
memory and forms the loss.  With --batches, a step's gradient is the mean over
that many batches, summed in fp32 by the products that form it.

    ids, weights            moe_route
    src2dst, start, counts  moe_sort_plan
    xs   = x, by expert     moe_sort_tokens
    h    = silu(g) u        moe_expert_gemm_swiglu     g | u = xs W13^T, kept for the gradient
    y    = h W2^T           moe_expert_gemm
    out  = weighted sum     moe_unsort_tokens
    dy, dweights            moe_unsort_tokens_backward
    dW2  = dy^T h           moe_expert_gemm_wgrad
    dgu                     moe_expert_gemm_dgrad_swiglu
    dW13 = dgu^T xs         moe_expert_gemm_wgrad
    dxs  = dgu W13          moe_expert_gemm_dgrad
    dx                      moe_unsort_tokens (no weights)
    W13, W2                 moe_adamw_step
"""

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import moe_expert_layer_ep_gb300 as M  # noqa: E402
import synth  # noqa: E402


class ExpertLayer:
    """Experts w13 [E, 2I, K], w2 [E, K, I] (bf16) with their gradients (grad_dtype), for batches of T tokens."""

    def __init__(self, w13, w2, T, topk, grad_dtype=torch.bfloat16):
        self.w13, self.w2 = w13, w2
        self.E, self.K, self.I = w13.shape[0], w13.shape[2], w2.shape[2]
        self.T, self.topk = T, topk
        self.rows = M.moe_compact_all_tokens(T * topk, self.E)
        dev, bf = w13.device, torch.bfloat16

        def rows(cols):
            return torch.empty((self.rows, cols), dtype=bf, device=dev)

        self.plan_ws = torch.empty(M.moe_sort_plan_workspace_size(T, topk, self.E), dtype=torch.uint8, device=dev)
        self.plan_status = self.plan_ws[:4].view(torch.int32)   # of the last plan
        self.status = torch.zeros(4, dtype=torch.int32, device=dev)   # of every call since
        self.src2dst = torch.empty((T, topk), dtype=torch.int32, device=dev)
        self.start = torch.empty(self.E, dtype=torch.int32, device=dev)
        self.counts = torch.empty(self.E, dtype=torch.int32, device=dev)
        self.xs, self.gu, self.h, self.y = rows(self.K), rows(2 * self.I), rows(self.I), rows(self.K)
        self.dy, self.dgu, self.dxs = rows(self.K), rows(2 * self.I), rows(self.K)
        self.dw13, self.dw2 = torch.empty_like(w13, dtype=grad_dtype), torch.empty_like(w2, dtype=grad_dtype)
        self.out = torch.empty((T, self.K), dtype=bf, device=dev)
        self.dx = torch.empty((T, self.K), dtype=bf, device=dev)
        self.dweights = torch.empty((T, topk), dtype=torch.float32, device=dev)

    @property
    def experts(self):
        return self.start, self.counts, self.status

    def forward(self, x, ids, weights):
        M.moe_sort_plan(ids, self.E, src2dst=self.src2dst, start=self.start, counts=self.counts, ws=self.plan_ws)
        torch.maximum(self.status[:1], self.plan_status, out=self.status[:1])   # (each plan clears its own)
        M.moe_sort_tokens(x, self.src2dst, out=self.xs)
        M.moe_expert_gemm_swiglu(self.xs, self.w13, *self.experts, h=self.h, gu=self.gu)
        M.moe_expert_gemm(self.h, self.w2, *self.experts, y=self.y)
        return M.moe_unsort_tokens(self.y, self.src2dst, weights, out=self.out)

    def backward(self, dout, weights, accumulate=False):
        """Gradients of w13, w2, x and the top-k weights, of the last forward()'s inputs.  accumulate: those of w13
        and w2 (in fp32) are added to what the last call left."""
        M.moe_unsort_tokens_backward(dout, self.y, self.src2dst, weights, dy=self.dy, dw=self.dweights)
        M.moe_expert_gemm_wgrad(self.dy, self.h, *self.experts, dw=self.dw2, accumulate=accumulate)
        M.moe_expert_gemm_dgrad_swiglu(self.dy, self.w2, self.gu, *self.experts, dgu=self.dgu)
        M.moe_expert_gemm_wgrad(self.dgu, self.xs, *self.experts, dw=self.dw13, accumulate=accumulate)
        M.moe_expert_gemm_dgrad(self.dgu, self.w13, *self.experts, dx=self.dxs)
        M.moe_unsort_tokens(self.dxs, self.src2dst, out=self.dx)
        return self.dw13, self.dw2, self.dx, self.dweights


def optimizer(layer, state_bits):
    """AdamW over the layer's weights: fp32 copies of them, states in 32 or 8 bits."""
    params, grads = [layer.w13, layer.w2], [layer.dw13, layer.dw2]
    masters = [p.float() for p in params]
    if state_bits == 32:
        m, v = [torch.zeros_like(w) for w in masters], [torch.zeros_like(w) for w in masters]
        return M.moe_adamw_create(params, grads, m, v, masters=masters)
    m = [torch.zeros(p.shape, dtype=torch.int8, device=p.device) for p in params]
    v = [torch.zeros(p.shape, dtype=torch.uint8, device=p.device) for p in params]
    scales = [[torch.zeros(-(-p.numel() // 256), device=p.device) for p in params] for _ in range(2)]
    return M.moe_adamw_create(params, grads, m, v, masters=masters, avg_scales=scales[0], sq_scales=scales[1])


def train(T=512, K=256, I=256, E=8, topk=2, steps=30, state_bits=8, lr=3e-3, clip=1.0, seed=1, batches_per_step=1):
    """Losses of `steps` training steps."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    layer = ExpertLayer(synth.bf16_expert_weights(E, 2 * I, K, seed, "cuda"), synth.bf16_expert_weights(E, K, I, seed + 1, "cuda"),
                        T, topk, torch.bfloat16 if batches_per_step == 1 else torch.float32)
    teacher = ExpertLayer(synth.bf16_expert_weights(E, 2 * I, K, seed + 2, "cuda") * 4,
                          synth.bf16_expert_weights(E, K, I, seed + 3, "cuda") * 4, T, topk)
    planes = M.moe_router_prepare(torch.randn((E, K), generator=g, device="cuda") * 0.1)
    opt = optimizer(layer, state_bits)
    # few batches, seen again and again
    batches = [synth.activations(T, K, seed + 10 + i, "cuda") for i in range(4)]
    losses = []
    for step in range(1, steps + 1):
        loss = 0.0
        for part in range(batches_per_step):
            x = batches[(step * batches_per_step + part) % len(batches)]
            ids, weights, _ = M.moe_route(x, planes, topk)
            want = teacher.forward(x, ids, weights).float()
            diff = layer.forward(x, ids, weights).float() - want
            loss = loss + diff.square().mean() / batches_per_step
            layer.backward((diff * (2.0 / diff.numel() * T / batches_per_step)).to(torch.bfloat16), weights,
                           accumulate=part > 0)
        losses.append(loss)
        norm = torch.stack([layer.dw13.float().norm(), layer.dw2.float().norm()]).norm()
        scale = (clip / norm).clamp(max=1.0).reshape(1)   # stays on the device
        M.moe_adamw_step(opt, step=step, lr=lr, beta2=0.95, weight_decay=0.01, grad_scale=scale)
    losses = [float(v) for v in losses]
    for part in (layer, teacher):
        status = M.moe_read_device_status(part.status)
        if status:
            raise RuntimeError(f"device status {M.STATUS_NAMES.get(status, status)}")
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    ap.add_argument("--batches", type=int, default=1, help="batches per step")
    a = ap.parse_args()
    losses = train(steps=a.steps, state_bits=a.state_bits, batches_per_step=a.batches)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i + 1:5d}  loss {losses[i]:.5f}")
    print(f"last        loss {losses[-1]:.5f}")


if __name__ == "__main__":
    main()
