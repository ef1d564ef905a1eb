"""Training the experts of an MoE layer, one step after another.

    python examples/train_experts.py [--steps N] [--state-bits 8|32] [--batches N] [--train-router] [--shared]

A student layer learns a teacher's outputs on synthetic tokens.  The router is
fixed (its top-k ids and weights are the layer's input), or, with
--train-router, learns too, with a load balance and a loss on the size of its
logits.  With --shared an expert that all tokens go to, with biases and
without a gate, is added to the routed ones.
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
    dx, dWr, losses         moe_route_backward        (--train-router: dx is added to)
    W13, W2, Wr ...         moe_adamw_step

and of the shared expert

    hs   = gelu(zs)         moe_expert_gemm_act       zs = x W1^T + b1, kept for the gradient
    out += hs W2^T + b2     moe_expert_gemm_act
    dW2, db2                moe_expert_gemm_wgrad, moe_expert_bias_grad
    dzs                     moe_expert_gemm_dgrad_act (through gelu)
    dW1, db1                moe_expert_gemm_wgrad, moe_expert_bias_grad
    dx  += dzs W1           moe_expert_gemm_dgrad_act
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


class SharedExpert:
    """w1 [I, K], w2 [K, I] (bf16) with fp32 biases, for batches of T tokens: gelu(x w1^T + b1) w2^T + b2."""

    dense = (None, None)   # one expert that has all rows: no start, no counts

    def __init__(self, w1, b1, w2, b2, T):
        self.w1, self.b1, self.w2, self.b2 = w1, b1, w2, b2
        I, K = w1.shape
        dev, bf = w1.device, torch.bfloat16
        self.status = torch.zeros(4, dtype=torch.int32, device=dev)
        self.z, self.h, self.dz = (torch.empty((T, I), dtype=bf, device=dev) for _ in range(3))
        self.dw1, self.dw2 = torch.empty((1, I, K), dtype=bf, device=dev), torch.empty((1, K, I), dtype=bf, device=dev)
        self.db1, self.db2 = torch.empty_like(b1), torch.empty_like(b2)

    def forward(self, x, out):
        """out += the expert's outputs."""
        at = (*self.dense, self.status)
        M.moe_expert_gemm_act(x, self.w1, *at, bias=self.b1, act="gelu", y=self.h, z=self.z)
        return M.moe_expert_gemm_act(self.h, self.w2, *at, bias=self.b2, residual=out, y=out)[0]

    def backward(self, dout, x, dx):
        """Gradients of w1, b1, w2 and b2; dx += that of x."""
        at = (*self.dense, self.status)
        M.moe_expert_gemm_wgrad(dout, self.h, *at, dw=self.dw2)
        M.moe_expert_bias_grad(dout, *at, db=self.db2)
        M.moe_expert_gemm_dgrad_act(dout, self.w2, *at, z=self.z, act="gelu", dx=self.dz)
        M.moe_expert_gemm_wgrad(self.dz, x, *at, dw=self.dw1)
        M.moe_expert_bias_grad(self.dz, *at, db=self.db1)
        M.moe_expert_gemm_dgrad_act(self.dz, self.w1, *at, residual=dx, dx=dx)
        return self.dw1, self.db1, self.dw2, self.db2


class Router:
    """fp32 weights [E, K] with their gradient, and the kernels' planes of them."""

    def __init__(self, w, T, topk, balance=0.01, zloss=0.001):
        E, K = w.shape
        self.w, self.topk, self.balance, self.zloss = w, topk, balance, zloss
        self.dw, self.losses = torch.empty_like(w), torch.empty(2, device=w.device)
        self.planes = torch.empty((3, E, K), dtype=torch.bfloat16, device=w.device)
        self.ws = torch.empty(M.moe_route_backward_workspace_size(T, K, E), dtype=torch.uint8, device=w.device)
        self.status = torch.zeros(4, dtype=torch.int32, device=w.device)   # of every gradient since

    def forward(self, x):
        M.moe_router_prepare(self.w, out=self.planes)
        self.ids, self.weights, self.logits = M.moe_route(x, self.planes, self.topk)
        return self.ids, self.weights

    def backward(self, x, dweights, dx, accumulate=False, batches=1):
        """Gradient of w; dx += that of x.  Of a mean over batches: the losses count 1 / batches, as dweights do."""
        M.moe_route_backward(x, self.planes, self.logits, self.ids, self.weights, dweights, balance=self.balance / batches,
                             zloss=self.zloss / batches, residual=dx, dx=dx, dw=self.dw, accumulate=accumulate, losses=self.losses,
                             ws=self.ws)
        torch.maximum(self.status[:1], self.ws[:4].view(torch.int32), out=self.status[:1])
        return self.dw


def optimizer(layer, state_bits, others=()):
    """AdamW over the layer's weights (fp32 copies of those in bf16) and others' [(param, grad)], states in 32 or 8
    bits."""
    params, grads = [layer.w13, layer.w2], [layer.dw13, layer.dw2]
    for p, g in others:
        params.append(p)
        grads.append(g)
    masters = [p.float() if p.dtype != torch.float32 else None for p in params]
    if state_bits == 32:
        m, v = ([torch.zeros(p.shape, device=p.device) for p in params] for _ in range(2))
        return M.moe_adamw_create(params, grads, m, v, masters=masters)
    m = [torch.zeros(p.shape, dtype=torch.int8, device=p.device) for p in params]
    v = [torch.zeros(p.shape, dtype=torch.uint8, device=p.device) for p in params]
    scales = [[torch.zeros(-(-p.numel() // 256), device=p.device) for p in params] for _ in range(2)]
    return M.moe_adamw_create(params, grads, m, v, masters=masters, avg_scales=scales[0], sq_scales=scales[1])


def train(T=512, K=256, I=256, E=8, topk=2, steps=30, state_bits=8, lr=3e-3, clip=1.0, seed=1, batches_per_step=1,
          train_router=False, shared=False):
    """Losses of `steps` training steps."""
    if shared and batches_per_step > 1:
        raise ValueError("the shared expert's gradients are those of one batch")
    g = torch.Generator(device="cuda").manual_seed(seed)
    layer = ExpertLayer(synth.bf16_expert_weights(E, 2 * I, K, seed, "cuda"), synth.bf16_expert_weights(E, K, I, seed + 1, "cuda"),
                        T, topk, torch.bfloat16 if batches_per_step == 1 else torch.float32)
    teacher = ExpertLayer(synth.bf16_expert_weights(E, 2 * I, K, seed + 2, "cuda") * 4,
                          synth.bf16_expert_weights(E, K, I, seed + 3, "cuda") * 4, T, topk)
    router = Router(torch.randn((E, K), generator=g, device="cuda") * 0.1, T, topk)
    planes = M.moe_router_prepare(router.w)   # the teacher's, and the student's where it does not learn
    others, more = [], None
    if train_router:
        router.w = router.w + torch.randn((E, K), generator=g, device="cuda") * 0.02
        others.append((router.w, router.dw))
    if shared:
        more = SharedExpert(synth.bf16_expert_weights(1, I, K, seed + 4, "cuda")[0], torch.zeros(I, device="cuda"),
                            synth.bf16_expert_weights(1, K, I, seed + 5, "cuda")[0], torch.zeros(K, device="cuda"), T)
        others += [(more.w1, more.dw1), (more.b1, more.db1), (more.w2, more.dw2), (more.b2, more.db2)]
    opt = optimizer(layer, state_bits, others)
    # few batches, seen again and again
    batches = [synth.activations(T, K, seed + 10 + i, "cuda") for i in range(4)]
    losses = []
    for step in range(1, steps + 1):
        loss = 0.0
        for part in range(batches_per_step):
            x = batches[(step * batches_per_step + part) % len(batches)]
            ids, weights, _ = M.moe_route(x, planes, topk)
            want = teacher.forward(x, ids, weights).float()
            if train_router:
                ids, weights = router.forward(x)
            out = layer.forward(x, ids, weights)
            if shared:
                more.forward(x, out)
            diff = out.float() - want
            loss = loss + diff.square().mean() / batches_per_step
            dout = (diff * (2.0 / diff.numel() * T / batches_per_step)).to(torch.bfloat16)
            layer.backward(dout, weights, accumulate=part > 0)
            if shared:
                more.backward(dout, x, layer.dx)
            if train_router:
                router.backward(x, layer.dweights, layer.dx, accumulate=part > 0, batches=batches_per_step)
        losses.append(loss)
        norm = torch.stack([g.float().norm() for g in (layer.dw13, layer.dw2, *(g for _, g in others))]).norm()
        scale = (clip / norm).clamp(max=1.0).reshape(1)   # stays on the device
        M.moe_adamw_step(opt, step=step, lr=lr, beta2=0.95, weight_decay=0.01, grad_scale=scale)
    losses = [float(v) for v in losses]
    for part in (layer, teacher, router, *([more] if shared else [])):
        status = M.moe_read_device_status(part.status)
        if status:
            raise RuntimeError(f"device status {M.STATUS_NAMES.get(status, status)}")
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    ap.add_argument("--batches", type=int, default=1, help="batches per step")
    ap.add_argument("--train-router", action="store_true", help="the router learns too")
    ap.add_argument("--shared", action="store_true", help="with an expert that all tokens go to")
    a = ap.parse_args()
    losses = train(steps=a.steps, state_bits=a.state_bits, batches_per_step=a.batches, train_router=a.train_router,
                   shared=a.shared)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i + 1:5d}  loss {losses[i]:.5f}")
    print(f"last        loss {losses[-1]:.5f}")


if __name__ == "__main__":
    main()
