"""An MoE block trained whole: router, experts, norms, gate and scales.

    y      = RMSnorm(x) n_1                              norm before the block
    logits = y W_r^T;  ids, w = route_scored(logits)     sigmoid scores, balance bias, top-k
    gate   = logistic(y W_g^T)                           one gate per token
    z, h   = y_perm W_gu^T, silu(z_g) z_u                grouped by expert, z kept
    rows   = h W_d^T                                     grouped by expert, float32
    c      = combine(rows, w)
    s      = x + a gate l (RMSnorm(c) p)                 norm after the block, gate, layer scale,
    out    = RMSnorm(s) n_2                              residual and the next norm in one pass

The backward gives the gradients of every parameter and of x, and a step clips them all to one
norm.  The experts' input gradient comes in float32 and is summed over a token's experts by the
combine itself, with weights of 1.

    python examples/moe_train.py [--tokens T] [--steps N]

Fits the block to a random target and prints the loss and the gradients' norm of each step (needs a
GB300 and the built library).
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mixture_experts_layer_04_gb300 as moe  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def empty(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def scratch(n):
    return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")


class TrainedMoEBlock:
    """Weights, plans and buffers of one block for batches of T tokens."""

    EPS = 1e-6

    def __init__(self, T, H=512, E=32, K=4, I=256, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF16)

        def vector(n, mean=1.0):
            return mean + 0.1 * torch.randn(n, generator=g, device="cuda")

        self.T, self.H, self.E, self.K = T, H, E, K
        self.params = dict(
            n_1=vector(H), w_r=randn(E, H, std=H ** -0.5), w_g=randn(1, H, std=H ** -0.5),
            w_gu=randn(E, 2 * I, H, std=H ** -0.5), w_d=randn(E, H, I, std=I ** -0.5),
            post=vector(H), scale=vector(H, 0.5), n_2=vector(H))
        self.bias = torch.zeros(E, device="cuda")

        self.cfg = moe.MoEConfig.make(T=T, H=H, E=E, K=K, I=I, dtype=moe.BF16)
        self.route = moe.RouteConfig.make(T, E, K, score=moe.SCORE_SIGMOID)
        self.lin_r = moe.LinearConfig.make(T, H, E, out_dtype=moe.F32)
        self.lin_g = moe.LinearConfig.make(T, H, 1, out_dtype=moe.F32)
        rows = T * K
        self.up = moe.GroupedConfig.make(rows, E, H, I, dx_dtype=moe.F32,
                                         activation=moe.ACT_SWIGLU)
        self.down = moe.GroupedConfig.make(rows, E, I, H, out_dtype=moe.F32)
        self.before = moe.BlockNormConfig.make(T, H, eps=self.EPS)
        self.after = moe.BlockNormConfig.make(T, H, eps=self.EPS, branch_scale=0.5,
                                              gate=moe.GATE_LOGISTIC)
        self.ws = scratch(max(
            moe.workspace_size(self.cfg),
            *(moe.linear_workspace_size(c) for c in (self.lin_r, self.lin_g)),
            *(moe.grouped_linear_workspace_size(c) for c in (self.up, self.down)),
            *(moe.block_norm_workspace_size(c) for c in (self.before, self.after))))

        self.y, self.c, self.s, self.out = (empty(T, H) for _ in range(4))
        self.logits, self.gate = empty(T, E, dtype=F32), empty(T, dtype=F32)
        self.ids, self.w = empty(T, K, dtype=I32), empty(T, K, dtype=F32)
        self.counts, self.offsets = empty(E, dtype=I32), empty(E + 1, dtype=I32)
        self.perm, self.inv = empty(rows, dtype=I32), empty(rows, dtype=I32)
        self.y_perm, self.rows = empty(rows, H), empty(rows, H, dtype=F32)
        self.z, self.h = empty(rows, 2 * I), empty(rows, I)
        self.ones = torch.ones(T, K, device="cuda")

        # gradients, and the list that clips them in place
        self.grads = {n: torch.empty_like(p) for n, p in self.params.items()}
        self.list = moe.GradList(self.grads.values(), self.grads.values())
        self.norm = empty(1, dtype=F32)
        self.clip_ws = scratch(moe.clip_grad_norm_workspace_size(self.list))

    def forward(self, x):
        p, ws = self.params, self.ws
        moe.block_norm(self.before, x, None, None, None, None, p["n_1"], None, self.y)
        moe.linear(self.lin_r, self.y, p["w_r"], None, None, self.logits, None, ws)
        moe.linear(self.lin_g, self.y, p["w_g"], None, None, self.gate, None, ws)
        moe.route_scored(self.route, self.logits, self.bias, self.ids, self.w)
        moe.permute(self.cfg, self.y, self.ids, self.counts, self.offsets, self.perm, self.inv,
                    self.y_perm, ws)
        moe.grouped_linear(self.up, self.y_perm, self.offsets, p["w_gu"], self.h, self.z, ws)
        moe.grouped_linear(self.down, self.h, self.offsets, p["w_d"], self.rows, None, ws)
        moe.combine(self.cfg, self.rows, self.inv, self.w, None, self.c)
        moe.block_norm(self.after, self.c, x, p["post"], self.gate, p["scale"], p["n_2"], self.s,
                       self.out)
        return self.out

    def backward(self, x, dout):
        """The parameters' gradients (self.grads) and dx, for the x of the last forward."""
        p, g, ws = self.params, self.grads, self.ws
        like = torch.empty_like
        dc, dx, dgate = like(self.c), like(x), like(self.gate)
        moe.block_norm_backward(self.after, dout, None, self.c, self.s, p["post"], self.gate,
                                p["scale"], p["n_2"], dc, dx, dgate, g["post"], g["scale"],
                                g["n_2"], ws)
        drows, dw = empty(*self.rows.shape), like(self.w)
        moe.combine_backward(self.cfg, dc, self.rows, self.inv, self.w, drows, dw)
        dh, dy_perm = like(self.h), like(self.rows)
        moe.grouped_linear_backward(self.down, drows, self.h, self.offsets, p["w_d"], None, dh,
                                    g["w_d"], ws)
        moe.grouped_linear_backward(self.up, dh, self.y_perm, self.offsets, p["w_gu"], self.z,
                                    dy_perm, g["w_gu"], ws)
        # what reaches y: through the experts, the router and the gate
        dy, dy_r, dy_g = like(self.y), like(self.y), like(self.y)
        dlogits = like(self.logits)
        moe.combine(self.cfg, dy_perm, self.inv, self.ones, None, dy)
        moe.route_scored_backward(self.route, self.logits, self.ids, dw, dlogits)
        moe.linear_backward(self.lin_r, dlogits, self.y, p["w_r"], None, dy_r, g["w_r"], None, ws)
        moe.linear_backward(self.lin_g, dgate, self.y, p["w_g"], None, dy_g, g["w_g"], None, ws)
        dy += dy_r
        dy += dy_g
        # the residual's gradient joins that of the first norm, in place
        moe.block_norm_backward(self.before, dy, dx, None, x, None, None, None, p["n_1"], None, dx,
                                None, None, None, g["n_1"], ws)
        return dx

    def step(self, lr, max_norm):
        """Clips the gradients to one norm and moves the parameters; the norm before clipping."""
        moe.clip_grad_norm(self.list, max_norm, self.norm, self.clip_ws)
        for n, t in self.params.items():
            t.copy_(t.float() - lr * self.grads[n].float())
        self.bias += 1e-3 * torch.sign(self.counts.float().mean() - self.counts.float())
        return self.norm


def fit(T=512, steps=10, lr=0.02, max_norm=1.0, seed=0):
    """A few steps of gradient descent on a random target; (loss, gradient norm) of each."""
    block = TrainedMoEBlock(T, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn(T, block.H, generator=g, device="cuda").to(BF16)
    target = torch.randn(T, block.H, generator=g, device="cuda")
    log = []
    for _ in range(steps):
        diff = block.forward(x).float() - target
        block.backward(x, (diff * (2.0 / diff.numel())).to(BF16))
        log.append(((diff * diff).mean().item(), block.step(lr, max_norm).item()))
    moe.sync_check()
    return log


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    for i, (loss, norm) in enumerate(fit(a.tokens, a.steps)):
        print(f"step {i}: loss {loss:.5f}, gradient norm {norm:.4f}")


if __name__ == "__main__":
    main()
