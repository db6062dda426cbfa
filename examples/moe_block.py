"""A transformer block's feed-forward half around the MoE layer, forward and backward.

    h      = x W_o^T + x                     attention output projection, residual in its epilogue
    logits = h W_r^T                         router logits in float32
    ids, w = route_scored(logits, bias)      sigmoid scores, balance bias, expert groups, top-k
    rows   = grouped FFN of the dispatched rows of h       (experts frozen, no gradient to h)
    c      = combine(rows, w)
    z      = h W_1^T + b_1;  u = silu(z)     dense branch
    y      = u W_2^T + c                     second product, the combined experts as residual

The backward gives the gradients of W_o, W_r, W_1, b_1 and W_2: the combine's gradient yields
the route weights', routing's gradient the logits', and the linear layers take it from there.
The experts' rows are a constant of h in it (a stop-gradient: they are frozen here, moe_train.py
trains them), so W_o's gradient is that of the dense branch, the router and the residual and
leaves out what h does through the experts.  After each step the balance bias moves against
the experts' load, as scores-plus-bias routing is trained.

    python examples/moe_block.py [--tokens T] [--steps N]

Fits the block to a random target and prints the loss of each step (needs a GB300 and the
built library).
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mixture_experts_layer_04_gb300 as moe  # noqa: E402

BF16 = torch.bfloat16


def _bytes(n):
    return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")


class MoEBlock:
    """Weights, plans and buffers of one block for batches of T tokens."""

    def __init__(self, T, H=512, E=64, K=6, I=256, dense=1024, groups=8, top_groups=4, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF16)

        self.T, self.H, self.E, self.K = T, H, E, K
        self.w_o = randn(H, H, std=0.5 * H ** -0.5)
        self.w_r = randn(E, H, std=H ** -0.5)
        self.bias = torch.zeros(E, device="cuda")
        self.w_gate_up = randn(E, 2 * I, H, std=H ** -0.5)
        self.w_down = randn(E, H, I, std=I ** -0.5)
        self.w_1 = randn(dense, H, std=H ** -0.5)
        self.b_1 = torch.zeros(dense, device="cuda")
        self.w_2 = randn(H, dense, std=dense ** -0.5)

        self.cfg = moe.MoEConfig.make(T=T, H=H, E=E, K=K, I=I, dtype=moe.BF16)
        self.route = moe.RouteConfig.make(T, E, K, groups, top_groups, group_rank=2,
                                          score=moe.SCORE_SIGMOID, scale=1.0)
        lin = moe.LinearConfig.make
        self.lin_o = lin(T, H, H)
        self.lin_r = lin(T, H, E, out_dtype=moe.F32)
        self.lin_1 = lin(T, H, dense, activation=moe.ACT_SILU)
        self.lin_2 = lin(T, dense, H)
        self.ws = _bytes(moe.workspace_size(self.cfg))
        self.lin_ws = _bytes(max(moe.linear_workspace_size(c) for c in
                                 (self.lin_o, self.lin_r, self.lin_1, self.lin_2)))

        def empty(*shape, dtype=BF16):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        f32, i32 = torch.float32, torch.int32
        self.h, self.c, self.y = empty(T, H), empty(T, H), empty(T, H)
        self.z, self.u = empty(T, dense), empty(T, dense)
        self.logits = empty(T, E, dtype=f32)
        self.ids, self.w = empty(T, K, dtype=i32), empty(T, K, dtype=f32)
        self.counts, self.offsets = empty(E, dtype=i32), empty(E + 1, dtype=i32)
        self.perm, self.inv = empty(T * K, dtype=i32), empty(T * K, dtype=i32)
        self.x_perm, self.rows = empty(T * K, H), empty(T * K, H, dtype=f32)

    def forward(self, x):
        ws, lws = self.ws, self.lin_ws
        moe.linear(self.lin_o, x, self.w_o, None, x, self.h, None, lws)
        moe.linear(self.lin_r, self.h, self.w_r, None, None, self.logits, None, lws)
        moe.route_scored(self.route, self.logits, self.bias, self.ids, self.w)
        moe.permute(self.cfg, self.h, self.ids, self.counts, self.offsets, self.perm, self.inv,
                    self.x_perm, ws)
        moe.grouped_ffn(self.cfg, self.x_perm, self.offsets, self.w_gate_up, self.w_down,
                        self.rows, ws)
        moe.combine(self.cfg, self.rows, self.inv, self.w, None, self.c)
        # u = silu(z) with z kept; its residual slot is free, the second product's takes c
        moe.linear(self.lin_1, self.h, self.w_1, self.b_1, None, self.u, self.z, lws)
        moe.linear(self.lin_2, self.u, self.w_2, None, self.c, self.y, None, lws)
        return self.y

    def backward(self, x, dy):
        """Gradients by name, for the x of the last forward, the experts' input held constant."""
        lws = self.lin_ws
        like = torch.empty_like
        du, dw_2 = like(self.u), like(self.w_2)
        moe.linear_backward(self.lin_2, dy, self.u, self.w_2, None, du, dw_2, None, lws)
        dh, dw_1, db_1 = like(self.h), like(self.w_1), like(self.b_1)
        moe.linear_backward(self.lin_1, du, self.h, self.w_1, self.z, dh, dw_1, db_1, lws)
        # the combine's gradient is dy itself: through the route weights to the logits
        d_w = like(self.w)
        moe.combine_backward(self.cfg, dy, self.rows, self.inv, self.w, None, d_w)
        d_logits = like(self.logits)
        moe.route_scored_backward(self.route, self.logits, self.ids, d_w, d_logits)
        dh_r, dw_r = like(self.h), like(self.w_r)
        moe.linear_backward(self.lin_r, d_logits, self.h, self.w_r, None, dh_r, dw_r, None, lws)
        dh += dh_r
        dw_o = like(self.w_o)
        moe.linear_backward(self.lin_o, dh, x, self.w_o, None, None, dw_o, None, lws)
        return dict(w_o=dw_o, w_r=dw_r, w_1=dw_1, b_1=db_1, w_2=dw_2)

    def balance(self, rate):
        """Move the bias against the load of the last batch."""
        self.bias += rate * torch.sign(self.counts.float().mean() - self.counts.float())


def fit(T=1024, steps=10, lr=0.05, seed=0):
    """A few steps of gradient descent on a random target; returns the losses."""
    block = MoEBlock(T, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn(T, block.H, generator=g, device="cuda").to(BF16)
    target = torch.randn(T, block.H, generator=g, device="cuda")
    losses = []
    for _ in range(steps):
        diff = block.forward(x).float() - target
        losses.append((diff * diff).mean().item())
        grads = block.backward(x, (diff * (2.0 / diff.shape[1])).to(BF16))
        for name, grad in grads.items():
            p = getattr(block, name)
            p.copy_(p.float() - lr / T ** 0.5 * grad.float())
        block.balance(1e-3)
    moe.sync_check()
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    for i, loss in enumerate(fit(a.tokens, a.steps)):
        print(f"step {i}: loss {loss:.5f}")


if __name__ == "__main__":
    main()
