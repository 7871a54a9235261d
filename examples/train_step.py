"""A training loop of one MoE layer on the library's operators:

  logits = x W_r^T                     (the caller's own projection)
  moe_route                            balance bias in the selection, expert groups, top-k, weights,
                                       routes per expert and normalised scores for the balance loss
  moe_fwd_routed / moe_bwd_routed      the experts on that routing, and their gradients
  moe_route_bwd                        the logits' gradient, from the weights' and the balance loss's
  moe_muon_update                      momentum and orthogonalised updates of the experts' matrices

The layer learns a random teacher layer's outputs.  Prints the loss and how
uneven the experts' load is (largest over mean).

    python examples/train_step.py [--steps N] [--tokens T]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import routing_grouped_expert_gemm_gb300 as rg  # noqa: E402

D, I, E, K, I_S = 512, 256, 16, 4, 256
GROUPS, KEPT = 4, 2
MATRICES = {"W_up": (E, I, D), "W_gate": (E, I, D), "W_down": (E, D, I),
            "Ws_up": (1, I_S, D), "Ws_gate": (1, I_S, D), "Ws_down": (1, D, I_S)}


class Layer:
    def __init__(self, T, seed, plan, route_plan):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.plan, self.route_plan = T, plan, route_plan
        self.W_r = torch.randn(E, D, generator=g, device="cuda") * D ** -0.5
        self.bias = torch.zeros(E, device="cuda")
        # fp32 masters; the layer computes with their bf16 copies
        self.master = {n: torch.randn(s, generator=g, device="cuda") * s[2] ** -0.5 for n, s in MATRICES.items()}
        self.w = {n: m.bfloat16() for n, m in self.master.items()}
        self.ws = torch.empty(rg.moe_workspace_bytes(plan, T), dtype=torch.uint8, device="cuda")
        self.route_ws = torch.empty(rg.moe_route_workspace_bytes(route_plan, T), dtype=torch.uint8, device="cuda")
        self.idx = torch.empty(T, K, dtype=torch.int32, device="cuda")
        self.wt = torch.empty(T, K, device="cuda")
        self.counts = torch.empty(E, dtype=torch.int32, device="cuda")
        self.prob_sum = torch.empty(E, device="cuda")
        self.out = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")

    def forward(self, x):
        self.logits = x.float() @ self.W_r.T
        rg.moe_route(self.route_plan, self.T, self.logits, self.bias, self.idx, self.wt, expert_counts=self.counts,
                     prob_sum=self.prob_sum, workspace=self.route_ws)
        rg.moe_fwd_routed(self.plan, self.T, x, self.w, self.idx, self.wt, self.out, self.ws)
        return self.out


class Trainer:
    def __init__(self, layer, lr=0.02, balance=1e-2, bias_step=2e-3):
        self.layer, self.lr, self.balance, self.bias_step = layer, lr, balance, bias_step
        T = layer.T
        self.grads = {"d" + n: torch.empty(s, dtype=torch.bfloat16, device="cuda") for n, s in MATRICES.items()}
        self.grads["dx"] = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
        self.bwd_ws = torch.empty(rg.moe_bwd_workspace_bytes(layer.plan, T), dtype=torch.uint8, device="cuda")
        self.d_wt = torch.empty(T, K, device="cuda")
        self.d_logits = torch.empty(T, E, device="cuda")
        self.momentum = {n: torch.zeros(s, device="cuda") for n, s in MATRICES.items()}
        self.update = {n: torch.empty(s, dtype=torch.bfloat16, device="cuda") for n, s in MATRICES.items()}
        self.muon = {n: rg.moe_muon_plan_create(*s) for n, s in MATRICES.items()}
        most = max(rg.moe_muon_workspace_bytes(p) for p in self.muon.values())
        self.muon_ws = torch.empty(most, dtype=torch.uint8, device="cuda")

    def step(self, x, target):
        m, T = self.layer, self.layer.T
        diff = m.forward(x).float() - target
        loss = diff.square().mean()
        d_out = (diff * (2.0 / diff.numel())).bfloat16()
        rg.moe_bwd_routed(m.plan, T, x, m.w, d_out, m.ws, self.grads, self.d_wt, self.bwd_ws)
        # balance loss: E / (K T^2) sum_e counts_e prob_sum_e, whose gradient goes through the scores only
        d_prob = m.counts.float() * (self.balance * loss.detach() * E / (K * T * T))
        rg.moe_route_bwd(m.route_plan, T, m.logits, m.idx, self.d_wt, self.d_logits, dprob_sum=d_prob)
        m.W_r -= 0.5 * (self.d_logits.T @ x.float())
        # the selection's bias follows the load
        m.bias += self.bias_step * torch.sign(T * K / E - m.counts.float())
        for n, (count, rows, cols) in MATRICES.items():
            scale = 0.2 * max(rows, cols) ** 0.5 * min(rows, cols) ** -0.5
            rg.moe_muon_update(self.muon[n], self.grads["d" + n], self.momentum[n], self.update[n], self.muon_ws, mu=0.9,
                               scale=scale)
            m.master[n].add_(self.update[n].float(), alpha=-self.lr)
            m.w[n].copy_(m.master[n])
        return loss


def train(steps=60, T=2048, seed=0):
    """Returns the losses and, per step, the largest expert's load over the mean."""
    plan = rg.moe_plan_create(T, D, I, E, K, I_S, minibatch=2048, dispatch="spread", mma_pair=1)
    route_plan = rg.moe_route_plan_create(E, K, score_fn="sigmoid", n_group=GROUPS, topk_group=KEPT, scale=1.0)
    teacher, layer = Layer(T, seed + 1, plan, route_plan), Layer(T, seed + 2, plan, route_plan)
    trainer = Trainer(layer)
    g = torch.Generator(device="cuda").manual_seed(seed)
    losses, load = [], []
    for _ in range(steps):
        x = torch.randn(T, D, generator=g, device="cuda").bfloat16()
        target = teacher.forward(x).float()
        losses.append(trainer.step(x, target))
        load.append(layer.counts.max() * (E / (T * K)))
    assert rg.moe_get_status(plan, layer.ws) == rg.MOE_STATUS_OK
    return [float(v) for v in losses], [float(v) for v in load]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=2048)
    a = ap.parse_args()
    losses, load = train(a.steps, a.tokens)
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.4f}  largest load {load[i]:.2f} x mean")
    print(f"step {a.steps - 1:4d}  loss {losses[-1]:.4f}  largest load {load[-1]:.2f} x mean")


if __name__ == "__main__":
    main()
