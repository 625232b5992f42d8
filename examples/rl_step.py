"""RL training steps around one MoE layer with router replay, on one GPU.

A tiny policy: embedding -> MoE layer (its routing replayed from a captured
payload, as the trainer of asynchronous RL does) -> head.  Each step runs

  moe_token_logprobs       the reference's and the sampler's log-probabilities
                           (once, before the update);
  layer.forward(train)     the replayed layer;
  moe_policy_loss          the clipped loss with its KL term and the gradient
                           in the vocabulary logits, written over them;
  layer.backward           the experts' gradients and those of the gates;
  layer.router_losses      dense router logits, balance and z losses with
                           per-expert counts, and the router's gradients;
  layer.norm_backward      with --norm (an RMS norm before the layer): its
                           gradient, the router's and the residual's joined in;

and a plain SGD update of the head, the embedding, the router and the norm (the
expert weights stay as quantised).  --ckpt8 keeps what the backward needs in 8
bits.  Run: python examples/rl_step.py [--norm] [--ckpt8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from block_scaled_fp8_router_gb300 import moe_r3 as L  # noqa: E402
from block_scaled_fp8_router_gb300.layer import MoELayerFP8, MoENorm, MoEWeightsFP8, quantize_weights  # noqa: E402


class TinyPolicy:
    """embedding [V, d] -> MoE layer with a residual -> head [V, d], bf16."""

    def __init__(self, V=4000, d=256, E=16, k=4, F=256, T_max=1024, seed=0, device="cuda", norm=False, ckpt8=False):
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s: torch.randn(*s, device=device, generator=g)
        self.emb = r(V, d).bfloat16()
        self.head = (0.05 * r(V, d)).bfloat16()
        w = MoEWeightsFP8((0.1 * r(E, d)).bfloat16(), *quantize_weights((0.06 * r(E, 2 * F, d)).bfloat16(),
                                                                        (0.06 * r(E, d, F)).bfloat16()))
        n = MoENorm(torch.ones(d, device=device)) if norm else None
        self.layer = MoELayerFP8(w, T_max, k, L.MOE_SCORE_SIGMOID, renorm=1, route_scale=2.5, norm=n, ckpt8=ckpt8)

    def hidden(self, tokens, replay_kT=None, capture_kT=None):
        self.x = self.emb[tokens]
        self.h = self.x + self.layer.forward(self.x, replay_kT=replay_kT, capture_kT=capture_kT, train=True)
        return self.h

    def logits(self, tokens, replay_kT=None, capture_kT=None):
        return self.hidden(tokens, replay_kT, capture_kT) @ self.head.t()


def rollout(policy, n_seqs, length, prompt, seed=1):
    """Prompts, sampled tokens and the captured routing of n_seqs samples (the
    inputs are random here; each position's sampled token is its target)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    V, T = policy.emb.shape[0], n_seqs * length
    tokens = torch.randint(0, V, (T,), device="cuda", generator=g)
    capture = torch.empty(policy.layer.k, T, dtype=torch.int32, device="cuda")
    logits = policy.logits(tokens, capture_kT=capture)
    u = torch.rand(T, V, device="cuda", generator=g).clamp_(1e-9, 1 - 1e-7)
    targets = (logits.float() - torch.log(-torch.log(u))).argmax(1)
    old, entropy = L.moe_token_logprobs(logits, targets, entropy=True)
    pos = torch.arange(T, device="cuda") % length
    weights = (pos >= prompt).float()                              # prompt tokens are not trained on
    reward = torch.randn(n_seqs, device="cuda", generator=g)
    adv = (reward - reward.mean()).repeat_interleave(length)       # one advantage per sample
    offsets = torch.arange(0, T + 1, length, dtype=torch.int32, device="cuda")
    return dict(tokens=tokens, targets=targets, old=old, ref=old.clone(), adv=adv, weights=weights, capture=capture,
                offsets=offsets, entropy=entropy)


def step(policy, b, lr=0.02, kl_coef=0.02, balance_coef=1e-2, z_coef=1e-4):
    """One update on the rollout b; returns (policy stats [6], router losses
    [2], counts [B, E])."""
    logits = policy.logits(b["tokens"], replay_kT=b["capture"])
    stats, _, dlogits = L.moe_policy_loss(logits, b["targets"], b["old"], b["adv"], ref_logprobs=b["ref"],
                                          weights=b["weights"], clip_low=0.2, clip_high=0.28, kl_coef=kl_coef,
                                          dlogits=logits, dev_status=policy.layer.dev_status)
    dh = dlogits @ policy.head
    d_head = dlogits.t().float() @ policy.h.float()
    dx_experts, d_gates = policy.layer.backward(dh)
    losses, counts, dx_router, dw = policy.layer.router_losses(balance_coef, z_coef, d_gates=d_gates,
                                                               token_mask=b["weights"] != 0, seq_offsets=b["offsets"])
    if policy.layer.norm is None:
        dx = dh.float() + dx_experts.float() + dx_router
    else:
        dx, d_norm, _ = policy.layer.norm_backward(dx_experts, dx_router, dres=dh)
        policy.layer.norm.weight.sub_(lr * d_norm)
    policy.head.sub_((lr * d_head).bfloat16())
    policy.emb.index_add_(0, b["tokens"], (-lr * dx).bfloat16())
    policy.layer.w.w_router.sub_((lr * dw).bfloat16())
    return stats, losses, counts


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--norm", action="store_true", help="an RMS norm before the layer")
    ap.add_argument("--ckpt8", action="store_true", help="what the backward needs, kept in 8 bits")
    a = ap.parse_args()
    policy = TinyPolicy(norm=a.norm, ckpt8=a.ckpt8)
    b = rollout(policy, n_seqs=8, length=96, prompt=24)
    for i in range(a.steps):
        stats, losses, counts = step(policy, b)
        s, r = stats.tolist(), losses.tolist()
        print(f"step {i}: loss {s[0]:+.5f} (pg {s[1]:+.5f}, kl {s[2]:.2e}, entropy {s[3]:.3f}, clipped {s[4]:.1%}); "
              f"balance {r[0]:.5f}, z {r[1]:.5f}, busiest expert {int(counts.sum(0).max())} of {int(counts.sum())} slots")
    status = L.check_status(policy.layer.dev_status)
    if status:
        raise SystemExit(f"device status {status:#x}")


if __name__ == "__main__":
    main()
