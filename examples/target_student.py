"""Trains the dense student on one chosen item a query, without its logits and
with its activations kept in 8 bits.

    python examples/target_student.py [--steps N]

Here nothing gives lists of scores: a query comes with the item that was chosen
(stood in for by the exact scorer's best).  The student is the one of
distill_student.py,

    h = gelu(norm(x) W1^T + b1) + x,   logits = norm(h) V^T + log-popularity

trained by the cross entropy of the chosen items over all of them.  The logits
are never held (``cross_entropy_step`` works in pieces of the items), and what
the gradients need of the forward pass is kept as e4m3 codes with a power of two
for every 32 values: the norms' sums, the layers' inputs and the pre-activation.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_embedding_exact_gb300 as sec  # noqa: E402
from examples.distill_student import WIDTH, features  # noqa: E402
from workload import CONFIGS, generate_rows  # noqa: E402

BF16 = torch.bfloat16


def forward_backward(h: sec.SparseCosine, p: dict, x: torch.Tensor, chosen: torch.Tensor, popularity: torch.Tensor,
                     mean: torch.Tensor, keep: bool = True):
    """(losses, {name: gradient}); keep: activations in 8 bits, else in 16."""
    w1, v = p["w1"].to(BF16), p["v"].to(BF16)
    pack = h.compress if keep else (lambda t: (t, None))
    y1, t1, r1 = h.rms_norm(x, p["g1"])
    if keep:
        a, pre, pre_scale = h.linear(y1, w1, bias=p["b1"], activation="gelu", compress_pre=True)
    else:
        (a, pre), pre_scale = h.linear(y1, w1, bias=p["b1"], activation="gelu", save_pre=True), None
    (y1, y1_scale), (t1, t1_scale) = pack(y1), pack(t1)
    y2, t2, r2 = h.rms_norm(a, p["g2"], residual=x)
    t2, t2_scale = pack(t2)
    losses, gy2, gv, _ = h.cross_entropy_step(y2, v, chosen, mean, bias=popularity)
    ga, gg2 = h.rms_norm_backward(gy2, t2, p["g2"], r2, total_scale=t2_scale)
    gy1, gw1, gb1 = h.linear_backward(ga, y1, w1, pre, "gelu", x_scale=y1_scale, pre_scale=pre_scale)
    _, gg1 = h.rms_norm_backward(gy1, t1, p["g1"], r1, total_scale=t1_scale)
    return losses, {"g1": gg1, "g2": gg2, "w1": gw1.float(), "b1": gb1, "v": gv.float()}


def start(n_i: int, dev: torch.device) -> dict:
    g = torch.Generator(device=dev).manual_seed(1)
    return {"g1": torch.ones(WIDTH, device=dev), "g2": torch.ones(WIDTH, device=dev),
            "w1": torch.randn(WIDTH, WIDTH, device=dev, generator=g) * WIDTH ** -0.5, "b1": torch.zeros(WIDTH, device=dev),
            "v": torch.randn(n_i, WIDTH, device=dev, generator=g) * WIDTH ** -0.5}


def chosen_items(h: sec.SparseCosine, n_q: int, n_i: int, dev: torch.device):
    """(features of the queries, the item of each, every item's log-popularity)."""
    cfg = CONFIGS["d65k_q1k_i10k"]
    queries, items = generate_rows(cfg, 0, 0, n_q), generate_rows(cfg, 1, 0, n_i)
    q, i = sec.DeviceCsr.from_host(queries, dev), sec.DeviceCsr.from_host(items, dev)
    _, best = h.topk_all(q, h.row_norms(q), i, h.row_norms(i), 1)
    chosen = best[:, 0].clone()
    popularity = torch.log(torch.bincount(chosen.clamp_min(0), minlength=n_i).float() + 1)
    return features(queries).to(dev), chosen, popularity


def train(steps: int = 200, n_q: int = 512, n_i: int = 10_000, rate: float = 0.01, device: int = 0):
    dev = torch.device("cuda", device)
    with sec.SparseCosine(CONFIGS["d65k_q1k_i10k"].dim, device=device) as h:
        x, chosen, popularity = chosen_items(h, n_q, n_i, dev)
        p, mean = start(n_i, dev), torch.full((n_q,), 1.0 / n_q, device=dev)
        m1, m2 = ({k: torch.zeros_like(v) for k, v in p.items()} for _ in range(2))
        losses = []
        for step in range(1, steps + 1):
            loss, grads = forward_backward(h, p, x, chosen, popularity, mean)
            losses.append(loss.mean())
            for name, grad in grads.items():  # Adam
                m1[name].lerp_(grad, 0.1)
                m2[name].lerp_(grad * grad, 0.01)
                p[name] -= rate * (m1[name] / (1 - 0.9 ** step)) / ((m2[name] / (1 - 0.99 ** step)).sqrt() + 1e-12)
        h.check_device()
        return torch.stack(losses).tolist()


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    args = ap.parse_args()
    losses = train(args.steps)
    for k in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {k:4d}  loss {losses[k]:.4f}")
    print(f"step {len(losses) - 1:4d}  loss {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
