"""Trains a dense student on the exact top-k lists and serves it in 8 bits.

    python examples/distill_student.py [--steps N]

The teacher is the exact scorer: the k items of largest cosine of every query
(``topk_all``).  The student sees dense features of a query's sparse row (a
fixed random projection), passes them through one block

    h = gelu(norm(x) W1^T + b1) + x,   logits = norm(h) V^T

with a learned vector in V for every item, and learns to give the teacher's
lists.  All of its arithmetic runs in the handle's dense operators: the norms,
linear layers and the distillation loss with their gradients.  Serving takes
one query at a time: the last norm writes 8-bit values with a scale, the items'
vectors are kept in 8 bits.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_embedding_exact_gb300 as sec  # noqa: E402
from workload import CONFIGS, generate_rows  # noqa: E402

WIDTH, K = 256, 10
TEACHER_TEMPERATURE = 0.1


def features(batch, seed: int = 0) -> torch.Tensor:
    """The rows' dense features: x V with a fixed random V, normalised."""
    rows = torch.repeat_interleave(torch.arange(batch.n_rows), torch.from_numpy(batch.indptr[1:] - batch.indptr[:-1]))
    g = torch.Generator().manual_seed(seed)
    table = torch.randn(batch.dim, WIDTH, generator=g)
    values = torch.from_numpy(batch.values)[:, None] * table[torch.from_numpy(batch.indices).long()]
    x = torch.zeros(batch.n_rows, WIDTH).index_add_(0, rows, values)
    return (x / x.pow(2).mean(1, keepdim=True).sqrt()).to(torch.bfloat16)


def train(steps: int = 200, n_q: int = 512, n_i: int = 10_000, rate: float = 0.01, device: int = 0):
    """(losses, share of the teacher's best items among the served student's
    ten best before training, the same after)."""
    dev = torch.device("cuda", device)
    cfg = CONFIGS["d65k_q1k_i10k"]
    queries, items = generate_rows(cfg, 0, 0, n_q), generate_rows(cfg, 1, 0, n_i)
    with sec.SparseCosine(cfg.dim, device=device) as h:
        q, i = sec.DeviceCsr.from_host(queries, dev), sec.DeviceCsr.from_host(items, dev)
        scores, best = h.topk_all(q, h.row_norms(q), i, h.row_norms(i), K)
        x = features(queries).to(dev)
        g = torch.Generator(device=dev).manual_seed(1)
        bf = torch.bfloat16
        # float32 weights, of which the layers take 16-bit copies
        p = {"g1": torch.ones(WIDTH, device=dev), "g2": torch.ones(WIDTH, device=dev),
             "w1": torch.randn(WIDTH, WIDTH, device=dev, generator=g) * WIDTH ** -0.5, "b1": torch.zeros(WIDTH, device=dev),
             "v": torch.randn(n_i, WIDTH, device=dev, generator=g) * WIDTH ** -0.5}
        m1, m2 = ({k: torch.zeros_like(v) for k, v in p.items()} for _ in range(2))
        mean = torch.full((n_q,), 1.0 / n_q, device=dev)

        def update(name: str, grad: torch.Tensor, step: int) -> None:
            """One step of Adam."""
            m1[name].lerp_(grad, 0.1)
            m2[name].lerp_(grad * grad, 0.01)
            p[name] -= rate * (m1[name] / (1 - 0.9 ** step)) / ((m2[name] / (1 - 0.99 ** step)).sqrt() + 1e-12)

        def serve() -> float:
            """One query at a time, the last layer in 8 bits."""
            scale = p["v"].abs().amax(1) / 448
            v8 = (p["v"] / scale[:, None]).to(torch.float8_e4m3fn)
            w1, hits = p["w1"].to(bf), 0
            for r in range(0, n_q, 8):
                y, _, _ = h.rms_norm(x[r : r + 1], p["g1"])
                a = h.linear(y, w1, bias=p["b1"], activation="gelu")
                y8, s8, _ = h.rms_norm_quantized(a, p["g2"], residual=x[r : r + 1])
                logits = h.linear(y8, v8, x_scale=s8, w_scale=scale, out_dtype=torch.float32)
                hits += int((logits.topk(K, dim=1).indices == best[r, 0]).any())
            return hits / len(range(0, n_q, 8))

        before, losses = serve(), []
        for step in range(1, steps + 1):
            w1, v = p["w1"].to(bf), p["v"].to(bf)
            y1, _, r1 = h.rms_norm(x, p["g1"])
            a, pre = h.linear(y1, w1, bias=p["b1"], activation="gelu", save_pre=True)
            y2, t2, r2 = h.rms_norm(a, p["g2"], residual=x)
            logits = h.linear(y2, v)
            loss, grad = h.distill_step(logits, scores, best, mean, teacher_temperature=TEACHER_TEMPERATURE, in_place=True)
            losses.append(loss.mean())
            gy2, gv, _ = h.linear_backward(grad, y2, v, grad_dtype=torch.float32)
            ga, gg2 = h.rms_norm_backward(gy2.to(bf), t2, p["g2"], r2)
            gy1, gw1, gb1 = h.linear_backward(ga, y1, w1, pre, "gelu", grad_dtype=torch.float32)
            _, gg1 = h.rms_norm_backward(gy1.to(bf), x, p["g1"], r1)
            for name, grad_p in (("g1", gg1), ("g2", gg2), ("w1", gw1), ("b1", gb1), ("v", gv)):
                update(name, grad_p, step)
        h.check_device()
        return torch.stack(losses).tolist(), before, serve()


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    args = ap.parse_args()
    losses, before, after = train(args.steps)
    for k in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {k:4d}  loss {losses[k]:.4f}")
    print(f"step {len(losses) - 1:4d}  loss {losses[-1]:.4f}")
    print(f"teacher's best item among the served student's ten best: {before:.1%} before, {after:.1%} after")


if __name__ == "__main__":
    main()
