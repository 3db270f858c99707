"""Distils a one-block language model into a narrower one, on one GPU.

Teacher and student are the same kind of model: token embedding (times a
factor), a gated block with a residual, logits through the student's own
embedding table (tied head), its vocabulary split over T logical shards. Each
step:

  teacher  vocab_logprobs     its top K tokens and their log probabilities
  student  vocab_embedding_scaled, swiglu_forward, head product
           vocab_distill_with_grad   loss and dlogits, in place
           head's gradients, swiglu_backward,
           vocab_embedding_backward  added to the head's part of the table gradient
           a step of gradient descent

and at the end vocab_logprobs scores the teacher's answers under the student. The head's
products are plain matrix products (torch.matmul); everything else is the
library's kernels.

    python examples/distill_gated_block.py [--steps 60] [--tokens 512]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tensor_transformer_mlp_columnparallel_gb300 as tp  # noqa: E402


class BlockLM:
    """embed -> x + gated(x) -> tied head, bf16."""

    def __init__(self, V, D, F, T, seed, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.V, self.D, self.F, self.T = V, D, F, T
        self.scale = 4.0

        def normal(r, c, std):
            return (torch.randn((r, c), generator=g, device=device) * std).to(torch.bfloat16)

        self.E = normal(V, D, D ** -0.5)
        Fs = F // T
        self.Wg = [normal(D, Fs, D ** -0.5) for _ in range(T)]
        self.Wu = [normal(D, Fs, D ** -0.5) for _ in range(T)]
        self.Wd = [normal(Fs, D, 3.0 * F ** -0.5) for _ in range(T)]

    def shards(self):
        return list(self.E.view(self.T, self.V // self.T, self.D))

    def forward(self, ids):
        x = tp.vocab_embedding_scaled(ids, self.shards(), self.scale)
        y, H, G, U = tp.swiglu_forward(x, self.Wg, self.Wu, self.Wd, save_gate_up=True)
        h = x + y
        return h @ self.E.t(), (ids, x, h, H, G, U)

    def backward(self, dlogits, saved):
        """Gradients (dE fp32, dWg, dWu, dWd) for the upstream dlogits."""
        ids, x, h, H, G, U = saved
        dh = dlogits @ self.E
        dE = (dlogits.t() @ h).float()                                  # the head's part
        dx, dWg, dWu, dWd = tp.swiglu_backward(x, self.Wg, self.Wu, self.Wd, H, G, U, dh)
        dx += dh                                                        # the residual
        tp.vocab_embedding_backward(ids, dx, self.V, self.T, scale=self.scale,
                                    accumulate_into=list(dE.view(self.T, self.V // self.T, self.D)))
        return dE, dWg, dWu, dWd

    def descend(self, grads, rate):
        """Steps of `rate` times each tensor's own size, along its gradient."""
        dE, dWg, dWu, dWd = grads
        for w, d in zip([self.E, *self.Wg, *self.Wu, *self.Wd], [dE, *dWg, *dWu, *dWd]):
            step = rate * w.float().norm() / (d.float().norm() + 1e-12)
            w -= (step * d.float()).to(w.dtype)


def distil(steps=60, tokens=512, V=4096, D=256, F=1024, T=4, K=32, tau=1.5, rate=0.05, seed=0):
    """Returns (loss of each step, and before and after: mean log probability and
    median rank of the teacher's most likely tokens under the student, and the
    student's mean entropy)."""
    teacher, student = BlockLM(V, 2 * D, 2 * F, T, seed + 1), BlockLM(V, D, F, T, seed + 2)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def batch():
        return torch.randint(0, V, (tokens,), generator=g, device="cuda")

    ids_held = batch()
    _, _, _, best, _ = tp.vocab_logprobs(teacher.forward(ids_held)[0], ids_held, T, top_k=1)
    answers = best[:, 0].long()

    def score():
        lp, rank, entropy, _, _ = tp.vocab_logprobs(student.forward(ids_held)[0], answers, T)
        return float(lp.mean()), float(rank.float().median()), float(entropy.mean())

    before, losses = score(), []
    for i in range(steps):
        ids = batch()
        z_teacher, _ = teacher.forward(ids)
        _, _, _, top, top_lp = tp.vocab_logprobs(z_teacher, ids, T, top_k=K)
        logits, saved = student.forward(ids)
        _, mean, _, dlogits = tp.vocab_distill_with_grad(logits, top, top_lp, T, temperature=tau,
                                                         grad_scale=1.0 / tokens, in_place=True)
        student.descend(student.backward(dlogits, saved), rate * (1 - i / steps))
        losses.append(mean)
    after = score()
    assert tp.tpmlp_check_device_error() == 0
    return [float(x) for x in losses], before, after


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args()
    losses, before, after = distil(steps=a.steps, tokens=a.tokens)
    print(f"distillation loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    for name, (lp, rank, ent) in (("before", before), ("after", after)):
        print(f"teacher's answers, {name}: log probability {lp:.3f}, median rank {rank:.0f}, entropy {ent:.3f}")
