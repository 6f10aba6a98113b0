"""On-policy distillation with the head's operators, on synthetic rows.

One step is what a trainer does with a student that has a layer norm before its
vocabulary head:

1. serving: the student's logits for one position per request go through the
   sampler's rules (penalties for repeated tokens, a bias, a grammar mask); a
   token is drawn, and its log-prob under the processed distribution is kept;
2. the teacher's top logits for the drawn positions are collected;
3. training: layer norm -> distillation through the head (the [T, V] logits never
   exist) -> gradients of the rows, the norm and the table, the table's summed in
   fp32 across the micro-batches.

    python examples/on_policy_distillation.py [--steps 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import chunked_lm_head_tcgen05_gb300 as lm  # noqa: E402
from chunked_lm_head_tcgen05_gb300 import autograd  # noqa: E402


def sample(student, rows, tokens, spans, allowed, temperature=1.0):
    """One token per request, and its log-prob under the processed distribution."""
    y, _, _ = lm.layernorm_forward(rows, student["norm_w"], student["norm_b"])
    logits = (y @ student["table"].t()).float()
    requests = logits.shape[0]
    ones = torch.ones(requests, device=rows.device)
    processed = lm.process_logits(
        logits, tokens, spans, repetition=1.2 * ones, frequency=0.1 * ones, presence=0.2 * ones,
        bias_offsets=torch.arange(requests + 1, device=rows.device),
        bias_ids=torch.zeros(requests, dtype=torch.int32, device=rows.device),
        bias_values=-2.0 * ones, allowed=allowed, out=logits)
    drawn = torch.multinomial(torch.softmax(processed / temperature, 1), 1)[:, 0].to(torch.int32)
    logp, entropy, lse = (torch.empty(requests, device=rows.device) for _ in range(3))
    status = lm.lmhead_score_logits_fwd(processed, drawn, None, temperature, logp, entropy, lse)
    if status:
        raise lm.LmheadError(status, "lmhead_score_logits_fwd")
    return drawn, logp


def teacher_top(teacher, rows, k):
    """The teacher's k top logits for each row, with its own log-sum-exp."""
    y = torch.nn.functional.layer_norm(rows.float(), rows.shape[1:], teacher["norm_w"].float(),
                                       teacher["norm_b"].float())
    logits = y @ teacher["table"].float().t()
    top = logits.topk(k, 1)
    return top.indices.to(torch.int32), top.values.contiguous(), torch.logsumexp(logits, 1)


def make_model(vocab, width, seed, device):
    g = torch.Generator(device=device).manual_seed(seed)
    return {"norm_w": torch.ones(width, device=device, dtype=torch.bfloat16),
            "norm_b": torch.zeros(width, device=device, dtype=torch.bfloat16),
            "table": (torch.randn(vocab, width, generator=g, device=device)
                      * 2.0 / width ** 0.5).to(torch.bfloat16)}


def main(steps=8, vocab=4096, width=256, requests=64, tokens_per_step=1024, k=32, seed=0,
         device="cuda"):
    """Returns the mean distillation loss of every step."""
    g = torch.Generator(device=device).manual_seed(seed)
    teacher = make_model(vocab, width, seed + 1, device)
    student = make_model(vocab, width, seed + 2, device)
    params = [student[n].requires_grad_(True) for n in ("norm_w", "norm_b")]
    table = student["table"].requires_grad_(True)
    table.main_grad = torch.zeros(vocab, width, device=device)
    master = table.detach().float()
    history = torch.randint(0, vocab, (requests, 48), generator=g, device=device,
                            dtype=torch.int32)
    allowed = torch.randint(-2 ** 31, 2 ** 31, (requests, (vocab + 31) // 32), generator=g,
                            device=device).to(torch.int32)
    begin = torch.arange(requests, device=device) * 48
    spans = torch.stack([begin, begin + 16, begin + 48], 1)
    losses = []
    for _ in range(steps):
        rows = torch.randn(tokens_per_step, width, generator=g, device=device).to(torch.bfloat16)
        with torch.no_grad():
            drawn, logp = sample(student, rows[:requests], history.reshape(-1), spans, allowed)
            assert torch.isfinite(logp).all() and (drawn >= 0).all()
        ids, top, lse = teacher_top(teacher, rows, k)
        mask = torch.ones(tokens_per_step, dtype=torch.uint8, device=device)
        mask[::7] = 0                                   # prompt tokens are not scored
        y = autograd.layer_norm(rows, student["norm_w"], student["norm_b"])
        loss = autograd.lmhead_distill(y, table, ids, top, mask, teacher_lse=lse, chunk_size=256)
        mean = loss.sum() / mask.sum()
        grads = torch.autograd.grad(mean, params + [table], allow_unused=True)
        with torch.no_grad():
            for p, d in zip(params, grads):
                p -= 0.5 * d
            master -= 150.0 * table.main_grad           # the table's gradient came here, in fp32
            table.copy_(master.to(torch.bfloat16))
            table.main_grad.zero_()
        losses.append(float(mean.detach()))
    return losses


if __name__ == "__main__":
    args = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    args.add_argument("--steps", type=int, default=8)
    lm.build()
    for i, value in enumerate(main(args.parse_args().steps)):
        print("step %d: distillation loss %.4f" % (i, value))
