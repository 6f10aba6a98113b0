"""Beam search of several requests, each with its own low-rank adapter, on synthetic weights.

One step is what a decoder does at its two ends, around whatever model lies between:

1. the last token of every beam goes in through the vocabulary table (``embedding_forward``,
   scaled) and joins the beam's state;
2. layer norm and the head's logits, to which each request's adapter adds its share in place
   (``adapters_forward``);
3. the sampler's penalties (``process_logits``);
4. the best continuations of each request's beams (``beam_select``), and the states moved to the
   beams that go on (``beam_reorder``): cache and token histories in place.

    python examples/beam_search_adapters.py [--steps 12]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import chunked_lm_head_tcgen05_gb300 as lm  # noqa: E402

EOS = 1


def make_model(vocab, width, adapters, rank, seed, device):
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=device)

    return {"table": (normal(vocab, width) / width ** 0.5).to(torch.bfloat16),
            "norm_w": torch.ones(width, device=device, dtype=torch.bfloat16),
            "norm_b": torch.zeros(width, device=device, dtype=torch.bfloat16),
            "down": (normal(adapters, rank, width) / width ** 0.5).to(torch.bfloat16),
            "up": normal(adapters, rank, vocab).to(torch.bfloat16),
            "scale": torch.full((adapters,), 0.5, device=device)}


def decode(model, first, adapter_of, beams=4, steps=12, penalty=1.1, trace=None):
    """Histories [R, steps + 1] and scores [requests, beams] of the best sequences that begin with
    first [requests]; row r = request * beams + beam.  trace: a list that gets every step's tensors."""
    device, requests = first.device, first.shape[0]
    rows, (vocab, width) = requests * beams, model["table"].shape
    table = model["table"].float()
    history = torch.zeros(rows, steps + 1, dtype=torch.int32, device=device)
    history[:, 0] = first.repeat_interleave(beams)
    cache = torch.zeros(rows, steps, width, dtype=torch.bfloat16, device=device)
    scores = torch.full((requests, beams), -float("inf"), device=device)
    scores[:, 0] = 0.0                       # all beams of a request begin as one
    finished = torch.zeros(requests, beams, dtype=torch.uint8, device=device)
    penalties = torch.full((rows,), penalty, device=device)
    adapters = adapter_of.repeat_interleave(beams).contiguous()
    begin = torch.arange(rows, device=device) * (steps + 1)
    for step in range(steps):
        cache[:, step] = lm.embedding_forward(history[:, step].contiguous(), model["table"],
                                              width ** 0.5)
        hidden = cache[:, :step + 1].float().mean(1).to(torch.bfloat16)    # the model between
        y, _, _ = lm.layernorm_forward(hidden, model["norm_w"], model["norm_b"])
        logits = y.float() @ table.t()
        lm.adapters_forward(logits, y, model["down"], model["up"], adapters, model["scale"],
                            out=logits)
        spans = torch.stack([begin, begin, begin + step + 1], 1)
        lm.process_logits(logits, history.view(-1), spans, repetition=penalties, out=logits)
        after = torch.empty_like(finished)
        old = scores
        scores, parents, tokens, _ = lm.beam_select(logits, scores.view(-1), beams,
                                                    finished=finished.view(-1), eos_id=EOS,
                                                    next_finished=after)
        before = history.clone() if trace is not None else None
        lm.beam_reorder(history, parents.view(-1), 0, history, beams)
        used = cache[:, :step + 1]
        lm.beam_reorder(used, parents.view(-1), 0, used, beams)
        history[:, step + 1] = tokens.view(-1)
        if trace is not None:
            trace.append(dict(hidden=hidden, y=y, logits=logits, old=old, finished=finished,
                              scores=scores, parents=parents, tokens=tokens, before=before,
                              after=after, history=history.clone(), cache=used.clone()))
        finished = after
    return history, scores


def main(steps=12, vocab=4096, width=256, requests=6, beams=4, adapters=3, rank=8, seed=0,
         device="cuda", trace=None):
    model = make_model(vocab, width, adapters, rank, seed, device)
    g = torch.Generator(device=device).manual_seed(seed + 1)
    first = torch.randint(2, vocab, (requests,), generator=g, device=device).to(torch.int32)
    adapter_of = (torch.arange(requests, device=device) % (adapters + 1) - 1).to(torch.int32)
    history, scores = decode(model, first, adapter_of, beams, steps, trace=trace)
    return model, adapter_of, history, scores


if __name__ == "__main__":
    args = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    args.add_argument("--steps", type=int, default=12)
    lm.build()
    _, _, sequences, totals = main(args.parse_args().steps)
    for request in range(totals.shape[0]):
        print("request %d: %.3f %s" % (request, float(totals[request, 0]),
                                       sequences[request * totals.shape[1]].tolist()))
