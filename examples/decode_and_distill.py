"""A teacher decodes under penalties and a mask, and a student is trained on what it answered.

    python examples/decode_and_distill.py [--requests 32] [--steps 24] [--epochs 40]

The operators of include/ls_row_ops.h as a program uses them, around the sampler:

* each decoding step: process_logits (penalties over the request's history, a
  bias against one id, a mask of allowed ids) -> sample_log_probs -> the ids are
  appended to the histories; top_log_probs of the same logits is what an API
  would return beside each token, and here the student's training target;
* training: distill (loss and gradient of the student's logits) over every
  position that was decoded.

Teacher and student are toy models (an embedding, a hidden layer, an output
projection) with random weights."""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import logits_sampling_gb300 as ls  # noqa: E402


class Model(torch.nn.Module):
    def __init__(self, vocab, width, seed):
        super().__init__()
        torch.manual_seed(seed)
        self.embed = torch.nn.Embedding(vocab, width)
        self.hidden = torch.nn.Linear(width, width)
        self.out = torch.nn.Linear(width, vocab, bias=False)

    def forward(self, ids):
        return self.out(torch.tanh(self.hidden(self.embed(ids)))) * 8.0


def decode(teacher, vocab, requests, steps, top, temperature):
    """Returns the ids that each position was fed, and the teacher's top ids and log-probs there."""
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(1)
    prompt = 4
    tokens = torch.zeros(requests, prompt + steps, dtype=torch.int32, device=dev)
    tokens[:, :prompt] = torch.randint(vocab, (requests, prompt), generator=gen, device=dev, dtype=torch.int32)
    prompt_lens = torch.full((requests,), prompt, dtype=torch.int32, device=dev)
    seq_lens = prompt_lens.clone()
    params = ls.LogitsParams(
        tokens=tokens, prompt_lens=prompt_lens, seq_lens=seq_lens,
        repetition_penalty=torch.full((requests,), 1.1, device=dev),
        presence_penalty=torch.full((requests,), 0.2, device=dev),
        frequency_penalty=torch.full((requests,), 0.1, device=dev),
        bias_offsets=torch.arange(requests + 1, dtype=torch.int32, device=dev),
        bias_ids=torch.zeros(requests, dtype=torch.int32, device=dev),        # id 0, say an end mark:
        bias_values=torch.full((requests,), -torch.inf, device=dev))          # not yet
    mask = torch.full((1, (vocab + 31) // 32), -1, dtype=torch.int32, device=dev)
    mask[0, -1] = 0x0000FFFF                                                  # the last ids are reserved
    mask_index = torch.zeros(requests, dtype=torch.int32, device=dev)
    sampling = ls.SamplingParams.from_host([0.8] * requests, [0] * requests, [0.95] * requests, range(requests))
    fed, top_ids, top_lps = [], [], []
    rows = torch.arange(requests, device=dev)
    for step in range(steps):
        last = tokens[rows, seq_lens.long() - 1].long()
        with torch.no_grad():
            logits = teacher(last).to(torch.bfloat16)
        ids, log_probs, _ = ls.top_log_probs(logits, top, temperature=temperature)
        fed.append(last)
        top_ids.append(ids)
        top_lps.append(log_probs)
        ls.process_logits(logits, requests, params, allowed_mask=mask, mask_index=mask_index, out=logits)
        new, _, _ = ls.sample_log_probs(logits, requests, sampling, step, True, False, want_log_probs=False)
        tokens[rows, seq_lens.long()] = new
        seq_lens += 1
    assert int((tokens[:, prompt:] == 0).sum()) == 0 and int(tokens.min()) >= 0
    return torch.cat(fed), torch.cat(top_ids), torch.cat(top_lps), tokens


def train(student, fed, top_ids, top_lps, epochs, temperature):
    optimizer = torch.optim.Adam(student.parameters(), lr=3e-3)
    losses = []
    for _ in range(epochs):
        optimizer.zero_grad()
        loss = ls.distill(student(fed), top_ids, top_lps, temperature=temperature, tail="bucket").mean()
        loss.backward()
        optimizer.step()
        losses.append(float(loss.detach()))
    return losses


def main(argv=None):
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--requests", type=int, default=32)
    parser.add_argument("--steps", type=int, default=24)
    parser.add_argument("--epochs", type=int, default=40)
    parser.add_argument("--vocab", type=int, default=32000)
    args = parser.parse_args(argv)
    temperature, top = 2.0, 64
    teacher = Model(args.vocab, 64, seed=0).cuda()
    student = Model(args.vocab, 64, seed=1).cuda()
    fed, top_ids, top_lps, tokens = decode(teacher, args.vocab, args.requests, args.steps, top, temperature)
    losses = train(student, fed, top_ids, top_lps, args.epochs, temperature)
    print(f"decoded {args.steps} tokens for {args.requests} requests, e.g. {tokens[0, 4:12].tolist()}")
    print(f"distillation loss over {len(fed)} positions: {losses[0]:.4f} -> {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    main()
