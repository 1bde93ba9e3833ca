"""A policy samples answers and is trained on them: by their rewards, then by pairs of them.

    python examples/train_on_samples.py [--prompts 16] [--length 12] [--updates 3]

The operators of include/ls_token_ops.h as a program uses them, behind the
sampler: answers are sampled, token_log_probs keeps their log-probs under the
sampling policy and under a reference, policy takes some steps on the clipped loss
with a KL term and an entropy bonus (advantages are an answer's reward against the
other answers to its prompt), and preference one more on the best and the worst
answer to each prompt.  The model is the toy model of decode_and_distill.py; an
answer's reward is how many of its ids are even."""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import logits_sampling_gb300 as ls  # noqa: E402
from decode_and_distill import Model  # noqa: E402

GROUP = 4  # answers to a prompt


def rollout(model, vocab, prompts, length):
    """Rows of all answers, one answer after another: what each position was fed, and the id it gave."""
    answers = prompts * GROUP
    gen = torch.Generator(device="cuda").manual_seed(1)
    last = torch.randint(vocab, (prompts,), generator=gen, device="cuda").repeat_interleave(GROUP)
    sampling = ls.SamplingParams.from_host([1.0] * answers, [0] * answers, [1.0] * answers, range(answers))
    fed, ids = [], []
    for step in range(length):
        with torch.no_grad():
            logits = model(last).to(torch.bfloat16)
        new = ls.sample(logits, answers, sampling, step, True, True)
        fed.append(last)
        ids.append(new)
        last = new.long()
    return torch.stack(fed, 1).reshape(-1), torch.stack(ids, 1).reshape(-1)


def batch_of(model, reference, vocab, prompts, length):
    fed, ids = rollout(model, vocab, prompts, length)
    reward = (ids % 2 == 0).float().view(prompts, GROUP, length).sum(2)
    advantage = (reward - reward.mean(1, keepdim=True)) / (reward.std(1, keepdim=True) + 1e-6)
    with torch.no_grad():
        old, _, _ = ls.token_log_probs(model(fed), ids)
        ref, _, _ = ls.token_log_probs(reference(fed), ids)
    best, worst = reward.argmax(1), reward.argmin(1)
    answer = torch.arange(prompts, device="cuda") * GROUP
    order = torch.stack([answer + best, answer + worst], 1).reshape(-1)  # chosen, rejected, chosen, ...
    rows = (order[:, None] * length + torch.arange(length, device="cuda")).reshape(-1)
    return {"fed": fed, "ids": ids, "old": old, "ref": ref, "advantages": advantage.reshape(-1).repeat_interleave(length),
            "weights": torch.full((len(ids),), 1.0 / len(ids), device="cuda"), "pair_rows": rows,
            "offsets": (torch.arange(2 * prompts + 1, device="cuda") * length).to(torch.int32)}


def policy_loss(model, batch):
    loss, metrics = ls.policy(model(batch["fed"]), batch["ids"], batch["advantages"], old_log_probs=batch["old"],
                              ref_log_probs=batch["ref"], weights=batch["weights"], clip_low=0.2, clip_high=0.28,
                              kl_coef=0.02, entropy_coef=0.01)
    return loss.sum(), metrics


def preference_loss(model, batch):
    rows = batch["pair_rows"]
    loss, _ = ls.preference(model(batch["fed"][rows]), batch["ids"][rows], batch["offsets"],
                            ref_log_probs=batch["ref"][rows], beta=0.1, label_smoothing=0.05)
    return loss.mean()


def main(argv=None):
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--prompts", type=int, default=16)
    parser.add_argument("--length", type=int, default=12)
    parser.add_argument("--updates", type=int, default=3)
    parser.add_argument("--vocab", type=int, default=32000)
    args = parser.parse_args(argv)
    model, reference = (Model(args.vocab, 64, seed=0).cuda() for _ in range(2))
    batch = batch_of(model, reference, args.vocab, args.prompts, args.length)
    optimizer = torch.optim.Adam(model.parameters(), lr=1e-3)
    for _ in range(args.updates):
        optimizer.zero_grad()
        loss, metrics = policy_loss(model, batch)
        loss.backward()
        optimizer.step()
        means = dict(zip(ls.POLICY_METRICS, metrics.mean(0).tolist()))
        print(f"policy loss {float(loss.detach()):.5f}  " + "  ".join(f"{k} {v:.4f}" for k, v in means.items()))
    optimizer.zero_grad()
    loss = preference_loss(model, batch)
    loss.backward()
    optimizer.step()
    print(f"preference loss {float(loss.detach()):.5f} over {args.prompts} pairs")
    return model, batch


if __name__ == "__main__":
    main()
