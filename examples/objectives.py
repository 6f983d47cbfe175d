"""The training objectives together, on a toy retriever and a toy answer model.

  python examples/objectives.py [steps]

A retriever scores 17 candidate documents per query with MaxSim and is
distilled from a teacher's scores of the 16 best.  A language model with a
vocabulary of 32000 first learns from a larger model's top tokens, then from
pairs of answers, then from rewards of tokens it sampled.  All data is random;
each stage prints its loss before and after.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from late_interaction_retrieval_gb300 import layers  # noqa: E402

VOCAB = 32000


class Answerer(torch.nn.Module):
    """Token embedding, one layer, logits over the vocabulary: enough to have gradients."""

    def __init__(self, dim=64):
        super().__init__()
        self.embed = torch.nn.Embedding(VOCAB, dim)
        self.mix = torch.nn.Linear(dim, dim)
        self.head = torch.nn.Linear(dim, VOCAB, bias=False)

    def forward(self, tokens):
        return self.head(torch.tanh(self.mix(self.embed(tokens))))


def _train(parameters, loss_of, steps, lr):
    optimizer = torch.optim.Adam(parameters, lr=lr)
    losses = []
    for _ in range(steps):
        optimizer.zero_grad()
        loss = loss_of()
        loss.backward()
        optimizer.step()
        losses.append(loss.detach())
    return float(losses[0]), float(losses[-1])


def retriever(steps, gen):
    """Candidate scores [queries, 17] distilled from a teacher that ranked 16 of them."""
    queries, candidates, dim = 64, 17, 64
    project = torch.nn.Linear(dim, dim, bias=False, device="cuda")
    q = torch.randn(queries, 16, dim, generator=gen, device="cuda")
    d = torch.randn(queries, candidates, 48, dim, generator=gen, device="cuda")
    teacher, index = torch.randn(queries, candidates, generator=gen, device="cuda").topk(candidates - 1, dim=1)
    maxsim, objective = layers.MaxSimKD(), layers.DistillTopK(scale=0.2)
    normal = torch.nn.functional.normalize

    def loss():
        return objective(maxsim(normal(project(q), dim=-1), normal(project(d), dim=-1)), index, teacher)

    return _train(project.parameters(), loss, steps, 1e-2)


def learn_from_a_larger_model(model, steps, gen):
    """The larger model's 32 likeliest tokens and its log-sum-exp, so that its probabilities are the true ones
    (and the loss, a sum over those tokens alone, may go below zero)."""
    tokens = torch.randint(0, VOCAB, (4, 32), generator=gen, device="cuda")
    larger = torch.randn(4, 32, VOCAB, generator=gen, device="cuda") * 2.0
    top, index = larger.topk(32, dim=-1)
    lse = torch.logsumexp(larger, dim=-1)
    objective = layers.DistillTopK()
    return _train(model.parameters(), lambda: objective(model(tokens).bfloat16(), index, top, lse), steps, 1e-2)


def learn_from_pairs(model, steps, gen):
    """Four pairs of answers of different lengths, packed: chosen ones first, prompt tokens (-100) not counted."""
    lengths = torch.tensor([9, 12, 7, 16, 11, 8, 13, 10])
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)]).to(torch.int32).cuda()
    rows = int(lengths.sum())
    tokens = torch.randint(0, VOCAB, (rows,), generator=gen, device="cuda")
    target = torch.randint(0, VOCAB, (rows,), generator=gen, device="cuda")
    target[offsets[:-1].long()] = -100
    with torch.no_grad():  # the reference model is the one training starts from
        reference = layers.preference_loss(model(tokens), target, offsets, return_rows=True)[2].clone()
    objective = layers.PreferenceLoss(beta=0.1)
    return _train(model.parameters(), lambda: objective(model(tokens), target, offsets, reference), steps, 1e-3)


def learn_from_rewards(model, steps, gen):
    """Tokens sampled once, rewarded at random; the KL term holds the model near the one that sampled."""
    tokens = torch.randint(0, VOCAB, (8, 24), generator=gen, device="cuda")
    with torch.no_grad():
        old = torch.log_softmax(model(tokens).float(), dim=-1)
        sampled = torch.multinomial(old.view(-1, VOCAB).exp(), 1, generator=gen).view(8, 24)
        old = old.gather(2, sampled[..., None])[..., 0]
    advantage = torch.randn(8, 24, generator=gen, device="cuda")
    objective = layers.PolicyLoss(kl_coef=0.02)
    return _train(model.parameters(), lambda: objective(model(tokens), sampled, old, advantage, old), steps, 1e-4)


def main(steps=30):
    gen = torch.Generator(device="cuda").manual_seed(0)
    torch.manual_seed(0)
    model = Answerer().cuda()
    result = {"retriever, from a teacher's scores": retriever(steps, gen)}
    for stage, run in (("answers, from a larger model", learn_from_a_larger_model),
                       ("answers, from pairs", learn_from_pairs), ("answers, from rewards", learn_from_rewards)):
        result[stage] = run(model, steps, gen)
    return result


if __name__ == "__main__":
    for stage, (before, after) in main(int(sys.argv[1]) if len(sys.argv) > 1 else 30).items():
        print(f"{stage:36s} loss {before:9.4f} -> {after:9.4f}")
