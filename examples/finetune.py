"""Fine-tunes a small bf16 language model with this library end to end: answers
are sampled from the model, their log-probabilities scored, and the model is
updated either on a reward (clipped policy loss with a KL term to the starting
model) or on pairs (preference loss).  Between the model's logits and its new
parameters everything runs in the library:

    policy:      logits -> policy_loss_logits -> logits' gradient
    preference:  logits -> token_logprob -> preference_loss -> logits' gradient
    both:        model's backward -> GlobalClip over both groups -> AnyPrecisionAdamW

    python examples/finetune.py policy --steps 30
    python examples/finetune.py preference --steps 30

The reward prefers tokens of the lower half of the vocabulary; it stands in
for a reward model.  Weights are random.
"""
import argparse
import copy
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from adamw_optimizer_step_sm_gb300 import losses as L
from adamw_optimizer_step_sm_gb300.optim import AnyPrecisionAdamW, GlobalClip

VOCAB, WIDTH, HEADS, LAYERS, PROMPT, ANSWER = 1003, 128, 4, 2, 8, 24


class Block(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.norm1, self.norm2 = torch.nn.LayerNorm(WIDTH), torch.nn.LayerNorm(WIDTH)
        self.qkv, self.out = torch.nn.Linear(WIDTH, 3 * WIDTH), torch.nn.Linear(WIDTH, WIDTH)
        self.up, self.down = torch.nn.Linear(WIDTH, 4 * WIDTH), torch.nn.Linear(4 * WIDTH, WIDTH)

    def forward(self, x):
        b, t, _ = x.shape
        q, k, v = self.qkv(self.norm1(x)).view(b, t, 3, HEADS, WIDTH // HEADS).permute(2, 0, 3, 1, 4)
        scores = (q @ k.transpose(-1, -2)) * (WIDTH // HEADS) ** -0.5
        future = torch.ones(t, t, dtype=torch.bool, device=x.device).triu(1)
        a = torch.softmax(scores.masked_fill(future, float("-inf")), -1) @ v
        x = x + self.out(a.transpose(1, 2).reshape(b, t, WIDTH))
        return x + self.down(F.relu(self.up(self.norm2(x))))


class Model(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.tokens = torch.nn.Embedding(VOCAB, WIDTH)
        self.places = torch.nn.Embedding(PROMPT + ANSWER, WIDTH)
        self.blocks = torch.nn.ModuleList(Block() for _ in range(LAYERS))
        self.norm = torch.nn.LayerNorm(WIDTH)
        for p in self.parameters():
            if p.dim() > 1:
                torch.nn.init.normal_(p, 0.0, 0.02)

    def forward(self, ids):
        x = self.tokens(ids) + self.places.weight[: ids.shape[1]]
        for b in self.blocks:
            x = b(x)
        return self.norm(x) @ self.tokens.weight.t()


@torch.no_grad()
def answer(model, prompts, temperature):
    ids = prompts
    for _ in range(ANSWER):
        logits = model(ids)[:, -1].float() / temperature
        ids = torch.cat([ids, torch.multinomial(torch.softmax(logits, -1), 1)], 1)
    return ids


def reward_of(ids):
    return (ids[:, PROMPT:] < VOCAB // 2).float().mean(1)


def answer_targets(ids):
    """Each token's successor, for the answer's tokens only."""
    targets = ids[:, 1:].clone()
    targets[:, : PROMPT - 1] = -100
    return targets


def train(kind="policy", steps=30, answers=32, lr=1e-3, seed=0, say=print):
    torch.manual_seed(seed)
    model = Model().cuda().bfloat16()
    frozen = copy.deepcopy(model).requires_grad_(False)
    params = list(model.parameters())
    opt = AnyPrecisionAdamW([{"params": [p for p in params if p.dim() > 1]},
                             {"params": [p for p in params if p.dim() == 1], "weight_decay": 0.0}],
                            lr=lr, weight_decay=0.01)
    clip = GlobalClip(opt)
    history = []
    for step in range(steps):
        prompts = torch.randint(0, VOCAB, (answers, PROMPT), device="cuda")
        ids = answer(model, prompts, 1.0)
        reward = reward_of(ids)
        if kind == "preference":   # the better answers of the batch over the worse ones
            order = reward.argsort(descending=True, stable=True)
            ids = ids[order]
        targets = answer_targets(ids)
        with torch.no_grad():
            old = L.token_logprob(model(ids)[:, :-1], targets).logp
            ref = L.token_logprob(frozen(ids)[:, :-1], targets).logp
        opt.zero_grad()
        logits = model(ids)
        if kind == "policy":
            advantages = (reward - reward.mean()) / (reward.std() + 1e-6)
            r = L.policy_loss_logits(logits[:, :-1], targets, old, advantages, ref_logp=ref, kl_coef=0.02,
                                     entropy_coef=0.001, clip_high=0.28, reduce="sequence")
            logits[:, :-1].backward(r.d_logits)
            entry = {"loss": r.stats[0], "kl": r.stats[2], "tokens": r.counts[0]}
        else:
            t = L.token_logprob(logits[:, :-1], targets)
            p = L.preference_loss(t.logp, ref, mask=targets != -100, beta=0.1)
            t.logp.backward(p.d_logp)
            entry = {"loss": p.stats[0], "right": p.stats[1]}
        norm = clip(1.0).norm.clone()
        opt.step()
        entry = {k: float(v) for k, v in dict(entry, reward=reward.mean(), norm=norm).items()}
        history.append(entry)
        say("step %3d  " % step + "  ".join("%s %.4f" % kv for kv in entry.items()))
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("kind", nargs="?", default="policy", choices=["policy", "preference"])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--answers", type=int, default=32)
    ap.add_argument("--lr", type=float, default=1e-3)
    a = ap.parse_args()
    train(a.kind, a.steps, a.answers, a.lr)
