"""Cases that measure the fine-tuning operators: token log-probabilities, the
preference and policy losses with their gradients, and the global gradient
clip.

``own`` false: each operator in its plain form (elementary torch operations in
32 bits, rounded once at the end).  ``own`` true: the calls that a user makes
of ``adamw_optimizer_step_sm_gb300.losses`` and ``.adamw_sm``.  ``exact`` is
the definition in 64 bits, row block by row block or on whole arrays.

Sizes: the vocabulary, the parameter lists and the flat tensor are this
repository's own workloads (OPT-1.3b's 50272 tokens and 388 tensors, the
1,048,576-element list); the rest are generic.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
IGNORE = -100
CLIP_LOW, CLIP_HIGH = 0.2, 0.28
BETA = 0.1


def listed():
    return [
        # log-probabilities of the tokens just sampled, three sequences decoding: latency
        dict(name="logprob_sampled", op="logprob", seqs=3, tokens=1, vocab=50272, dtype="fp32",
             backward=False, entropy=True, shifted=False, pad=0, ignored=0.0, masked=0, temperature=0.7),
        # a frozen reference model's scores of a batch of answers
        dict(name="logprob_reference", op="logprob", seqs=8, tokens=1023, vocab=50272, dtype="bf16",
             backward=False, entropy=False, shifted=True, pad=0, ignored=0.25, masked=0, temperature=1.0),
        # a supervised step: logits shifted by one token, prompts ignored, the whole gradient
        dict(name="logprob_train", op="logprob", seqs=4, tokens=1023, vocab=50272, dtype="bf16",
             backward=True, entropy=False, shifted=True, pad=0, ignored=0.25, masked=0, temperature=1.0),
        # an odd vocabulary in padded rows, some of its entries masked out, with an entropy bonus
        dict(name="logprob_odd", op="logprob", seqs=1, tokens=1021, vocab=32003, dtype="fp16",
             backward=True, entropy=True, shifted=False, pad=5, ignored=0.1, masked=301, temperature=1.3),
        # one small batch of answers
        dict(name="policy_small", op="policy", seqs=8, tokens=1000, packed=False, mask=0.3, ref=True,
             entropy=False, kl="k3", reduce="token", adv_per_token=False, dual=0.0),
        # a large rollout of ragged answers (some empty), per-token advantages
        dict(name="policy_rollout", op="policy", seqs=2048, tokens=2097189, packed=True, mask=0.4, ref=True,
             entropy=True, kl="k3", reduce="sequence", adv_per_token=True, dual=3.0),
        # a micro-batch of one short answer, from logits to their gradient
        dict(name="policy_logits_short", op="policy_logits", seqs=1, tokens=64, vocab=50272, dtype="bf16",
             shifted=True, pad=0, ignored=0.25, ref=True, entropy=False, kl="k3", reduce="token", dual=0.0),
        # the largest: a batch of long answers, from logits to their gradient
        dict(name="policy_logits_long", op="policy_logits", seqs=8, tokens=2047, vocab=50272, dtype="bf16",
             shifted=True, pad=0, ignored=0.25, ref=True, entropy=True, kl="k3", reduce="sequence", dual=0.0),
        # four pairs of short answers
        dict(name="preference_small", op="preference", pairs=4, tokens=2000, packed=False, mask=0.3,
             kind="sigmoid", smoothing=0.1, ref="token", average=False),
        # many pairs of ragged answers
        dict(name="preference_many", op="preference", pairs=1024, tokens=2097143, packed=True, mask=0.4,
             kind="ipo", smoothing=0.0, ref="token", average=True),
        # a flat list of a million accumulated gradients in 37 odd tensors of two types
        dict(name="clip_1m", op="clip", tensors=37, total=1048576, hidden=0, layers=0, vocab=0,
             src="mixed", dst="bf16", norm="l2", clipped=True),
        # OPT-1.3b's whole list, accumulated in fp32, into the bf16 gradients that the optimizer reads
        dict(name="clip_1.3b", op="clip", tensors=0, total=0, hidden=2048, layers=24, vocab=50272,
             src="fp32", dst="bf16", norm="l2", clipped=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["logprob", "policy", "policy_logits", "preference", "clip"])
    if op in ("logprob", "policy_logits"):
        vocab = _log(rng, 300, 160000)
        rows = _log(rng, 1, min(16384, 400_000_000 // vocab))
        seqs = max(1, min(rows, _log(rng, 1, 16)))
        c = dict(op=op, seqs=seqs, tokens=max(1, rows // seqs), vocab=vocab,
                 dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), shifted=rng.random() < 0.5,
                 pad=rng.choice([0, 0, 3, 8]), ignored=round(rng.uniform(0.0, 0.5), 2), entropy=rng.random() < 0.5)
        if op == "logprob":
            return dict(c, backward=rng.random() < 0.6, masked=rng.choice([0, vocab // 50]),
                        temperature=round(rng.uniform(0.5, 1.5), 2))
        return dict(c, ref=rng.random() < 0.7, kl=rng.choice(["k1", "k2", "k3"]),
                    reduce=rng.choice(["token", "sequence", "fixed"]), dual=rng.choice([0.0, 3.0]))
    if op == "policy":
        seqs = _log(rng, 1, 4096)
        return dict(op=op, seqs=seqs, tokens=seqs * _log(rng, 2, 1 + 2_000_000 // seqs), packed=rng.random() < 0.6,
                    mask=round(rng.uniform(0.0, 0.6), 2), ref=rng.random() < 0.7, entropy=rng.random() < 0.5,
                    kl=rng.choice(["k1", "k2", "k3"]), reduce=rng.choice(["token", "sequence", "fixed"]),
                    adv_per_token=rng.random() < 0.5, dual=rng.choice([0.0, 3.0]))
    if op == "preference":
        pairs = _log(rng, 1, 2048)
        ref = rng.choice(["token", "token", "sequence", "none"])
        # without the reference's own tokens the two sums of a pair are large and nearly cancel: answers stay short
        longest = min(32768, 2 + 1_000_000 // pairs) if ref == "token" else min(128, 2 + 1_000_000 // pairs)
        return dict(op=op, pairs=pairs, tokens=2 * pairs * _log(rng, 2, longest),
                    packed=rng.random() < 0.6, mask=round(rng.uniform(0.0, 0.6), 2),
                    kind=rng.choice(["sigmoid", "hinge", "ipo"]), smoothing=0.0,
                    ref=ref, average=rng.random() < 0.5)
    return dict(op=op, tensors=_log(rng, 1, 400), total=_log(rng, 3000, 300_000_000), hidden=0, layers=0, vocab=0,
                src=rng.choice(["bf16", "fp16", "fp32", "mixed"]), dst=rng.choice(["bf16", "fp32"]),
                norm=rng.choice(["l2", "l2", "max"]), clipped=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs --

def _numels(c):
    """The list's tensor sizes: an OPT-shaped model's, or `total` elements in
    `tensors` parts, cut anywhere (a case has the same list whatever the seed)."""
    if c["hidden"]:
        h = c["hidden"]
        layer = [h * h, h] * 4 + [h, h] + [4 * h * h, 4 * h, 4 * h * h, h] + [h, h]
        return [c["vocab"] * h, 2050 * h] + layer * c["layers"] + [h, h]
    rng = random.Random(c["total"] * 1009 + c["tensors"])
    cuts = sorted(rng.randrange(c["total"] + 1) for _ in range(c["tensors"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [c["total"]])]


def _src_types(c, numels):
    """The type of each tensor of the list: mixed lists hold their smaller
    tensors in fp32, the larger ones in bf16."""
    if c["src"] != "mixed":
        return [c["src"]] * len(numels)
    middle = sorted(numels)[len(numels) // 2]
    return ["fp32" if n < middle else "bf16" for n in numels]


def _rows(c):
    return c["seqs"] * c["tokens"]


def _valid(c):
    return _rows(c) - int(round(c["ignored"] * _rows(c)))


def _block_mask(n, share, g):
    """Tokens that count: runs of 16 (prompts, padding and tool output are left out)."""
    on = torch.rand(n // 16 + 1, generator=g, device="cuda") >= share
    return on.repeat_interleave(16)[:n].contiguous()


def _offsets(n, rows, g):
    """Row starts of `n` packed tokens in `rows` rows of random lengths, some of them empty."""
    cuts = torch.randint(0, n + 1, (rows - 1,), generator=g, device="cuda", dtype=torch.int64).sort().values
    ends = torch.tensor([0, n], dtype=torch.int64, device="cuda")
    return torch.cat([ends[:1], cuts, ends[1:]])


def _logit_inputs(c, g):
    s, t, v, dt = c["seqs"], c["tokens"], c["vocab"], DT[c["dtype"]]
    extra = 1 if c["shifted"] else 0
    buf = torch.randn((s, t + extra, v + c["pad"]), generator=g, device="cuda", dtype=dt)
    buf.mul_(2.0)
    logits = buf[:, :t, :v]
    n = s * t
    targets = torch.randint(0, v - c.get("masked", 0), (n,), generator=g, device="cuda", dtype=torch.int64)
    # most tokens are ones that the model expects
    likely = (torch.rand(n, generator=g, device="cuda") < 0.7).to(dt) * 9.0
    at = torch.arange(n, device="cuda")
    logits[at // t, at % t, targets] += likely
    if c.get("masked", 0):  # entries of the vocabulary that are never to be produced
        logits[:, :, v - c["masked"]:] = -math.inf
    out = torch.randperm(n, generator=g, device="cuda")[: n - _valid(c)]
    targets[out] = IGNORE
    return logits, targets.view(s, t)


def _expected_logp(logits, targets):
    """log-probabilities in blocks of rows, to make a policy's earlier ones from."""
    s, t, v = logits.shape
    n = s * t
    out = torch.empty(n, device="cuda")
    flat = targets.reshape(-1).clamp(min=0)
    step = max(1, 100_000_000 // v)
    for a in range(0, n, step):
        at = torch.arange(a, min(n, a + step), device="cuda")
        x = logits[at // t, at % t].float()
        out[a:a + step] = x.gather(1, flat[at, None])[:, 0] - torch.logsumexp(x, 1)
    return out


def prepare(case, seed):
    c, s = case, {"case": case}
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    op = c["op"]
    if op in ("logprob", "policy_logits"):
        s["logits"], s["targets"] = _logit_inputs(c, g)
        n = _rows(c)
        if op == "logprob":
            s["d_logp"] = -torch.rand(c["seqs"], c["tokens"], generator=g, device="cuda") / n
            s["d_entropy"] = -0.01 * torch.rand(c["seqs"], c["tokens"], generator=g, device="cuda") / n if c["entropy"] else None
            return s
        logp = _expected_logp(s["logits"], s["targets"])
        d = torch.randn(n, generator=g, device="cuda") * 0.15
        # no token on the clip's edge, where the last bit of a log-probability decides
        for edge in (math.log1p(-CLIP_LOW), math.log1p(CLIP_HIGH), math.log(3.0)):
            d = torch.where((d - edge).abs() < 1e-3, d + 4e-3, d)
        s["old"] = (logp - d).view(c["seqs"], c["tokens"])
        s["ref"] = (logp + torch.randn(n, generator=g, device="cuda") * 0.2).view(c["seqs"], c["tokens"]) if c["ref"] else None
        s["adv"] = torch.randn(c["seqs"], generator=g, device="cuda") + 0.25
        return s
    if op in ("policy", "preference"):
        rows = c["seqs"] if op == "policy" else 2 * c["pairs"]
        n = c["tokens"]
        shape = (n,) if c["packed"] else (rows, n // rows)
        # on a grid of 2^-12, so that differences are exact and no token is on the clip's edge
        grid = lambda x: (x * 4096).round() / 4096
        logp = -grid(torch.rand(n, generator=g, device="cuda").pow(3) * 8)
        s["logp"] = logp.view(shape)
        s["mask"] = _block_mask(n, c["mask"], g).view(shape) if c["mask"] else None
        s["offsets"] = _offsets(n, rows, g) if c["packed"] else None
        if op == "policy":
            s["old"] = (logp - grid(torch.randn(n, generator=g, device="cuda") * 0.15)).view(shape)
            s["ref"] = (logp + grid(torch.randn(n, generator=g, device="cuda") * 0.2)).view(shape) if c["ref"] else None
            s["entropy"] = (torch.rand(n, generator=g, device="cuda") * 4).view(shape) if c["entropy"] else None
            s["adv"] = (torch.randn(n if c["adv_per_token"] else rows, generator=g, device="cuda") + 0.25)
            if c["adv_per_token"]:
                s["adv"] = s["adv"].view(shape)
        elif c["ref"] == "token":
            s["ref"] = (logp + grid(torch.randn(n, generator=g, device="cuda") * 0.2)).view(shape)
        elif c["ref"] == "sequence":
            s["ref"] = -1.4 * n / rows * torch.rand(rows, generator=g, device="cuda")
        else:
            s["ref"] = None
        return s
    numels = _numels(c)
    types = _src_types(c, numels)
    s["src"], s["dst"], views, outs = [], [], [], []
    place = {}
    for name in sorted(set(types)):
        # flat buffers, each tensor at a 16-byte boundary, as the optimizers lay out their gradients
        at = {}
        end = 0
        for k, (m, t) in enumerate(zip(numels, types)):
            if t == name:
                at[k] = end
                end += -(-m // 8) * 8
        src = torch.zeros(end, dtype=DT[name], device="cuda")
        for k, o in at.items():
            src[o:o + numels[k]].normal_(0.0, 1e-2, generator=g)
        dst = torch.zeros(end, dtype=DT[c["dst"]], device="cuda")
        s["src"].append(src)
        s["dst"].append(dst)
        place.update({k: (src[o:o + numels[k]], dst[o:o + numels[k]]) for k, o in at.items()})
    for k in range(len(numels)):
        views.append(place[k][0])
        outs.append(place[k][1])
    total = sum(numels)
    norm = 1e-2 * math.sqrt(total) if c["norm"] == "l2" else 0.05
    s["max_norm"] = norm / 7 if c["clipped"] else norm * 7
    s["views"], s["outs"] = views, outs
    if own:
        from adamw_optimizer_step_sm_gb300 import adamw_sm as A
        s["plan"] = A.ClipPlan(views, outs)  # a training run builds it once
    return s


# ------------------------------------------------------------- plain forms --

def _plain_logprob(s, c, d_logp=None, d_entropy=None, want_entropy=False, scale=1.0):
    """(logp, entropy, gradient of the logits) of all rows, in 32 bits."""
    t = s["targets"]
    counts = t != IGNORE
    x = s["logits"].float() * scale
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    lp = x - m - torch.log(z)
    at = t.clamp(min=0)[..., None]
    logp = torch.where(counts, lp.gather(-1, at)[..., 0], 0.0)
    p = e / z
    entropy = None
    if want_entropy:
        plp = torch.where(p > 0, p * lp, 0.0)
        entropy = torch.where(counts, -plp.sum(-1), 0.0)
    grad = lambda dl, dh: _plain_logits_grad(s, p, plp if want_entropy and dh is not None else None, entropy, at, counts, dl, dh, scale)
    return logp, entropy, grad


def _plain_logits_grad(s, p, plp, entropy, at, counts, d_logp, d_entropy, scale):
    dl = torch.where(counts, d_logp, 0.0)[..., None]
    g = p * -dl
    g.scatter_add_(-1, at, dl)
    if plp is not None:
        g = g - torch.where(counts, d_entropy, 0.0)[..., None] * (plp + p * entropy[..., None])
    return (g * scale).to(s["logits"].dtype)


def _row_of(n, offsets, rows):
    at = torch.arange(n, device="cuda")
    return torch.searchsorted(offsets, at, right=True) - 1 if offsets is not None else at // (n // rows)


def _per_row(values, row, rows, packed):
    """Sums by row; of packed rows in two levels (runs of 256 tokens first),
    so that a long row's 32-bit sum keeps its last digits."""
    if not packed:
        return values.view(rows, -1).sum(1)
    run = row + torch.arange(values.numel(), device="cuda") // 256
    runs = rows + values.numel() // 256 + 1
    row_of_run = torch.zeros(runs, dtype=torch.int64, device="cuda").index_put_((run,), row)
    part = torch.zeros(runs, device="cuda").index_add_(0, run, values)
    return torch.zeros(rows, device="cuda").index_add_(0, row_of_run, part)


def _plain_policy(c, logp, old, ref, adv, entropy, mask, offsets, rows, kl_coef, entropy_coef):
    """(stats, counts, d_logp, d_entropy) of flat tokens, in 32 bits."""
    n = logp.numel()
    row = _row_of(n, offsets, rows)
    a = adv if adv.numel() == n and adv.numel() != rows else adv[row]
    on = mask if mask is not None else torch.ones(n, dtype=torch.bool, device="cuda")
    f = on.float()
    per_row = _per_row(f, row, rows, offsets is not None)
    tokens, filled = per_row.sum(), (per_row > 0).float().sum()
    if c["reduce"] == "token":
        w = f / tokens.clamp(min=1)
    elif c["reduce"] == "sequence":
        w = f / (per_row.clamp(min=1)[row] * filled.clamp(min=1))
    else:
        w = f / float(n)
    d = logp - old
    r = torch.exp(d)
    low, high = math.log1p(-CLIP_LOW), math.log1p(CLIP_HIGH)
    rc = torch.where(d > high, 1 + CLIP_HIGH, torch.where(d < low, 1 - CLIP_LOW, r))
    pg = torch.maximum(-a * r, -a * rc)
    off = ((a > 0) & (d > high)) | ((a < 0) & (d < low))
    if c["dual"]:
        capped = (a < 0) & (d > math.log(c["dual"]))
        pg = torch.where(capped, -a * c["dual"], pg)
        off = off | capped
    g = torch.where(off, 0.0, -a * r)
    zero = torch.zeros((), device="cuda")
    kl = zero
    if ref is not None:
        k = logp - ref
        if c["kl"] == "k1":
            kl, dk = k, torch.ones_like(k)
        elif c["kl"] == "k2":
            kl, dk = 0.5 * k * k, k
        else:
            kl, dk = torch.expm1(-k) + k, -torch.expm1(-k)
        g = g + kl_coef * dk
    mean = lambda v: (torch.where(on, v, 0.0) * w).sum()
    pgm, klm = mean(pg), mean(kl) if ref is not None else zero
    em = mean(entropy) if entropy is not None else zero
    loss = pgm + kl_coef * klm - entropy_coef * em
    stats = torch.stack([loss, pgm, klm, em, mean(off.float()), mean(torch.expm1(d) - d)])
    counts = torch.stack([tokens, filled]).to(torch.int64)
    d_logp = torch.where(on, g, 0.0) * w
    return stats, counts, d_logp, (-entropy_coef * w if entropy is not None else None)


def _plain_preference(c, s):
    n, rows, b = c["tokens"], 2 * c["pairs"], c["pairs"]
    logp = s["logp"].reshape(-1)
    on = s["mask"].reshape(-1) if s["mask"] is not None else torch.ones(n, dtype=torch.bool, device="cuda")
    row = _row_of(n, s["offsets"], rows)
    ref = s["ref"].reshape(-1) if s["ref"] is not None else None
    d = logp - ref if c["ref"] == "token" else logp
    total = _per_row(torch.where(on, d, 0.0), row, rows, c["packed"])
    if c["ref"] == "sequence":
        total = total - ref
    per_row = _per_row(on.float(), row, rows, c["packed"]).clamp(min=1) if c["average"] else torch.ones(rows, device="cuda")
    total = total / per_row
    delta = total[:b] - total[b:]
    h = BETA * delta
    eps = c["smoothing"]
    if c["kind"] == "sigmoid":
        soft = lambda v: torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
        losses = (1 - eps) * soft(-h) + eps * soft(h)
        up = 1 / (1 + torch.exp(-h))
        dd = BETA * (eps * up - (1 - eps) / (1 + torch.exp(h)))
    elif c["kind"] == "hinge":
        losses = (1 - h).clamp(min=0)
        dd = torch.where(h < 1, -BETA, 0.0)
    else:
        losses = (delta - 1 / (2 * BETA)).square()
        dd = 2 * (delta - 1 / (2 * BETA))
    stats = torch.stack([losses.mean(), (delta > 0).float().mean(), h.mean()])
    per_token = (torch.cat([dd, -dd]) / b / per_row)[row]
    return [stats, losses, BETA * total, torch.where(on, per_token, 0.0)]


def _plain_clip(c, s):
    x = [v.float() for v in s["src"]]
    if c["norm"] == "l2":
        norm = torch.sqrt(sum(v.square().sum() for v in x))
    else:
        norm = torch.stack([v.abs().amax() for v in x if v.numel()]).amax()
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return [norm, coef, (~torch.isfinite(norm)).to(torch.int32)] + [(v * coef).to(DT[c["dst"]]) for v in x]


def _coefs(c):
    return (0.05 if c["ref"] else 0.0), (0.01 if c["entropy"] else 0.0)


def run(state):
    s, c = state, state["case"]
    return _run_own(s, c) if own else _run_plain(s, c)


def _run_plain(s, c):
    op = c["op"]
    if op == "logprob":
        logp, entropy, grad = _plain_logprob(s, c, want_entropy=c["entropy"], scale=1 / c["temperature"])
        return [logp, entropy, grad(s["d_logp"], s["d_entropy"])] if c["backward"] else [logp, entropy]
    if op == "policy_logits":
        logp, entropy, grad = _plain_logprob(s, c, want_entropy=c["entropy"])
        kl, ent = _coefs(c)
        flat = lambda v: v.reshape(-1) if v is not None else None
        stats, counts, dl, dh = _plain_policy(c, flat(logp), flat(s["old"]), flat(s["ref"]), s["adv"], flat(entropy),
                                              flat(s["targets"] != IGNORE), None, c["seqs"], kl, ent)
        shape = s["targets"].shape
        return [stats, counts, logp, entropy, grad(dl.view(shape), dh.view(shape) if dh is not None else None)]
    if op == "policy":
        kl, ent = _coefs(c)
        flat = lambda v: v.reshape(-1) if v is not None else None
        shape = s["logp"].shape
        stats, counts, dl, dh = _plain_policy(c, flat(s["logp"]), flat(s["old"]), flat(s["ref"]), flat(s["adv"]),
                                              flat(s["entropy"]), flat(s["mask"]), s["offsets"], c["seqs"], kl, ent)
        return [stats, counts, dl.view(shape), dh.view(shape) if dh is not None else None]
    if op == "preference":
        stats, losses, rewards, d = _plain_preference(c, s)
        return [stats, losses, rewards, d.view(s["logp"].shape)]
    return _plain_clip(c, s)


def _run_own(s, c):
    from adamw_optimizer_step_sm_gb300 import losses as L
    op = c["op"]
    if op == "logprob":
        r = L.token_logprob(s["logits"], s["targets"], ignore_index=IGNORE, temperature=c["temperature"], entropy=c["entropy"])
        if not c["backward"]:
            return [r.logp, r.entropy]
        d = L.token_logprob_backward(s["logits"], s["targets"], r, s["d_logp"], s["d_entropy"], ignore_index=IGNORE,
                                     temperature=c["temperature"])
        return [r.logp, r.entropy, d]
    if op == "policy_logits":
        kl, ent = _coefs(c)
        r = L.policy_loss_logits(s["logits"], s["targets"], s["old"], s["adv"], ref_logp=s["ref"], entropy=c["entropy"],
                                 ignore_index=IGNORE, clip_low=CLIP_LOW, clip_high=CLIP_HIGH, dual_clip=c["dual"],
                                 kl=c["kl"], kl_coef=kl, entropy_coef=ent, reduce=c["reduce"],
                                 divisor=float(_rows(c)))
        return [r.stats, r.counts, r.logp, r.entropy, r.d_logits]
    if op == "policy":
        kl, ent = _coefs(c)
        r = L.policy_loss(s["logp"], s["old"], s["adv"], ref_logp=s["ref"], entropy=s["entropy"], mask=s["mask"],
                          offsets=s["offsets"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH, dual_clip=c["dual"],
                          kl=c["kl"], kl_coef=kl, entropy_coef=ent, reduce=c["reduce"], divisor=float(c["tokens"]))
        return [r.stats, r.counts, r.d_logp, r.d_entropy]
    if op == "preference":
        r = L.preference_loss(s["logp"], s["ref"], mask=s["mask"], offsets=s["offsets"], beta=BETA, kind=c["kind"],
                              label_smoothing=c["smoothing"], length_average=c["average"])
        return [r.stats, r.losses, r.rewards, r.d_logp]
    r = s["plan"].clip(s["max_norm"], norm=c["norm"])
    return [r.norm, r.coef, r.nonfinite] + s["dst"]


# ------------------------------------------------------------------- work --

def work(case):
    c, op = case, case["op"]
    if op in ("logprob", "policy_logits"):
        n, v, e = _rows(c), c["vocab"], SIZE[c["dtype"]]
        read = _valid(c) * v * e + 8 * n
        small = 4 * n * (1 + bool(c["entropy"]))
        ops = (6 if c["entropy"] else 4) * _valid(c) * v
        if op == "policy_logits":
            return {"bytes": read + n * v * e + small + 4 * n * (1 + bool(c["ref"])) + 4 * c["seqs"],
                    "flops": ops + (9 if c["entropy"] else 5) * _valid(c) * v}
        if not c["backward"]:
            return {"bytes": read + small, "flops": ops}
        return {"bytes": read + n * v * e + 2 * small, "flops": ops + (9 if c["entropy"] else 5) * _valid(c) * v}
    if op == "policy":
        n = c["tokens"]
        arrays = 2 + bool(c["ref"]) + bool(c["entropy"]) + bool(c["adv_per_token"]) + 1 + bool(c["entropy"])
        return {"bytes": 4 * n * arrays + (n if c["mask"] else 0) + 8 * c["seqs"], "flops": 40 * n}
    if op == "preference":
        n = c["tokens"]
        return {"bytes": 4 * n * (2 + (c["ref"] == "token")) + (n if c["mask"] else 0) + 32 * c["pairs"], "flops": 4 * n}
    numels = _numels(c)
    read = sum(n * SIZE[t] for n, t in zip(numels, _src_types(c, numels)))
    return {"bytes": read + sum(numels) * SIZE[c["dst"]], "flops": 3 * sum(numels)}


# ------------------------------------------------------------ 64-bit values --

def _exact_rows(s, c, want_entropy, scale, weights):
    """The definition row by row in blocks, in 64 bits.  weights(logp,
    entropy) gives the gradients with respect to the two, or None."""
    logits, t = s["logits"], s["targets"].reshape(-1)
    seqs, toks, v = logits.shape
    n = seqs * toks
    logp = torch.zeros(n, dtype=torch.float64, device="cuda")
    ent = torch.zeros(n, dtype=torch.float64, device="cuda")
    lse = torch.zeros(n, dtype=torch.float64, device="cuda")
    step = max(1, 40_000_000 // v)
    keep = (t != IGNORE).nonzero()[:, 0]
    for a in range(0, keep.numel(), step):
        at = keep[a:a + step]
        x = logits[at // toks, at % toks].double() * scale
        z = torch.logsumexp(x, 1)
        lse[at] = z
        logp[at] = x.gather(1, t[at, None])[:, 0] - z
        if want_entropy:
            q = torch.exp(x - z[:, None])
            ent[at] = z - torch.where(q > 0, q * x, 0.0).sum(1)
    got = weights(logp, ent)
    grad = None
    if got is not None:
        gl, gh = got
        grad = torch.zeros((n, v), dtype=torch.float64, device="cuda")
        for a in range(0, keep.numel(), step):
            at = keep[a:a + step]
            lp = logits[at // toks, at % toks].double() * scale - lse[at, None]
            q = torch.exp(lp)
            part = -gl[at, None] * q
            part[torch.arange(at.numel(), device="cuda"), t[at]] += gl[at]
            if gh is not None:
                part -= gh[at, None] * torch.where(q > 0, q * (lp + ent[at, None]), 0.0)
            grad[at] = part * scale
        grad = grad.view(seqs, toks, v)
    shape = (seqs, toks)
    return logp.view(shape), ent.view(shape) if want_entropy else None, grad


def _exact_policy(c, logp, old, ref, adv, entropy, on, offsets, rows, kl_coef, entropy_coef):
    n = logp.numel()
    starts = offsets if offsets is not None else torch.arange(rows + 1, device="cuda") * (n // rows)
    row = torch.repeat_interleave(torch.arange(rows, device="cuda"), starts[1:] - starts[:-1])
    total = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), on.to(torch.int64).cumsum(0)])
    per_row = (total[starts[1:]] - total[starts[:-1]]).double()
    filled = (per_row > 0).sum()
    tokens = on.sum()
    w = {"token": lambda: 1.0 / max(1, int(tokens)) * torch.ones(n, dtype=torch.float64, device="cuda"),
         "sequence": lambda: 1.0 / (per_row.clamp(min=1) * max(1, int(filled)))[row],
         "fixed": lambda: torch.full((n,), 1.0 / n, dtype=torch.float64, device="cuda")}[c["reduce"]]() * on
    a = adv.double() if adv.numel() == n and n != rows else adv.double()[row]
    d = torch.where(on, logp.double() - old.double(), 0.0)
    r = torch.exp(d)
    bounded = r.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH)
    gain = torch.minimum(a * r, a * bounded)
    off = a * bounded < a * r
    if c["dual"]:
        floor = a * c["dual"]
        off = off | ((a < 0) & (gain < floor))
        gain = torch.where(a < 0, torch.maximum(gain, floor), gain)
    dl = torch.where(off, 0.0, -a * r)
    kl = torch.zeros(n, dtype=torch.float64, device="cuda")
    if ref is not None:
        k = torch.where(on, logp.double() - ref.double(), 0.0)
        kl, dk = {"k1": (k, torch.ones_like(k)), "k2": (k * k / 2, k),
                  "k3": (torch.exp(-k) - 1 + k, 1 - torch.exp(-k))}[c["kl"]]
        dl = dl + kl_coef * dk
    ent = entropy.double() if entropy is not None else torch.zeros(n, dtype=torch.float64, device="cuda")
    parts = [(v * w).sum() for v in (-gain, kl, torch.where(on, ent, 0.0), off.double(), r - 1 - d)]
    loss = parts[0] + kl_coef * parts[1] - entropy_coef * parts[2]
    counts = torch.stack([tokens, filled]).to(torch.int64)
    return torch.stack([loss] + parts), counts, dl * w, -entropy_coef * w


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    op = c["op"]
    flat = lambda v: v.reshape(-1) if v is not None else None
    if op == "logprob":
        scale = 1 / c["temperature"]
        back = (lambda lp, h: (s["d_logp"].reshape(-1).double(), flat(s["d_entropy"].double()) if c["entropy"] else None)) \
            if c["backward"] else (lambda lp, h: None)
        logp, ent, grad = _exact_rows(s, c, c["entropy"], scale, back)
        return [logp, ent, grad] if c["backward"] else [logp, ent]
    if op == "policy_logits":
        kl, ec = _coefs(c)
        kept = {}

        def weights(lp, h):
            kept["r"] = _exact_policy(c, lp, flat(s["old"]), flat(s["ref"]), s["adv"], h if c["entropy"] else None,
                                      flat(s["targets"]) != IGNORE, None, c["seqs"], kl, ec)
            return kept["r"][2], kept["r"][3] if c["entropy"] else None
        logp, ent, grad = _exact_rows(s, c, c["entropy"], 1.0, weights)
        return [kept["r"][0], kept["r"][1], logp, ent, grad]
    if op == "policy":
        kl, ec = _coefs(c)
        on = flat(s["mask"]) if s["mask"] is not None else torch.ones(c["tokens"], dtype=torch.bool, device="cuda")
        stats, counts, dl, dh = _exact_policy(c, flat(s["logp"]), flat(s["old"]), flat(s["ref"]), flat(s["adv"]),
                                              flat(s["entropy"]), on, s["offsets"], c["seqs"], kl, ec)
        shape = s["logp"].shape
        return [stats, counts, dl.view(shape), dh.view(shape) if c["entropy"] else None]
    if op == "preference":
        n, b = c["tokens"], c["pairs"]
        starts = s["offsets"] if s["offsets"] is not None else torch.arange(2 * b + 1, device="cuda") * (n // (2 * b))
        on = flat(s["mask"]) if s["mask"] is not None else torch.ones(n, dtype=torch.bool, device="cuda")
        x = flat(s["logp"]).double()
        if c["ref"] == "token":
            x = x - flat(s["ref"]).double()
        zero = torch.zeros(1, dtype=torch.float64, device="cuda")
        run_sum = torch.cat([zero, torch.where(on, x, 0.0).cumsum(0)])
        run_on = torch.cat([zero, on.double().cumsum(0)])
        total = run_sum[starts[1:]] - run_sum[starts[:-1]]
        if c["ref"] == "sequence":
            total = total - s["ref"].double()
        share = (run_on[starts[1:]] - run_on[starts[:-1]]).clamp(min=1) if c["average"] else torch.ones_like(total)
        total = total / share
        delta = total[:b] - total[b:]
        leaf = delta.clone().requires_grad_(True)
        h = BETA * leaf
        if c["kind"] == "sigmoid":
            losses = -(1 - c["smoothing"]) * torch.nn.functional.logsigmoid(h) \
                - c["smoothing"] * torch.nn.functional.logsigmoid(-h)
        elif c["kind"] == "hinge":
            losses = torch.relu(1 - h)
        else:
            losses = (leaf - 0.5 / BETA) ** 2
        losses.mean().backward()
        g = torch.cat([leaf.grad, -leaf.grad]) / share
        row = torch.repeat_interleave(torch.arange(2 * b, device="cuda"), starts[1:] - starts[:-1])
        stats = torch.stack([losses.mean().detach(), (delta > 0).double().mean(), BETA * delta.mean()])
        return [stats, losses.detach(), BETA * total, torch.where(on, g[row], 0.0).view(s["logp"].shape)]
    norm = torch.zeros((), dtype=torch.float64, device="cuda")
    for v in s["src"]:
        for part in v.split(1 << 26):
            q = part.double().abs()
            norm = norm + q.square().sum() if c["norm"] == "l2" else torch.maximum(norm, q.amax())
    norm = norm.sqrt() if c["norm"] == "l2" else norm
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return [norm, coef, torch.zeros((), dtype=torch.int32, device="cuda")] + [v.double() * coef for v in s["src"]]
