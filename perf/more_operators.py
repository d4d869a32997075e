"""Cases that measure the matrix operators of a training step: orthogonalising
matrices by Newton-Schulz products, the Muon step built on it, and products
grouped by expert with their gradients.

``own`` false: each operator in its plain form (elementary torch operations in
32 bits, rounded once at the end).  ``own`` true: the calls that a user makes
of ``adamw_optimizer_step_sm_gb300.matrix`` and ``.optim``.  ``exact`` is the
definition in 64 bits; it multiplies the small Gram matrices through all steps
and the matrix itself once, where the plain form multiplies the matrix in
every step.

Sizes: 2048 and 8192 are OPT-1.3b's width and feed-forward width, 128 that of
the model in ``examples/finetune.py``, 20000 packed tokens a batch of ragged
answers; the rest are generic.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
COEFS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
# fine-tuning: a small rate, the update's size that of an AdamW step's
LR, MOMENTUM, DECAY = 2e-5, 0.95, 0.1


def listed():
    return [
        # one small matrix (an adapter's factor): latency
        dict(name="ortho_adapter", op="ortho", batch=1, rows=64, cols=128, dtype="bf16", steps=5, rank=64),
        # odd sizes, fp32 gradients
        dict(name="ortho_odd", op="ortho", batch=3, rows=515, cols=1031, dtype="fp32", steps=5, rank=515),
        # the attention matrices of a few layers
        dict(name="ortho_square", op="ortho", batch=16, rows=2048, cols=2048, dtype="bf16", steps=5, rank=256),
        # a layer's feed-forward matrix, taller than wide
        dict(name="ortho_tall", op="ortho", batch=1, rows=8192, cols=2048, dtype="bf16", steps=5, rank=256),
        # the small model's list: latency of a whole step
        dict(name="muon_small", op="muon", hidden=128, ffn=512, layers=2, experts=0, momentum="fp32"),
        # three layers of OPT-1.3b (the largest)
        dict(name="muon_layers", op="muon", hidden=2048, ffn=8192, layers=3, experts=0, momentum="fp32"),
        # a layer whose feed-forward part is 16 experts, a momentum of 16 bits
        dict(name="muon_experts", op="muon", hidden=1024, ffn=512, layers=1, experts=16, momentum="bf16"),
        # eight tokens decoding, each through its experts: the weights are streamed once
        dict(name="experts_token", op="experts", tokens=8, experts=16, active=7, n=8192, k=2048, dtype="bf16",
             backward=False, spread=1.0),
        # a prompt through a few large experts
        dict(name="experts_prompt", op="experts", tokens=3001, experts=8, active=8, n=8192, k=2048, dtype="bf16",
             backward=False, spread=0.5),
        # a training batch of ragged answers: product and both gradients
        dict(name="experts_train", op="experts", tokens=20000, experts=16, active=16, n=8192, k=2048, dtype="bf16",
             backward=True, spread=0.5),
        # many small experts, some without a token
        dict(name="experts_many", op="experts", tokens=16384, experts=128, active=120, n=768, k=2048, dtype="bf16",
             backward=True, spread=1.0),
        # odd sizes in fp16
        dict(name="experts_odd", op="experts", tokens=1021, experts=5, active=4, n=1003, k=515, dtype="fp16",
             backward=True, spread=1.0),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["ortho", "muon", "experts"])
    if op == "ortho":
        rows, cols = _log(rng, 8, 4096), _log(rng, 8, 4096)
        m = min(rows, cols)
        most = int(2e12 // (20 * m * m * max(rows, cols))) + 1
        return dict(op=op, batch=min(most, _log(rng, 1, 64)), rows=rows, cols=cols,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), steps=rng.choice([3, 5, 5]),
                    rank=max(1, m // rng.choice([1, 4, 16])))
    if op == "muon":
        hidden = _log(rng, 48, 2048)
        ffn = max(8, int(hidden * rng.choice([0.5, 1.3, 4])))
        experts = rng.choice([0, 0, _log(rng, 2, 16)])
        return dict(op=op, hidden=hidden, ffn=ffn, layers=rng.choice([1, 2]) if not experts else 1,
                    experts=experts if ffn <= hidden else min(experts, 4), momentum=rng.choice(["fp32", "bf16"]))
    k, n, experts = _log(rng, 48, 8192), _log(rng, 48, 8192), _log(rng, 1, 128)
    experts = max(1, min(experts, 600_000_000 // (k * n)))
    tokens = max(1, min(_log(rng, 1, 32768), 400_000_000_000 // (k * n)))
    return dict(op=op, tokens=tokens, experts=experts, active=max(1, min(experts, tokens, int(experts * rng.uniform(0.6, 1.1)))),
                n=n, k=k, dtype=rng.choice(["bf16", "bf16", "fp16"]), backward=rng.random() < 0.5,
                spread=rng.choice([0.0, 0.5, 1.0]))


# ------------------------------------------------------------------ inputs --

def _shapes(c):
    """The parameters of a list of layers: four attention matrices, and the two
    of the feed-forward part, or of its experts."""
    h, f, e = c["hidden"], c["ffn"], c["experts"]
    wide = [(e, f, h), (e, h, f)] if e else [(f, h), (h, f)]
    return ([(h, h)] * 4 + wide) * c["layers"]


def _gradient(shape, rank, g):
    """A gradient's shape of spectrum: a few strong directions over noise."""
    *batch, m, n = shape
    decay = torch.arange(1, rank + 1, device="cuda").float().rsqrt()
    u = torch.randn(*batch, m, rank, generator=g, device="cuda") * decay
    v = torch.randn(*batch, rank, n, generator=g, device="cuda")
    x = torch.matmul(u, v)
    x += 0.5 * torch.randn(*batch, m, n, generator=g, device="cuda")
    return x.mul_(1e-3)


def _lengths(c, seed):
    """Tokens of each expert: `active` of them have at least one."""
    rng = random.Random(seed * 31 + 7)
    some = sorted(rng.sample(range(c["experts"]), c["active"]))
    weight = [math.exp(c["spread"] * rng.gauss(0, 1)) for _ in some]
    left = c["tokens"] - len(some)
    cuts = [int(left * sum(weight[:i]) / sum(weight)) for i in range(len(some))] + [left]
    lens = [0] * c["experts"]
    for e, a, b in zip(some, cuts, cuts[1:]):
        lens[e] = 1 + b - a
    return lens


def prepare(case, seed):
    c, s = case, {"case": case}
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)
    if c["op"] == "ortho":
        s["x"] = _gradient((c["batch"], c["rows"], c["cols"]), c["rank"], g).to(DT[c["dtype"]])
        return s
    if c["op"] == "experts":
        lens = _lengths(c, int(seed))
        ends = [sum(lens[:i]) for i in range(len(lens) + 1)]
        s["ends"] = ends  # a program that routes knows them, or keeps them on the device
        s["offsets"] = torch.tensor(ends, dtype=torch.int64, device="cuda")
        dt = DT[c["dtype"]]
        s["x"] = torch.randn(c["tokens"], c["k"], generator=g, device="cuda", dtype=dt)
        s["w"] = torch.randn(c["experts"], c["n"], c["k"], generator=g, device="cuda", dtype=dt).mul_(c["k"] ** -0.5)
        if c["backward"]:
            s["dy"] = torch.randn(c["tokens"], c["n"], generator=g, device="cuda", dtype=dt)
            s["x"].requires_grad_(True)
            s["w"].requires_grad_(True)
        return s
    shapes = _shapes(c)
    rank = max(1, min(c["hidden"], c["ffn"]) // 8)
    grads, moments, masters = [], [], []
    for shape in shapes:
        grads.append(_gradient(shape, rank, g).bfloat16())
        moments.append(_gradient(shape, rank, g).to(DT[c["momentum"]]))
        masters.append(0.02 * torch.randn(*shape, generator=g, device="cuda"))
    s["params"] = [torch.nn.Parameter(m.bfloat16()) for m in masters]
    if own:
        from adamw_optimizer_step_sm_gb300.optim import Muon
        for p, d in zip(s["params"], grads):
            p.grad = d
        s["opt"] = Muon(s["params"], lr=LR, momentum=MOMENTUM, weight_decay=DECAY, nesterov=True, steps=5,
                        coefficients=COEFS, eps=EPS, scale="rms", momentum_dtype=DT[c["momentum"]])
        for p, b, m in zip(s["params"], moments, masters):
            s["opt"].state[p]["momentum"].copy_(b)
            s["opt"].state[p]["master"].copy_(m)
        s["moments"] = [s["opt"].state[p]["momentum"] for p in s["params"]]
        s["masters"] = [s["opt"].state[p]["master"] for p in s["params"]]
    else:
        s["grads"], s["moments"], s["masters"] = grads, moments, masters
    return s


# ------------------------------------------------------------- plain forms --

def _plain_ortho(x, steps):
    """Newton-Schulz steps of the matrices of x, in 32 bits."""
    x = x.float()
    x = x / x.square().sum((-2, -1), keepdim=True).sqrt().clamp(min=EPS)
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT
    a, b, c = COEFS
    for _ in range(steps):
        gram = x @ x.mT
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.mT if tall else x


def _plain_step(s):
    for p, d, m, w in zip(s["params"], s["grads"], s["moments"], s["masters"]):
        d = d.float()
        b = torch.lerp(m.float(), d, 1 - MOMENTUM)
        u = _plain_ortho(torch.lerp(d, b, MOMENTUM), 5)
        m.copy_(b)
        w.mul_(1 - LR * DECAY).sub_(u, alpha=LR * 0.2 * math.sqrt(max(p.shape[-2:])))
        p.detach().copy_(w)


def run(state):
    s, c = state, state["case"]
    if c["op"] == "ortho":
        if own:
            from adamw_optimizer_step_sm_gb300 import matrix
            return matrix.orthogonalize(s["x"], steps=c["steps"], coefficients=COEFS, eps=EPS)
        return _plain_ortho(s["x"], c["steps"]).bfloat16()
    if c["op"] == "muon":
        if own:
            s["opt"].step()
        else:
            _plain_step(s)
        return [[p.detach() for p in s["params"]], s["masters"], s["moments"]]
    if own:
        from adamw_optimizer_step_sm_gb300 import matrix
        y = matrix.expert_linear(s["x"], s["w"], s["offsets"])
        if c["backward"]:
            return [y.detach(), *torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])]
        return [y]
    x, w, ends = s["x"].detach(), s["w"].detach(), s["ends"]
    y = x.new_empty(c["tokens"], c["n"])
    dx, dw = (torch.empty_like(x), torch.zeros_like(w)) if c["backward"] else (None, None)
    for e, (a, b) in enumerate(zip(ends, ends[1:])):  # a library product for each expert that has tokens
        if a == b:
            continue
        xe, we = x[a:b].float(), w[e].float()
        y[a:b] = xe @ we.t()
        if c["backward"]:
            de = s["dy"][a:b].float()
            dx[a:b] = de @ we
            dw[e] = de.t() @ xe
    return [y, dx, dw] if c["backward"] else [y]


def work(case):
    c = case
    if c["op"] == "ortho":
        m, n = sorted((c["rows"], c["cols"]))
        # symmetric products count once for each pair of entries
        flops = c["steps"] * (m * m * n + m ** 3 + 2 * m * m * n) * c["batch"]
        return {"bytes": c["batch"] * m * n * (SIZE[c["dtype"]] + 2), "flops": flops}
    if c["op"] == "muon":
        total = flops = 0
        for *batch, m, n in _shapes(c):
            count = math.prod(batch)
            m, n = sorted((m, n))
            total += count * m * n
            flops += 5 * (m * m * n + m ** 3 + 2 * m * m * n) * count
        # the gradient; momentum and master read and written; the parameter written
        return {"bytes": total * (2 + 2 * SIZE[c["momentum"]] + 8 + 2), "flops": flops}
    t, e, n, k = c["tokens"], c["active"], c["n"], c["k"]
    size = SIZE[c["dtype"]]
    if not c["backward"]:
        return {"bytes": size * (t * k + t * n + e * n * k), "flops": 2 * t * n * k}
    # x, w, dy read; y, dx and the gradient of every expert written
    return {"bytes": size * (2 * t * k + 2 * t * n + e * n * k + c["experts"] * n * k), "flops": 6 * t * n * k}


# -------------------------------------------------------------- definition --

def _exact_ortho(x, steps):
    """In 64 bits, through the small Gram matrix: G <- Q G Q, P <- Q P with
    Q = a + b G + c G^2, and P X once at the end."""
    x = x.double()
    x = x / torch.linalg.matrix_norm(x).clamp(min=EPS)[..., None, None]
    wide = x.shape[-1] >= x.shape[-2]
    gram = x @ x.mT if wide else x.mT @ x
    one = torch.eye(gram.shape[-1], dtype=torch.float64, device=x.device)
    whole = one
    a, b, c = COEFS
    for k in range(steps):
        q = torch.matmul(gram, b * one + c * gram) + a * one
        whole = q @ whole
        if k + 1 < steps:
            gram = q @ gram @ q
    return whole @ x if wide else x @ whole


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "ortho":
        return _exact_ortho(s["x"], c["steps"])
    if c["op"] == "muon":
        params, masters, moments = [], [], []
        for d, m, w in zip(s["grads"], s["moments"], s["masters"]):
            d = d.double()
            m = MOMENTUM * m.double() + (1 - MOMENTUM) * d
            u = _exact_ortho((1 - MOMENTUM) * d + MOMENTUM * m, 5)
            w = w.double() * (1 - LR * DECAY) - LR * 0.2 * math.sqrt(max(w.shape[-2:])) * u
            masters.append(w)
            params.append(w)
            moments.append(m)
        return [params, masters, moments]
    x, w = s["x"].detach().double(), s["w"].detach()
    owner = torch.bucketize(torch.arange(c["tokens"], device="cuda"), s["offsets"][1:], right=True)
    y = torch.zeros(c["tokens"], c["n"], dtype=torch.float64, device="cuda")
    dx, dw = torch.zeros_like(x), torch.zeros(w.shape, dtype=torch.float64, device="cuda")
    for e in owner.unique().tolist():
        at = (owner == e).nonzero()[:, 0]
        we = w[e].double()
        y[at] = torch.einsum("tk,nk->tn", x[at], we)
        if c["backward"]:
            de = s["dy"][at].double()
            dx[at] = torch.einsum("tn,nk->tk", de, we)
            dw[e] = torch.einsum("tn,tk->nk", de, x[at])
    return [y, dx, dw] if c["backward"] else [y]
