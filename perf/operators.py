"""Operators that close a quantization-aware training step around the E8 projection, measured.

* token log probabilities of a model's output logits (with entropy and the k
  most likely alternatives), and their gradient: the loss end of a step, and
  what a served model reports per token;
* the embedding lookup with scaling and its gradient: the input end;
* the update of the bf16 latents along the orthogonalized momentum
  (Newton-Schulz products): the optimizer step of the latent weights.

``run`` computes a case in plain torch operations (``own`` false) or with the
library's entry points (``own`` true).
"""

import math

import numpy as np
import torch

own = False

# Newton-Schulz polynomial sigma -> a sigma + b sigma^3 + c sigma^5: steep at 0,
# and within [0.68, 1.21] of 1 after five steps for singular values above 1e-2.
COEFFS = (3.4445, -4.7750, 2.0315)
STEPS = 5


def listed():
    return [
        # one generated token: the sampled token's log probability and the eight best alternatives, some tokens banned
        {"name": "logprobs_1x131072_bf16_top8", "op": "logprobs", "rows": 1, "vocab": 131072, "pad": 0,
         "dtype": "bf16", "tokens": 1, "top": 8, "scale": 1.0, "banned": True, "index": "i64"},
        # a served batch at temperature 1/1.25 with float32 logits out of a wider (padded) buffer, an odd vocabulary
        {"name": "logprobs_48x50001_f32_top20", "op": "logprobs", "rows": 48, "vocab": 50001, "pad": 175,
         "dtype": "f32", "tokens": 1, "top": 20, "scale": 1.25, "banned": True, "index": "i32"},
        # scoring given continuations: four candidate tokens per position, entropy, no alternatives
        {"name": "logprobs_4096x32768_bf16_score4", "op": "logprobs", "rows": 4096, "vocab": 32768, "pad": 0,
         "dtype": "bf16", "tokens": 4, "top": 0, "scale": 1.0, "banned": False, "index": "i64"},
        # training through log probability and entropy with upstream gradients: forward call, then backward call
        {"name": "logprobs_train_301x32003_f32", "op": "logprobs_train", "rows": 301, "vocab": 32003, "pad": 0,
         "dtype": "f32", "tokens": 1, "scale": 1.0, "entropy": True, "index": "i64"},
        # the loss of a training step whose token weights are known beforehand: loss terms and gradient in one call
        {"name": "logprobs_loss_8192x131072_bf16", "op": "logprobs_loss", "rows": 8192, "vocab": 131072, "pad": 0,
         "dtype": "bf16", "tokens": 1, "scale": 1.0, "entropy": False, "index": "i64"},
        # the lookup of a decode step: a few tokens
        {"name": "embed_7x4096_bf16", "op": "embed", "tokens": 7, "vocab": 131072, "dim": 4096, "dtype": "bf16",
         "out": "bf16", "scale": 64.0, "index": "i64"},
        # a small training batch, odd vocabulary and width, float32 table and gradients
        {"name": "embed_train_999x1001_f32", "op": "embed_train", "tokens": 999, "vocab": 50001, "dim": 1001,
         "dtype": "f32", "out": "f32", "scale": 1.0, "index": "i32"},
        # a full training batch of text (a few tokens make up much of it): bf16 table, float32 gradient of the table
        {"name": "embed_train_32768x4096_bf16", "op": "embed_train", "tokens": 32768, "vocab": 131072, "dim": 4096,
         "dtype": "bf16", "out": "f32", "scale": 64.0, "index": "i64"},
        # one small matrix: launch bound
        {"name": "orthogonalize_256x256_f32", "op": "orthogonalize", "batch": 1, "rows": 256, "cols": 256,
         "dtype": "f32"},
        # the 128 experts' gate projections of the mixture-of-experts workload
        {"name": "orthogonalize_128x768x2048_bf16", "op": "orthogonalize", "batch": 128, "rows": 768, "cols": 2048,
         "dtype": "bf16"},
        # a tall matrix of the dense decoder, an odd number of rows kept (a shard)
        {"name": "orthogonalize_5503x4096_bf16", "op": "orthogonalize", "batch": 1, "rows": 5503, "cols": 4096,
         "dtype": "bf16"},
        # the whole optimizer step of the training workload's latent matrix: momentum, orthogonalization, latents
        {"name": "orthogonal_step_4096x14336_bf16", "op": "orthogonal_step", "batch": 1, "rows": 4096, "cols": 14336,
         "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs_train", "logprobs_loss", "embed", "embed_train",
                     "orthogonalize", "orthogonal_step"])
    if op.startswith("logprobs"):
        rows, vocab = _log_int(rng, 1, 8192), _log_int(rng, 512, 131072)
        if op == "logprobs":
            rows = min(rows, max(1, (1 << 27) // vocab))
            return {"op": op, "rows": rows, "vocab": vocab, "pad": rng.choice([0, 0, rng.randrange(1, 200)]),
                    "dtype": rng.choice(["bf16", "f32"]), "tokens": rng.choice([1, 1, 2, 5]),
                    "top": rng.choice([0, 1, 5, 20, 50]), "scale": rng.choice([1.0, 0.7, 1.25]),
                    "banned": rng.random() < 0.5, "index": rng.choice(["i64", "i32"])}
        dtype = rng.choice(["bf16", "f32"])
        rows = min(rows, (8192 * 131072 // (2 if dtype == "f32" else 1)) // vocab)
        return {"op": op, "rows": rows, "vocab": vocab, "pad": rng.choice([0, 0, rng.randrange(1, 200)]),
                "dtype": dtype, "tokens": rng.choice([1, 1, 3]), "scale": rng.choice([1.0, 0.7]),
                "entropy": rng.random() < 0.5, "index": rng.choice(["i64", "i32"])}
    if op.startswith("embed"):
        tokens = _log_int(rng, 1, 256) if op == "embed" else _log_int(rng, 64, 32768)
        return {"op": op, "tokens": tokens, "vocab": _log_int(rng, 500, 131072), "dim": _log_int(rng, 64, 4096),
                "dtype": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"]),
                "scale": rng.choice([1.0, 45.25]), "index": rng.choice(["i64", "i32"])}
    rows, cols = _log_int(rng, 64, 4096), 8 * _log_int(rng, 8, 1791)
    if rng.random() < 0.3:
        rows, cols = cols + rng.randrange(8), max(8, rows // 8 * 8)
    most = 4096 * 4096 * 14336 // 4
    batch = min(rng.choice([1, 1, 1, 2, 7, 32]), max(1, most // (min(rows, cols) * rows * cols)))
    return {"op": op, "batch": batch, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "f32"])}


# ---------------------------------------------------------------- inputs

_DT = {"bf16": torch.bfloat16, "f32": torch.float32, "i64": torch.int64, "i32": torch.int32}


def _logits(case, g):
    """Logits of a language model: wide normal values with a few likely tokens per row."""
    rows, vocab = case["rows"], case["vocab"]
    x = torch.empty((rows, vocab + case["pad"]), dtype=_DT[case["dtype"]], device="cuda")
    x.normal_(0.0, 2.0, generator=g)
    # one likely token in each twelfth of the vocabulary (distinct, so that the scatter has one value per place)
    best = torch.randint(0, vocab // 12, (rows, 12), generator=g, device="cuda")
    best += torch.arange(12, device="cuda") * (vocab // 12)
    lift = torch.rand((rows, 12), generator=g, device="cuda") * 8.0 + 6.0
    x.scatter_(1, best, lift.to(x.dtype))
    if case.get("banned"):
        x[:, vocab // 7: vocab // 7 + max(1, vocab // 50)] = -math.inf
    tok = torch.randint(0, vocab, (rows, case["tokens"]), generator=g, device="cuda")
    pick = torch.rand((rows, case["tokens"]), generator=g, device="cuda") < 0.8       # mostly likely tokens
    liked = torch.gather(best, 1, torch.randint(0, 12, tok.shape, generator=g, device="cuda"))
    tok = torch.where(pick, liked, tok)
    if rows > 16:
        tok[torch.rand(rows, generator=g, device="cuda") < 0.05] = -1                 # positions without a target
    return x, tok.to(_DT[case["index"]])


def _token_ids(case, g):
    """Token ids of text: frequency about 1 / rank, ranks spread over the vocabulary; a few padded positions."""
    u = torch.rand(case["tokens"], generator=g, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(case["vocab"] + 1.0)).long().clamp_(1, case["vocab"]) - 1
    tok = (rank * 40503 + 17) % case["vocab"]
    if case["tokens"] > 16:
        tok[torch.rand(case["tokens"], generator=g, device="cuda") < 0.03] = -1
    return tok.to(_DT[case["index"]])


def _gradient(shape, g):
    """A weight gradient: a part of low rank with falling strength, and the noise of a batch."""
    b, r, c = shape
    k = max(1, min(r, c) // 8)
    left = torch.randn((b, r, k), generator=g, device="cuda")
    left *= torch.linspace(1.0, 0.1, k, device="cuda") / math.sqrt(k)
    right = torch.randn((b, k, c), generator=g, device="cuda")
    return (torch.matmul(left, right) + torch.randn(shape, generator=g, device="cuda")) * 1e-4


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, s = case["op"], {"case": dict(case)}
    f32 = {"dtype": torch.float32, "device": "cuda"}
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op.startswith("logprobs"):
        full, s["tokens"] = _logits(case, g)
        rows, n = case["rows"], case["tokens"]
        s["logits"] = full[:, :case["vocab"]]
        s["logprob"], s["lse"], s["entropy"] = torch.empty((rows, n), **f32), torch.empty(rows, **f32), torch.empty(rows, **f32)
        if case.get("top"):
            s["top_idx"] = torch.empty((rows, case["top"]), dtype=torch.int32, device="cuda")
            s["top_logprob"] = torch.empty((rows, case["top"]), **f32)
        if op != "logprobs":
            s["grad_logprob"] = -torch.rand((rows, n), generator=g, **f32) - 0.5
            s["grad_entropy"] = 0.1 * torch.rand(rows, generator=g, **f32) if case["entropy"] else None
            s["grad_logits"] = torch.empty_like(full)[:, :case["vocab"]]
    elif op.startswith("embed"):
        dt, out = _DT[case["dtype"]], _DT[case["out"]]
        s["tokens"] = _token_ids(case, g)
        s["table"] = (torch.randn((case["vocab"], case["dim"]), generator=g, device="cuda") * 0.02).to(dt)
        s["out"] = torch.empty((case["tokens"], case["dim"]), dtype=dt, device="cuda")
        if op == "embed_train":
            s["grad_out"] = (torch.randn((case["tokens"], case["dim"]), generator=g, device="cuda") * 1e-3).to(dt)
            s["grad_table"] = torch.empty((case["vocab"], case["dim"]), dtype=out, device="cuda")
    else:
        shape = (case["batch"], case["rows"], case["cols"])
        s["grad"] = _gradient(shape, g).to(_DT[case["dtype"]])
        if op == "orthogonal_step":
            s["momentum"] = _gradient(shape, g)
            s["w"] = (torch.randn(shape, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
            s["momentum_out"], s["w_out"] = torch.empty_like(s["momentum"]), torch.empty_like(s["w"])
        else:
            s["update"] = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

MU, LR, DECAY = 0.95, 0.02, 0.01


def _gamma(case):
    return math.sqrt(max(1.0, case["rows"] / case["cols"]))


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _workspace(s, e8q):
    """The device scratch that a program keeps for its calls: made on the first pass."""
    if "ws" not in s:
        case = s["case"]
        if case["op"].startswith("logprobs"):
            size = e8q.e8q_token_logprobs_workspace_size(case["rows"], case["vocab"], case.get("top", 0))
        elif case["op"] == "embed_train":
            size = e8q.e8q_embed_backward_workspace_size(case["tokens"], case["vocab"], case["dim"])
        else:
            size = e8q.e8q_orthogonalize_workspace_size(case["batch"], case["rows"], case["cols"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s["ws"]


def _run_own(s):
    import bit_e8_lattice_amd as e8q
    case = s["case"]
    op = case["op"]
    if op == "embed":
        e8q.e8q_embed(s["table"], s["tokens"], s["out"], s["status"], scale=case["scale"])
        return s["out"]
    ws = _workspace(s, e8q)
    if op == "logprobs":
        e8q.e8q_token_logprobs(s["logits"], ws, s["status"], tokens=s["tokens"], scale=case["scale"],
                               logprob_out=s["logprob"], lse_out=s["lse"], entropy_out=s["entropy"],
                               top_idx_out=s.get("top_idx"), top_logprob_out=s.get("top_logprob"))
        out = {"logprob": s["logprob"], "lse": s["lse"], "entropy": s["entropy"]}
        if case["top"]:
            out["top_idx"], out["top_logprob"] = s["top_idx"], s["top_logprob"]
        return out
    if op == "logprobs_train":
        e8q.e8q_token_logprobs(s["logits"], ws, s["status"], tokens=s["tokens"], scale=case["scale"],
                               logprob_out=s["logprob"], lse_out=s["lse"], entropy_out=s["entropy"])
        e8q.e8q_token_logprobs_backward(s["logits"], s["lse"], s["grad_logits"], s["status"],
                                        tokens=s["tokens"], grad_logprob=s["grad_logprob"], scale=case["scale"],
                                        entropy=s["entropy"] if case["entropy"] else None,
                                        grad_entropy=s["grad_entropy"])
        return {"logprob": s["logprob"], "entropy": s["entropy"], "grad_logits": s["grad_logits"]}
    if op == "logprobs_loss":
        e8q.e8q_token_logprobs_grad(s["logits"], s["tokens"], s["grad_logprob"], s["grad_logits"], ws, s["status"],
                                    grad_entropy=s["grad_entropy"], scale=case["scale"], logprob_out=s["logprob"],
                                    entropy_out=s["entropy"])
        return {"logprob": s["logprob"], "entropy": s["entropy"], "grad_logits": s["grad_logits"]}
    if op == "embed_train":
        e8q.e8q_embed(s["table"], s["tokens"], s["out"], s["status"], scale=case["scale"])
        e8q.e8q_embed_backward(s["grad_out"], s["tokens"], case["vocab"], ws, s["status"], scale=case["scale"],
                               grad_table=s["grad_table"])
        return {"out": s["out"], "grad_table": s["grad_table"]}
    if op == "orthogonalize":
        e8q.e8q_orthogonalize(s["grad"], s["update"], ws, s["status"], steps=STEPS, coeffs=COEFFS)
        return s["update"]
    e8q.e8q_orthogonal_step(s["w"], s["grad"], s["momentum"], ws, s["status"], mu=MU, nesterov=True, lr=LR,
                            decay=DECAY, gamma=_gamma(case), steps=STEPS, coeffs=COEFFS, w_out=s["w_out"],
                            momentum_out=s["momentum_out"])
    return {"w": s["w_out"], "momentum": s["momentum_out"]}


def _plain_logprobs(s):
    case, tok = s["case"], s["tokens"].long()
    y = s["logits"].float() * case["scale"]
    m = y.amax(dim=1, keepdim=True)
    e = torch.exp(y - m)
    total = e.sum(dim=1, keepdim=True)
    lse = m + torch.log(total)
    p = e / total
    lp = y - lse
    entropy = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(dim=1)
    live = tok >= 0
    logprob = torch.where(live, torch.gather(lp, 1, tok.clamp(min=0)), torch.zeros_like(tok, dtype=torch.float32))
    return live, lse[:, 0], p, lp, entropy, logprob


def _plain_logit_gradient(s, live, p, lp, entropy):
    """Gradient of sum(grad_logprob * logprob) + sum(grad_entropy * entropy) with respect to the logits."""
    g = torch.where(live, s["grad_logprob"], torch.zeros_like(s["grad_logprob"]))
    d = -g.sum(dim=1, keepdim=True) * p
    if s["grad_entropy"] is not None:
        d -= s["grad_entropy"][:, None] * torch.where(p > 0, p * (lp + entropy[:, None]), torch.zeros_like(p))
    d.scatter_add_(1, s["tokens"].long().clamp(min=0), g)
    return (d * s["case"]["scale"]).to(s["logits"].dtype)


def _orthogonal(x, steps):
    """Newton-Schulz steps on the matrices of x (float32 or float64), scaled to unit Frobenius norm first."""
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.mT.contiguous()
    x = x / torch.sqrt((x * x).sum(dim=(1, 2), keepdim=True))
    a, b, c = COEFFS
    for _ in range(steps):
        gram = torch.matmul(x, x.mT.contiguous())
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    return x.mT.contiguous() if tall else x


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op.startswith("logprobs"):
        live, lse, p, lp, entropy, logprob = _plain_logprobs(s)
        if op == "logprobs":
            out = {"logprob": logprob, "lse": lse, "entropy": entropy}
            if case["top"]:
                # equal logits in the order of their index
                order = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True).indices[:, :case["top"]]
                out["top_idx"] = order.to(torch.int32)
                out["top_logprob"] = torch.gather(lp, 1, order)
            return out
        return {"logprob": logprob, "entropy": entropy,
                "grad_logits": _plain_logit_gradient(s, live, p, lp, entropy)}
    if op.startswith("embed"):
        tok = s["tokens"].long()
        live = (tok >= 0)[:, None]
        out = s["table"][tok.clamp(min=0)].float() * case["scale"]
        out = torch.where(live, out, torch.zeros_like(out)).to(s["out"].dtype)
        if op == "embed":
            return out
        grad = torch.zeros((case["vocab"] + 1, case["dim"]), dtype=torch.float32, device="cuda")
        grad.index_add_(0, torch.where(tok >= 0, tok, case["vocab"]), s["grad_out"].float())
        return {"out": out, "grad_table": (grad[:-1] * case["scale"]).to(s["grad_table"].dtype)}
    if op == "orthogonalize":
        return _orthogonal(s["grad"].float(), STEPS).to(torch.bfloat16)
    grad = s["grad"].float()
    momentum = MU * s["momentum"] + grad
    update = _orthogonal(grad + MU * momentum, STEPS)
    w = s["w"].float() * (1.0 - LR * DECAY) - (LR * _gamma(case)) * update
    return {"w": w.to(torch.bfloat16), "momentum": momentum}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op.startswith("logprobs"):
        es = 2 if case["dtype"] == "bf16" else 4
        ix = 8 if case["index"] == "i64" else 4
        cells = case["rows"] * case["vocab"]
        small = case["rows"] * (case["tokens"] * (ix + 4) + 8 + case.get("top", 0) * 8)
        if op == "logprobs":
            return {"bytes": cells * es + small, "flops": 6 * cells}
        small += case["rows"] * (case["tokens"] * 4 + (4 if case["entropy"] else 0))
        return {"bytes": 2 * cells * es + small, "flops": 10 * cells}
    if op.startswith("embed"):
        es, ix = (2 if case["dtype"] == "bf16" else 4), (8 if case["index"] == "i64" else 4)
        n, dim, vocab = case["tokens"], case["dim"], case["vocab"]
        # rows that the ids touch: expected number of distinct ids at frequency 1 / (rank ln(V + 1))
        k = torch.arange(1, vocab + 1, dtype=torch.float64)
        distinct = float((-torch.expm1(n * torch.log1p(-(torch.log1p(1 / k) / math.log(vocab + 1.0))))).sum())
        total = n * ix + (distinct + n) * dim * es
        flops = n * dim
        if op == "embed_train":
            total += n * dim * es + vocab * dim * (2 if case["out"] == "bf16" else 4)
            flops += 2 * n * dim
        return {"bytes": total, "flops": flops}
    b, n, m = case["batch"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
    # a symmetric product has half its entries; the steps by X <- (aI + bA + cA^2) X, or all but the first and the
    # last product on the n x n side (A <- M A M, Q <- M Q, O = Q X), whichever is less
    direct = STEPS * (3 * n * n * m + n ** 3)
    gram = 3 * n * n * m + (4 * STEPS - 3) * n ** 3
    es = 2 if case["dtype"] == "bf16" else 4
    cells = b * n * m
    moved = cells * (es + 2) if op == "orthogonalize" else cells * (es + 8 + 4)
    return {"bytes": moved, "flops": b * min(direct, gram)}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("logprobs"):
        return _exact_logprobs(case, s)
    if op.startswith("embed"):
        tok = s["tokens"].cpu().numpy().astype(np.int64)
        keep = np.flatnonzero(tok >= 0)
        at = torch.from_numpy(tok[keep]).cuda()
        rows = torch.from_numpy(keep).cuda()
        out = torch.zeros((case["tokens"], case["dim"]), dtype=torch.float64, device="cuda")
        out[rows] = s["table"].index_select(0, at).double() * case["scale"]
        if op == "embed":
            return out
        grad = torch.zeros((case["vocab"], case["dim"]), dtype=torch.float64, device="cuda")
        grad.index_put_((at,), s["grad_out"].double()[rows] * case["scale"], accumulate=True)
        return {"out": out, "grad_table": grad}
    g = s["grad"].double()
    if op == "orthogonalize":
        return _exact_polar(g)
    momentum = MU * s["momentum"].double() + g
    u = _exact_polar(g + MU * momentum)
    return {"w": s["w"].double() - LR * (DECAY * s["w"].double() + _gamma(case) * u), "momentum": momentum}


def _exact_logprobs(case, s):
    x, tok = s["logits"], s["tokens"].long()
    rows, vocab, n = case["rows"], case["vocab"], case["tokens"]
    res = {"logprob": torch.zeros((rows, n), dtype=torch.float64, device="cuda"),
           "entropy": torch.zeros(rows, dtype=torch.float64, device="cuda")}
    top = case.get("top", 0)
    if case["op"] == "logprobs":
        res["lse"] = torch.zeros(rows, dtype=torch.float64, device="cuda")
        if top:
            res["top_idx"] = None
            res["top_logprob"] = torch.zeros((rows, top), dtype=torch.float64, device="cuda")
    else:
        res["grad_logits"] = torch.zeros((rows, vocab), dtype=torch.float64, device="cuda")
    step = max(1, (1 << 28) // vocab)
    for lo in range(0, rows, step):
        sl = slice(lo, min(rows, lo + step))
        y = x[sl].double() * case["scale"]
        lp = torch.log_softmax(y, dim=1)
        p = lp.exp()
        ent = torch.special.entr(p).sum(dim=1)
        t = tok[sl]
        res["entropy"][sl] = ent
        res["logprob"][sl] = torch.where(t >= 0, torch.take_along_dim(lp, t.clamp(min=0), 1), 0.0)
        if case["op"] == "logprobs":
            res["lse"][sl] = torch.logsumexp(y, dim=1)
            if top:
                res["top_logprob"][sl] = torch.topk(lp, top, dim=1).values
            continue
        up = torch.where(t >= 0, s["grad_logprob"][sl].double(), 0.0)
        d = torch.zeros_like(p).scatter_add_(1, t.clamp(min=0), up) - up.sum(dim=1, keepdim=True) * p
        if s["grad_entropy"] is not None:
            d += s["grad_entropy"][sl].double()[:, None] * (torch.special.entr(p) - ent[:, None] * p)
        res["grad_logits"][sl] = d * case["scale"]
    return res


def _exact_polar(g):
    """The singular values of g / |g| through STEPS polynomial steps, in float64, on the smaller side's
    eigenvectors' span: O = q(S) g / |g| with S = (g g^T) / |g|^2 and q built up by its factors."""
    tall = g.shape[1] > g.shape[2]
    x = (g.transpose(1, 2) if tall else g).contiguous()
    x = x / torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True)
    gram = torch.bmm(x, x.transpose(1, 2).contiguous())
    eye = torch.eye(gram.shape[1], dtype=torch.float64, device=g.device).expand_as(gram)
    total = None
    for _ in range(STEPS):
        factor = COEFFS[0] * eye + COEFFS[1] * gram + COEFFS[2] * torch.bmm(gram, gram)
        total = factor if total is None else torch.bmm(factor, total)
        gram = torch.bmm(factor, torch.bmm(gram, factor))
    o = torch.bmm(total, x)
    return (o.transpose(1, 2) if tall else o).contiguous()
