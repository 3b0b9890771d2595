"""Operators around an exported mixture-of-experts model and the model distilled from it, measured.

* the mixture-of-experts layer of a few tokens straight from the exported form
  (16-bit core indices of 8-weight groups and escape records): router, the
  chosen experts' gate, up and down products, their weighted sum;
* the adjustment of output logits before a token is chosen: penalties for
  tokens of the row's history, biases of given tokens, a grammar's bit mask;
* the distillation loss against a teacher's top logits and its gradient.

``run`` computes a case in plain torch operations (``own`` false) or with the
library's entry points (``own`` true).
"""

import functools
import math

import numpy as np
import torch

own = False


def listed():
    moe = {"op": "moe", "experts": 128, "hidden": 2048, "inter": 768, "top_k": 8, "bound": 16, "alpha": 3.0,
           "had_in": 128, "had_down": 128, "act": "silu", "normalize": True, "router": "bf16", "x": "bf16", "y": "bf16"}
    return [
        # one sequence's decode step through a layer of the mixture-of-experts workload
        {"name": "moe_1x128e_2048x768", **moe, "tokens": 1},
        # a few sequences (or drafted tokens) through a small layer of odd sizes: a wider core, small rotation blocks
        {"name": "moe_5x9e_520x328_f32", **moe, "tokens": 5, "experts": 9, "hidden": 520, "inter": 328, "top_k": 2,
         "bound": 24, "alpha": 2.5, "had_in": 8, "had_down": 8, "act": "gelu_tanh", "normalize": False,
         "router": "f32", "x": "f32", "y": "f32"},
        # a small served batch: about half of the experts are met, by one or two tokens each
        {"name": "moe_16x128e_2048x768", **moe, "tokens": 16},
        # a full served batch: nearly every expert, four tokens each
        {"name": "moe_64x128e_2048x768", **moe, "tokens": 64},
        # one sequence: penalties from 700 tokens of history, a few biased tokens
        {"name": "adjust_1x131072_bf16", "op": "adjust", "rows": 1, "vocab": 131072, "pad": 0, "dtype": "bf16",
         "history": 700, "repetition": True, "counts": True, "bias": 16, "mask": False, "index": "i64"},
        # constrained decoding of a served batch with an odd vocabulary out of a wider buffer
        {"name": "adjust_48x50001_f32_mask", "op": "adjust", "rows": 48, "vocab": 50001, "pad": 175, "dtype": "f32",
         "history": 1500, "repetition": False, "counts": True, "bias": 300, "mask": True, "index": "i32"},
        # a large served batch with long histories, everything at once
        {"name": "adjust_512x131072_bf16_all", "op": "adjust", "rows": 512, "vocab": 131072, "pad": 0,
         "dtype": "bf16", "history": 8192, "repetition": True, "counts": True, "bias": 64, "mask": True,
         "index": "i64"},
        # held-out loss against a stored teacher, a small batch
        {"name": "distill_eval_64x50001_f32_k20", "op": "distill_eval", "rows": 64, "vocab": 50001, "pad": 175,
         "dtype": "f32", "k": 20, "scale": 1.0, "tail": "none", "index": "i32"},
        # training through the loss with upstream gradients: forward call, then backward call, rest of the mass kept
        {"name": "distill_train_301x32003_f32_k16", "op": "distill_train", "rows": 301, "vocab": 32003, "pad": 0,
         "dtype": "f32", "k": 16, "scale": 0.5, "tail": "rest", "index": "i64"},
        # a training step whose row weights are known beforehand: loss and gradient in one call
        {"name": "distill_grad_4096x32768_bf16_k32", "op": "distill_grad", "rows": 4096, "vocab": 32768, "pad": 0,
         "dtype": "bf16", "k": 32, "scale": 1.0, "tail": "renorm", "index": "i32"},
        # the same at a large vocabulary
        {"name": "distill_grad_8192x131072_bf16_k64", "op": "distill_grad", "rows": 8192, "vocab": 131072, "pad": 0,
         "dtype": "bf16", "k": 64, "scale": 1.0, "tail": "rest", "index": "i32"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["moe", "moe", "adjust", "adjust", "distill_eval", "distill_train", "distill_grad"])
    if op == "moe":
        had_in, had_down = rng.choice([0, 8, 32, 128, 128, 256]), rng.choice([0, 8, 64, 128, 128])
        step_in, step_down = max(8, had_in), max(8, had_down)
        hidden = step_in * max(1, _log_int(rng, 64, 4096) // step_in)
        inter = step_down * max(1, _log_int(rng, 64, 2048) // step_down)
        experts = _log_int(rng, 2, 128)
        experts = max(2, min(experts, 128 * 2048 * 768 // (hidden * inter)))
        return {"op": op, "experts": experts, "hidden": hidden, "inter": inter,
                "top_k": rng.randrange(1, min(8, experts) + 1), "bound": rng.choice([8, 16, 16, 24, 40]),
                "alpha": rng.choice([2.5, 3.0, 3.0]), "had_in": had_in, "had_down": had_down,
                "act": rng.choice(["silu", "silu", "gelu_tanh"]), "normalize": rng.random() < 0.7,
                "router": rng.choice(["bf16", "f32"]), "x": rng.choice(["bf16", "f32"]),
                "y": rng.choice(["bf16", "f32"]), "tokens": _log_int(rng, 1, 64)}
    rows, vocab = _log_int(rng, 1, 8192), _log_int(rng, 512, 131072)
    pad, dtype, index = rng.choice([0, 0, rng.randrange(1, 200)]), rng.choice(["bf16", "f32"]), rng.choice(["i64", "i32"])
    if op == "adjust":
        rows = max(1, min(rows, 512 * 131072 // (2 if dtype == "f32" else 1) // vocab))
        history = min(_log_int(rng, 1, 8192), max(1, (1 << 22) // rows))
        return {"op": op, "rows": rows, "vocab": vocab, "pad": pad, "dtype": dtype, "history": history,
                "repetition": rng.random() < 0.6, "counts": rng.random() < 0.8, "bias": rng.choice([0, 1, 20, 300]),
                "mask": rng.random() < 0.5, "index": index}
    most = 8192 * 131072 // (2 if dtype == "f32" else 1)
    if op == "distill_eval":
        most //= 4
    return {"op": op, "rows": max(1, min(rows, most // vocab)), "vocab": vocab, "pad": pad, "dtype": dtype,
            "k": rng.choice([1, 5, 16, 50, 128]), "scale": rng.choice([1.0, 0.5]),
            "tail": rng.choice(["none", "renorm", "rest"]), "index": index}


# ---------------------------------------------------------------- inputs

_DT = {"bf16": torch.bfloat16, "f32": torch.float32, "i64": torch.int64, "i32": torch.int32}
_TAIL = {"none": 0, "renorm": 1, "rest": 2}
_ACT = {"silu": 0, "gelu_tanh": 1}


@functools.lru_cache(maxsize=None)
def _core_points(bound):
    """2z of the E8 points with |2z|^2 <= bound in lexicographic order, int8 [n, 8]."""
    most = math.isqrt(bound)
    found = []
    for parity in (0, 1):
        values = np.array([v for v in range(-most, most + 1) if v % 2 == parity], dtype=np.int8)
        if not len(values):
            continue
        pts = np.zeros((1, 0), dtype=np.int8)
        for _ in range(8):                                   # prefixes within the bound
            pts = np.concatenate([np.repeat(pts, len(values), axis=0), np.tile(values, len(pts))[:, None]], axis=1)
            pts = pts[(pts.astype(np.int32) ** 2).sum(axis=1) <= bound]
        found.append(pts[pts.astype(np.int32).sum(axis=1) % 4 == 0])
    pts = np.concatenate(found)
    return pts[np.lexsort(pts.T[::-1])]


def _nearest_e8(x):
    """2z (int64) of the E8 point nearest to each row of x [n, 8]: the better of the nearest points of D8 and D8 + 1/2."""
    best = None
    for shift in (0.0, 0.5):
        n = torch.round(x - shift)
        err = x - shift - n
        worst = err.abs().argmax(dim=1, keepdim=True)
        move = torch.where(torch.gather(err, 1, worst) >= 0, 1.0, -1.0)
        odd = (n.sum(dim=1, keepdim=True) % 2 != 0).to(x.dtype)
        y = n.scatter_add(1, worst, move * odd) + shift
        d = ((x - y) ** 2).sum(dim=1, keepdim=True)
        best = (y, d) if best is None else (torch.where(d < best[1], y, best[0]), torch.minimum(d, best[1]))
    return (2 * best[0]).long()


def _exported(experts, rows, cols, bound, alpha, g):
    """The exported form of [experts, rows, cols] weights that are normal with deviation 0.02 in the rotated basis (as
    rotated weights are), at scale alpha x row RMS: core indices, escape records, their counts and the row scales."""
    pts = torch.from_numpy(_core_points(bound)).cuda().long()
    weights = 128 ** torch.arange(7, -1, -1, device="cuda")
    keys = ((pts + 64) * weights).sum(dim=1)
    idx = torch.empty((experts, rows * cols // 8), dtype=torch.int16, device="cuda")
    records, counts = [], []
    for e in range(experts):
        z = _nearest_e8(torch.randn((rows * cols // 8, 8), generator=g, device="cuda") / alpha)
        key = ((z + 64) * weights).sum(dim=1)
        at = torch.searchsorted(keys, key).clamp_(max=len(keys) - 1)
        core = keys[at] == key
        idx[e] = torch.where(core, at, 0xFFFF).to(torch.int16)
        out = (~core).nonzero()[:, 0]
        rec = torch.empty((len(out), 5), dtype=torch.int32, device="cuda")
        rec[:, 0] = out.to(torch.int32)
        rec[:, 1:] = z[out].to(torch.int16).view(torch.int32)
        records.append(rec)
        counts.append(len(out))
    spread = 1.0 + 0.1 * torch.randn(experts * rows, generator=g, device="cuda").clamp(-3, 3)
    return {"core_idx": idx.view(-1), "esc": torch.cat(records).view(torch.uint8).view(-1),
            "esc_count": torch.tensor(counts, dtype=torch.int64, device="cuda"),
            "row_scale": 0.02 * alpha * spread, "shape": (experts, rows, cols)}


def _signs(cols, had, g):
    if not had:
        return None
    return (torch.randint(0, 2, (cols,), generator=g, device="cuda") * 2 - 1).to(torch.int8)


def _prepare_moe(case, g, s):
    e, h, f, t = case["experts"], case["hidden"], case["inter"], case["tokens"]
    for name, rows, cols in (("gate", f, h), ("up", f, h), ("down", h, f)):
        s[name] = _exported(e, rows, cols, case["bound"], case["alpha"], g)
    s["signs_in"], s["signs_down"] = _signs(h, case["had_in"], g), _signs(f, case["had_down"], g)
    x = torch.randn((t, h), generator=g, device="cuda")
    x[:, torch.randint(0, h, (max(1, h // 500),), generator=g, device="cuda")] *= 12.0      # a few strong channels
    s["x"] = x.to(_DT[case["x"]])
    s["router"] = (torch.randn((e, h), generator=g, device="cuda") / math.sqrt(h)).to(_DT[case["router"]])
    s["expert_idx"] = torch.empty((t, case["top_k"]), dtype=torch.int32, device="cuda")
    s["expert_weight"] = torch.empty((t, case["top_k"]), dtype=torch.float32, device="cuda")
    s["y"] = torch.empty((t, h), dtype=_DT[case["y"]], device="cuda")


def _text(shape, vocab, g):
    """Token ids of text: frequency about 1 / rank, ranks spread over the vocabulary."""
    u = torch.rand(shape, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(vocab + 1.0)).long().clamp_(1, vocab) - 1
    return (rank * 40503 + 17) % vocab


def _prepare_adjust(case, g, s):
    rows, vocab, ix = case["rows"], case["vocab"], _DT[case["index"]]
    full = torch.empty((rows, vocab + case["pad"]), dtype=_DT[case["dtype"]], device="cuda").normal_(0.0, 3.0, generator=g)
    s["logits"], s["out"] = full[:, :vocab], torch.empty_like(full)[:, :vocab]
    n = case["history"]
    s["history"] = _text((rows, n), vocab, g).to(ix)
    length = torch.randint(0 if rows > 4 else n, n + 1, (rows,), generator=g, device="cuda")
    prompt = (torch.rand(rows, generator=g, device="cuda") * (length + 1)).long()
    s["history_len"], s["prompt_len"] = length.to(torch.int32), prompt.to(torch.int32)
    pick = lambda lo, hi: lo + (hi - lo) * torch.rand(rows, generator=g, device="cuda")  # noqa: E731
    s["repetition"] = pick(1.0, 1.3) if case["repetition"] else None
    s["frequency"] = pick(0.0, 0.8) if case["counts"] else None
    s["presence"] = pick(-0.2, 0.8) if case["counts"] else None
    s["bias_idx"] = s["bias"] = s["mask"] = None
    if case["bias"]:
        s["bias_idx"] = torch.randint(0, vocab, (rows, case["bias"]), generator=g, device="cuda").to(ix)
        s["bias"] = 4.0 * torch.randn((rows, case["bias"]), generator=g, device="cuda")
    if case["mask"]:
        # a grammar allows a few tokens of some rows and nearly all of others
        words = (vocab + 31) // 32
        rate = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.5, 0.002, 0.95)
        mask = torch.zeros((rows, words), dtype=torch.int32, device="cuda")
        for b in range(32):
            bit = torch.rand((rows, words), generator=g, device="cuda") < rate[:, None]
            mask |= bit.to(torch.int32) << b
        s["mask"] = mask


def _prepare_distill(case, g, s):
    rows, vocab, k = case["rows"], case["vocab"], case["k"]
    x = torch.empty((rows, vocab + case["pad"]), dtype=_DT[case["dtype"]], device="cuda").normal_(0.0, 2.0, generator=g)
    # the teacher's places: one in each k-th of the vocabulary (distinct), falling probabilities, a rest of 1 to 30 percent
    step = max(1, vocab // k)
    idx = torch.randint(0, step, (rows, k), generator=g, device="cuda") + torch.arange(k, device="cuda") * step
    idx = torch.gather(idx, 1, torch.argsort(torch.rand((rows, k), generator=g, device="cuda"), dim=1))
    z = 6.0 * torch.rand((rows, k), generator=g, device="cuda")
    rest = 0.01 + 0.29 * torch.rand((rows, 1), generator=g, device="cuda")
    lp, order = torch.sort(torch.log_softmax(z, dim=1) + torch.log1p(-rest), dim=1, descending=True)
    idx = torch.gather(idx, 1, order)
    # the student likes about the same tokens
    lift = (z + 7.0 + torch.randn((rows, k), generator=g, device="cuda")) / case["scale"]
    x.scatter_(1, idx, torch.gather(lift, 1, order).to(x.dtype))
    if rows > 16:
        idx[torch.rand(rows, generator=g, device="cuda") < 0.05] = -1                 # positions without a target
        short = torch.rand((rows, 1), generator=g, device="cuda") < 0.1               # rows with fewer places
        idx = torch.where(short & (torch.arange(k, device="cuda") >= (k + 1) // 2), -1, idx)
    s["logits"] = x[:, :vocab]
    s["teacher_idx"], s["teacher_logprob"] = idx.to(_DT[case["index"]]), lp
    f32 = {"dtype": torch.float32, "device": "cuda"}
    s["loss"] = torch.empty(rows, **f32)
    if case["op"] == "distill_eval":
        s["logprob"] = torch.empty((rows, k), **f32)
    else:
        s["stats"] = torch.empty((rows, 4), **f32)
        s["grad_loss"] = torch.rand(rows, generator=g, **f32) + 0.5
        s["grad_logits"] = torch.empty_like(x)[:, :vocab]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": dict(case), "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["op"] == "moe":
        _prepare_moe(case, g, s)
    elif case["op"] == "adjust":
        _prepare_adjust(case, g, s)
    else:
        _prepare_distill(case, g, s)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _workspace(s, e8q):
    """The device scratch that a program keeps for its calls: made on the first pass."""
    if "ws" not in s:
        case = s["case"]
        if case["op"] == "moe":
            size = e8q.e8q_moe_workspace_size(case["experts"], case["hidden"], case["inter"], case["tokens"],
                                              case["top_k"])
        else:
            size = e8q.e8q_distill_workspace_size(case["rows"], case["vocab"], case["k"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s["ws"]


def _run_own(s):
    import bit_e8_lattice_amd as e8q
    case = s["case"]
    op = case["op"]
    if op == "moe":
        if "experts" not in s:
            s["experts"] = [e8q.Experts(s[n]["core_idx"], s[n]["esc"], s[n]["esc_count"], s[n]["row_scale"], s[n]["shape"])
                            for n in ("gate", "up", "down")]
        e8q.e8q_moe_core_escape(*s["experts"], case["bound"], s["x"], s["expert_idx"], s["expert_weight"], s["y"],
                                _workspace(s, e8q), s["status"], router=s["router"], signs_in=s["signs_in"],
                                had_block_in=case["had_in"], signs_down=s["signs_down"],
                                had_block_down=case["had_down"], activation=_ACT[case["act"]],
                                normalize=case["normalize"])
        return {"y": s["y"], "expert_idx": s["expert_idx"], "expert_weight": s["expert_weight"]}
    if op == "adjust":
        e8q.e8q_adjust_logits(s["logits"], s["out"], s["status"], history=s["history"], history_len=s["history_len"],
                              prompt_len=s["prompt_len"], repetition=s["repetition"], frequency=s["frequency"],
                              presence=s["presence"], bias_idx=s["bias_idx"], bias=s["bias"], mask=s["mask"])
        return s["out"]
    ws, tail = _workspace(s, e8q), _TAIL[case["tail"]]
    if op == "distill_eval":
        e8q.e8q_distill(s["logits"], s["teacher_idx"], s["teacher_logprob"], ws, s["status"], scale=case["scale"],
                        tail=tail, loss_out=s["loss"], logprob_out=s["logprob"])
        return {"loss": s["loss"], "logprob": s["logprob"]}
    if op == "distill_train":
        e8q.e8q_distill(s["logits"], s["teacher_idx"], s["teacher_logprob"], ws, s["status"], scale=case["scale"],
                        tail=tail, loss_out=s["loss"], stats_out=s["stats"])
        e8q.e8q_distill_backward(s["logits"], s["teacher_idx"], s["teacher_logprob"], s["stats"], s["grad_loss"],
                                 s["grad_logits"], s["status"], scale=case["scale"], tail=tail)
    else:
        e8q.e8q_distill_grad(s["logits"], s["teacher_idx"], s["teacher_logprob"], s["grad_loss"], s["grad_logits"], ws,
                             s["status"], scale=case["scale"], tail=tail, loss_out=s["loss"])
    return {"loss": s["loss"], "grad_logits": s["grad_logits"]}


# ---------------------------------------------------------------- the plain forms

def _rotate(x, signs, block):
    """kappa H (sign * x) in blocks of the last axis."""
    if signs is None:
        return x
    n = x.shape[-1]
    v = (x * signs).reshape(-1, n // block, block)
    width = 1
    while width < block:
        v = v.reshape(v.shape[0], n // block, block // (2 * width), 2, width)
        v = torch.stack((v[:, :, :, 0] + v[:, :, :, 1], v[:, :, :, 0] - v[:, :, :, 1]), dim=3)
        v = v.reshape(v.shape[0], n // block, block)
        width *= 2
    return v.reshape(x.shape) * (1.0 / math.sqrt(block))


def _plain_products(m, points, which, vectors):
    """W_hat x in the rotated basis of each route: expert which[i] on vectors[i]; a few routes at a time."""
    experts, rows, cols = m["shape"]
    groups = rows * cols // 8
    rec = m["esc"].view(torch.int32).view(-1, 5)
    owner = torch.repeat_interleave(torch.arange(experts, device="cuda"), m["esc_count"], output_size=len(rec))
    table = torch.cat([points, rec[:, 1:].contiguous().view(torch.int16).float()])
    idx = m["core_idx"].to(torch.int32).bitwise_and(0xFFFF)
    idx.index_copy_(0, owner * groups + rec[:, 0].long(), torch.arange(len(rec), dtype=torch.int32, device="cuda") + len(points))
    idx, scale = idx.view(experts, groups), m["row_scale"].view(experts, rows)
    out = torch.empty((len(which), rows), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (rows * cols))
    for lo in range(0, len(which), step):
        e = which[lo:lo + step]
        z = table.index_select(0, idx.index_select(0, e).view(-1)).view(-1, rows, cols)
        out[lo:lo + step] = torch.matmul(z, vectors[lo:lo + step, :, None])[:, :, 0] * (0.5 * scale.index_select(0, e))
    return out


def _plain_moe(s):
    case = s["case"]
    t, k = case["tokens"], case["top_k"]
    # logits next to the border of the chosen ones: 64 bits
    logits = torch.matmul(s["x"].double(), s["router"].double().t().contiguous())
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    prob = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    weight = torch.gather(prob, 1, order)
    weight = (weight / (weight if case["normalize"] else prob).sum(dim=1, keepdim=True)).float()
    points = torch.from_numpy(_core_points(case["bound"])).cuda().float()
    which = order.reshape(-1)
    x = _rotate(s["x"].float(), s["signs_in"], case["had_in"]).repeat_interleave(k, dim=0)
    gate, up = (_plain_products(s[n], points, which, x) for n in ("gate", "up"))
    if case["act"] == "silu":
        act = gate / (1.0 + torch.exp(-gate))
    else:
        act = 0.5 * gate * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (gate + 0.044715 * gate * gate * gate)))
    down = _plain_products(s["down"], points, which, _rotate(act * up, s["signs_down"], case["had_down"]))
    y = (down.view(t, k, -1) * weight[:, :, None]).sum(dim=1)
    return {"y": y.to(s["y"].dtype), "expert_idx": order.to(torch.int32), "expert_weight": weight}


def _plain_adjust(s):
    case = s["case"]
    x = s["logits"].float()
    rows, vocab = x.shape
    hist = s["history"].long()
    at = torch.arange(hist.shape[1], device="cuda")
    live, made = at < s["history_len"][:, None], at >= s["prompt_len"][:, None]
    if case["repetition"]:
        seen = torch.zeros((rows, vocab), dtype=torch.float32, device="cuda").scatter_add_(1, hist, live.float()) > 0
        r = s["repetition"][:, None]
        x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    if case["counts"]:
        count = torch.zeros((rows, vocab), dtype=torch.float32, device="cuda").scatter_add_(1, hist, (live & made).float())
        x = x - (s["frequency"][:, None] * count + s["presence"][:, None] * (count > 0))
    if case["bias"]:
        x = x.scatter_add(1, s["bias_idx"].long(), s["bias"])
    if case["mask"]:
        col = torch.arange(vocab, device="cuda")
        bit = (s["mask"][:, col >> 5] >> (col & 31).to(torch.int32)) & 1
        x = torch.where(bit != 0, x, -math.inf)
    return x.to(s["out"].dtype)


def _plain_distill(s):
    case = s["case"]
    y = s["logits"].float() * case["scale"]
    m = y.amax(dim=1, keepdim=True)
    e = torch.exp(y - m)
    total = e.sum(dim=1, keepdim=True)
    lse = m + torch.log(total)
    idx = s["teacher_idx"].long()
    live = idx >= 0
    at = idx.clamp(min=0)
    t_lp = s["teacher_logprob"]
    p = torch.where(live, torch.exp(t_lp), 0.0)
    mass = p.sum(dim=1, keepdim=True)
    if case["tail"] == "renorm":
        t_lp = t_lp - torch.log(mass)
        p = torch.where(live, p / mass, 0.0)
    lq = torch.where(live, torch.gather(y, 1, at) - lse, 0.0)
    loss = torch.where(live, p * (t_lp - lq), 0.0).sum(dim=1)
    if case["tail"] == "rest":
        out = torch.cat([e, torch.zeros_like(total)], dim=1).scatter_(1, torch.where(live, at, y.shape[1]), 0.0)[:, :-1]
        rest = out.sum(dim=1, keepdim=True) / total
        p_rest = (1.0 - mass).clamp(min=0.0)
        loss = loss + torch.where(p_rest > 0, p_rest * (torch.log(p_rest) - torch.log(rest)), 0.0)[:, 0]
    if case["op"] == "distill_eval":
        return {"loss": loss, "logprob": lq}
    g = s["grad_loss"][:, None] * case["scale"]
    if case["tail"] == "rest":
        d = out / total * (1.0 - p_rest / rest)
        d = torch.cat([d, torch.zeros_like(total)], dim=1)
        d = d.scatter_(1, torch.where(live, at, y.shape[1]), torch.exp(lq) - p)[:, :-1]
    else:
        d = (e / total * p.sum(dim=1, keepdim=True)).scatter_add(1, at, -p)
    return {"loss": loss, "grad_logits": (d * g).to(s["logits"].dtype)}


def _run_plain(s):
    op = s["case"]["op"]
    return _plain_moe(s) if op == "moe" else _plain_adjust(s) if op == "adjust" else _plain_distill(s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "moe":
        e, h, f, t, k = (case[n] for n in ("experts", "hidden", "inter", "tokens", "top_k"))
        met = e * (1.0 - (1.0 - k / e) ** t)                  # experts that some token chooses, on average
        weights = met * 3 * h * f
        moved = (weights / 4 + met * (2 * f + h) * 4 + e * h * (2 if case["router"] == "bf16" else 4) +
                 t * h * ((2 if case["x"] == "bf16" else 4) + (2 if case["y"] == "bf16" else 4)) + t * k * 8)
        return {"bytes": int(moved), "flops": 2 * t * (3 * k * h * f + e * h)}
    es, ix = (2 if case["dtype"] == "bf16" else 4), (8 if case["index"] == "i64" else 4)
    rows, cells = case["rows"], case["rows"] * case["vocab"]
    if op == "adjust":
        used = case["history"] // 2 if rows > 4 else case["history"]
        small = rows * ((used * ix if case["repetition"] or case["counts"] else 0) + case["bias"] * (ix + 4) + 20)
        return {"bytes": 2 * cells * es + (cells // 8 if case["mask"] else 0) + small, "flops": cells}
    small = rows * (case["k"] * (ix + 4) + 8)
    if op == "distill_eval":
        return {"bytes": cells * es + small + rows * case["k"] * 4, "flops": 4 * cells}
    return {"bytes": 2 * cells * es + small, "flops": 7 * cells}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "moe":
        return _exact_moe(case, s)
    if case["op"] == "adjust":
        return _exact_adjust(case, s)
    return _exact_distill(case, s)


def _restored(m, e, bound, signs, block):
    """The expert's restored weights R^T (s z) in float64 [rows, cols]."""
    _, rows, cols = m["shape"]
    pts = torch.from_numpy(_core_points(bound)).cuda()
    idx = m["core_idx"].view(m["shape"][0], -1)[e].long() % 65536
    core = idx < len(pts)
    z = torch.where(core[:, None], pts[idx.clamp(max=len(pts) - 1)], 0).double()
    first = int(m["esc_count"][:e].sum())
    rec = m["esc"].view(-1, 20)[first:first + int(m["esc_count"][e])].contiguous()
    z[rec[:, :4].contiguous().view(torch.int32)[:, 0].long()] = rec[:, 4:].contiguous().view(torch.int16).double()
    w = z.view(rows, cols) * (0.5 * m["row_scale"].view(-1, rows)[e].double())[:, None]
    if signs is None:
        return w
    h = torch.ones((1, 1), dtype=torch.float64, device="cuda")
    while h.shape[0] < block:
        h = torch.kron(torch.tensor([[1.0, 1.0], [1.0, -1.0]], dtype=torch.float64, device="cuda"), h)
    w = torch.mm(w.view(-1, block), h).view(rows, cols) / math.sqrt(block)
    return w * signs.double()


def _exact_moe(case, s):
    t, k = case["tokens"], case["top_k"]
    x = s["x"].double()
    prob = torch.softmax(torch.mm(x, s["router"].double().t().contiguous()), dim=1)
    weight, which = torch.topk(prob, k, dim=1)
    if case["normalize"]:
        weight = weight / weight.sum(dim=1, keepdim=True)
    y = torch.zeros((t, case["hidden"]), dtype=torch.float64, device="cuda")
    for e in torch.unique(which).tolist():
        tok, place = (which == e).nonzero(as_tuple=True)
        gate, up = (torch.mm(x[tok], _restored(s[n], e, case["bound"], s["signs_in"], case["had_in"]).t().contiguous())
                    for n in ("gate", "up"))
        if case["act"] == "silu":
            h = torch.nn.functional.silu(gate) * up
        else:
            h = torch.nn.functional.gelu(gate, approximate="tanh") * up
        down = torch.mm(h, _restored(s["down"], e, case["bound"], s["signs_down"], case["had_down"]).t().contiguous())
        y.index_add_(0, tok, down * weight[tok, place][:, None])
    return {"y": y, "expert_idx": None, "expert_weight": weight}


def _exact_adjust(case, s):
    rows, vocab = case["rows"], case["vocab"]
    res = torch.empty((rows, vocab), dtype=torch.float64, device="cuda")
    step = max(1, (1 << 27) // vocab)
    at = torch.arange(case["history"], device="cuda")
    for lo in range(0, rows, step):
        sl = slice(lo, min(rows, lo + step))
        x = s["logits"][sl].double()
        n = x.shape[0]
        row = torch.arange(n, device="cuda")[:, None].expand(n, case["history"])
        hist, live = s["history"][sl].long(), at < s["history_len"][sl][:, None]
        made = live & (at >= s["prompt_len"][sl][:, None])
        if case["repetition"]:
            seen = torch.zeros((n, vocab), dtype=torch.bool, device="cuda")
            seen[row[live], hist[live]] = True
            r = s["repetition"][sl].double()[:, None]
            x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
        if case["counts"]:
            count = torch.bincount(row[made] * vocab + hist[made], minlength=n * vocab).view(n, vocab).double()
            x = x - s["frequency"][sl].double()[:, None] * count
            x = x - s["presence"][sl].double()[:, None] * (count > 0).double()
        if case["bias"]:
            where = torch.arange(n, device="cuda")[:, None].expand(n, case["bias"])
            x = x.index_put((where, s["bias_idx"][sl].long()), s["bias"][sl].double(), accumulate=True)
        if case["mask"]:
            bits = (s["mask"][sl][:, :, None] >> torch.arange(32, dtype=torch.int32, device="cuda")) & 1
            x = x.masked_fill(bits.reshape(n, -1)[:, :vocab] == 0, -math.inf)
        res[sl] = x
    return res


def _exact_distill(case, s):
    rows, vocab, k = case["rows"], case["vocab"], case["k"]
    f64 = {"dtype": torch.float64, "device": "cuda"}
    res = {"loss": torch.empty(rows, **f64)}
    if case["op"] == "distill_eval":
        res["logprob"] = torch.empty((rows, k), **f64)
    else:
        res["grad_logits"] = torch.empty((rows, vocab), **f64)
    step = max(1, (1 << 27) // vocab)
    for lo in range(0, rows, step):
        sl = slice(lo, min(rows, lo + step))
        lq_all = torch.log_softmax(s["logits"][sl].double() * case["scale"], dim=1)
        n = lq_all.shape[0]
        idx = s["teacher_idx"][sl].long()
        live = idx >= 0
        p = torch.where(live, s["teacher_logprob"][sl].double().exp(), 0.0)
        if case["tail"] == "renorm":
            p = p / p.sum(dim=1, keepdim=True).clamp(min=1e-300)
        lq = torch.where(live, torch.take_along_dim(lq_all, idx.clamp(min=0), 1), 0.0)
        loss = torch.xlogy(p, p).sum(dim=1) - (p * lq).sum(dim=1)
        named = torch.zeros((n, vocab + 1), dtype=torch.bool, device="cuda")
        named.scatter_(1, torch.where(live, idx, vocab), True)
        named = named[:, :vocab]
        if case["tail"] == "rest":
            lq_rest = torch.logsumexp(lq_all.masked_fill(named, -math.inf), dim=1)
            p_rest = (1.0 - p.sum(dim=1)).clamp(min=0.0)
            loss = loss + torch.xlogy(p_rest, p_rest) - p_rest * lq_rest
        res["loss"][sl] = loss
        if case["op"] == "distill_eval":
            res["logprob"][sl] = lq
            continue
        # d loss / d y = q sum(p) - p, and of the rest - p_rest (q in the rest / q_rest - q)
        q = lq_all.exp()
        total = torch.zeros((n, vocab + 1), **f64).scatter_add_(1, torch.where(live, idx, vocab), p)[:, :vocab]
        d = q * p.sum(dim=1, keepdim=True) - total
        if case["tail"] == "rest":
            d = d - p_rest[:, None] * (torch.exp(lq_all - lq_rest[:, None]).masked_fill(named, 0.0) - q)
        res["grad_logits"][sl] = d * (s["grad_loss"][sl].double()[:, None] * case["scale"])
    return res
