"""Measured cases of the operators that sit around the vocabulary head.

Three families, each in both directions:

* layer norm of the rows that the head reads (``norm_fwd``, ``norm_bwd``);
* distillation from a teacher's top logits, on logits the caller holds
  (``distill_logits_fwd``, ``distill_logits_bwd``) and through the head, whose
  [T, V] logits never exist (``distill_head_fwd``, ``distill_head_train``);
* penalties for repeated tokens, biases and grammar masks on logits
  (``process_fwd``, ``process_bwd``).

``run`` computes a case with elementary torch operations in 32 bits, or, when
``own`` is true, with the calls a user makes of this package.  ``exact`` is the
definition in 64 bits.
"""
import math

import torch

own = False

_DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
_BYTES = {"float32": 4, "bfloat16": 2, "float16": 2}
_EPS = 1e-5


def listed():
    return [
        # The final norm of one decoded token before the head's scores.
        {"name": "norm fwd, one token", "op": "norm_fwd", "rows": 1, "width": 2560,
         "dtype": "bfloat16", "bias": True},
        # The final norm of a training batch of sixteen 4,096-token rows.
        {"name": "norm fwd, 65536 rows", "op": "norm_fwd", "rows": 65536, "width": 2560,
         "dtype": "bfloat16", "bias": True},
        # Its backward for one 4,096-token row: the head hands over fp32 gradients.
        {"name": "norm bwd, 4096 rows", "op": "norm_bwd", "rows": 4096, "width": 2560,
         "dtype": "bfloat16", "grad_dtype": "float32", "bias": True},
        # An odd width in fp32, without a bias, on a packed row of odd length.
        {"name": "norm bwd, odd fp32", "op": "norm_bwd", "rows": 5431, "width": 1111,
         "dtype": "float32", "grad_dtype": "float32", "bias": False},
        # The distillation loss of the last three tokens of a trace, whose table is padded.
        {"name": "distill logits fwd, 3 rows", "op": "distill_logits_fwd", "rows": 3,
         "vocab": 151936, "pad": 64, "k": 20, "dtype": "bfloat16", "tau": 1.0, "mask": 0.0,
         "normalised": False},
        # One 512-token chunk of a chunked trainer that holds the chunk's fp32 logits.
        {"name": "distill logits fwd, chunk", "op": "distill_logits_fwd", "rows": 512,
         "vocab": 151936, "pad": 0, "k": 64, "dtype": "float32", "tau": 0.7, "mask": 0.0,
         "normalised": True},
        # The gradient of four such chunks in bf16, a quarter of the tokens unscored.
        {"name": "distill logits bwd, 2048 rows", "op": "distill_logits_bwd", "rows": 2048,
         "vocab": 151936, "pad": 0, "k": 128, "dtype": "bfloat16", "tau": 0.7, "mask": 0.25,
         "normalised": False},
        # The loss alone (evaluation) of a 4,096-token row through the head.
        {"name": "distill head fwd, 4096 rows", "op": "distill_head_fwd", "rows": 4096,
         "width": 2560, "vocab": 151936, "k": 64, "tau": 1.0, "mask": 0.0, "normalised": True},
        # A training step's loss and gradients, with the prompt's tokens unscored.
        {"name": "distill head train, 2048 rows", "op": "distill_head_train", "rows": 2048,
         "width": 2560, "vocab": 151936, "k": 64, "tau": 0.7, "mask": 0.3, "normalised": False},
        # One request's next token: 900 tokens of history, a grammar, a few biases.
        {"name": "process fwd, one request", "op": "process_fwd", "rows": 1, "vocab": 151936,
         "dtype": "float32", "history": 900, "shared": False, "biases": 12, "grammar": 1.0},
        # One step of a large batch: ragged histories, a grammar on half of the rows.
        {"name": "process fwd, 256 requests", "op": "process_fwd", "rows": 256, "vocab": 151936,
         "dtype": "bfloat16", "history": 8192, "shared": False, "biases": 300, "grammar": 0.5},
        # Scoring a sampled trace under the sampler's penalties: every position's history is
        # a prefix of the same tokens; the vocabulary is odd.
        {"name": "process bwd, 512 positions", "op": "process_bwd", "rows": 512, "vocab": 50257,
         "dtype": "float32", "history": 2048, "shared": True, "biases": 0, "grammar": 0.25},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "distill_logits_fwd", "distill_logits_bwd",
                     "distill_head_fwd", "distill_head_train", "process_fwd", "process_bwd"])
    if op.startswith("norm"):
        width = _log(rng, 64, 8192)
        width = width if rng.random() < 0.4 else max(64, width // 64 * 64)
        c = {"op": op, "rows": min(_log(rng, 1, 65536), 65536 * 2560 // width), "width": width,
             "dtype": rng.choice(sorted(_DTYPES)), "bias": rng.random() < 0.7}
        if op == "norm_bwd":
            c["grad_dtype"] = rng.choice(["float32", c["dtype"]])
        return c
    if op.startswith("distill_logits"):
        vocab = _log(rng, 1000, 151936)
        return {"op": op, "rows": min(_log(rng, 1, 8192), 2048 * 151936 // 2 // vocab),
                "vocab": vocab, "pad": rng.choice([0, 0, 1, 64]), "k": _log(rng, 1, 256),
                "dtype": rng.choice(sorted(_DTYPES)), "tau": rng.choice([1.0, 0.7, 2.0]),
                "mask": rng.choice([0.0, 0.3]), "normalised": rng.random() < 0.5}
    if op.startswith("distill_head"):
        vocab, width = _log(rng, 2000, 151936), 64 * _log(rng, 4, 64)
        most = 2048 * 2560 * 151936 // (vocab * width)
        return {"op": op, "rows": max(256, min(_log(rng, 256, 4096), most)), "width": min(width, 2560)
                if most < 256 else width, "vocab": vocab, "k": _log(rng, 1, 128),
                "tau": rng.choice([1.0, 0.7]), "mask": rng.choice([0.0, 0.3]),
                "normalised": rng.random() < 0.5}
    vocab = _log(rng, 1000, 151936)
    shared = rng.random() < 0.4
    return {"op": op, "rows": min(_log(rng, 1, 2048), 256 * 151936 // vocab), "vocab": vocab,
            "dtype": rng.choice(sorted(_DTYPES)),
            "history": _log(rng, 1, 1024 if shared else 8192), "shared": shared,
            "biases": rng.choice([0, 1, 40, 300]), "grammar": rng.choice([0.0, 0.5, 1.0])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _teacher(g, rows, vocab, k, normalised):
    """A teacher's top logits: distinct ids, falling values, some rows cut short (-inf)."""
    gaps = torch.randint(1, max(2, vocab // (k + 1)), (rows, k), generator=g, device="cuda")
    start = torch.randint(0, vocab, (rows, 1), generator=g, device="cuda")
    ids = ((start + gaps.cumsum(1)) % vocab).to(torch.int32)
    fall = torch.rand(rows, k, generator=g, device="cuda") * (8.0 / k)
    top = 12.0 + _randn(g, rows, 1) - fall.cumsum(1) - 1.5 * torch.log1p(
        torch.arange(k, device="cuda", dtype=torch.float32))
    kept = torch.randint(k // 2 + 1, k + 1, (rows, 1), generator=g, device="cuda")
    top = top.masked_fill(torch.arange(k, device="cuda") >= kept, -math.inf).contiguous()
    lse = None
    if not normalised:   # the teacher's own log-sum-exp: its top entries hold about 9 / 10
        lse = torch.logsumexp(top.double(), 1).float() + 0.1 * torch.rand(
            rows, generator=g, device="cuda")
    return ids.contiguous(), top, lse


def _loss_mask(g, rows, share):
    if share == 0.0:
        return None
    m = (torch.rand(rows, generator=g, device="cuda") >= share).to(torch.uint8)
    m[rows // 2] = 1
    return m


def _prepare_norm(c, g):
    rows, width, dt = c["rows"], c["width"], _DTYPES[c["dtype"]]
    s = {"x": (_randn(g, rows, width) * 1.7 + 0.3 * _randn(g, rows, 1)).to(dt),
         "weight": (1.0 + 0.2 * _randn(g, width)).to(dt),
         "bias": (0.1 * _randn(g, width)).to(dt) if c["bias"] else None}
    if c["op"] == "norm_bwd":
        s["grad"] = (0.01 * _randn(g, rows, width)).to(_DTYPES[c["grad_dtype"]])
        x = s["x"].float()
        mean = x.mean(1)
        s["mean"], s["rstd"] = mean, torch.rsqrt((x - mean[:, None]).square().mean(1) + _EPS)
    return s


def _prepare_logits(c, g):
    rows, vocab, k = c["rows"], c["vocab"], c["k"]
    ids, top, tlse = _teacher(g, rows, vocab, k, c["normalised"])
    z = 2.0 * _randn(g, rows, vocab + c["pad"])
    at = ids.long()
    z.scatter_(1, at, 0.8 * top.clamp_min(-4.0) + 0.7 * _randn(g, rows, k))
    z = z.to(_DTYPES[c["dtype"]])
    s = {"logits": z[:, :vocab], "ids": ids, "top": top, "teacher_lse": tlse,
         "mask": _loss_mask(g, rows, c["mask"])}
    if c["op"] == "distill_logits_bwd":
        s["grad"] = _randn(g, rows) / rows
        s["lse"] = torch.logsumexp(s["logits"].float() / c["tau"], 1)
        if s["mask"] is not None:
            s["lse"] = torch.where(s["mask"] != 0, s["lse"], torch.zeros_like(s["lse"]))
    return s


def _prepare_head(c, g):
    rows, width, vocab, k = c["rows"], c["width"], c["vocab"], c["k"]
    ids, top, tlse = _teacher(g, rows, vocab, k, c["normalised"])
    weight = (_randn(g, vocab, width) * (2.0 / math.sqrt(width))).to(torch.bfloat16)
    hidden = _randn(g, rows, width) + 2.0 * weight[ids[:, 0].long()].float()
    s = {"hidden": hidden.to(torch.bfloat16), "weight": weight, "ids": ids, "top": top,
         "teacher_lse": tlse, "mask": _loss_mask(g, rows, c["mask"])}
    if c["op"] == "distill_head_train":
        s["grad"] = _randn(g, rows).abs() / rows
        s["hidden"].requires_grad_(True)
        s["weight"].requires_grad_(True)
    return s


def _prepare_process(c, g):
    rows, vocab = c["rows"], c["vocab"]
    # ids as text has them: few frequent, many rare
    def text(n):
        u = torch.rand(n, generator=g, device="cuda")
        return (vocab * u.pow(4)).long().clamp_max(vocab - 1).to(torch.int32)

    if c["shared"]:   # positions of one trace: prompt, then a growing output
        n = c["history"] + rows
        spans = torch.empty(rows, 3, dtype=torch.int64, device="cuda")
        spans[:, 0] = 0
        spans[:, 1] = c["history"]
        spans[:, 2] = c["history"] + torch.arange(rows, device="cuda")
        total = rows * c["history"] + rows * (rows - 1) // 2
    else:             # requests of their own, ragged; one of them has no history yet
        cpu = torch.Generator().manual_seed(g.initial_seed())
        lens = torch.randint(c["history"] // 4 + 1, c["history"] + 1, (rows,), generator=cpu)
        if rows > 1:
            lens[rows // 2] = 0
        ends = lens.cumsum(0)
        begin = ends - lens
        split = begin + (lens * torch.rand(rows, generator=cpu, dtype=torch.float64)).long()
        spans = torch.stack([begin, split, ends], 1).cuda().contiguous()
        total = n = int(ends[-1])
    s = {"logits": (3.0 * _randn(g, rows, vocab)).to(_DTYPES[c["dtype"]]),
         "tokens": text(max(n, 1)), "spans": spans, "total": total,
         "repetition": 1.0 + 0.3 * torch.rand(rows, generator=g, device="cuda"),
         "frequency": 0.2 * torch.rand(rows, generator=g, device="cuda"),
         "presence": 0.5 * torch.rand(rows, generator=g, device="cuda"),
         "bias_offsets": None, "bias_ids": None, "bias_values": None,
         "allowed": None, "allowed_rows": None}
    if c["biases"]:
        nb = min(c["biases"], vocab // 4)
        gaps = torch.randint(1, vocab // (nb + 1) + 1, (rows, nb), generator=g, device="cuda")
        s["bias_ids"] = ((gaps.cumsum(1) * 7919 % vocab) if math.gcd(7919, vocab) == 1 else
                         gaps.cumsum(1) % vocab).to(torch.int32).reshape(-1).contiguous()
        s["bias_values"] = 4.0 * _randn(g, rows * nb)
        s["bias_offsets"] = torch.arange(rows + 1, device="cuda", dtype=torch.int64) * nb
    if c["grammar"] > 0.0:
        words = (vocab + 31) // 32
        m = max(1, rows // 2)
        bits = torch.randint(0, 1 << 32, (m, words), generator=g, device="cuda")
        keep = torch.randint(0, 1 << 32, (m, words), generator=g, device="cuda")
        bits = (bits & keep) & 0xFFFFFFFF   # a quarter of the ids stays allowed
        s["allowed"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
        with_grammar = torch.rand(rows, generator=g, device="cuda") < c["grammar"]
        pick = torch.randint(0, m, (rows,), generator=g, device="cuda")
        s["allowed_rows"] = torch.where(with_grammar, pick, -torch.ones_like(pick)).to(torch.int32)
    if c["op"] == "process_bwd":
        s["grad"] = (0.01 * _randn(g, rows, vocab)).to(_DTYPES[c["dtype"]])
    return s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op.startswith("norm"):
        s = _prepare_norm(case, g)
    elif op.startswith("distill_logits"):
        s = _prepare_logits(case, g)
    elif op.startswith("distill_head"):
        s = _prepare_head(case, g)
    else:
        s = _prepare_process(case, g)
    s["case"] = case
    return s


# ------------------------------------------------------------------ plain forms, 32 bits
def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = torch.rsqrt((xc * xc).mean(1) + _EPS)
    y = xc * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_bwd(s):
    x, dy, w = s["x"].float(), s["grad"].float(), s["weight"].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    wdy = dy * w
    c1 = (wdy * xh).mean(1, keepdim=True)
    c2 = wdy.mean(1, keepdim=True)
    dx = (wdy - c2 - xh * c1) * s["rstd"][:, None]
    out = {"dx": dx.to(s["x"].dtype), "d_weight": (dy * xh).sum(0)}
    if s["bias"] is not None:
        out["d_bias"] = dy.sum(0)
    return out


def _plain_teacher(s):
    """p [T, K] and log p [T, K] (0 where p = 0)."""
    a = s["top"].float()
    lse = s["teacher_lse"]
    if lse is None:
        m = a.max(1).values
        lse = m + torch.log(torch.exp(a - m[:, None]).sum(1))
    logp = a - lse[:, None]
    live = a > -math.inf
    return torch.where(live, torch.exp(logp), 0.0), torch.where(live, logp, 0.0), live


def _plain_lse(z):
    m = z.max(1).values
    return m + torch.log(torch.exp(z - m[:, None]).sum(1))


def _plain_loss(s, z):
    p, logp, live = _plain_teacher(s)
    lse = _plain_lse(z)
    zt = torch.where(live, torch.gather(z, 1, s["ids"].long()), 0.0)   # absent entries: 0
    loss = (p * torch.where(live, logp - (zt - lse[:, None]), 0.0)).sum(1)
    if s["mask"] is not None:
        on = s["mask"] != 0
        loss, lse = torch.where(on, loss, 0.0), torch.where(on, lse, 0.0)
        zt = torch.where(on[:, None], zt, 0.0)
    return loss, lse, zt, p


def _plain_dz(s, z, lse, p, tau):
    """Cotangent of the logits before the temperature."""
    g = s["grad"] / tau
    if s["mask"] is not None:
        g = torch.where(s["mask"] != 0, g, 0.0)
    dz = torch.exp(z - lse[:, None]) * (g * p.sum(1))[:, None]
    return dz.scatter_add_(1, s["ids"].long(), -g[:, None] * p)


def _plain_distill_logits_fwd(s):
    loss, lse, _, _ = _plain_loss(s, s["logits"].float() / s["case"]["tau"])
    return {"loss": loss, "lse": lse}


def _plain_distill_logits_bwd(s):
    tau = s["case"]["tau"]
    p, _, _ = _plain_teacher(s)
    dz = _plain_dz(s, s["logits"].float() / tau, s["lse"], p, tau)
    return {"d_logits": dz.to(s["logits"].dtype)}


def _plain_distill_head(s):
    tau = s["case"]["tau"]
    with torch.no_grad():
        h, w = s["hidden"].float(), s["weight"].float()
        z = h @ w.t() / tau
        loss, lse, zt, p = _plain_loss(s, z)
        if s["case"]["op"] == "distill_head_fwd":
            return {"loss": loss, "lse": lse, "z_top": zt}
        dz = _plain_dz(s, z, lse, p, tau)
        return {"loss": loss, "d_hidden": (dz @ w).to(torch.bfloat16),
                "d_weight": (dz.t() @ h).to(torch.bfloat16)}


def _plain_counts(s):
    """Per (row, id): occurrences in the outputs, and whether it occurs at all."""
    rows, vocab = s["logits"].shape
    begin, split, end = s["spans"].unbind(1)
    lens = end - begin
    row = torch.repeat_interleave(torch.arange(rows, device="cuda"), lens, output_size=s["total"])
    at = torch.arange(s["total"], device="cuda") - (lens.cumsum(0) - lens)[row] + begin[row]
    cell = row * vocab + s["tokens"][at].long()
    is_out = (at >= split[row]).to(torch.int32)
    counts = torch.zeros(rows * vocab, dtype=torch.int32, device="cuda")
    seen = torch.zeros(rows * vocab, dtype=torch.int32, device="cuda")
    counts.scatter_add_(0, cell, is_out)
    seen.scatter_add_(0, cell, torch.ones_like(is_out))
    return counts.view(rows, vocab), seen.view(rows, vocab) > 0


def _plain_allowed(s):
    vocab = s["logits"].shape[1]
    v = torch.arange(vocab, device="cuda")
    pick = s["allowed_rows"].long()
    words = s["allowed"][pick.clamp_min(0)][:, v // 32]
    return ((words >> (v % 32).to(torch.int32)) & 1).bool() | (pick < 0)[:, None]


def _plain_process_fwd(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    counts, seen = _plain_counts(s)
    r = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    x = x - (s["frequency"][:, None] * counts + s["presence"][:, None] * (counts > 0))
    if s["bias_ids"] is not None:
        per = s["bias_ids"].numel() // rows
        bias = torch.zeros_like(x).scatter_(1, s["bias_ids"].view(rows, per).long(),
                                            s["bias_values"].view(rows, per))
        x = x + bias
    if s["allowed"] is not None:
        x = torch.where(_plain_allowed(s), x, -math.inf)
    return {"out": x.to(s["logits"].dtype)}


def _plain_process_bwd(s):
    x, g = s["logits"].float(), s["grad"].float()
    _, seen = _plain_counts(s)
    r = s["repetition"][:, None]
    g = torch.where(seen, torch.where(x > 0, g / r, g * r), g)
    if s["allowed"] is not None:
        g = torch.where(_plain_allowed(s), g, 0.0)
    return {"d_logits": g.to(s["logits"].dtype)}


_PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd,
          "distill_logits_fwd": _plain_distill_logits_fwd,
          "distill_logits_bwd": _plain_distill_logits_bwd,
          "distill_head_fwd": _plain_distill_head, "distill_head_train": _plain_distill_head,
          "process_fwd": _plain_process_fwd, "process_bwd": _plain_process_bwd}


# ------------------------------------------------------------------ the package's calls
def _own_run(s):
    import chunked_lm_head_tcgen05_gb300 as lm
    from chunked_lm_head_tcgen05_gb300 import autograd

    c, op = s["case"], s["case"]["op"]
    if op == "norm_fwd":
        y, mean, rstd = lm.layernorm_forward(s["x"], s["weight"], s["bias"], _EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        dx, dw, db = lm.layernorm_backward(s["grad"], s["x"], s["weight"], s["mean"], s["rstd"],
                                           with_bias=s["bias"] is not None)
        out = {"dx": dx, "d_weight": dw}
        if db is not None:
            out["d_bias"] = db
        return out
    if op == "distill_logits_fwd":
        loss, lse = lm.distill_logits_forward(s["logits"], s["ids"], s["top"], s["mask"],
                                              c["tau"], 1.0, s["teacher_lse"])
        return {"loss": loss, "lse": lse}
    if op == "distill_logits_bwd":
        return {"d_logits": lm.distill_logits_backward(
            s["logits"], s["ids"], s["top"], s["mask"], c["tau"], 1.0, s["grad"], s["lse"],
            s["teacher_lse"])}
    if op == "distill_head_fwd":
        loss, lse, zt = lm.distill_forward(s["hidden"], s["weight"], s["ids"], s["top"],
                                           s["mask"], c["tau"], 1.0, 512, s["teacher_lse"])
        return {"loss": loss, "lse": lse, "z_top": zt}
    if op == "distill_head_train":
        loss = autograd.lmhead_distill(s["hidden"], s["weight"], s["ids"], s["top"], s["mask"],
                                       c["tau"], 1.0, 512, s["teacher_lse"])
        dh, dw = torch.autograd.grad(loss, (s["hidden"], s["weight"]), s["grad"])
        return {"loss": loss.detach(), "d_hidden": dh, "d_weight": dw}
    rules = dict(tokens=s["tokens"], spans=s["spans"], repetition=s["repetition"],
                 allowed=s["allowed"], allowed_rows=s["allowed_rows"])
    if op == "process_fwd":
        return {"out": lm.process_logits(s["logits"], frequency=s["frequency"],
                                         presence=s["presence"], bias_offsets=s["bias_offsets"],
                                         bias_ids=s["bias_ids"], bias_values=s["bias_values"],
                                         **rules)}
    return {"d_logits": lm.process_logits_backward(s["grad"], s["logits"], **rules)}


def run(state):
    return _own_run(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, b = case["op"], _BYTES.get(case.get("dtype"), 2)
    r = case["rows"]
    if op.startswith("norm"):
        n, w = r * case["width"], case["width"]
        params = (2 if case["bias"] else 1) * w
        if op == "norm_fwd":
            return {"bytes": 2 * n * b + params * b + 8 * r, "flops": 8 * n}
        return {"bytes": n * (2 * b + _BYTES[case["grad_dtype"]]) + w * b + 8 * r + 4 * params,
                "flops": 14 * n}
    if op.startswith("distill"):
        live = r * (1.0 - case["mask"])
        v, k = case["vocab"], case["k"]
        teacher = live * (8 * k + 12)
        if op == "distill_logits_fwd":
            return {"bytes": live * v * b + teacher, "flops": live * 4 * v}
        if op == "distill_logits_bwd":
            return {"bytes": live * v * b + r * v * b + teacher, "flops": live * 4 * v}
        h = case["width"]
        if op == "distill_head_fwd":
            return {"bytes": 2 * live * h + 2 * v * h + teacher + 4 * r * k,
                    "flops": 2 * live * h * v}
        return {"bytes": 2 * live * h + 2 * r * h + 4 * v * h + teacher, "flops": 6 * live * h * v}
    v = case["vocab"]   # forward: logits and results; backward: both gradients (logits at few ids)
    if case["shared"]:
        tokens = case["history"] + r
    else:
        tokens = 0.625 * case["history"] * r
    grammar = (max(1, r // 2) * ((v + 31) // 32) * 4 + 4 * r) if case["grammar"] else 0
    biases = 8 * case["biases"] * r if op == "process_fwd" else 0
    return {"bytes": 2 * r * v * b + 4 * tokens + 36 * r + grammar + biases,
            "flops": 2 * r * v}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_norm(s, case):
    x, w = s["x"].double(), s["weight"].double()
    if case["op"] == "norm_fwd":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + _EPS) ** -0.5
        y = (x - mean.unsqueeze(1)) / torch.sqrt(var + _EPS).unsqueeze(1) * w
        return {"y": y if s["bias"] is None else y + s["bias"].double(), "mean": mean,
                "rstd": rstd}
    n = x.shape[1]
    dy, mean, rstd = s["grad"].double(), s["mean"].double(), s["rstd"].double()
    xh = torch.einsum("tn,t->tn", x - mean.unsqueeze(1), rstd)
    gh = dy * w                       # gradient of the normalised row
    along = torch.einsum("tn,tn->t", gh, xh) / n
    dx = rstd.unsqueeze(1) * (gh - gh.sum(1, keepdim=True) / n - xh * along.unsqueeze(1))
    out = {"dx": dx, "d_weight": torch.einsum("tn,tn->n", dy, xh)}
    if s["bias"] is not None:
        out["d_bias"] = dy.sum(0)
    return out


def _exact_rows(s, z, g, lse_given, tau):
    """Loss, lse, z at the top ids and cotangent of some rows; z in 64 bits, already / tau."""
    a, ids = s["top"].double(), s["ids"].long()
    tl = torch.logsumexp(a, 1) if s["teacher_lse"] is None else s["teacher_lse"].double()
    logp = a - tl.unsqueeze(1)
    p = logp.exp()
    lse = torch.logsumexp(z, 1)
    zt = z.gather(1, ids)
    logq = zt - lse.unsqueeze(1)
    loss = torch.special.xlogy(p, p).sum(1) - torch.where(p > 0, p * logq, 0.0).sum(1)
    dz = None
    if g is not None:
        use = lse if lse_given is None else lse_given.double()
        q = torch.exp(z - use.unsqueeze(1))
        onehots = torch.zeros_like(z).scatter_add_(1, ids, p)
        dz = (p.sum(1, keepdim=True) * q - onehots) * (g / tau).unsqueeze(1)
    return loss, lse, torch.where(torch.isneginf(a), 0.0, zt), dz


def _part(s, rows, names):
    return {n: None if s.get(n) is None else s[n].detach()[rows] for n in names}


def _exact_distill(s, case):
    tau, rows = case["tau"], case["rows"]
    head = case["op"].startswith("distill_head")
    want = case["op"] in ("distill_logits_bwd", "distill_head_train")
    got, w = [], s["weight"].detach().double() if head else None
    dw = torch.zeros_like(w) if head and want else None
    for at in range(0, rows, 512):
        part = slice(at, min(rows, at + 512))
        t = _part(s, part, ("ids", "top", "teacher_lse", "mask", "grad", "lse", "hidden", "logits"))
        x = t["hidden"].double() if head else t["logits"].double()
        z = (x @ w.T if head else x) / tau
        loss, lse, zt, dz = _exact_rows(t, z, t["grad"].double() if want else None, t["lse"], tau)
        if t["mask"] is not None:
            on = t["mask"].double()
            loss, lse, zt = loss * on, lse * on, zt * on.unsqueeze(1)
            dz = None if dz is None else dz * on.unsqueeze(1)
        del z
        row = {"loss": loss, "lse": lse, "z_top": zt}
        if want and head:
            row["d_hidden"] = dz @ w
            dw += dz.T @ x
        elif want:
            row["d_logits"] = dz
        keep = {"distill_logits_fwd": ("loss", "lse"), "distill_logits_bwd": ("d_logits",),
                "distill_head_fwd": ("loss", "lse", "z_top"),
                "distill_head_train": ("loss", "d_hidden")}[case["op"]]
        got.append({n: row[n] for n in keep})
    out = {n: torch.cat([r[n] for r in got]) for n in got[0]}
    if dw is not None:
        out["d_weight"] = dw
    return out


def _exact_process(s, case):
    rows, vocab = s["logits"].shape
    spans = s["spans"].cpu().tolist()
    offsets = None if s["bias_offsets"] is None else s["bias_offsets"].cpu().tolist()
    pick = None if s["allowed_rows"] is None else s["allowed_rows"].cpu().tolist()
    bit = torch.arange(32, device="cuda", dtype=torch.int64)
    got = torch.empty(rows, vocab, dtype=torch.float64, device="cuda")
    for r in range(rows):
        b, m, e = spans[r]
        made = torch.bincount(s["tokens"][m:e].long(), minlength=vocab)
        met = torch.bincount(s["tokens"][b:e].long(), minlength=vocab) > 0
        x, rho = s["logits"][r].double(), s["repetition"][r].double()
        factor = torch.where(met, torch.where(x > 0, 1.0 / rho, rho), 1.0)
        if case["op"] == "process_bwd":
            v = s["grad"][r].double() * factor
            off = 0.0
        else:
            v = x * factor - s["frequency"][r].double() * made \
                - s["presence"][r].double() * made.clamp_max(1)
            if offsets is not None:
                mine = slice(offsets[r], offsets[r + 1])
                v.index_add_(0, s["bias_ids"][mine].long(), s["bias_values"][mine].double())
            off = -math.inf
        if pick is not None and pick[r] >= 0:
            word = s["allowed"][pick[r]].long() & 0xFFFFFFFF
            on = (word.unsqueeze(1) >> bit & 1).reshape(-1)[:vocab] == 1
            v = v.masked_fill(~on, off)
        got[r] = v
    return {"out" if case["op"] == "process_fwd" else "d_logits": got}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s, case)
    if case["op"].startswith("distill"):
        return _exact_distill(s, case)
    return _exact_process(s, case)
