"""Measured cases of the operators at both ends of a decoded or trained token.

Three families:

* embedding rows with scaling and their gradient (``embed_fwd``, ``embed_bwd``): the
  vocabulary table read at the model's other end;
* low-rank adapters of many requests beside a shared projection, in both directions
  (``adapters_fwd``, ``adapters_bwd``): the projection's result is at hand, each row
  names its adapter;
* one step of beam search (``beam_select``, ``beam_reorder``): the best continuations
  over beams and vocabulary, and the states moved to the beams that go on.

``run`` computes a case with elementary torch operations in 32 bits (scores of beams in
64, where two continuations may be close), or, when ``own`` is true, with the calls a
user makes of this package.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

_DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
_BYTES = {"float32": 4, "bfloat16": 2, "float16": 2}


def listed():
    return [
        # The next tokens of a small decoding batch.
        {"name": "embed fwd, 16 tokens", "op": "embed_fwd", "tokens": 16, "vocab": 151936,
         "width": 2560, "dtype": "bfloat16", "scale": 1.0},
        # A training batch of sixteen 4,096-token rows, scaled by the square root of the width.
        {"name": "embed fwd, 65536 tokens", "op": "embed_fwd", "tokens": 65536, "vocab": 151936,
         "width": 2560, "dtype": "bfloat16", "scale": 50.596},
        # The same batch's gradient of a bf16 table: frequent ids hold thousands of tokens.
        {"name": "embed bwd, 65536 tokens", "op": "embed_bwd", "tokens": 65536, "vocab": 151936,
         "width": 2560, "dtype": "bfloat16", "grad_dtype": "bfloat16", "scale": 50.596,
         "padding": True},
        # A packed row of odd length and width, fp32 throughout.
        {"name": "embed bwd, odd fp32", "op": "embed_bwd", "tokens": 5431, "vocab": 50257,
         "width": 1111, "dtype": "float32", "grad_dtype": "float32", "scale": 1.0,
         "padding": False},
        # One decoding step of 64 requests with 16 adapters on the vocabulary head.
        {"name": "adapters fwd, 64 requests", "op": "adapters_fwd", "rows": 64, "width": 2560,
         "vocab": 151936, "rank": 16, "adapters": 16, "bare": 0.1, "runs": False,
         "dtype": "bfloat16"},
        # Four fine-tuned models trained at once on one 2,048-token chunk's logits.
        {"name": "adapters fwd, 2048 rows", "op": "adapters_fwd", "rows": 2048, "width": 2560,
         "vocab": 151936, "rank": 32, "adapters": 4, "bare": 0.0, "runs": True,
         "dtype": "bfloat16"},
        # The gradients of that chunk.
        {"name": "adapters bwd, 2048 rows", "op": "adapters_bwd", "rows": 2048, "width": 2560,
         "vocab": 151936, "rank": 32, "adapters": 4, "bare": 0.0, "runs": True,
         "dtype": "bfloat16"},
        # A square projection of ragged size with fp32 cotangents.
        {"name": "adapters bwd, ragged fp32", "op": "adapters_bwd", "rows": 777, "width": 1088,
         "vocab": 2491, "rank": 8, "adapters": 3, "bare": 0.2, "runs": True,
         "dtype": "float32"},
        # One request's step: four beams, twice as many continuations.
        {"name": "beam select, 4 beams", "op": "beam_select", "groups": 1, "beams": 4,
         "vocab": 151936, "take": 8, "dtype": "float32", "tau": 1.0, "finished": 0.0},
        # 32 requests of eight beams, a few of which have ended.
        {"name": "beam select, 32 x 8 beams", "op": "beam_select", "groups": 32, "beams": 8,
         "vocab": 151936, "take": 16, "dtype": "bfloat16", "tau": 0.7, "finished": 0.1},
        # One request's cache of a small layer after 300 tokens.
        {"name": "beam reorder, 4 beams", "op": "beam_reorder", "layers": 2, "groups": 1,
         "beams": 4, "heads": 4, "room": 512, "used": 300, "dim": 64, "dtype": "bfloat16",
         "keep": 0.5, "in_place": True},
        # Keys and values of one layer of 16 requests, 1,501 tokens of 2,048 in use.
        {"name": "beam reorder, 16 x 4 beams", "op": "beam_reorder", "layers": 2, "groups": 16,
         "beams": 4, "heads": 8, "room": 2048, "used": 1501, "dim": 128, "dtype": "bfloat16",
         "keep": 0.5, "in_place": True},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(max(low, high))))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "adapters_fwd", "adapters_bwd", "beam_select",
                     "beam_reorder"])
    dtype = rng.choice(sorted(_DTYPES))
    if op.startswith("embed"):
        width = _log(rng, 64, 8192)
        width = width if rng.random() < 0.4 else max(64, width // 64 * 64)
        c = {"op": op, "tokens": _log(rng, 1, min(65536, 65536 * 1280 // width)),
             "vocab": _log(rng, 1000, min(151936, 151936 * 1280 // width)), "width": width,
             "dtype": dtype, "scale": rng.choice([1.0, round(math.sqrt(width), 3)])}
        if op == "embed_bwd":
            c["grad_dtype"] = rng.choice(["float32", "bfloat16"])
            c["padding"] = rng.random() < 0.5
        return c
    if op.startswith("adapters"):
        vocab = _log(rng, 1000, 151936)
        vocab = vocab if rng.random() < 0.4 else vocab // 64 * 64 + 64
        width = 64 * _log(rng, 4, 64)
        rows = _log(rng, 1, min(4096, 1024 * 151936 // vocab))
        n = _log(rng, 1, 16)
        rank = min(_log(rng, 1, 64), max(1, 128 // n)) if rng.random() < 0.5 else \
            min(rng.choice([8, 16, 32]), 128 // n)
        return {"op": op, "rows": rows, "width": width, "vocab": vocab, "rank": rank,
                "adapters": n, "bare": rng.choice([0.0, 0.2]), "runs": rng.random() < 0.5,
                "dtype": dtype}
    beams = _log(rng, 1, 16)
    if op == "beam_select":
        vocab = _log(rng, 1000, 151936)
        return {"op": op, "groups": _log(rng, 1, 256 // beams), "beams": beams, "vocab": vocab,
                "take": rng.choice([beams, 2 * beams]), "dtype": dtype,
                "tau": rng.choice([1.0, 0.7, 2.0]), "finished": rng.choice([0.0, 0.2])}
    groups = _log(rng, 1, 64 // beams)
    room = _log(rng, 16, 2048)
    return {"op": op, "layers": rng.choice([1, 2, 4]), "groups": groups, "beams": beams,
            "heads": rng.choice([1, 2, 4, 8]), "room": room, "used": rng.randint(1, room),
            "dim": rng.choice([33, 64, 80, 128]), "dtype": dtype,
            "keep": rng.choice([0.25, 0.5, 0.75]), "in_place": rng.random() < 0.6}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _prepare_embed(c, g):
    n, vocab, width, dt = c["tokens"], c["vocab"], c["width"], _DTYPES[c["dtype"]]
    # ids as text has them: few frequent, many rare
    u = torch.rand(n, generator=g, device="cuda")
    ids = (vocab * u.pow(4)).long().clamp_max(vocab - 1).to(torch.int32)
    if c["op"] == "embed_fwd":
        return {"ids": ids, "weight": (0.02 * _randn(g, vocab, width)).to(dt)}
    if c["padding"]:   # the last eighth of a padded batch
        ids[n - n // 8:] = 3
    return {"ids": ids, "grad": (0.01 * _randn(g, n, width)).to(dt)}


def _prepare_adapters(c, g):
    rows, width, vocab = c["rows"], c["width"], c["vocab"]
    rank, n, dt = c["rank"], c["adapters"], _DTYPES[c["dtype"]]
    of = torch.randint(0, n, (rows,), generator=g, device="cuda")
    if c["runs"]:      # every request's rows lie together
        of = of.sort().values
    of = torch.where(torch.rand(rows, generator=g, device="cuda") < c["bare"],
                     torch.full_like(of, -1), of)   # rows of the shared model itself
    s = {"x": _randn(g, rows, width).to(torch.bfloat16),
         "down": (_randn(g, n, rank, width) / math.sqrt(width)).to(torch.bfloat16),
         "up": (0.3 * _randn(g, n, rank, vocab) / math.sqrt(rank)).to(torch.bfloat16),
         "of": of.to(torch.int32),
         "scale": 0.5 + torch.rand(n, generator=g, device="cuda")}
    if c["op"] == "adapters_fwd":
        s["base"] = (2.0 * _randn(g, rows, vocab)).to(dt)
    else:
        s["grad"] = (0.01 * _randn(g, rows, vocab)).to(dt)
    return s


def _prepare_select(c, g):
    rows, vocab = c["groups"] * c["beams"], c["vocab"]
    z = 2.0 * _randn(g, rows, vocab)
    # a model's few likely tokens stand out
    likely = torch.randint(0, vocab, (rows, 12), generator=g, device="cuda")
    z.scatter_(1, likely, 12.0 + 2.0 * _randn(g, rows, 12))
    s = {"logits": z.to(_DTYPES[c["dtype"]]),
         "scores": -20.0 * torch.rand(rows, generator=g, device="cuda"), "finished": None}
    if c["finished"] > 0.0:
        s["finished"] = (torch.rand(rows, generator=g, device="cuda")
                         < c["finished"]).to(torch.uint8)
    return s


def _survivors(c):
    return max(1, int(c["beams"] * c["keep"]))


def _prepare_reorder(c, g):
    rows, beams = c["groups"] * c["beams"], c["beams"]
    cache = _randn(g, c["layers"], rows, c["heads"], c["room"], c["dim"]).to(_DTYPES[c["dtype"]])
    # beams that go on stay where they are, the others take over one of those
    order = torch.rand(c["groups"], beams, generator=g, device="cuda").argsort(1)
    kept = order[:, :_survivors(c)]
    pick = torch.randint(0, _survivors(c), (c["groups"], beams), generator=g, device="cuda")
    parents = kept.gather(1, pick).scatter_(1, kept, kept)
    parents = parents + beams * torch.arange(c["groups"], device="cuda")[:, None]
    return {"cache": cache, "parents": parents.reshape(-1).to(torch.int32)}


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op.startswith("embed"):
        s = _prepare_embed(case, g)
    elif op.startswith("adapters"):
        s = _prepare_adapters(case, g)
    elif op == "beam_select":
        s = _prepare_select(case, g)
    else:
        s = _prepare_reorder(case, g)
    s["case"] = case
    return s


# ------------------------------------------------------------------ plain forms
def _plain_embed_fwd(s):
    rows = s["weight"][s["ids"].long()].float() * s["case"]["scale"]
    return {"y": rows.to(s["weight"].dtype)}


def _plain_embed_bwd(s):
    c = s["case"]
    dy = s["grad"].float() * c["scale"]
    if c["padding"]:
        dy = torch.where((s["ids"] == 3)[:, None], 0.0, dy)
    d = torch.zeros(c["vocab"], c["width"], dtype=torch.float32, device="cuda")
    return {"d_weight": d.index_add_(0, s["ids"].long(), dy).to(_DTYPES[c["grad_dtype"]])}


def _plain_share(s, wide, factor):
    """[T, adapters * rank]: wide . factor^T, scaled, where the row has that adapter, else 0."""
    n, rank, _ = factor.shape
    u = (wide.float() @ factor.float().reshape(n * rank, -1).t()).view(-1, n, rank)
    mine = s["of"][:, None] == torch.arange(n, device="cuda")
    return torch.where(mine[:, :, None], u * s["scale"][:, None], 0.0).reshape(-1, n * rank)


def _plain_adapters_fwd(s):
    n, rank, vocab = s["up"].shape
    u = _plain_share(s, s["x"], s["down"])
    y = s["base"].float() + u @ s["up"].float().reshape(n * rank, vocab)
    return {"y": y.to(s["base"].dtype)}


def _plain_adapters_bwd(s):
    n, rank, vocab = s["up"].shape
    u, du = _plain_share(s, s["x"], s["down"]), _plain_share(s, s["grad"], s["up"])
    return {"dx": du @ s["down"].float().reshape(n * rank, -1),
            "d_down": (du.t() @ s["x"].float()).view(s["down"].shape),
            "d_up": (u.t() @ s["grad"].float()).view(n, rank, vocab)}


def _plain_beam_select(s):
    c = s["case"]
    beams, take, vocab = c["beams"], c["take"], c["vocab"]
    rows = c["groups"] * beams
    x = s["logits"].float() + 0.0     # one zero
    z = x.double() / c["tau"]
    m = z.max(1).values
    lse = m + torch.log(torch.exp(z - m[:, None]).sum(1))
    # order of the logits and, among equals, of the ids, as one integer
    bits = x.view(torch.int32).long()
    key = torch.where(bits >= 0, bits, -2147483648 - bits) * vocab + (
        vocab - 1 - torch.arange(vocab, device="cuda"))
    best = torch.topk(key, take, dim=1).values
    token = vocab - 1 - best % vocab
    score = s["scores"].double()[:, None] + z.gather(1, token) - lse[:, None]
    if s["finished"] is not None:     # an ended beam goes on with the end token alone
        ended = (s["finished"] != 0)[:, None]
        first = torch.arange(take, device="cuda") == 0
        score = torch.where(ended, torch.where(first, s["scores"].double()[:, None], -math.inf),
                            score)
        token = torch.where(ended, 2, token)
        lse = torch.where(s["finished"] != 0, 0.0, lse)
    parent = torch.arange(rows, device="cuda")[:, None].expand(rows, take)
    score, at = torch.sort(score.view(c["groups"], beams * take), dim=1, descending=True,
                           stable=True)
    score, at = score[:, :take], at[:, :take]
    found = score > -math.inf         # fewer continuations than asked for: -1
    parent = parent.reshape(c["groups"], -1).gather(1, at)
    token = token.reshape(c["groups"], -1).gather(1, at)
    return {"scores": score.float(), "parents": torch.where(found, parent, -1).to(torch.int32),
            "tokens": torch.where(found, token, -1).to(torch.int32), "lse": lse.float()}


def _used(s):
    return s["cache"][:, :, :, :s["case"]["used"]]


def _plain_beam_reorder(s):
    moved = _used(s).index_select(1, s["parents"].long())
    return {"cache": _used(s).copy_(moved) if s["case"]["in_place"] else moved}


_PLAIN = {"embed_fwd": _plain_embed_fwd, "embed_bwd": _plain_embed_bwd,
          "adapters_fwd": _plain_adapters_fwd, "adapters_bwd": _plain_adapters_bwd,
          "beam_select": _plain_beam_select, "beam_reorder": _plain_beam_reorder}


# ------------------------------------------------------------------ the package's calls
def _own_run(s):
    import chunked_lm_head_tcgen05_gb300 as lm

    c, op = s["case"], s["case"]["op"]
    if op == "embed_fwd":
        return {"y": lm.embedding_forward(s["ids"], s["weight"], c["scale"])}
    if op == "embed_bwd":
        return {"d_weight": lm.embedding_backward(s["grad"], s["ids"], c["vocab"], c["scale"],
                                                  padding_id=3 if c["padding"] else None,
                                                  dtype=_DTYPES[c["grad_dtype"]])}
    if op == "adapters_fwd":
        return {"y": lm.adapters_forward(s["base"], s["x"], s["down"], s["up"], s["of"],
                                         s["scale"])}
    if op == "adapters_bwd":
        dx, d_down, d_up = lm.adapters_backward(s["grad"], s["x"], s["down"], s["up"], s["of"],
                                                s["scale"])
        return {"dx": dx, "d_down": d_down, "d_up": d_up}
    if op == "beam_select":
        scores, parents, tokens, lse = lm.beam_select(s["logits"], s["scores"], c["beams"],
                                                      c["take"], c["tau"],
                                                      finished=s["finished"], eos_id=2)
        return {"scores": scores, "parents": parents, "tokens": tokens, "lse": lse}
    if c["in_place"]:
        return {"cache": lm.beam_reorder(_used(s), s["parents"], 1, beams=c["beams"],
                                         out=_used(s))}
    return {"cache": lm.beam_reorder(_used(s), s["parents"], 1)}


def run(state):
    return _own_run(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, b = case["op"], _BYTES[case["dtype"]]
    if op.startswith("embed"):
        n, vocab, width = case["tokens"], case["vocab"], case["width"]
        # ids are vocab u^4 with u uniform: an id's share is the length of its u interval
        met = min(n, vocab)
        if vocab > 1:
            few = 4096
            edges = [(i / few) ** 0.25 for i in range(few + 1)]
            met = sum(vocab / few * (1.0 - math.exp(-n * (q - p) * few / vocab))
                      for p, q in zip(edges, edges[1:]))
        if op == "embed_fwd":
            return {"bytes": (min(met, n) + n) * width * b + 4 * n, "flops": n * width}
        live = n - n // 8 if case["padding"] else n
        return {"bytes": live * width * b + vocab * width * _BYTES[case["grad_dtype"]] + 4 * n,
                "flops": 2 * live * width}
    if op.startswith("adapters"):
        t, h, v, r, n = (case[k] for k in ("rows", "width", "vocab", "rank", "adapters"))
        live = t * (1.0 - case["bare"])
        met = n * (1.0 - (1.0 - 1.0 / n) ** live)
        if op == "adapters_fwd":
            return {"bytes": 2 * t * v * b + 2 * live * h + 2 * met * r * (h + v) + 4 * t,
                    "flops": 2 * live * r * (h + v)}
        return {"bytes": live * v * b + 2 * live * h + 4 * t * h + 2 * met * r * (h + v)
                + 4 * n * r * (h + v) + 4 * t,
                "flops": 2 * live * r * (3 * h + 2 * v)}
    rows = case["groups"] * case["beams"]
    if op == "beam_select":
        live = rows * (1.0 - case["finished"])
        return {"bytes": live * case["vocab"] * b + 9 * rows + 12 * case["groups"] * case["take"],
                "flops": 4 * live * case["vocab"]}
    row = case["layers"] * case["heads"] * case["used"] * case["dim"] * b
    stay = _survivors(case)
    if case["in_place"]:
        moved = case["beams"] - stay
        return {"bytes": case["groups"] * (moved + min(moved, stay)) * row + 4 * rows, "flops": 0}
    return {"bytes": case["groups"] * (case["beams"] + stay) * row + 4 * rows, "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_embed(s, case):
    if case["op"] == "embed_fwd":
        picked = torch.nn.functional.embedding(s["ids"].long(), s["weight"]).double()
        return {"y": picked.mul_(case["scale"])}
    ids, order = s["ids"].long().sort()
    live = ids != 3 if case["padding"] else torch.ones_like(ids, dtype=torch.bool)
    ids, order = ids[live], order[live]
    d = torch.zeros(case["vocab"], case["width"], dtype=torch.float64, device="cuda")
    for at in range(0, ids.numel(), 8192):
        some = slice(at, at + 8192)
        d.index_put_((ids[some],), s["grad"][order[some]].double(), accumulate=True)
    return {"d_weight": d.mul_(case["scale"])}


def _exact_adapters(s, case):
    forward = case["op"] == "adapters_fwd"
    out = {"y": s["base"].double()} if forward else {
        "dx": torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda"),
        "d_down": torch.zeros(s["down"].shape, dtype=torch.float64, device="cuda"),
        "d_up": torch.zeros(s["up"].shape, dtype=torch.float64, device="cuda")}
    for a in range(case["adapters"]):
        rows = (s["of"] == a).nonzero().flatten()
        x, down, up = s["x"][rows].double(), s["down"][a].double(), s["up"][a].double()
        sigma = s["scale"][a].double()
        inner = torch.einsum("th,rh->tr", x, down) * sigma
        if forward:
            out["y"].index_add_(0, rows, torch.einsum("tr,rv->tv", inner, up))
            continue
        g = s["grad"][rows].double()
        d_inner = torch.einsum("tv,rv->tr", g, up) * sigma
        out["dx"][rows] = torch.einsum("tr,rh->th", d_inner, down)
        out["d_down"][a] = torch.einsum("tr,th->rh", d_inner, x)
        out["d_up"][a] = torch.einsum("tr,tv->rv", inner, g)
    return out


def _exact_select(s, case):
    beams, take, vocab = case["beams"], case["take"], case["vocab"]
    got = {"scores": [], "parents": [], "tokens": [], "lse": []}
    for group in range(case["groups"]):
        rows = slice(group * beams, (group + 1) * beams)
        z = s["logits"][rows].double() / case["tau"]
        total = s["scores"][rows].double().unsqueeze(1) + torch.log_softmax(z, 1)
        got["lse"].append(torch.logsumexp(z, 1))
        if s["finished"] is not None:
            over = s["finished"][rows] != 0
            total[over] = -math.inf
            total[over, 2] = s["scores"][rows][over].double()
            got["lse"][-1][over] = 0.0
        score, at = total.flatten().sort(descending=True, stable=True)
        score, at = score[:take], at[:take]
        none = torch.isneginf(score)
        got["scores"].append(score)
        got["parents"].append((at // vocab + group * beams).masked_fill(none, -1).to(torch.int32))
        got["tokens"].append((at % vocab).masked_fill(none, -1).to(torch.int32))
    return {k: torch.cat(v) if k == "lse" else torch.stack(v) for k, v in got.items()}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("embed"):
        return _exact_embed(s, case)
    if case["op"].startswith("adapters"):
        return _exact_adapters(s, case)
    if case["op"] == "beam_select":
        return _exact_select(s, case)
    rows = [s["cache"][:, p, :, :case["used"]] for p in s["parents"].tolist()]
    return {"cache": torch.stack(rows, 1).double()}
