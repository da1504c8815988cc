"""More language-model operators: what is measured of each, in its plain form and in the library's.

What an adapter step needs whose frozen weights are held in 4 bits, and whose lost accuracy a
teacher is to bring back:

  project   a shared projection with 4-bit weights, with low-rank adapters of many requests or
            probes beside it
  quantize  the 4-bit codes and group scales of a matrix, and the values that they stand for
  distill   the divergence of a teacher's top logits from the model's distribution, per row,
            with its gradient with respect to the model's logits
  head      log probabilities of given tokens from hidden states and the unembedding matrix,
            with the gradients with respect to both

4-bit weights.  W[f, k] = scales[k // group, f] * (q[f, k] - zeros[k // group, f]), zeros 8 where
there are none.  Codes lie in blocks of 16 features x 128 values of k, 1024 bytes each:
[features / 16][k / 128][8 k: four][feature: 16][32 k: four][4 bytes], the four bytes holding eight
neighbouring values of k as their (low, high) halves: (0, 2), (4, 6), (1, 3), (5, 7).

A row whose target is IGNORE counts for nothing: its log probability, loss and gradients are 0.
"""
import math
import random

import torch

own = False

IGNORE = -100
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
VOCAB = 50272


def listed():
    return [
        # the next token of one sequence, no adapters: latency counts
        {"name": "project 1 token", "op": "project", "groups": 1, "length": 1, "d_in": 5120,
         "d_out": 5120, "group": 128, "zeros": False, "rank": 0, "adapters": 0, "probes": 0, "dtype": "bf16"},
        # one token of each of 32 requests through the widest model's widened projection, an
        # adapter for each
        {"name": "project 32 requests", "op": "project", "groups": 32, "length": 1, "d_in": 7168,
         "d_out": 28672, "group": 128, "zeros": False, "rank": 16, "adapters": 32, "probes": 0, "dtype": "bf16"},
        # a small model in fp32, both signs of 16 probes and the clean pass; codes with zero points
        {"name": "project fp32 probes", "op": "project", "groups": 33, "length": 64, "d_in": 768,
         "d_out": 2304, "group": 32, "zeros": True, "rank": 8, "adapters": 1, "probes": 16, "dtype": "fp32"},
        # both signs of 32 probes and the clean pass, a short batch for each, widened projection
        {"name": "project 32 probes", "op": "project", "groups": 65, "length": 64, "d_in": 5120,
         "d_out": 20480, "group": 128, "zeros": False, "rank": 16, "adapters": 1, "probes": 32, "dtype": "bf16"},
        # a small model's matrix, in fp32
        {"name": "quantize fp32", "op": "quantize", "d_in": 768, "d_out": 2304, "group": 32, "dtype": "fp32"},
        # the widest model's widened projection
        {"name": "quantize 30b", "op": "quantize", "d_in": 7168, "d_out": 28672, "group": 128, "dtype": "bf16"},
        # the loss alone, of 33 probes' short batches: what a forward-only step takes
        {"name": "distill loss", "op": "distill", "rows": 1056, "vocab": VOCAB, "pad": 0, "dtype": "bf16",
         "top": 20, "ignore": 0.0, "masked": 0.0, "temperature": 1.0, "grad": False},
        # odd sizes, part of the vocabulary masked off, prompts ignored, a softened teacher
        {"name": "distill fp32 odd", "op": "distill", "rows": 515, "vocab": 32003, "pad": 2, "dtype": "fp32",
         "top": 5, "ignore": 0.5, "masked": 0.1, "temperature": 2.0, "grad": True},
        # every token of 64 sequences of 128, with the gradient
        {"name": "distill 8k rows", "op": "distill", "rows": 8192, "vocab": VOCAB, "pad": 0, "dtype": "bf16",
         "top": 32, "ignore": 0.0, "masked": 0.0, "temperature": 1.0, "grad": True},
        # a few answers
        {"name": "head 8 rows", "op": "head", "rows": 8, "vocab": VOCAB, "dim": 5120, "dtype": "bf16",
         "ignore": 0.0},
        # a small model in fp32, all tokens of a batch
        {"name": "head fp32", "op": "head", "rows": 2048, "vocab": VOCAB, "dim": 768, "dtype": "fp32",
         "ignore": 0.0},
        # the widest model's batch of 64 sequences of 128, prompts ignored
        {"name": "head 8k rows", "op": "head", "rows": 8192, "vocab": VOCAB, "dim": 7168, "dtype": "bf16",
         "ignore": 0.5},
    ]


def _between(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["project", "project", "project", "quantize", "distill", "distill", "head", "head"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    slower = 12 if dtype == "fp32" else 1
    if op == "project":
        group = rng.choice([32, 64, 128])
        d_in, d_out = group * _between(rng, 2, 7168 // group), 8 * _between(rng, 8, 3584)
        most = 4160 * 5120 * 20480 // 2 // (d_in * d_out * slower)
        rows = _between(rng, 1, max(1, min(8192, most)))
        probes = rng.choice([0, 0, 1, 8, 32])
        groups = 2 * probes + 1 if probes else _between(rng, 1, 64)
        rank = rng.choice([8, 16, 24, 32, 64]) if probes else rng.choice([0, 8, 16, 64])
        adapters = 1 if probes else _between(rng, 1, min(32, groups)) if rank else 0
        return {"op": op, "groups": groups, "length": max(1, rows // groups), "d_in": d_in, "d_out": d_out,
                "group": group, "zeros": rng.random() < 0.3, "rank": rank, "adapters": adapters,
                "probes": probes, "dtype": dtype}
    if op == "quantize":
        group = rng.choice([32, 64, 128])
        return {"op": op, "d_in": group * _between(rng, 2, 7168 // group), "d_out": 8 * _between(rng, 8, 3584),
                "group": group, "dtype": dtype}
    ignore = rng.choice([0.0, 0.25, 0.5, 0.75])
    if op == "distill":
        vocab = _between(rng, 1000, 200000)
        size = 4 if dtype == "fp32" else 2
        rows = _between(rng, 1, min(8192, 8192 * VOCAB * 2 // (vocab * size)))
        return {"op": op, "rows": rows, "vocab": vocab, "pad": rng.choice([0, 0, 1, 8]), "dtype": dtype,
                "top": rng.choice([1, 4, 8, 20, 32, 64]), "ignore": ignore, "masked": rng.choice([0.0, 0.0, 0.2]),
                "temperature": rng.choice([1.0, 1.0, 0.5, 2.0]), "grad": rng.random() < 0.7}
    vocab, dim = _between(rng, 1000, 131072), 8 * _between(rng, 8, 896)
    most = 8192 * VOCAB * 7168 // 2 // (vocab * dim * slower)
    return {"op": op, "rows": _between(rng, 1, max(1, min(8192, most))), "vocab": vocab, "dim": dim,
            "dtype": dtype, "ignore": ignore}


def _lengths(case):
    """Ragged lengths of the groups, about the case's mean: the same for every seed."""
    rng = random.Random(case["groups"] * 4099 + case["length"])
    mean = case["length"]
    return [rng.randint(mean - mean // 2, mean + mean // 2) for _ in range(case["groups"])]


def _counted(case, rows):
    """Which rows count: of each sequence of 128, the first ones are a prompt."""
    length = min(128, rows)
    first = int(length * case["ignore"])
    return [r % length >= first for r in range(rows)]


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "project":
        rows, d_in, d_out, rank = sum(_lengths(case)), case["d_in"], case["d_out"], case["rank"]
        params = case["adapters"] * rank * (d_in + d_out)
        scales = d_in // case["group"] * d_out * (2 if case["zeros"] else 1)
        return {"bytes": d_in * d_out // 2 + (rows * (d_in + d_out) + scales + d_out + params) * size
                + case["probes"] * params // 8,
                "flops": 2 * rows * (d_in * d_out + rank * (d_in + d_out))}
    if case["op"] == "quantize":
        n = case["d_in"] * case["d_out"]
        return {"bytes": 2 * n * size + n // 2 + n // case["group"] * size, "flops": 6 * n}
    rows = sum(_counted(case, case["rows"]))
    if case["op"] == "distill":
        out = rows * case["vocab"] * size + (case["rows"] - rows) * case["vocab"] * size
        return {"bytes": rows * (case["vocab"] * size + case["top"] * 12) + case["rows"] * 16
                + (out if case["grad"] else 0),
                "flops": (9 if case["grad"] else 4) * rows * case["vocab"]}
    return {"bytes": (rows + case["rows"] + 2 * case["vocab"]) * case["dim"] * size + case["rows"] * 16,
            "flops": 6 * rows * case["dim"] * case["vocab"]}


def _targets(case, rows, vocab, gen):
    t = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    keep = torch.tensor(_counted(case, rows), device="cuda")
    return torch.where(keep, t, torch.full_like(t, IGNORE))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    state, dtype = {"case": case}, TYPES[case["dtype"]]
    if case["op"] == "project":
        d_in, d_out, rank, groups = case["d_in"], case["d_out"], case["rank"], case["groups"]
        lengths = _lengths(case)
        rows, params = sum(lengths), case["adapters"] * rank * (d_in + d_out)
        state["lengths"] = lengths
        state["starts"] = torch.tensor([sum(lengths[:g]) for g in range(groups + 1)], device="cuda")
        state["x"] = normal(rows, d_in, dtype=dtype)
        # codes of a bell curve in groups, as quantizing gives them: about eight, seldom at the ends
        halves = [(normal(-(-d_out // 16), -(-d_in // 128), 1024, std=2.5) + 8.0).round().clamp(1, 15).to(torch.uint8)
                  for _ in range(2)]
        state["codes"] = halves[0] | (halves[1] << 4)
        state["scales"] = (0.008 * (1.0 + 0.25 * normal(d_in // case["group"], d_out).clamp(-3, 3))).to(dtype)
        state["zeros"] = (8.0 + normal(d_in // case["group"], d_out)).to(dtype) if case["zeros"] else None
        state["bias"] = normal(d_out, std=0.02, dtype=dtype)
        if rank:
            state["adapters"] = normal(params, std=0.02, dtype=dtype)
            state["scale"] = 2.0
            if case["probes"]:
                # both signs of each probe, then the clean pass, of the one adapter
                which = [g // 2 if g < 2 * case["probes"] else -1 for g in range(groups)]
                alpha = [0.0 if p < 0 else (1e-3 if g % 2 == 0 else -1e-3) for g, p in enumerate(which)]
                ids = [0] * groups
                state["probes"] = torch.tensor(which, dtype=torch.int32, device="cuda")
                state["alphas"] = torch.tensor(alpha, dtype=torch.float32, device="cuda")
                state["bits"] = torch.randint(0, 256, (case["probes"], -(-params // 128) * 16),
                                              generator=gen, device="cuda", dtype=torch.uint8)
            else:
                # some requests come without an adapter
                rng = random.Random(seed)
                ids = [rng.randrange(case["adapters"]) if rng.random() < 0.9 else -1 for _ in range(groups)]
            state["ids"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
    elif case["op"] == "quantize":
        state["weight"] = normal(case["d_out"], case["d_in"], std=0.02, dtype=dtype)
    elif case["op"] == "distill":
        rows, vocab, top = case["rows"], case["vocab"], case["top"]
        x = normal(rows, vocab + case["pad"], std=2.5)
        if case["masked"]:
            off = torch.rand(vocab + case["pad"], generator=gen, device="cuda") < case["masked"]
            off[: 64] = False
            x = x.masked_fill(off, -math.inf)
        state["logits"] = x.to(dtype)[:, :vocab]
        # the teacher's alternatives, distinct in a row, in falling order; a few rows have fewer
        reach = 64 if case["masked"] else vocab
        first = torch.randint(0, reach, (rows, 1), generator=gen, device="cuda")
        stride = reach // top
        step = torch.randint(1, stride + 1, (rows, 1), generator=gen, device="cuda") if stride > 1 else 1
        ids = (first + step * torch.arange(top, device="cuda")) % reach
        few = torch.rand(rows, 1, generator=gen, device="cuda") < 0.05
        last = few & (torch.arange(top, device="cuda") >= max(1, top // 2))
        state["teacher_ids"] = ids.masked_fill(last, -1)
        state["teacher_logits"] = normal(rows, top, std=2.5).sort(dim=1, descending=True).values
        state["targets"] = _targets(case, rows, reach, gen)
        state["row_grad"] = (0.5 + torch.rand(rows, generator=gen, device="cuda")) / rows
    else:
        state["hidden"] = normal(case["rows"], case["dim"], dtype=dtype)
        state["weight"] = normal(case["vocab"], case["dim"], std=2.5 / math.sqrt(case["dim"]), dtype=dtype)
        state["targets"] = _targets(case, case["rows"], case["vocab"], gen)
        state["row_grad"] = (0.5 + torch.rand(case["rows"], generator=gen, device="cuda")) / case["rows"]
    return state


_kept = {}


def _context():
    import forward_only_amd as zo
    if "ctx" not in _kept:
        _kept["ctx"] = zo.zo_init(0)
    return zo, _kept["ctx"]


def run(state):
    op = state["case"]["op"]
    if op == "project":
        return _project(state)
    if op == "quantize":
        return _quantize(state)
    if op == "distill":
        return _distill(state)
    return _head(state)


def _values(codes, d_out, d_in):
    """The codes [d_out, d_in] as whole numbers, from their blocks."""
    nf, nk = codes.shape[:2]
    halves = torch.stack((codes & 15, codes >> 4), dim=-1)
    # [nf, nk, 8 k: q, feature, 32 k: c, byte, half]: the eight values in the order of k are
    # halves (byte, half) of 0 = (0, 0), 1 = (2, 0), 2 = (0, 1), 3 = (2, 1), 4 = (1, 0), ...
    v = halves.view(nf, nk, 4, 16, 4, 2, 2, 2)          # byte = 2 * odd + pair
    v = v.permute(0, 3, 1, 4, 2, 6, 7, 5)               # feature | k: c, q, pair, half, odd
    return v.reshape(nf * 16, nk * 128)[:d_out, :d_in]


def _weights(state, dtype):
    case = state["case"]
    q = _values(state["codes"], case["d_out"], case["d_in"]).to(dtype)
    q = q.view(case["d_out"], -1, case["group"])
    s, z = state["scales"].to(dtype).t()[:, :, None], 8.0
    if case["zeros"]:
        z = state["zeros"].to(dtype).t()[:, :, None]
    return ((q - z) * s).view(case["d_out"], case["d_in"])


def _project(state):
    case = state["case"]
    if own:
        zo, ctx = _context()
        more = {}
        if case["rank"]:
            more = {"adapters": state["adapters"], "rank": case["rank"], "starts": state["starts"],
                    "ids": state["ids"], "scale": state["scale"]}
            if case["probes"]:
                more |= {"probes": state["probes"], "alphas": state["alphas"], "bits": state["bits"]}
        weight = zo.Q4Weight(state["codes"], state["scales"], state["zeros"], case["d_in"])
        return {"y": zo.zo_q4_project(ctx, state["x"], weight, bias=state["bias"], **more)}
    d_in, d_out, rank, groups = case["d_in"], case["d_out"], case["rank"], case["groups"]
    x, dtype = state["x"].float(), state["x"].dtype
    y = x @ _weights(state, torch.float32).t() + state["bias"].float()
    if not rank:
        return {"y": y.to(dtype)}
    theta = state["adapters"].float().view(case["adapters"], rank * (d_in + d_out))
    ids = state["ids"].long()
    if case["probes"]:
        # each group's own parameters, moved along its probe and rounded as they are stored
        at = state["probes"].long().clamp(min=0)
        signs = (state["bits"][:, :, None] >> torch.arange(8, device="cuda", dtype=torch.uint8)) & 1
        signs = signs.view(case["probes"], -1)[:, : theta.numel()].float() * 2 - 1
        theta = (theta + signs[at] * state["alphas"][:, None]).to(dtype).float()
    else:
        theta = theta[ids.clamp(min=0)]
    theta = theta * (ids >= 0).float()[:, None]
    a = theta[:, : rank * d_in].reshape(groups, rank, d_in)
    b = theta[:, rank * d_in:].reshape(groups, d_out, rank)
    # groups padded to the longest: padding repeats the last row and is left out afterwards
    longest, starts = max(state["lengths"]), state["starts"]
    rows = starts[:-1, None] + torch.arange(longest, device="cuda")
    valid = rows < starts[1:, None]
    u = torch.bmm(x[rows.clamp(max=x.shape[0] - 1)], a.transpose(1, 2).contiguous())
    low = torch.bmm(u, b.transpose(1, 2).contiguous())[valid]
    return {"y": (y + state["scale"] * low).to(dtype)}


def _quantize(state):
    case, weight = state["case"], state["weight"]
    if own:
        zo, ctx = _context()
        q4 = zo.zo_q4_quantize(ctx, weight, case["group"])
        return {"scales": q4.scales, "weight": zo.zo_q4_unpack(ctx, q4)}
    # in 64 bits: values lie next to the border between two codes
    w = weight.double().view(case["d_out"], -1, case["group"])
    s = (w.abs().amax(dim=2, keepdim=True) / 7.0).to(weight.dtype).double()
    q = torch.where(s > 0, torch.round(w / s), torch.zeros_like(w)).clamp(-8, 7)
    return {"scales": s[:, :, 0].t().contiguous().to(weight.dtype), "weight": (q * s).view(weight.shape).to(weight.dtype)}


def _counting(state):
    """The rows that count, and a function that puts their values among all rows."""
    targets = state["targets"]
    if not state["case"]["ignore"]:
        return None, lambda value: value
    keep = (targets != IGNORE).nonzero()[:, 0]

    def put(value):
        whole = torch.zeros((targets.numel(),) + value.shape[1:], dtype=value.dtype, device=value.device)
        return whole.index_copy(0, keep, value)

    return keep, put


def _distill(state):
    case, logits, ids = state["case"], state["logits"], state["teacher_ids"]
    heights, given, temperature = state["teacher_logits"], state["row_grad"], case["temperature"]
    if own:
        zo, ctx = _context()
        out = zo.zo_distill_loss(ctx, logits, ids, heights, targets=state["targets"], temperature=temperature,
                                 grad=case["grad"], row_grad=given if case["grad"] else None)
        return {"loss": out.loss, "grad": out.grad}
    keep, put = _counting(state)
    if keep is not None:
        logits, ids, heights, given = logits[keep], ids[keep], heights[keep], given[keep]
    x = logits.float() / temperature
    there = ids >= 0
    t = (heights / temperature).masked_fill(~there, -math.inf)
    t = t - t.amax(dim=1, keepdim=True)
    p = torch.exp(t)
    total = p.sum(dim=1, keepdim=True)
    p, logp = p / total, t - torch.log(total)
    x = x - x.amax(dim=1, keepdim=True)
    e = torch.exp(x)
    s = e.sum(dim=1, keepdim=True)
    logq = torch.gather(x, 1, ids.clamp(min=0)) - torch.log(s)
    loss = torch.where(there, p * (logp - logq), torch.zeros_like(p)).sum(dim=1) * temperature ** 2
    grad = None
    if case["grad"]:
        q = e.div_(s).scatter_add_(1, ids.clamp(min=0), torch.where(there, -p, torch.zeros_like(p)))
        grad = put(q.mul_((given * temperature)[:, None]).to(logits.dtype))
    return {"loss": put(loss), "grad": grad}


def _head(state):
    hidden, weight, targets, given = state["hidden"], state["weight"], state["targets"], state["row_grad"]
    if own:
        zo, ctx = _context()
        return zo.zo_head_grad(ctx, hidden, weight, targets, row_grad=given)._asdict()
    keep, put = _counting(state)
    if keep is not None:
        hidden, targets, given = hidden[keep], targets[keep], given[keep]
    h, w = hidden.float(), weight.float()
    x = h @ w.t()
    x -= x.amax(dim=1, keepdim=True)
    e = torch.exp(x)
    s = e.sum(dim=1, keepdim=True)
    logp = (torch.gather(x, 1, targets[:, None]) - torch.log(s))[:, 0]
    d = e.div_(s).scatter_add_(1, targets[:, None], torch.full_like(s, -1.0)).mul_(given[:, None])
    return {"logp": put(logp), "hidden_grad": put((d @ w).to(hidden.dtype)),
            "weight_grad": (d.t() @ h).to(weight.dtype)}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "project":
        return _exact_project(state)
    if case["op"] == "quantize":
        w = state["weight"].double().view(case["d_out"], -1, case["group"])
        s = (w.abs().amax(dim=2) / 7.0).to(state["weight"].dtype).double()
        q = torch.where(s[:, :, None] > 0, torch.round(w / s[:, :, None]), torch.zeros_like(w))
        return {"scales": s.t(), "weight": (q * s[:, :, None]).view(case["d_out"], case["d_in"])}
    if case["op"] == "distill":
        losses, grads = [], []
        for at in range(0, case["rows"], 1024):
            rows = slice(at, at + 1024)
            mask = state["targets"][rows] != IGNORE
            ids, t = state["teacher_ids"][rows], case["temperature"]
            q = torch.log_softmax(state["logits"][rows].double() / t, dim=1)
            p = torch.log_softmax((state["teacher_logits"][rows].double() / t).masked_fill(ids < 0, -math.inf), dim=1)
            at_ids = torch.where(ids < 0, torch.zeros_like(p), p.exp() * (p - q.gather(1, ids.clamp(min=0))))
            losses.append((t * t * at_ids.sum(dim=1)).masked_fill(~mask, 0.0))
            if case["grad"]:
                g = q.exp()
                g.scatter_add_(1, ids.clamp(min=0), -p.exp().masked_fill(ids < 0, 0.0))
                g *= (t * state["row_grad"][rows].double())[:, None]
                grads.append(g.masked_fill_(~mask[:, None], 0.0))
        return {"loss": torch.cat(losses), "grad": torch.cat(grads) if grads else None}
    rows, w = case["rows"], state["weight"].double()
    wt = w.t().contiguous()
    logp, dh, dw = [], [], torch.zeros_like(w)
    for at in range(0, rows, 2048):
        h, t = state["hidden"][at: at + 2048].double(), state["targets"][at: at + 2048]
        mask = t != IGNORE
        p = torch.log_softmax(h @ wt, dim=1)
        logp.append(p.gather(1, t.clamp(min=0)[:, None])[:, 0].masked_fill(~mask, 0.0))
        d = p.exp_()
        d[torch.arange(t.numel(), device="cuda"), t.clamp(min=0)] -= 1.0
        d *= (state["row_grad"][at: at + 2048].double() * mask)[:, None]
        dh.append(d @ w)
        dw += d.t().contiguous() @ h
    return {"logp": torch.cat(logp), "hidden_grad": torch.cat(dh), "weight_grad": dw}


def _exact_project(state):
    case = state["case"]
    d_in, d_out, rank = case["d_in"], case["d_out"], case["rank"]
    # each code by where its block keeps it
    f, k = torch.arange(d_out, device="cuda")[:, None], torch.arange(d_in, device="cuda")[None, :]
    j = k % 8
    place = (k % 32 // 8 * 16 + f % 16) * 16 + k % 128 // 32 * 4 + j % 2 * 2 + j // 4
    byte = state["codes"].view(-1)[(f // 16 * state["codes"].shape[1] + k // 128) * 1024 + place]
    q = ((byte >> (j // 2 % 2 * 4).to(torch.uint8)) & 15).double()
    z = state["zeros"].double() if case["zeros"] else torch.full_like(state["scales"], 8.0).double()
    at = torch.arange(d_in, device="cuda") // case["group"]
    w = (q.t() - z[at]) * state["scales"].double()[at]
    y, at, per = [], 0, rank * (d_in + d_out)
    for g, length in enumerate(state["lengths"]):
        x = state["x"][at: at + length].double()
        at += length
        out = x @ w + state["bias"].double()
        i = int(state["ids"][g]) if rank else -1
        if i >= 0:
            theta = state["adapters"][i * per: (i + 1) * per]
            p = int(state["probes"][g]) if case["probes"] else -1
            if p >= 0:
                row = state["bits"][p][:, None] >> torch.arange(8, dtype=torch.uint8, device="cuda")
                z = (row & 1).reshape(-1)[i * per: (i + 1) * per].float() * 2 - 1
                theta = (theta.float() + z * state["alphas"][g]).to(theta.dtype)
            theta = theta.double()
            a, b = theta[: rank * d_in].view(rank, d_in), theta[rank * d_in:].view(d_out, rank)
            out = out + state["scale"] * ((x @ a.t().contiguous()) @ b.t().contiguous())
        y.append(out)
    return {"y": torch.cat(y)}
