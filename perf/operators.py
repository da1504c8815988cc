"""The language-model operators: what is measured of each, in its plain form and in the library's.

Four operators, used together by a forward-only training step with low-rank adapters, and
one by one when scoring text:

  token    log probabilities of given tokens, with entropy and the top alternatives, from logits
  head     the same log probabilities and entropies from hidden states and the unembedding matrix
  adapter  a shared projection with low-rank adapters of many requests or probes beside it
  group    the mean negative log probability of each group of rows, in 64 bits

A row whose target is IGNORE counts for nothing: its log probability and entropy are 0, its
alternatives -1 and 0.
"""
import math
import random

import numpy as np
import torch

own = False

IGNORE = -100
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
VOCAB = 50272


def listed():
    return [
        # the next token of one sequence: entropy and alternatives only, latency counts
        {"name": "token 1 row", "op": "token", "rows": 1, "vocab": VOCAB, "pad": 0, "dtype": "bf16",
         "given": False, "ignore": 0.0, "masked": 0.0, "top": 20},
        # answers of odd length over an odd vocabulary, part of it masked off, prompts ignored
        {"name": "token fp32 odd", "op": "token", "rows": 2051, "vocab": 32003, "pad": 2,
         "dtype": "fp32", "given": True, "ignore": 0.5, "masked": 0.1, "top": 5},
        # every token of 128 sequences of 128
        {"name": "token 16k rows", "op": "token", "rows": 16384, "vocab": VOCAB, "pad": 0,
         "dtype": "bf16", "given": True, "ignore": 0.0, "masked": 0.0, "top": 0},
        # a few candidate answers: the unembedding matrix is read once
        {"name": "head 8 rows", "op": "head", "rows": 8, "vocab": VOCAB, "dim": 5120,
         "dtype": "bf16", "ignore": 0.0},
        # a small model in fp32, all tokens of a batch
        {"name": "head fp32", "op": "head", "rows": 2048, "vocab": VOCAB, "dim": 768,
         "dtype": "fp32", "ignore": 0.0},
        # the widest model's batch of 128 sequences of 128, prompts ignored
        {"name": "head 16k rows", "op": "head", "rows": 16384, "vocab": VOCAB, "dim": 7168,
         "dtype": "bf16", "ignore": 0.75},
        # one token of each of 32 requests, an adapter for each
        {"name": "adapter 32 requests", "op": "adapter", "groups": 32, "length": 1, "d_in": 5120,
         "d_out": 5120, "rank": 16, "adapters": 32, "probes": 0, "dtype": "bf16"},
        # both signs of 32 probes of one adapter and the clean pass, a short batch for each
        {"name": "adapter 32 probes", "op": "adapter", "groups": 65, "length": 48, "d_in": 5120,
         "d_out": 5120, "rank": 16, "adapters": 1, "probes": 32, "dtype": "bf16"},
        # the same of a small model in fp32
        {"name": "adapter fp32 probes", "op": "adapter", "groups": 33, "length": 64, "d_in": 768,
         "d_out": 768, "rank": 8, "adapters": 1, "probes": 16, "dtype": "fp32"},
        # long prompts of several requests through the widened projection
        {"name": "adapter prompts", "op": "adapter", "groups": 8, "length": 1024, "d_in": 5120,
         "d_out": 20480, "rank": 32, "adapters": 5, "probes": 0, "dtype": "bf16"},
        # 16 probes of both signs and the clean pass, one short sequence for each
        {"name": "group short", "op": "group", "groups": 33, "length": 32, "ignore": 0.5},
        # 160 probes of both signs and the clean pass, a batch of 2048 tokens for each
        {"name": "group long", "op": "group", "groups": 321, "length": 2048, "ignore": 0.25},
    ]


def _between(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["token", "token", "head", "head", "adapter", "adapter", "group"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    ignore = rng.choice([0.0, 0.25, 0.5, 0.75])
    if op == "token":
        vocab = _between(rng, 1000, 200000)
        size = 4 if dtype == "fp32" else 2
        rows = _between(rng, 1, min(16384, 16384 * VOCAB * 2 // (vocab * size)))
        return {"op": op, "rows": rows, "vocab": vocab, "pad": rng.choice([0, 0, 1, 8]),
                "dtype": dtype, "given": rng.random() < 0.8, "ignore": ignore,
                "masked": rng.choice([0.0, 0.0, 0.2]), "top": rng.choice([0, 0, 1, 4, 8, 20, 32])}
    if op == "head":
        vocab, dim = _between(rng, 1000, 131072), 8 * _between(rng, 8, 896)
        most = 16384 * VOCAB * 7168 // 4 // (vocab * dim * (12 if dtype == "fp32" else 1))
        return {"op": op, "rows": _between(rng, 1, max(1, min(16384, most))), "vocab": vocab,
                "dim": dim, "dtype": dtype, "ignore": ignore}
    if op == "adapter":
        d_in, d_out = 8 * _between(rng, 8, 896), 8 * _between(rng, 8, 2560)
        most = 8192 * 5120 * 20480 // 2 // (d_in * d_out * (12 if dtype == "fp32" else 1))
        rows = _between(rng, 1, max(1, min(8192, most)))
        probes = rng.choice([0, 1, 8, 32])
        groups = 2 * probes + 1 if probes else _between(rng, 1, 64)
        adapters = 1 if probes else _between(rng, 1, min(32, groups))
        return {"op": op, "groups": groups, "length": max(1, rows // groups), "d_in": d_in,
                "d_out": d_out, "rank": rng.choice([8, 16, 24, 32, 64]), "adapters": adapters,
                "probes": probes, "dtype": dtype}
    return {"op": op, "groups": _between(rng, 1, 321), "length": _between(rng, 8, 2048),
            "ignore": ignore}


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
    if case["op"] == "token":
        rows = sum(_counted(case, case["rows"]))
        size = 4 if case["dtype"] == "fp32" else 2
        out = 4 + 12 * case["top"] + (4 if case["given"] else 0)
        return {"bytes": rows * case["vocab"] * size + case["rows"] * (8 * case["given"] + out),
                "flops": 5 * rows * case["vocab"]}
    if case["op"] == "head":
        rows = sum(_counted(case, case["rows"]))
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": (rows + case["vocab"]) * case["dim"] * size + case["rows"] * 16,
                "flops": 2 * rows * case["dim"] * case["vocab"]}
    if case["op"] == "adapter":
        rows, d_in, d_out, rank = sum(_lengths(case)), case["d_in"], case["d_out"], case["rank"]
        size = 4 if case["dtype"] == "fp32" else 2
        params = case["adapters"] * rank * (d_in + d_out)
        return {"bytes": (rows * (d_in + d_out) + d_in * d_out + d_out + params) * size
                + case["probes"] * params // 8,
                "flops": 2 * rows * (d_in * d_out + rank * (d_in + d_out))}
    rows = sum(_lengths(case))
    return {"bytes": rows * 12 + case["groups"] * 16, "flops": 2 * rows}


def _targets(case, rows, vocab, gen):
    t = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    keep = torch.tensor(_counted(case, rows), device="cuda")
    return torch.where(keep, t, torch.full_like(t, IGNORE))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    state = {"case": case}
    if case["op"] == "token":
        rows, vocab = case["rows"], case["vocab"]
        dtype = TYPES[case["dtype"]]
        x = normal(rows, vocab + case["pad"], std=2.5)
        if case["masked"]:
            off = torch.rand(vocab + case["pad"], generator=gen, device="cuda") < case["masked"]
            off[: 64] = False
            x = x.masked_fill(off, -math.inf)
        state["logits"] = x.to(dtype)[:, :vocab]
        state["targets"] = _targets(case, rows, 64 if case["masked"] else vocab, gen) if case["given"] else None
    elif case["op"] == "head":
        dtype = TYPES[case["dtype"]]
        state["hidden"] = normal(case["rows"], case["dim"], dtype=dtype)
        state["weight"] = normal(case["vocab"], case["dim"], std=2.5 / math.sqrt(case["dim"]), dtype=dtype)
        state["targets"] = _targets(case, case["rows"], case["vocab"], gen)
    elif case["op"] == "adapter":
        dtype, rank = TYPES[case["dtype"]], case["rank"]
        d_in, d_out, adapters, groups = case["d_in"], case["d_out"], case["adapters"], case["groups"]
        lengths = _lengths(case)
        rows, params = sum(lengths), case["adapters"] * rank * (d_in + d_out)
        state["lengths"] = lengths
        state["starts"] = torch.tensor([sum(lengths[:g]) for g in range(groups + 1)], device="cuda")
        state["x"] = normal(rows, d_in, dtype=dtype)
        state["weight"] = normal(d_out, d_in, std=0.02, dtype=dtype)
        state["bias"] = normal(d_out, std=0.02, dtype=dtype)
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
            ids = [rng.randrange(adapters) if rng.random() < 0.9 else -1 for _ in range(groups)]
        state["ids"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
    else:
        lengths = _lengths(case)
        rows = sum(lengths)
        state["starts"] = torch.tensor([0] + lengths, device="cuda").cumsum(0)
        state["logp"] = -torch.rand(rows, generator=gen, device="cuda").mul(6.0).add(0.01)
        state["targets"] = _targets(case, rows, VOCAB, gen)
    return state


_kept = {}


def _context():
    import forward_only_amd as zo
    if "ctx" not in _kept:
        _kept["ctx"] = zo.zo_init(0)
    return zo, _kept["ctx"]


def run(state):
    case = state["case"]
    if case["op"] == "token":
        return _token(state)
    if case["op"] == "head":
        return _head(state)
    if case["op"] == "adapter":
        return _adapter(state)
    return _group(state)


def _counting(state):
    """The rows that count, and a function that puts their values among all rows; None for all."""
    targets = state["targets"]
    if targets is None or not state["case"]["ignore"]:
        return None, targets, lambda value, rest: value
    keep = (targets != IGNORE).nonzero()[:, 0]

    def put(value, rest):
        whole = torch.full((targets.numel(),) + value.shape[1:], rest, dtype=value.dtype, device=value.device)
        return whole.index_copy(0, keep, value)

    return keep, targets[keep], put


def _statistics(x, targets):
    """The logarithm of the sum of e^x, log probability of the targets, and entropy, 32 bits."""
    top = x.amax(dim=1, keepdim=True)
    e = torch.exp(x - top)
    s = e.sum(dim=1, keepdim=True)
    less = torch.where(e > 0, (x - top) * e, torch.zeros_like(e)).sum(dim=1, keepdim=True)
    norm = top + torch.log(s)
    entropy = (torch.log(s) - less / s)[:, 0]
    if targets is None:
        return norm, None, entropy
    return norm, (torch.gather(x, 1, targets[:, None]) - norm)[:, 0], entropy


def _token(state):
    case, logits = state["case"], state["logits"]
    if own:
        zo, ctx = _context()
        return zo.zo_token_logprobs(ctx, logits, state["targets"], top_k=case["top"])._asdict()
    keep, targets, put = _counting(state)
    x = (logits if keep is None else logits[keep]).float()
    norm, logp, entropy = _statistics(x, targets)
    out = {"logp": None if logp is None else put(logp, 0.0), "entropy": put(entropy, 0.0)}
    if case["top"]:
        # the value in the high half in an order of whole numbers, the index counted down in the low
        b = (x + 0.0).view(torch.int32)
        b = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long()
        low = torch.arange(case["vocab"] - 1, -1, -1, device=x.device)
        key = torch.topk(b * (1 << 32) + low, case["top"], dim=1).values
        ids = case["vocab"] - 1 - (key & 0xFFFFFFFF)
        out["top_ids"], out["top_logp"] = put(ids, -1), put(torch.gather(x, 1, ids) - norm, 0.0)
    return out


def _head(state):
    hidden, weight = state["hidden"], state["weight"]
    if own:
        zo, ctx = _context()
        return zo.zo_head_logprobs(ctx, hidden, weight, state["targets"])._asdict()
    keep, targets, put = _counting(state)
    x = (hidden if keep is None else hidden[keep]).float()
    _, logp, entropy = _statistics(x @ weight.float().t(), targets)
    return {"logp": put(logp, 0.0), "entropy": put(entropy, 0.0)}


def _adapter(state):
    case = state["case"]
    if own:
        zo, ctx = _context()
        more = {}
        if case["probes"]:
            more = {"probes": state["probes"], "alphas": state["alphas"], "bits": state["bits"]}
        return {"y": zo.zo_adapter_project(ctx, state["x"], state["weight"], state["adapters"],
                                           case["rank"], state["starts"], state["ids"],
                                           scale=state["scale"], bias=state["bias"], **more)}
    d_in, d_out, rank, groups = case["d_in"], case["d_out"], case["rank"], case["groups"]
    x, dtype = state["x"].float(), state["x"].dtype
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
    y = x @ state["weight"].float().t() + state["bias"].float() + state["scale"] * low
    return {"y": y.to(dtype)}


def _group(state):
    if own:
        zo, ctx = _context()
        return {"loss": zo.zo_group_loss(ctx, state["logp"], state["targets"], state["starts"])}
    starts, groups = state["starts"], state["case"]["groups"]
    count = state["targets"] != IGNORE
    lost = torch.where(count, -state["logp"], torch.zeros_like(state["logp"])).double()
    which = torch.repeat_interleave(torch.arange(groups, device="cuda"), starts[1:] - starts[:-1],
                                    output_size=lost.numel())
    zero = torch.zeros(groups, dtype=torch.float64, device="cuda")
    total = zero.index_add(0, which, lost)
    return {"loss": total / zero.index_add(0, which, count.double())}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] in ("token", "head"):
        rows, targets = case["rows"], state["targets"]
        logp, entropy = [], []
        tops = [] if case.get("top") else None
        w = state["weight"].double().t().contiguous() if case["op"] == "head" else None
        for at in range(0, rows, 4096):
            if w is None:
                x = state["logits"][at: at + 4096].double()
            else:
                x = state["hidden"][at: at + 4096].double() @ w
            p = torch.log_softmax(x, dim=1)
            h = -(p.exp() * p.clamp(min=-1e300)).sum(dim=1)
            if targets is None:
                mask = torch.ones(x.shape[0], dtype=torch.bool, device="cuda")
            else:
                t = targets[at: at + 4096]
                mask = t != IGNORE
                logp.append(p.gather(1, t.clamp(min=0)[:, None])[:, 0].masked_fill(~mask, 0.0))
            entropy.append(h.masked_fill(~mask, 0.0))
            if tops is not None:
                best = p.sort(dim=1, descending=True).values[:, : case["top"]]
                tops.append(best.masked_fill(~mask[:, None], 0.0))
        out = {"logp": torch.cat(logp) if logp else None, "entropy": torch.cat(entropy)}
        if tops is not None:
            out["top_ids"], out["top_logp"] = None, torch.cat(tops)
        return out
    if case["op"] == "adapter":
        d_in, d_out, rank = case["d_in"], case["d_out"], case["rank"]
        w, bias = state["weight"].double().t().contiguous(), state["bias"].double()
        per, y, at = rank * (d_in + d_out), [], 0
        for g, length in enumerate(state["lengths"]):
            x = state["x"][at: at + length].double()
            at += length
            out = x @ w + bias
            i = int(state["ids"][g])
            if i >= 0:
                theta = state["adapters"][i * per: (i + 1) * per]
                p = int(state["probes"][g]) if case["probes"] else -1
                if p >= 0:
                    row = state["bits"][p].cpu().numpy()
                    z = np.unpackbits(row, bitorder="little")[i * per: (i + 1) * per].astype("f4") * 2 - 1
                    step = torch.from_numpy(z).cuda() * state["alphas"][g]
                    theta = (theta.float() + step).to(theta.dtype)
                theta = theta.double()
                a, b = theta[: rank * d_in].view(rank, d_in), theta[rank * d_in:].view(d_out, rank)
                out = out + state["scale"] * ((x @ a.t().contiguous()) @ b.t().contiguous())
            y.append(out)
        return {"y": torch.cat(y)}
    starts = state["starts"].tolist()
    loss = []
    for g in range(case["groups"]):
        lp, t = state["logp"][starts[g]: starts[g + 1]], state["targets"][starts[g]: starts[g + 1]]
        lp = lp[t != IGNORE].double()
        loss.append(-lp.sum() / lp.numel())
    return {"loss": torch.stack(loss)}
