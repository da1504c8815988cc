"""Plain 64-bit references of the language-model operators and the error bounds they are held to.

Bounds (u = 2^-24, half an fp32 step; u_bf16 = 2^-8, half a bf16 step, both relative):
  * softmax sums.  A term e^d with d = x - m <= 0 carries the rounding of d log2(e) (2 u |d|
    of the exponent, the constant's and the product's) and of the exponential (at most 2 u);
    sum_v p_v |d_v| <= log V <= 13 for V < 4e5, so the sum's relative error is below 32 u from
    its terms, and below (V / 256 + 32) u from adding them: at most V / 256 terms one after
    another in each of 256 threads, then a tree, each merge rescaling once more.  Hence
      E = (V / 256 + 64) u   bounds the absolute error of log s,
      logp: E + u (|x_t - m| + |logp|),  entropy: E (1 + |t / s|) + E |t / s|, |t / s| <= 13.
    Where E is not a sum of worst cases: rows of up to 12 KB are added by 64 threads, up to
    V / 64 = 96 terms one after another, worst case 96 + 64 against E = 88 u at V = 6144; and the
    head adds up to 32 features in a lane and then joins parts.  There E counts on roundings of
    random sign: an error uniform within u of a partial sum that grows to the whole gives eight
    standard deviations of 8 sqrt(96 / 9) u = 26 u for 96 terms, which with the terms' 32 u stays
    below E.
  * a product of k terms summed in fp32: rounding errors of random sign, k of them, each at
    most u times a partial sum; 8 sqrt(k) u |x| |w| (2-norms) is eight standard deviations
    or more.
"""
from __future__ import annotations

import math

import torch

IGNORE = -100
U32 = 2.0 ** -24
UBF = 2.0 ** -8


def log_stats(x):
    """(max, log s, t / s) of the rows of a float64 matrix; terms of probability 0 drop out."""
    m = x.max(dim=1, keepdim=True).values
    d = x - m
    e = torch.exp(d)
    s = e.sum(dim=1)
    t = torch.where(e == 0, torch.zeros_like(e), e * d).sum(dim=1)
    return m[:, 0], torch.log(s), t / s


def token(x, targets, top_k):
    """logp, entropy, ids, alternatives' logp from logits (any float type, CPU), in 64 bits."""
    x64 = x.double()
    m, logs, ts = log_stats(x64)
    rows, vocab = x.shape
    # (x - m) - log s: at the type's lowest values m + log s would be m even in 64 bits, and
    # the equal logits' -log V be lost; then to the range of fp32, where max - min is infinite
    lp = ((x64 - m[:, None]) - logs[:, None]).clamp(-1e39, 1e39)
    lp = torch.where(lp < -torch.finfo(torch.float32).max, torch.full_like(lp, -math.inf), lp)
    entropy = logs - ts
    logp = None
    if targets is not None:
        ok = (targets >= 0) & (targets < vocab)
        at = torch.where(ok, targets, torch.zeros_like(targets))
        logp = lp.gather(1, at[:, None])[:, 0]
        logp = torch.where(ok, logp, torch.full_like(logp, math.nan))
    # stable ascending sort of the negated values: ties lowest index first; NaN first of all
    key = torch.where(torch.isnan(x64), torch.full_like(x64, math.inf), x64 + 0.0)
    nan_first = torch.isnan(x64).double()
    order = torch.argsort(-key, dim=1, stable=True)
    order = order.gather(1, torch.argsort(-nan_first.gather(1, order), dim=1, stable=True))
    ids = order[:, :top_k]
    top = lp.gather(1, ids)
    if targets is not None:
        skip = targets == IGNORE
        logp = logp.masked_fill(skip, 0.0)
        entropy = entropy.masked_fill(skip, 0.0)
        ids = ids.masked_fill(skip[:, None], -1)
        top = top.masked_fill(skip[:, None], 0.0)
    return logp, entropy, ids, top


def token_bound(vocab):
    return (vocab / 256 + 64) * U32


def assert_close(got, ref, bound, what):
    """|got - ref| <= bound where ref is finite; NaN and infinities exactly alike."""
    g, r = got.double().cpu(), ref.double().cpu()
    assert g.shape == r.shape, (what, g.shape, r.shape)
    fin = torch.isfinite(r)
    same = torch.where(torch.isnan(r), torch.isnan(g), g == r)
    assert bool((same | fin).all()), f"{what}: NaN or infinity in the wrong place"
    b = torch.as_tensor(bound, dtype=torch.float64).expand_as(r) if not torch.is_tensor(bound) \
        else bound.double().cpu().expand_as(r)
    err = (g - r).abs()
    bad = fin & ~(err <= b)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds; worst "
                                 f"{float((err / b)[bad].max()):.3g} times the bound")


def signs(bits, n):
    """+/-1 of packed rows (uint8 [probes, stride], CPU) over n parameters."""
    b = (bits[:, :, None] >> torch.arange(8, dtype=torch.uint8)) & 1
    return b.reshape(bits.shape[0], -1)[:, :n].float() * 2 - 1


def project(x, w, bias, adapters, rank, starts, ids, scale, probes=None, alphas=None, z=None):
    """(y, the low-rank part's magnitude, bound of the sums) in 64 bits for CPU tensors; rows of
    no group are NaN in y."""
    d_in, d_out = x.shape[1], w.shape[0]
    per = rank * (d_in + d_out)
    X, W = x.double(), w.double()
    base = X @ W.t()
    if bias is not None:
        base = base + bias.double()
    y = torch.full_like(base, math.nan)
    low = torch.zeros_like(base)
    norms = torch.linalg.vector_norm(X, dim=1)[:, None] * torch.linalg.vector_norm(W, dim=1)[None, :]
    bound = 8 * math.sqrt(d_in) * U32 * norms
    for g in range(len(ids)):
        lo, hi = int(starts[g]), int(starts[g + 1])
        if hi <= lo:
            continue
        y[lo:hi] = base[lo:hi]
        i = int(ids[g])
        if i < 0:
            continue
        th = adapters[i * per:(i + 1) * per]
        if probes is not None and int(probes[g]) >= 0:
            th = (th.float() + z[int(probes[g])][i * per:(i + 1) * per] * alphas[g]).to(th.dtype)
        th = th.double()
        a, b = th[:rank * d_in].view(rank, d_in), th[rank * d_in:].view(d_out, rank)
        u = X[lo:hi] @ a.t()
        d = scale * (u @ b.t())
        y[lo:hi] += d
        mag = abs(scale) * (u.abs() @ b.abs().t())
        low[lo:hi] = mag
        un = (torch.linalg.vector_norm(X[lo:hi], dim=1)[:, None]
              * torch.linalg.vector_norm(a, dim=1)[None, :])
        bound[lo:hi] += abs(scale) * 8 * math.sqrt(d_in) * U32 * (un @ b.abs().t())
    return y, low, bound
