"""Plain 64-bit references of the 4-bit projection and the distillation loss, with their bounds
(u = 2^-24 and the bf16 half step as in lm_ref).

  * 4-bit projection, weights as they are held.  A group's sum of x (o + q) (bf16: o = 16; fp32: 0) and
    of x is at most |x_g| |o + q| and |x_g| sqrt(G) (2-norms), each rounded G times: 8 sqrt(G) u of
    these is eight standard deviations of roundings of random sign.  Their difference, formed by one
    fused multiply-add, and the scale's product round once more each, of values no larger.  With
    |o + q| <= sqrt(G) (o + 15) and zero points |o + z|,
      |error of a group| <= s (8 sqrt(G) + 2) u |x_g| sqrt(G) (2 o + 15 + |z|);
    groups add up in fp32: 8 sqrt(d_in / G) u times the sum of the groups' values, which
    sqrt(sum of squares) bounds, is within 8 sqrt(d_in) u |x| |w|.
  * unpacked weights: rounded to the type by the reference too; the product's bound is lm_ref's.
  * distillation.  E = (V / 256 + 128) u bounds the error of log s: at most V / 256 terms one after another, a
    tree of ten, and each term's exponent off by 3 u |d|, sum q |d| <= log V <= 13.  A teacher's
    share carries 4 u |t - max| / T + 160 u relative (128 terms, a tree, a quotient).  Then
      loss: T^2 sum p (E + 4 u (|x - m| + |t - max|) / T + 200 u) + T^2 sum p |log p - log q| (4 u |t - max| / T + 170 u)
      gradient / (g T): q (E + 4 u (|x - m| / T + |log s|) + 8 u) + sum p (4 u |t - max| / T + 170 u),
    and one rounding to the type.
"""
from __future__ import annotations

import math

import torch

from lm_ref import IGNORE, U32, UBF  # noqa: F401


def code_places(d_out, d_in):
    """(byte, shift) of every code [d_out, d_in] among the codes' bytes, as include/zo.h states it."""
    f, k = torch.arange(d_out)[:, None], torch.arange(d_in)[None, :]
    block = (f // 16) * (-(-d_in // 128)) + k // 128
    byte = 16 * (16 * (k // 8 % 4) + f % 16) + 4 * (k // 32 % 4) + 2 * (k % 2) + k // 4 % 2
    return block * 1024 + byte, 4 * (k // 2 % 2)


def pack(values):
    d_out, d_in = values.shape
    codes = torch.zeros(-(-d_out // 16) * -(-d_in // 128) * 1024, dtype=torch.int32)
    at, shift = code_places(d_out, d_in)
    codes.index_add_(0, at.reshape(-1), (values.int() << shift.int()).reshape(-1))
    return codes.to(torch.uint8).view(-(-d_out // 16), -(-d_in // 128), 1024)


def values_of(codes, d_out, d_in):
    at, shift = code_places(d_out, d_in)
    return codes.reshape(-1).int()[at] >> shift & 15


def weights(values, scales, zeros):
    """s (q - z) in 64 bits, [d_out, d_in]."""
    d_out, d_in = values.shape
    group = d_in // scales.shape[0]
    at = torch.arange(d_in) // group
    z = 8.0 if zeros is None else zeros.double().t()[:, at]
    return (values.double() - z) * scales.double().t()[:, at]


def quantize(w, group):
    """(values, scales) of w, by the definition in 64 bits."""
    d_out, d_in = w.shape
    g = w.double().view(d_out, -1, group)
    s = (g.abs().amax(dim=2) / 7.0).to(w.dtype)
    s = torch.where(torch.isfinite(g.sum(dim=2)) & torch.isfinite(g.abs().amax(dim=2)), s, torch.full_like(s, math.nan))
    q = torch.round(g / s.double()[:, :, None]).clamp(-8, 7) + 8
    q = torch.where((s > 0)[:, :, None], q, torch.full_like(q, 8))
    return q.view(d_out, d_in).to(torch.uint8), s.t().contiguous()


def q4_bound(x, scales, zeros, dtype):
    """The 4-bit sums' bound [rows, d_out]."""
    d_in = x.shape[1]
    groups = scales.shape[0]
    size = d_in // groups
    o = 16.0 if dtype == torch.bfloat16 else 0.0
    xg = torch.linalg.vector_norm(x.double().view(x.shape[0], groups, size), dim=2)
    z = torch.full_like(scales, 8.0).double() if zeros is None else zeros.double().abs()
    each = scales.double().abs() * (8 * math.sqrt(size) + 2) * U32 * math.sqrt(size) * (2 * o + 15 + z)
    return xg @ each


def distill(x, ids, t, targets, temperature):
    """(loss, q - p's, bound of the loss, bound of the gradient, both over g = 1) in 64 bits, CPU."""
    rows, vocab = x.shape
    T, X = temperature, x.double()
    there = ids != -1
    ok = (ids >= 0) & (ids < vocab)
    at = torch.where(ok, ids, torch.zeros_like(ids))
    h = t.double().masked_fill(~there, -math.inf)
    top = h.amax(dim=1, keepdim=True) if ids.shape[1] else torch.zeros(rows, 1).double()
    p = torch.softmax(h / T, dim=1)
    logp = torch.log_softmax(h / T, dim=1)
    m = X.amax(dim=1, keepdim=True)
    s = torch.exp((X - m) / T).sum(dim=1, keepdim=True)
    logq = (X - m) / T - torch.log(s)
    q = logq.exp()
    d = logp - logq.gather(1, at)
    terms = torch.where(there & (p != 0), p * d, torch.zeros_like(p))
    loss = T * T * terms.sum(dim=1)
    E = (vocab / 256 + 128) * U32
    dt = torch.where(there, ((h - top) / T).abs(), torch.zeros_like(h)).nan_to_num(posinf=0.0)
    dx = ((X.gather(1, at) - m) / T).abs().nan_to_num(posinf=0.0)
    keep = torch.where(there, p, torch.zeros_like(p)).nan_to_num(0.0)
    share = 4 * U32 * dt + 170 * U32
    lb = T * T * (keep * (E + 4 * U32 * (dx + dt) + 200 * U32)).sum(dim=1) \
        + T * T * (keep * d.abs().nan_to_num(posinf=0.0, neginf=0.0) * share).sum(dim=1)
    grad = q.clone()
    grad.scatter_add_(1, at, torch.where(there, -p, torch.zeros_like(p)))
    dv = ((X - m) / T).abs().nan_to_num(posinf=0.0)
    gb = q.nan_to_num(0.0) * (E + 4 * U32 * (dv + torch.log(s).abs().nan_to_num(0.0)) + 8 * U32)
    gb = gb.scatter_add(1, at, keep * share)
    # a bad id, or a teacher without a distribution, leaves nothing of the row
    bad = (there & (~ok | torch.isnan(p))).any(dim=1)
    loss = loss.masked_fill(bad, math.nan)
    grad = grad.masked_fill(bad[:, None], math.nan)
    none = ~there.any(dim=1)
    if targets is not None:
        none = none | (targets == IGNORE)
    loss, grad = loss.masked_fill(none, 0.0), T * grad.masked_fill(none[:, None], 0.0)
    return loss, grad, lb, T * gb


def head_grad(h, w, targets, g, dtype):
    """(logp, dh, dW, bounds of the three) in 64 bits, CPU.

    The logits carry lm_ref's bound of a product, e = 8 sqrt(d) u |h| |w| (at most over a row's
    features), and log s E as in lm_ref: a share p is off by p (2 e + E + 4 u (|l - m| + |log s|)) or
    less, D by that, its product with g and the rounding to the type.  The products add
    8 sqrt(terms) u of their operands' 2-norms."""
    H, W, G = h.double(), w.double(), g.double()
    rows, d = h.shape
    vocab = w.shape[0]
    half = UBF if dtype == torch.bfloat16 else U32
    count = targets != IGNORE
    H = torch.where(count[:, None], H, torch.zeros_like(H))
    ok = (targets >= 0) & (targets < vocab)
    at = torch.where(ok, targets, torch.zeros_like(targets))
    x = H @ W.t()
    m = x.amax(dim=1, keepdim=True)
    logs = torch.log(torch.exp(x - m).sum(dim=1, keepdim=True))
    p = torch.exp((x - m) - logs)
    e = 8 * math.sqrt(d) * U32 * torch.linalg.vector_norm(H, dim=1) * torch.linalg.vector_norm(W, dim=1).max()
    E = (vocab / 256 + 64) * U32
    logp = (x - m - logs).gather(1, at[:, None])[:, 0]
    D = p.clone()
    D[torch.arange(rows), at] -= 1.0
    gz = torch.where(count, G, torch.zeros_like(G))[:, None]
    D = D * gz
    off = gz.abs() * p * (2 * e[:, None] + E + 4 * U32 * ((x - m).abs() + logs.abs())) + (half + 3 * U32) * D.abs() \
        + gz.abs() * U32 * p
    norm = torch.linalg.vector_norm
    dh, dw = D @ W, D.t() @ H
    bh = off @ W.abs() + 8 * math.sqrt(vocab) * U32 * norm(D, dim=1)[:, None] * norm(W, dim=0)[None, :] + half * dh.abs()
    bw = off.t() @ H.abs() + 8 * math.sqrt(rows) * U32 * norm(D, dim=0)[:, None] * norm(H, dim=0)[None, :] + half * dw.abs()
    bl = 2 * e + E + 2 * U32 * ((x - m).gather(1, at[:, None])[:, 0].abs() + logp.abs())
    bad = count & ~ok
    logp = logp.masked_fill(bad, math.nan).masked_fill(~count, 0.0)
    dh = dh.masked_fill(bad[:, None], math.nan)
    if bool(bad.any()):
        dw = torch.full_like(dw, math.nan)
    return logp, dh, dw, bl, bh, bw
