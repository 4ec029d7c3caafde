"""Plain 64-bit implementations of routing by scores and of the layer with experts in 8 bits,
written from their definitions in occ.h; the tests compare the kernels with them and their
gradients with differences.  CPU torch and Python; the choice is a sort of tuples."""
from __future__ import annotations

import math

import torch

from block_reference import U, half_step

SOFTMAX, SIGMOID = 0, 1
TINY = 2.0 ** -100


def left_out(logits):
    return torch.isnan(logits) | (logits == -math.inf)


def scores(logits, kind):
    """s in 64 bits, 0 for an expert that is left out."""
    out = left_out(logits)
    v = torch.where(out, torch.zeros_like(logits), logits).double()
    if kind == SIGMOID:
        s = torch.where(v >= 0, 1 / (1 + torch.exp(-v.abs())),
                        torch.exp(-v.abs()) / (1 + torch.exp(-v.abs())))
        return torch.where(out, torch.zeros_like(s), s)
    v = torch.where(out, torch.full_like(v, -math.inf), v)
    top = v.amax(1, keepdim=True)
    e = torch.where(v == -math.inf, torch.zeros_like(v), torch.exp(v - torch.where(
        top == -math.inf, torch.zeros_like(top), top)))
    total = e.sum(1, keepdim=True)
    return torch.where(total > 0, e / torch.where(total > 0, total, torch.ones_like(total)), e)


def shares(logits, ids, kind):
    """s / (sum of the chosen s) of the chosen, from the scores' logarithms (a softmax's but for a
    term that cancels), which do not vanish; 0 where all of them are left out."""
    v = logits.gather(1, ids.long())
    dead = left_out(v)
    v = torch.where(dead, torch.zeros_like(v), v).double()
    if kind == SIGMOID:
        v = v.clamp(max=0) - torch.log1p(torch.exp(-v.abs()))
    v = torch.where(dead, torch.full_like(v, -math.inf), v)
    top = v.amax(1, keepdim=True)
    e = torch.exp(v - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(1, keepdim=True)
    return torch.where(total > 0, e / torch.where(total > 0, total, torch.ones_like(total)), e)


def route(logits, bias, placement, k, kind, top_groups, group_best, renormalise, scale):
    """ids (T x k) and w in 64 bits."""
    T, Ne = logits.shape
    s = scores(logits, kind)
    dead = left_out(logits)
    order = s + bias.double() if bias is not None else logits.double()
    group_of = s + bias.double() if bias is not None else s
    ids, w = torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        c = [-math.inf if dead[t, e] else float(order[t, e]) for e in range(Ne)]
        allowed = set(range(Ne))
        if top_groups < len(placement):
            ranked = []
            for g, members in enumerate(placement):
                best = sorted((float(group_of[t, e]) for e in members if not dead[t, e]),
                              reverse=True)[:group_best]
                ranked.append((-sum(best) if best else math.inf, g))
            allowed = {int(e) for _, g in sorted(ranked)[:top_groups] for e in placement[g]}
        pick = sorted((-c[e], e) for e in allowed)[:k]
        for j, (_, e) in enumerate(pick):
            ids[t, j], w[t, j] = e, s[t, e]
    if renormalise:
        w = shares(logits, ids, kind)
    return ids, scale * w


def route_back(logits, ids, dw, kind, renormalise, scale):
    """The gradient in the logits, by formula, and the magnitudes that it is made of."""
    T, Ne = logits.shape
    s, dead = scores(logits, kind), left_out(logits)
    grad, mag = torch.zeros(T, Ne, dtype=torch.float64), torch.zeros(T, Ne, dtype=torch.float64)
    good = (ids >= 0) & (ids < Ne)
    at = torch.where(good, ids, torch.zeros_like(ids)).long()
    good = good & ~dead.gather(1, at)
    sj = torch.where(good, s.gather(1, at), torch.zeros(T, ids.shape[1], dtype=torch.float64))
    g = torch.where(good, dw.double(), torch.zeros_like(dw, dtype=torch.float64))
    if kind == SOFTMAX and not renormalise:
        chosen = torch.zeros_like(grad).scatter_add_(1, at, g)
        size = torch.zeros_like(grad).scatter_add_(1, at, g.abs())
        sub, subm = (g * sj).sum(1, keepdim=True), (g * sj).abs().sum(1, keepdim=True)
        return scale * s * (chosen - sub), abs(scale) * s * (size + subm)
    r = sj
    if renormalise:  # of those that count: others read as left out
        r = shares(torch.where(good, logits.gather(1, at), torch.full_like(logits[:1, :1], -math.inf)),
                   torch.arange(ids.shape[1]).expand_as(ids), kind)
    rest = 1.0
    if kind == SIGMOID:  # 1 - s without its cancellation
        x = torch.where(good, logits.gather(1, at), torch.zeros_like(sj, dtype=logits.dtype)).double()
        rest = 1 / (1 + torch.exp(x.clamp(max=700)))
    mean = (g * r).sum(1, keepdim=True) if renormalise else 0.0
    meanm = (g * r).abs().sum(1, keepdim=True) if renormalise else 0.0
    grad.scatter_add_(1, at, scale * r * rest * (g - mean))
    mag.scatter_add_(1, at, abs(scale) * r * rest * (g.abs() + meanm))
    return grad, mag


def bias_step(ids, valid, bias, Ne, rate):
    rows = ids if valid is None else ids[valid.bool()]
    flat = rows.flatten().long()
    counts = torch.bincount(flat[(flat >= 0) & (flat < Ne)], minlength=Ne)
    over = counts.sum() - Ne * counts
    new = bias + torch.tensor(rate, dtype=torch.float32) * torch.sign(over).float()
    return torch.cat([counts, torch.tensor([rows.shape[0]])]).int(), new


def quantise(x):
    """codes (int8) and scales of the rows of x by the definition's own fp32 arithmetic."""
    x = x.float()
    a = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    held = ~bad & (a >= TINY)
    safe = torch.where(held, a, torch.ones_like(a))
    # (a number over a tensor is torch's reciprocal times the number: two roundings, not a quotient)
    top = torch.full_like(a, 127.0)
    inv = torch.where(held, top / safe, torch.zeros_like(a))
    q = torch.round(torch.where(bad[..., None], torch.zeros_like(x), x) * inv[..., None]).clamp(-127, 127)
    scale = torch.where(bad, torch.full_like(a, math.nan),
                        torch.where(held, a / top, torch.zeros_like(a)))
    return q.to(torch.int8), scale


def sanitise(ids, w, Ne):
    """An id out of range or repeated becomes the lowest unused expert with weight 0."""
    ids, w = ids.clone(), w.clone()
    for t in range(ids.shape[0]):
        seen = []
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < Ne or e in seen:
                e = next(c for c in range(Ne) if c not in seen)
                ids[t, j], w[t, j] = e, 0.0
            seen.append(e)
    return ids, w


def expert8(xq, xs, gate, up, down, w):
    """Terms of y for rows of codes through one expert, in 64 bits, and a bound on how far a
    kernel's fp32 arithmetic may be from them before the terms are rounded.

    h is off by at most n u |h|: the scales' products and acc (4 roundings), exp of |g| in base
    2 (|g| + 2), the reciprocal and the products (6), so that n = |g| + 12.  A code h * (127 / a)
    is then off by at most (n_h + n_a + 2) u |v|, v the code before its rounding (n_a of the
    row's largest); where v lies that near the middle of two codes either may be taken, which
    moves a term by one code's weight.  The scale is off by n_a + 1, and a term's own product of
    scales and sum by 3 roundings more."""
    x = xq.double() * xs.double()[:, None]
    g = x @ (gate[0].double() * gate[1].double()[:, None]).t()
    u = x @ (up[0].double() * up[1].double()[:, None]).t()
    h = w.double()[:, None] * g * torch.sigmoid(g) * u
    n = g.abs() + 12
    a = h.abs().amax(1, keepdim=True)
    # the row's largest may be another element within the rounding: the largest n of the row
    n_a = n.amax(1, keepdim=True)
    held = a >= TINY
    unit = torch.where(held, a / 127, torch.zeros_like(a))
    v = torch.where(held, h / torch.where(held, unit, torch.ones_like(unit)), torch.zeros_like(h))
    code = torch.round(v)
    near = ((v - torch.floor(v) - 0.5).abs() <= (n + n_a + 2) * U * v.abs()).double()
    wide = down[0].double()
    term = (code @ wide.t()) * unit * down[1].double()
    moved = (near @ wide.abs().t()) * unit * down[1].double().abs()
    return term, moved + (n_a + 4) * U * term.abs()


def layer8(x, ids, w, experts, shared):
    """y in 64 bits and the bound of a bf16 y that is made as occ.h says."""
    xq, xs = quantise(x)
    ids, w = sanitise(ids, w, experts[0][0].shape[0])
    T, d = x.shape
    y, far, size = (torch.zeros(T, d, dtype=torch.float64) for _ in range(3))

    def add(rows, term, off):
        y.index_add_(0, rows, term)
        far.index_add_(0, rows, off + half_step(torch.bfloat16) * (term.abs() + off))
        size.index_add_(0, rows, term.abs() + off)

    for e in range(experts[0][0].shape[0]):
        rows, slot = (ids == e).nonzero(as_tuple=True)
        if rows.numel():
            add(rows, *expert8(xq[rows], xs[rows], *[(q[e], s[e]) for q, s in experts], w[rows, slot]))
    n_shared = shared[0][0].shape[0] if shared else 0
    for e in range(n_shared):
        add(torch.arange(T), *expert8(xq, xs, *[(q[e], s[e]) for q, s in shared], torch.ones(T)))
    far = far + (ids.shape[1] + n_shared) * U * size
    return y, far + half_step(torch.bfloat16) * (y.abs() + far)
