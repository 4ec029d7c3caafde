"""Plain 64-bit implementations of the operators around the layer (norms, router losses, gate
projection, AdamW), written from their definitions in occ.h, with their gradients by formula; the
tests compare the kernels with them and them with differences.  Device-agnostic torch."""
from __future__ import annotations

import torch

U = 2.0 ** -24  # half a step of fp32 relative to the value


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def unit_rows(v, eps):
    rstd = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    return v * rstd, rstd


def as_rows(gate, kind):
    """A gate as something that multiplies rows: kind 0 none, 1 per channel, 2 per token."""
    return 1.0 if kind == 0 else gate.double() if kind == 1 else gate.double()[:, None]


def block_norm(x, y, w_post, gate, w_pre, kind, eps, scale):
    """(r, h), with the sum of the magnitudes that make up r."""
    x = x.double()
    r, mag = x, x.abs()
    if y is not None:
        z = y.double()
        if w_post is not None:
            z = unit_rows(z, eps)[0] * w_post.double()
        z = scale * as_rows(gate, kind) * z
        r, mag = x + z, x.abs() + z.abs()
    h = None if w_pre is None else unit_rows(r, eps)[0] * w_pre.double()
    return r, h, mag


def block_norm_back(dr, dh, r, y, w_post, gate, w_pre, kind, eps, scale):
    """Gradients and, under the same names, the sums of magnitudes behind them (for error
    bounds): dicts of dx, dy, dw_post, dgate, dw_pre."""
    like = (dr if dr is not None else dh).double()
    g = dr.double() if dr is not None else torch.zeros_like(like)
    mag = g.abs()
    out, m = {}, {}
    if w_pre is not None:
        n, rstd = unit_rows(r.double(), eps)
        q = dh.double() * w_pre.double()
        g = g + rstd * (q - n * (q * n).mean(1, keepdim=True))
        mag = mag + rstd * (q.abs() + n.abs() * (q * n).abs().mean(1, keepdim=True))
        out["dw_pre"], m["dw_pre"] = (dh.double() * n).sum(0), (dh.double() * n).abs().sum(0)
    out["dx"], m["dx"] = g, mag
    if y is None:
        return out, m
    yd, ga = y.double(), as_rows(gate, kind)
    n, rstd = unit_rows(yd, eps) if w_post is not None else (yd, None)
    w = w_post.double() if w_post is not None else 1.0
    dz, dzm = scale * g, abs(scale) * mag
    if kind:
        axis = 0 if kind == 1 else 1
        out["dgate"], m["dgate"] = (dz * n * w).sum(axis), (dzm * (n * w).abs()).sum(axis)
    q, qm = dz * ga, dzm * abs(ga)
    if w_post is not None:
        out["dw_post"], m["dw_post"] = (q * n).sum(0), (qm * n.abs()).sum(0)
        q, qm = q * w, qm * abs(w)
        q = rstd * (q - n * (q * n).mean(1, keepdim=True))
        qm = rstd * (qm + n.abs() * (qm * n.abs()).mean(1, keepdim=True))
    out["dy"], m["dy"] = q, qm
    return out, m


def softmax_rows(logits):
    """(p, lse) by rows; a row of -inf alone has p = 0 and lse = 0."""
    l = logits.double()
    top = l.max(1, keepdim=True).values
    empty = torch.isneginf(top)
    top = torch.where(empty, torch.zeros_like(top), top)
    e = torch.exp(l - top)
    s = e.sum(1, keepdim=True)
    p = torch.where(empty, torch.zeros_like(e), e / torch.where(empty, torch.ones_like(s), s))
    lse = torch.where(empty, torch.zeros_like(s), top + torch.log(s))
    return p, lse


def balance(logits, ids, valid, group_of, k, coef):
    """(loss[4], probs, counts of Ne + 1) and what the gradient needs; group_of: each expert's
    group."""
    T, Ne = logits.shape
    rows = (torch.ones(T, dtype=torch.bool, device=logits.device) if valid is None
            else valid.bool())
    n = int(rows.sum())
    flat = ids[rows].flatten().long()
    flat = flat[(flat >= 0) & (flat < Ne)]
    cnt = torch.bincount(flat, minlength=Ne)
    counts = torch.cat([cnt, cnt.new_tensor([n])])
    Nd = int(group_of.max()) + 1
    zero = torch.zeros(Nd, dtype=torch.float64, device=logits.device)
    if n == 0:
        return torch.zeros(4, dtype=torch.float64), zero.new_zeros(Ne), counts, None
    p, lse = softmax_rows(logits[rows])
    probs = p.mean(0)
    f = cnt.double() * Ne / (k * n)
    members = zero.index_add(0, group_of, torch.ones(Ne, dtype=torch.float64, device=zero.device))
    F = zero.index_add(0, group_of, f) / members
    terms = torch.stack([coef[0] * (f * probs).sum(),
                         coef[1] * (F * zero.index_add(0, group_of, probs)).sum(),
                         coef[2] * (lse * lse).mean()])
    return torch.cat([terms.sum()[None], terms]), probs, counts, (rows, n, p, lse, f, F[group_of])


def balance_back(logits, kept, coef, dloss, dlogits_in):
    """(dlogits, magnitude behind it)."""
    out = (torch.zeros(logits.shape, dtype=torch.float64, device=logits.device)
           if dlogits_in is None else dlogits_in.double().clone())
    mag = out.abs()
    if kept is None:
        return out, mag
    rows, n, p, lse, f, F = kept
    c = coef[0] * f + coef[1] * F
    g = dloss / n * p * (c - (p * c).sum(1, keepdim=True) + 2 * coef[2] * lse)
    size = coef[0] * (f + 1) + coef[1] * (F + 1)
    gm = abs(dloss) / n * p * (size + (p * size).sum(1, keepdim=True) + 2 * coef[2] * lse.abs())
    out[rows] += g
    mag[rows] += gm
    return out, mag


def gate_back(dlogits, x, w_router, dx_in):
    """(dx, dw) and their magnitudes."""
    dl, w, xd = dlogits.double(), w_router.double(), x.double()
    dx, dxm = dl @ w, dl.abs() @ w.abs()
    if dx_in is not None:
        dx, dxm = dx + dx_in.double(), dxm + dx_in.double().abs()
    dlt = dl.t().contiguous()
    return dx, dxm, dlt @ xd, dlt.abs() @ xd.abs()


def adamw(p, g, m, v, a):
    """New (p, m, v) and the step taken, from fp64 values; a: the descriptor's fields."""
    g = g * a["grad_scale"]
    m = a["beta1"] * m + (1 - a["beta1"]) * g
    v = a["beta2"] * v + (1 - a["beta2"]) * g * g
    mh, vh = m / (1 - a["beta1"] ** a["step"]), v / (1 - a["beta2"] ** a["step"])
    step = a["lr"] * mh / (torch.sqrt(vh) + a["eps"])
    return p * (1 - a["lr"] * a["weight_decay"]) - step, m, v, step


def blocks(v, size=256):
    """v (1-D) in rows of `size`, zeros behind the last."""
    rows = torch.zeros(-(-v.numel() // size) * size, dtype=v.dtype, device=v.device)
    rows[:v.numel()] = v
    return rows.view(-1, size)


def quantise(v, keep_nonzero):
    """fp64 values as (e4m3 codes, fp32 units)."""
    rows = blocks(v)
    top = rows.abs().max(1).values
    unit = torch.where(top < 2.0 ** -100, torch.zeros_like(top), top / 448).float()
    safe = torch.where(unit > 0, unit.double(), torch.ones_like(top))[:, None]
    code = torch.where(unit[:, None] > 0, rows / safe, torch.zeros_like(rows)).clamp(-448, 448)
    if keep_nonzero:
        code = torch.where((rows > 0) & (unit[:, None] > 0), code.clamp(min=2.0 ** -9), code)
    return code.flatten()[:v.numel()].float().to(torch.float8_e4m3fn), unit


def dequantise(code, unit):
    return code.float().double() * unit.double().repeat_interleave(256)[:code.numel()]
