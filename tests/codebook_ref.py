"""64-bit definitions of the codebook calls (lookup, its gradient, balance
loss, its gradient) for the tests, and the error bounds of the kernels.

u is half a step of fp32 relative to the value (2^-24), h(t) half a step of
the output type.  The bounds count roundings:

* lookup: one fp32 product (u), one rounding to the output (h);
* gradient sums of n rows: n additions in any order, then the scale and the
  addition to the old row: (n + 2) u of the sum of magnitudes, then h;
* exponentials: the argument (z - m) log2 e is an fp32 fused product with m
  log2 e rounded and log2 e itself rounded, so it is off by at most
  u (|m| + 3 |z - m|) log2 e; 2^x is good to 4 u.  With every finite |z| of a row
  at most R, |z - m| <= 2 R: a relative error of at most u (7 R + 4);
* a row's sum: at most 32 additions in a lane, 5 between lanes, 8 between
  warps, and the warps' factors (one more exponential): u (7 R + 4 + 45 + 8);
* a column sum: at most 1,024 rows in a lane, 5 between lanes, 8 between
  warps; blocks are added in fp64.
"""
import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Spacing of the subnormals (absolute rounding error near 0)."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def lookup(T, ids, scale):
    """T B x K x D, ids B x N (any label outside [0, K) names nothing)."""
    B, K, D = T.shape
    out = torch.zeros(ids.shape + (D,), dtype=torch.float64)
    for b in range(B):
        ok = (ids[b] >= 0) & (ids[b] < K)
        out[b, ok] = T[b].double()[ids[b][ok].long()] * scale
    return out


def lookup_grad(dY, ids, K, scale):
    """(the gradient, the sums of magnitudes, the counts), B x K (x D)."""
    B, N, D = dY.shape
    g = torch.zeros(B, K, D, dtype=torch.float64)
    mag = torch.zeros(B, K, D, dtype=torch.float64)
    cnt = torch.zeros(B, K, dtype=torch.float64)
    for b in range(B):
        ok = (ids[b] >= 0) & (ids[b] < K)
        i, y = ids[b][ok].long(), dY[b][ok].double()
        g[b].index_add_(0, i, y * scale)
        mag[b].index_add_(0, i, (y * scale).abs())
        cnt[b].index_add_(0, i, torch.ones(len(i), dtype=torch.float64))
    return g, mag, cnt


def lookup_grad_tol(g, mag, cnt, out, old=None):
    m = mag if old is None else mag + old.abs()
    v = g if old is None else g + old
    e = (cnt[..., None] + 2) * U * m
    return 1.001 * (e + half_step(out) * (v.abs() + e) + tiny(out) + tiny(torch.float32) * (cnt[..., None] + 2))


def balance(Z, ids, mask, coef):
    """Z B x N x E, ids B x N x M, mask B x N or None; everything in fp64."""
    B, N, E = Z.shape
    M = ids.shape[2]
    z = Z.double()
    on = ~(z == -float("inf")).all(dim=2)
    if mask is not None:
        on &= mask.bool()
    zz = torch.where(on[..., None], z, torch.zeros((), dtype=torch.float64))
    lse = torch.logsumexp(zz, dim=2)
    p = torch.where(on[..., None], torch.exp(zz - lse[..., None]), torch.zeros((), dtype=torch.float64))
    n = on.sum(1)
    P = p.sum(1) / n.clamp(min=1)[:, None]
    counts = torch.zeros(B, E, dtype=torch.int32)
    for b in range(B):
        c = ids[b][on[b]].reshape(-1).long()
        c = c[(c >= 0) & (c < E)]
        counts[b] = torch.bincount(c, minlength=E).int()
    f = counts.double() / (M * n.clamp(min=1))[:, None]
    loss = coef * E * (f * P).sum(1)
    lse = torch.where(on, lse, torch.full((), float("inf"), dtype=torch.float64))
    return {"loss": loss, "counts": counts, "tokens": n.int(), "meanp": P, "lse": lse, "p": p, "f": f, "on": on}


def balance_grad(r, gloss, coef):
    """dZ from balance()'s result r; gloss B."""
    p, f = r["p"], r["f"][:, None, :]
    E = p.shape[2]
    k = gloss.double() * coef * E / r["tokens"].clamp(min=1)
    return k[:, None, None] * p * (f - (f * p).sum(2, keepdim=True))


def row_range(Z):
    """R: the largest finite |z| of each row (0 where there is none) among the
    logits within 110 of the row's largest; exp of the others is below 2^-126 and
    counts as 0 on both sides but for the flush that balance_tol adds."""
    z = Z.double()
    top = torch.where(torch.isfinite(z), z, torch.full((), -float("inf"), dtype=torch.float64)).amax(2, keepdim=True)
    near = torch.isfinite(z) & (z >= top - 110)
    return torch.where(near, z.abs(), torch.zeros((), dtype=torch.float64)).amax(2)


def balance_tol(Z, r):
    """Bounds of (loss, meanp, lse) of the kernel against balance()'s r."""
    R = row_range(Z)
    s = U * (14 * R + 70)  # relative error of a row's probabilities: two exponentials, the sum, the quotient
    worst = s.amax(1)[:, None]
    rel = worst + (1024 + 13 + 4) * U
    n = r["tokens"].clamp(min=1)[:, None].double()
    P = rel * r["meanp"] + 2 * U * r["meanp"] + 2.0 ** -126 * 2  # results below 2^-126 are flushed
    loss = (rel[:, 0] + 4 * U) * r["loss"].abs() + 1e-37 + 0 * n[:, 0]
    lse = s + U * (3 * R + 8) + 4 * U * torch.where(torch.isfinite(r["lse"]), r["lse"], torch.zeros((), dtype=torch.float64)).abs()
    return 1.01 * loss, 1.01 * P, 1.01 * lse


def balance_grad_tol(Z, r, gloss, coef, dtype):
    p, f = r["p"], r["f"][:, None, :]
    E = p.shape[2]
    k = (gloss.double() * coef * E / r["tokens"].clamp(min=1)).abs()[:, None, None]
    # lse is an fp32 value (its own error, balance_tol, moves every p of the row), then z - lse, the product
    # with log2 e, 2^x
    e = (U * (24 * row_range(Z) + 120))[..., None]
    dot = (f * p).sum(2, keepdim=True)
    g = k * p * (f - dot)
    err = k * p * ((e + 6 * U) * (f - dot).abs() + (e + 50 * U) * dot + 3 * U * f)
    return 1.01 * (err + half_step(dtype) * (g.abs() + err) + tiny(dtype) + k * 2.0 ** -126 * 2)
