"""Error bounds of fk_balance and fk_balance_grad row by row, the 64-bit
definition on any device, and the kernels' spreads of a row (which compiled
kernel a number of columns and an alignment reach).

u is half a step of fp32 relative to the value (2^-24).  For a row with maximum
m let d_e = m - z_e and D = sum_e p_e d_e.  The kernels never work on z itself
but on differences, so the bounds hold at any magnitude of the logits.

Forward, p_e = 2^t w q / sum with t = (z_e - own) log2 e of a lane's own
maximum, w = 2^((own - m) log2 e) and, for rows of several warps, q = 2^((m_w - m)
log2 e).  The three arguments' magnitudes add up to d_e log2 e.  Each is off by
a rounded difference, a rounded constant and a rounded product (3 u relative),
which 2^x turns into 3 u d_e ln 2 log2 e = 3 u d_e; each 2^x is good to 4 u (12
in all), their products and the quotient take 8 u.  The sum is off by the
p-weighted mean of those, 3 u D + 20 u, and by its own additions: 32 in a lane,
5 between lanes, 8 between warps.  So a probability is off by
u (3 d_e + 3 D + 100) relative to itself, and lse by u (3 D + 70), by 2 u
|lse - m| <= 20 u of the logarithm and u |lse| of its last addition.
A column mean adds min(N, 1024) rows in a lane, 5 between lanes, 8 between
owners (blocks are added in fp64), then rounds once.
Results below 2^-126 are flushed on the way: an absolute 2^-120.

Backward, p_e = 2^((z_e - lse) log2 e), with the row normalised again where
|lse| > 64.  Nearer 0 the error of lse counts, u (3 D + 90 + 64); else the sum's
counts, u (3 D + 100).  |z_e - lse| <= d_e + 30 (ln E, and the rounding of a far
lse, which is no larger than that or leaves lse = m).  So p is off by
u (3 d_e + 3 D + 300).  k f takes 8 roundings, the dot product 45 additions.
"""
import torch

U = 2.0 ** -24
INF = float("inf")


def balance(Z, ids, mask, coef):
    """The definition in fp64: Z B x N x E, ids B x N x M, mask B x N or None."""
    B, N, E = Z.shape
    M = ids.shape[2]
    z = Z.double()
    on = ~(z == -INF).all(dim=2)
    if mask is not None:
        on &= mask != 0
    z = torch.where(on[..., None], z, torch.zeros_like(z))
    m = z.amax(2)
    lse = m + torch.log(torch.exp(z - m[..., None]).sum(2))
    p = torch.exp(z - m[..., None])
    p = torch.where(on[..., None], p / p.sum(2, keepdim=True), torch.zeros_like(z))
    n = on.sum(1)
    P = p.sum(1) / n.clamp(min=1)[:, None]
    ok = (ids >= 0) & (ids < E) & on[..., None]
    flat = torch.where(ok, ids.long() + E * torch.arange(B, device=Z.device)[:, None, None], B * E)
    counts = torch.bincount(flat.reshape(-1), minlength=B * E + 1)[:B * E].view(B, E)
    f = counts.double() / (M * n.clamp(min=1))[:, None]
    d = torch.where(torch.isfinite(z) & on[..., None], m[..., None] - z, torch.zeros_like(z))
    d = torch.where(p > 0, d, torch.zeros_like(z))
    return {"loss": coef * E * (f * P).sum(1), "counts": counts.int(), "tokens": n.int(), "meanp": P,
            "lse": torch.where(on, lse, torch.full_like(lse, INF)), "p": p, "f": f, "on": on, "d": d,
            "D": (p * d).sum(2, keepdim=True)}


def balance_grad(r, gloss, coef):
    p, f = r["p"], r["f"][:, None, :]
    k = gloss.double() * coef * p.shape[2] / r["tokens"].clamp(min=1)
    return k[:, None, None] * p * (f - (f * p).sum(2, keepdim=True))


def tol(r, coef):
    """Absolute bounds of (loss, meanp, lse)."""
    p, N, E = r["p"], r["p"].shape[1], r["p"].shape[2]
    n = r["tokens"].clamp(min=1)[:, None].double()
    rel = U * (3 * r["d"] + 3 * r["D"] + 100)
    P = (p * rel).sum(1) / n + U * (min(N, 1024) + 20) * r["meanp"] + 2.0 ** -120
    loss = coef * E * (r["f"] * P).sum(1) + 8 * U * r["loss"].abs() + 2.0 ** -120
    lse = U * (3 * r["D"][..., 0] + 90 + torch.where(r["on"], r["lse"].abs(), torch.zeros_like(r["lse"])))
    return 1.01 * loss, 1.01 * P, 1.01 * lse


def grad_tol(r, gloss, coef, dtype):
    p, f = r["p"], r["f"][:, None, :]
    k = (gloss.double() * coef * p.shape[2] / r["tokens"].clamp(min=1)).abs()[:, None, None]
    rel = U * (3 * r["d"] + 3 * r["D"] + 300)
    dot = (f * p).sum(2, keepdim=True)
    errdot = (f * p * (rel + 60 * U)).sum(2, keepdim=True)
    g = k * p * (f - dot)
    err = k * p * ((f - dot).abs() * (rel + 10 * U) + errdot + 10 * U * f + 4 * U * dot)
    h = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    return 1.01 * (err + h * (g.abs() + err) + tiny + k * 2.0 ** -120)


def spread(E, size, aligned):
    """(columns of a pack, packs of a lane, log2 of the lanes of a team) for rows
    of E logits of `size` bytes at pointers of `aligned` bytes; a lane holds at
    most 32 columns, a warp's about 16."""
    row = E * size
    unit = 16 if row % 16 == 0 and aligned % 16 == 0 else 4 if row % 4 == 0 and aligned % 4 == 0 else 2
    VL = max(1, unit // size)
    packs = -(-E // VL)
    wide = packs > 32 * (32 // VL)
    logg, per = (6, 32 // VL) if wide else (0, 16 // VL)
    while (wide or logg < 5) and per << logg < packs:
        logg += 1
    P = 1
    while P << logg < packs:
        P += P if P < 8 else 8 if wide else 4
    return VL, P, logg


def spreads(size):
    """Every spread of a type of `size` bytes, {spread: its numbers of columns},
    at pointers aligned to its packs and no further."""
    out = {}
    for aligned in (16, 4) if size == 4 else (16, 4, 2):
        for E in range(1, 8193):
            s = spread(E, size, aligned)
            if s[0] * size == aligned:
                out.setdefault(s, []).append(E)
    return out


def step_rows(s):
    """(rows of an owner's step, owners of a block) of a spread: from 64 lanes on a
    team has several warps and a row, else a warp's teams have one or two each."""
    VL, P, logg = s
    lanes = max(32, 1 << logg)
    return (lanes >> logg) * (2 if VL * P <= 16 else 1), 256 // lanes
