"""The codebook operators as they are measured: inputs, plain forms, work.

Four operators around a codebook (or embedding table) T of K rows and the
labels that name its rows:

* ``lookup``        Y[i] = scale * T[ids[i]]                       (fk_lookup)
* ``lookup_grad``   dT[k] = scale * sum of dY[i] over ids[i] = k   (fk_lookup_grad)
* ``balance``       the balance loss of N rows of E logits with M chosen
                    columns each, per-column counts, mean
                    probabilities and row log-sum-exps             (fk_balance)
* ``balance_grad``  its gradient with respect to the logits        (fk_balance_grad)

``run`` computes them with elementary torch operations, or, where ``own`` is
true, through the library's calls.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one new token in serving: the smallest call, latency alone
        {"name": "lookup one token", "op": "lookup", "B": 1, "N": 1, "D": 1024, "K": 65536, "dt": "bf16", "out": "bf16",
         "ids": "uniform", "pad": 0.0},
        # the embedding workload's points replaced by their centroids (vector quantisation)
        {"name": "lookup embed", "op": "lookup", "B": 1, "N": 1 << 20, "D": 128, "K": 1024, "dt": "f16", "out": "f16",
         "ids": "uniform", "pad": 0.0},
        # a ragged padded batch of rows that are no whole number of 16 bytes, fp32 master table, bf16 activations
        {"name": "lookup ragged", "op": "lookup", "B": 1, "N": 50001, "D": 1002, "K": 32001, "dt": "f32", "out": "bf16",
         "ids": "zipf", "pad": 0.11},
        # a small training batch: few tokens, a wide row each
        {"name": "grad small batch", "op": "lookup_grad", "B": 1, "N": 500, "D": 1024, "K": 8192, "dt": "bf16",
         "out": "f32", "ids": "zipf", "pad": 0.05},
        # the batched token-clustering workload: 32 codebooks of 256 rows
        {"name": "grad batched", "op": "lookup_grad", "B": 32, "N": 32768, "D": 128, "K": 256, "dt": "bf16",
         "out": "f32", "ids": "uniform", "pad": 0.0},
        # the Zipf workload's codebook: 65,536 rows, a fifth of the tokens on one of them
        {"name": "grad zipf", "op": "lookup_grad", "B": 1, "N": 1 << 21, "D": 128, "K": 65536, "dt": "bf16",
         "out": "f32", "ids": "zipf", "pad": 0.0},
        # a language-model batch: a large vocabulary, most of whose rows no token names
        {"name": "grad vocabulary", "op": "lookup_grad", "B": 1, "N": 16384, "D": 2048, "K": 131072, "dt": "bf16",
         "out": "bf16", "ids": "zipf", "pad": 0.02},
        # a router over a few experts on one short sequence
        {"name": "balance short", "op": "balance", "B": 1, "N": 300, "E": 8, "M": 2, "dt": "f32", "pad": 0.0, "off": 0},
        # a router over 64 experts, two chosen, padded sequences, three experts switched off by -inf logits
        {"name": "balance router", "op": "balance", "B": 16, "N": 32768, "E": 64, "M": 2, "dt": "bf16", "pad": 0.13,
         "off": 3},
        # use of a 1,024-row codebook by the embedding workload's points, one label each
        {"name": "balance codes", "op": "balance", "B": 1, "N": 262144, "E": 1024, "M": 1, "dt": "f16", "pad": 0.0,
         "off": 0},
        # the router's backward pass
        {"name": "balance_grad router", "op": "balance_grad", "B": 16, "N": 32768, "E": 64, "M": 2, "dt": "bf16",
         "pad": 0.13, "off": 3},
        # the backward pass in fp32, an odd number of columns
        {"name": "balance_grad odd", "op": "balance_grad", "B": 1, "N": 100003, "E": 515, "M": 4, "dt": "f32",
         "pad": 0.02, "off": 0},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, uniform in its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["lookup", "lookup_grad", "balance", "balance_grad"])
    dt = rng.choice(["f32", "f16", "bf16"])
    B = rng.choice([1, 1, 1, _log(rng, 2, 32)])
    pad = rng.choice([0.0, round(rng.uniform(0.0, 0.4), 3)])
    if op.startswith("lookup"):
        D = _log(rng, 8, 4096)
        if rng.random() < 0.6:  # mostly whole 16-byte rows, as models have them
            D = max(8, D // 8 * 8)
        K = max(1, min(_log(rng, 16, 131072), (1 << 26) // (B * D)))
        N = max(1, min(_log(rng, 1, 1 << 20), (1 << 26) // D) // B)
        return {"op": op, "B": B, "N": N, "D": D, "K": K, "dt": dt,
                "out": rng.choice([dt, dt, "f32", "bf16"]), "ids": rng.choice(["uniform", "zipf"]), "pad": pad}
    E = _log(rng, 2, 4096)
    if rng.random() < 0.6 and E > 8:
        E = E // 8 * 8
    M = rng.choice([1, 1, 2, 4, 8])
    N = max(1, min(_log(rng, 16, 1 << 19), (1 << 26) // E) // B)
    return {"op": op, "B": B, "N": N, "E": E, "M": min(M, E), "dt": dt, "pad": pad,
            "off": rng.choice([0, min(3, E - 1)])}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ids(g, case, n, k):
    """n labels below k, uniform or with Zipf(1.2) masses; a `pad` share of them -1 (no row)."""
    if case.get("ids", "uniform") == "zipf":
        mass = torch.arange(1, k + 1, device="cuda", dtype=torch.float64) ** -1.2
        cdf = torch.cumsum(mass, 0) / mass.sum()
        u = torch.rand(n, device="cuda", dtype=torch.float64, generator=g)
        ids = torch.searchsorted(cdf, u).clamp_(max=k - 1).int()
    else:
        ids = torch.randint(0, k, (n,), device="cuda", dtype=torch.int32, generator=g)
    if case["pad"]:
        ids[torch.rand(n, device="cuda", generator=g) < case["pad"]] = -1
    return ids


def prepare(case, seed):
    g = _gen(seed)
    B, N, dt = case["B"], case["N"], DT[case["dt"]]
    s = dict(case)
    if case["op"].startswith("lookup"):
        D, K = case["D"], case["K"]
        s["scale"] = math.sqrt(D) if case["op"] == "lookup" else 1.0 / math.sqrt(D)
        s["labels"] = _ids(g, case, B * N, K).view(B, N) if B > 1 else _ids(g, case, N, K)
        rows, key = (K, "T") if case["op"] == "lookup" else (N, "dY")
        shape = (B, rows, D) if B > 1 else (rows, D)
        s[key] = torch.empty(shape, dtype=dt, device="cuda")
        flat, step = s[key].view(-1), 1 << 26
        for i in range(0, flat.numel(), step):
            n = min(step, flat.numel() - i)
            flat[i:i + n] = torch.randn(n, device="cuda", generator=g) * 0.02
        return s
    E, M = case["E"], case["M"]
    lead = (B, N) if B > 1 else (N,)
    # logits of a router that already prefers some columns
    Z = torch.randn(lead + (E,), device="cuda", generator=g) * 1.5
    Z += torch.randn(E, device="cuda", generator=g)
    if case["off"]:
        Z[..., torch.randperm(E, device="cuda", generator=g)[:case["off"]]] = -math.inf
    s["Z"] = Z.to(dt)
    # the chosen columns: the M largest logits (M may exceed the columns that are switched on)
    ids = torch.topk(Z, M, dim=-1).indices.int()
    if M > 1:  # some second choices dropped, as by a capacity limit
        drop = torch.rand(lead, device="cuda", generator=g) < 0.03
        ids[..., M - 1][drop] = -1
    s["labels"] = ids if M > 1 else ids[..., 0].contiguous()
    s["mask"] = None
    if case["pad"]:
        # sequences of different lengths in a padded batch
        length = (torch.rand(B, 1, device="cuda", generator=g) * 2 * case["pad"] * N).long()
        s["mask"] = (torch.arange(N, device="cuda")[None, :] < N - length).view(lead)
    s["coef"] = 0.01
    if case["op"] == "balance_grad":
        f = _balance(s["Z"], s["labels"], s["mask"], B, N, E, M, 0.01)
        s["counts"], s["tokens"], s["lse"] = f["counts"], f["tokens"], f["lse"]
        # the loss's own gradient: a loss scale, as fp16 training uses
        s["gloss"] = torch.full((B,) if B > 1 else (), 65536.0, device="cuda")
    return s


# ------------------------------------------------------------- plain forms --
def _flat_ids(labels, B, N, K):
    """Row numbers in the B*K rows of the batch, and which labels name one."""
    ids = labels.long().view(B, -1)
    ok = (ids >= 0).view(-1)
    ids = (ids.clamp(min=0) + torch.arange(B, device=ids.device)[:, None] * K).view(-1)
    return ids, ok


def _lookup(T, labels, B, N, D, K, scale, out):
    ids, ok = _flat_ids(labels, B, N, K)
    rows = T.view(B * K, D)[ids].float() * scale
    rows = torch.where(ok[:, None], rows, torch.zeros((), device=rows.device))
    return rows.to(out).view(labels.shape + (D,))


def _lookup_grad(dY, labels, B, N, D, K, scale, out):
    ids, ok = _flat_ids(labels, B, N, K)
    ids = torch.where(ok, ids, torch.full_like(ids, B * K))
    # long sums (a hot row takes a fifth of the tokens): in 64 bits
    acc = torch.zeros(B * K + 1, D, dtype=torch.float64, device=dY.device)
    acc.index_add_(0, ids, dY.view(B * N, D).double())
    return (acc[:B * K] * scale).to(out).view(dY.shape[:-2] + (K, D))


def _balance(Z, labels, mask, B, N, E, M, coef):
    z = Z.float().view(B, N, E)
    m = z.max(dim=2).values
    on = m > -math.inf
    if mask is not None:
        on = on & mask.view(B, N)
    m = torch.where(on, m, torch.zeros((), device=z.device))
    e = torch.exp(z - m[:, :, None])
    s = e.sum(dim=2)
    p = torch.where(on[:, :, None], e / s[:, :, None], torch.zeros((), device=z.device))
    lse = torch.where(on, m + torch.log(s), torch.full((), math.inf, device=z.device))
    tokens = on.sum(dim=1)
    used = tokens.clamp(min=1).double()
    meanp = p.sum(dim=1, dtype=torch.float64) / used[:, None]
    ids, ok = _flat_ids(labels, B, N, E)
    ok = ok & on.view(B * N, 1).expand(B * N, M).reshape(-1)
    counts = torch.zeros(B * E, dtype=torch.int32, device=z.device)
    counts.index_add_(0, ids, ok.int())
    counts = counts.view(B, E)
    f = counts.double() / (M * used)[:, None]
    loss = coef * E * (f * meanp).sum(dim=1)
    lead = Z.shape[:-2]
    return {"loss": loss.float().view(lead), "counts": counts.view(lead + (E,)), "tokens": tokens.int().view(lead),
            "meanp": meanp.float().view(lead + (E,)), "lse": lse.view(lead + (N,))}


def _balance_grad(Z, counts, tokens, lse, gloss, B, N, E, M, coef):
    z, l = Z.float().view(B, N, E), lse.view(B, N, 1)
    on = l < math.inf
    p = torch.where(on, torch.exp(z - torch.where(on, l, torch.zeros((), device=z.device))),
                    torch.zeros((), device=z.device))
    used = tokens.view(B, 1).clamp(min=1).double()
    f = (counts.view(B, E).double() / (M * used)).float()[:, None, :]
    k = (gloss.view(B, 1).double() * coef * E / used).float()[:, :, None]
    return (k * p * (f - (f * p).sum(dim=2, keepdim=True))).to(Z.dtype).view(Z.shape)


def run(state):
    s = state
    B, N = s["B"], s["N"]
    if s["op"] == "lookup":
        if own:
            import distance_argmin_flashassign_b200 as fk
            return fk.fk_lookup(s["T"], s["labels"], s["scale"], dtype=DT[s["out"]])
        return _lookup(s["T"], s["labels"], B, N, s["D"], s["K"], s["scale"], DT[s["out"]])
    if s["op"] == "lookup_grad":
        if own:
            import distance_argmin_flashassign_b200 as fk
            return fk.fk_lookup_grad(s["dY"], s["labels"], s["K"], s["scale"], dtype=DT[s["out"]])
        return _lookup_grad(s["dY"], s["labels"], B, N, s["D"], s["K"], s["scale"], DT[s["out"]])
    E, M, coef = s["E"], s["M"], s["coef"]
    if s["op"] == "balance":
        if own:
            import distance_argmin_flashassign_b200 as fk
            loss, counts, tokens, meanp, lse = fk.fk_balance(s["Z"], s["labels"], mask=s["mask"], coef=coef)
            return {"loss": loss, "counts": counts, "tokens": tokens, "meanp": meanp, "lse": lse}
        return _balance(s["Z"], s["labels"], s["mask"], B, N, E, M, coef)
    if own:
        import distance_argmin_flashassign_b200 as fk
        return fk.fk_balance_grad(s["Z"], s["counts"], s["tokens"], s["lse"], M, coef=coef, gloss=s["gloss"])
    return _balance_grad(s["Z"], s["counts"], s["tokens"], s["lse"], s["gloss"], B, N, E, M, coef)


def work(case):
    B, N, b = case["B"], case["N"], BYTES[case["dt"]]
    if case["op"] == "lookup":
        D = case["D"]
        rows = B * min(N, case["K"])
        return {"bytes": 4 * B * N + rows * D * b + B * N * D * BYTES[case["out"]], "flops": B * N * D}
    if case["op"] == "lookup_grad":
        D = case["D"]
        return {"bytes": 4 * B * N + B * N * D * b + B * case["K"] * D * BYTES[case["out"]], "flops": B * N * D}
    E, M = case["E"], case["M"]
    n = B * N
    if case["op"] == "balance":
        return {"bytes": n * E * b + 4 * n * M + (n if case["pad"] else 0) + 4 * n + 8 * B * E + 8 * B,
                "flops": 5 * n * E}
    return {"bytes": 2 * n * E * b + 4 * n + 4 * B * E + 8 * B, "flops": 6 * n * E}


# ------------------------------------------------------- from the definition --
def exact(case, seed):
    s = prepare(case, seed)
    B, N = case["B"], case["N"]
    if case["op"] == "lookup":
        D, K = case["D"], case["K"]
        T, labels = s["T"].view(B, K, D), s["labels"].view(B, N).long()
        out = torch.zeros(B, N, D, dtype=torch.float64, device="cuda")
        for b in range(B):
            at = torch.nonzero(labels[b] >= 0)[:, 0]
            out[b, at] = T[b].index_select(0, labels[b, at]).double() * s["scale"]
        return out.view(s["labels"].shape + (D,))
    if case["op"] == "lookup_grad":
        D, K = case["D"], case["K"]
        dY, labels = s["dY"].view(B, N, D), s["labels"].view(B, N).long()
        out = torch.zeros(B, K, D, dtype=torch.float64, device="cuda")
        for b in range(B):  # running sums of the rows in label order, and their differences at each label's ends
            lab, order = torch.sort(labels[b], stable=True)
            ends = torch.searchsorted(lab, torch.arange(-1, K, device="cuda"), right=True)
            for c in range(0, D, 256):
                run_ = torch.zeros(N + 1, min(256, D - c), dtype=torch.float64, device="cuda")
                torch.cumsum(dY[b, :, c:c + 256][order].double(), 0, out=run_[1:])
                out[b, :, c:c + 256] = (run_[ends[1:]] - run_[ends[:-1]]) * s["scale"]
        return out.view(s["dY"].shape[:-2] + (K, D))
    E, M = case["E"], case["M"]
    Z, ids = s["Z"].view(B, N, E), s["labels"].view(B, N, M).long()
    mask = None if s["mask"] is None else s["mask"].view(B, N)
    if case["op"] == "balance":
        out = {k: [] for k in ("loss", "counts", "tokens", "meanp", "lse")}
        for b in range(B):
            z = Z[b].double()
            lse = torch.logsumexp(z, dim=1)
            on = (lse > -math.inf) if mask is None else (lse > -math.inf) & mask[b]
            n = int(on.sum())
            P = torch.exp(z[on] - lse[on][:, None]).sum(0) / max(n, 1)
            chosen = ids[b][on].reshape(-1)
            c = torch.bincount(chosen[chosen >= 0], minlength=E)
            out["loss"].append(s["coef"] * E * torch.dot(c.double() / (M * max(n, 1)), P))
            out["counts"].append(c.int())
            out["tokens"].append(torch.tensor(n, dtype=torch.int32, device="cuda"))
            out["meanp"].append(P)
            out["lse"].append(torch.where(on, lse, torch.full_like(lse, math.inf)))
        lead = s["Z"].shape[:-2]
        return {k: torch.stack(v).view(lead + v[0].shape) for k, v in out.items()}
    dZ = torch.zeros(B, N, E, dtype=torch.float64, device="cuda")
    counts, tokens, lse = s["counts"].view(B, E), s["tokens"].view(B), s["lse"].view(B, N).double()
    for b in range(B):
        n = max(int(tokens[b]), 1)
        f = counts[b].double() / (M * n)
        on = torch.nonzero(torch.isfinite(lse[b]))[:, 0]
        p = torch.exp(Z[b, on].double() - lse[b, on, None])
        dZ[b, on] = float(s["gloss"].view(-1)[b]) * s["coef"] * E / n * p * (f[None, :] - (p @ f)[:, None])
    return dZ.view(s["Z"].shape)
