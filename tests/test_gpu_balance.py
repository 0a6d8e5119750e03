"""fk_balance and fk_balance_grad through every kernel they are compiled to,
against the 64-bit definition with the bounds of tests/balance_bounds.py."""
import pytest
import torch

import distance_argmin_flashassign_b200 as fk
from tests import balance_bounds as bb
from tests.parity import TORCH_DT
from tests.test_gpu_codebook import BAL, _bal_case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF, NAN = float("inf"), float("nan")
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def logits(B, N, E, dt, seed):
    """Rows of a router with every kind of mask: columns switched off by -inf and
    by the type's lowest value, padded rows of NaN, rows that are -inf
    throughout, rows of one value (the lowest, fills of -1e4 and -1e9: even
    choices), rows that jump by hundreds and thousands."""
    t = TORCH_DT[dt]
    g = torch.Generator(device=DEV).manual_seed(seed)
    Z = torch.randn(B, N, E, device=DEV, generator=g) * 2 + torch.randn(E, device=DEV, generator=g)
    low = torch.finfo(t).min
    i = torch.arange(N, device=DEV)
    Z[:, i % 7 == 3] += 200.0
    Z[:, i % 7 == 5] -= 3000.0
    if E > 4:
        Z[..., E // 2] = -INF
        Z[..., E - 1] = low
    for at, value in ((4, -INF), (6, low), (8, -1e4), (10, max(low, -1e9))):
        Z[:, i % 16 == at] = value
    if E > 2:
        Z[:, i % 32 == 6, 1] = -INF  # even over the rest
    mask = torch.rand(B, N, device=DEV, generator=g) < 0.9
    if N < 8:
        mask[:, 0] = True
    ids = torch.randint(-1, E, (B, N, 1 + E % 3), device=DEV, generator=g, dtype=torch.int32)
    Z = Z.to(t)
    Z[~mask] = NAN
    return Z, ids, mask


def placed(t, by):
    """t `by` elements behind a 256-byte border."""
    v = torch.empty(t.numel() + by, dtype=t.dtype, device=DEV)[by:].view(t.shape)
    return v.copy_(t)


def check(Z, ids, mask, by, coef=0.7):
    """One forward and one backward call, each result within its bound."""
    B = Z.shape[0]
    Zd = placed(Z, by)
    out = dict(zip(("loss", "counts", "tokens", "meanp", "lse"), fk.fk_balance(Zd, ids, mask=mask, coef=coef)))
    fk.fk_sync()
    Zc = torch.where(mask[..., None], Z, torch.zeros_like(Z))  # rows left out are not looked at
    r = bb.balance(Zc, ids, mask, coef)
    loss, P, lse = bb.tol(r, coef)
    assert torch.equal(out["counts"], r["counts"]) and torch.equal(out["tokens"], r["tokens"])
    assert torch.equal(out["lse"] == INF, ~r["on"])
    at = r["on"]
    assert bool(((out["lse"].double() - r["lse"]).abs()[at] <= lse[at]).all())
    assert bool(((out["meanp"].double() - r["meanp"]).abs() <= P).all())
    assert bool(((out["loss"].double() - r["loss"]).abs() <= loss).all())
    gl = torch.linspace(0.5, 300.0, B, device=DEV)
    dZ = placed(torch.full_like(Z, 77.0), by)
    fk.fk_balance_grad(Zd, out["counts"], out["tokens"], out["lse"], ids.shape[2], coef=coef, gloss=gl, dZ=dZ)
    fk.fk_sync()
    want = bb.balance_grad(r, gl, coef)
    assert bool(((dZ.double() - want).abs() <= bb.grad_tol(r, gl, coef, Z.dtype)).all())
    assert bool((dZ[~at] == 0).all())


CASES = [(dt, s) for dt in SIZE for s in bb.spreads(SIZE[dt])]


@pytest.mark.parametrize("dt,s", CASES, ids=lambda v: v if isinstance(v, str) else "x".join(map(str, v)))
def test_every_spread_of_a_row(dt, s):
    """The fewest columns of each kernel and the most (16-byte packs) or some
    between: one block, a few of two problems, and all of the machine with
    several tiles an owner."""
    cols = bb.spreads(SIZE[dt])[s]
    rows, owners = bb.step_rows(s)
    for E in {cols[0], cols[-1] if s[0] * SIZE[dt] == 16 else cols[2 * len(cols) // 3]}:
        many = min(148 * 3 * owners * rows * 3 + 7, (1 << 23) // E)
        for B, N in ((1, 5), (2, 2 * rows * owners + 3), (1, many)):
            check(*logits(B, N, E, dt, E + N), s[0] if s[0] * SIZE[dt] < 16 else 0)


@pytest.mark.parametrize("E", [2, 8, 64, 515, 1024, 2050, 8192])
@pytest.mark.parametrize("dt", list(SIZE))
def test_gradient_of_rows_far_from_zero(dt, E):
    """Rows of one value far from 0, as masks leave them: lse, an fp32 number,
    does not resolve ln E there, and the choice is even all the same.  And
    rows of two values a step of the type apart."""
    low = torch.finfo(TORCH_DT[dt]).min
    values = [low, max(low, -1e30), max(low, -1e9), -6e4, -1e4, -512.0, 512.0, 6e4, -low]
    Z = torch.tensor(values, device=DEV).to(TORCH_DT[dt])[:, None].expand(-1, E).contiguous()[None]
    Z = torch.cat([Z, Z], 1)
    Z[:, len(values):, ::2] = (Z[:, len(values):, ::2].double() * (1 - torch.finfo(Z.dtype).eps)).to(Z.dtype)
    N = Z.shape[1]
    ids = torch.zeros(1, N, 1, dtype=torch.int32, device=DEV)
    ids[0, :5] = E - 1
    check(Z, ids, torch.ones(1, N, dtype=torch.bool, device=DEV), 0)


@pytest.mark.parametrize("dt", list(SIZE))
@pytest.mark.parametrize("case", BAL, ids=lambda c: "x".join(map(str, c)))
def test_cases_of_the_calls_own_tests(case, dt):
    """The cases of tests/test_gpu_codebook.py, whose bounds there grow with |z|,
    and so with the type's lowest value in one of their rows."""
    Z, ids, mask = _bal_case(case, dt)
    check(Z.to(DEV), ids.to(DEV), mask.to(DEV), case[4])


def _all_offset(E, N, M, by, dt):
    """Inputs whose arrays all start `by` elements behind a 256-byte border."""
    Z, _, mask = logits(1, N, E, dt, 7 * E + by)
    g = torch.Generator(device=DEV).manual_seed(by)
    ids = torch.randint(-1, E, (1, N, M), device=DEV, generator=g, dtype=torch.int32)
    return Z, placed(ids, by), placed(mask, by)


@pytest.mark.parametrize("by", [1, 3, 13])
@pytest.mark.parametrize("dt,E,N,M", [("f32", 3, 300000, 1), ("bf16", 1, 700000, 1), ("f16", 33, 100000, 3), ("bf16", 515, 30000, 2),
                                      ("f32", 1027, 3000, 1), ("f32", 5, 20, 3), ("bf16", 1, 1, 1), ("bf16", 2, 3, 1)])
def test_arrays_that_start_and_end_inside_16_bytes(dt, E, N, M, by):
    """The first and last bytes of each array, which no 16-byte piece of it
    covers, come to their places apart from the rest; the owner of the first
    rows then uses these places again.  Labels, mask, logits and lse alike,
    the same bits on every run."""
    Z, ids, mask = _all_offset(E, N, M, by, dt)
    check(Z, ids, mask, by)
    Zd, lse = placed(Z, by), placed(torch.zeros(1, N, device=DEV), by)
    first = None
    for _ in range(10):
        loss, counts, tokens, meanp, _ = fk.fk_balance(Zd, ids, mask=mask, lse=lse)
        out = [loss, counts, tokens, meanp, lse.clone(), fk.fk_balance_grad(Zd, counts, tokens, lse, M, dZ=placed(Zd, by))]
        if first is None:
            first = out
        assert all(torch.equal(a, b) for a, b in zip(out, first))
    # and the same from lse wherever it lies
    assert torch.equal(fk.fk_balance_grad(Zd, counts, tokens, lse.clone(), M, dZ=placed(Zd, by)), first[5])


def test_the_library_has_no_scratch_for_the_per_thread_stream():
    """cudaStreamPerThread is one handle for a stream of each thread: two threads'
    kernels would share scratch.  Refused on the host, nothing is written."""
    X, ids = torch.randn(100, 8, device=DEV), torch.zeros(100, dtype=torch.int32, device=DEV)
    out = [torch.full((8, 8), 7.0, device=DEV), torch.full((1,), 7.0, device=DEV), torch.full((8,), 7, dtype=torch.int32, device=DEV),
           torch.full((1,), 7, dtype=torch.int32, device=DEV)]
    dT, loss, counts, tokens = [t.data_ptr() for t in out]
    torch.cuda.synchronize()
    x, i, f32 = X.data_ptr(), ids.data_ptr(), fk.FK_F32
    for st in (fk.lib.fk_lookup_grad(x, 1, 100, 8, f32, i, 8, 1.0, dT, f32, 0, None, 0, 2),
               fk.lib.fk_balance(x, 1, 100, 8, f32, i, 1, None, 1.0, loss, counts, tokens, None, None, None, 0, 2)):
        assert st == fk.FK_ERR_UNSUPPORTED
        assert "cudaStreamPerThread" in fk.lib.fk_last_error_message().decode()
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in out)
