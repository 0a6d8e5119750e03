"""Codebook calls on the GPU against their 64-bit definitions
(tests/codebook_ref.py, where the tolerances are derived)."""
import threading

import pytest
import torch

import distance_argmin_flashassign_b200 as fk
from tests import codebook_ref as ref
from tests.parity import TORCH_DT

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF, NAN = float("inf"), float("nan")
DTS = ["f32", "f16", "bf16"]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def labels(shape, K, seed, none=0.1, hot=0.0):
    """Labels below K, a share of them -1 and a share of them one label."""
    g = gen(seed)
    ids = torch.randint(0, K, shape, generator=g, dtype=torch.int32)
    ids[torch.rand(shape, generator=g) < hot] = K // 3
    ids[torch.rand(shape, generator=g) < none] = -1
    return ids


def offset(t, by):
    """t on the device, `by` elements behind an aligned address."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=DEV)
    v = buf[by:].view(t.shape)
    v.copy_(t)
    return v


def guarded(shape, dtype, by=0):
    """An output of `shape` between two guards, and a check that they still stand."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + 128 + by,), 77.0, dtype=dtype, device=DEV)

    def check():
        assert bool((buf[:64 + by] == 77).all()) and bool((buf[64 + by + n:] == 77).all())
    return buf[64 + by:64 + by + n].view(shape), check


# ------------------------------------------------------------------ lookup --
LOOK = [  # (B, N, K, D, offset of the pointers in elements)
    (1, 1, 7, 128, 0), (1, 1000, 50, 128, 0), (1, 333, 9, 1, 0), (1, 77, 30, 2, 0), (1, 129, 40, 100, 0), (1, 65, 20, 1002, 0),
    (1, 200, 30, 127, 0), (3, 257, 11, 64, 0), (5, 31, 4, 40, 0), (1, 100, 20, 128, 1), (1, 100, 20, 128, 2), (1, 40, 6, 16384, 0),
    (2, 10, 3, 5000, 0), (1, 50, (1 << 22) - 1, 1, 0), (1, 2, 1, 8, 0),
]


@pytest.mark.parametrize("out", DTS)
@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("case", LOOK, ids=lambda c: "x".join(map(str, c)))
def test_lookup(case, dt, out):
    B, N, K, D, by = case
    T = (torch.randn(B, K, D, generator=gen(D + K)) * 3).to(TORCH_DT[dt])
    ids = labels((B, N), K, N)
    scale = 1.7
    Y, check = guarded((B, N, D), TORCH_DT[out], by)
    if B == 1:
        fk.fk_lookup(offset(T, by)[0], ids[0].to(DEV), scale, Y=Y[0])
    else:
        fk.fk_lookup(offset(T, by), ids.to(DEV), scale, Y=Y)
    fk.fk_sync()
    check()
    want = ref.lookup(T, ids, float(torch.tensor(scale)))
    err = (Y.double().cpu() - want).abs()
    h, t = ref.half_step(TORCH_DT[out]), ref.tiny(TORCH_DT[out])
    # the scale rounded to fp32, the product, the rounding to the output
    assert bool((err <= 1.001 * ((2 * ref.U + h) * want.abs() + t)).all())
    assert bool((Y.cpu()[ids < 0] == 0).all())


def test_lookup_of_one_is_exact():
    """Scale 1 in the table's own type copies the rows bit for bit, NaN and infinities included."""
    T = torch.randn(20, 64, generator=gen(1)).bfloat16()
    T[3, 5], T[4, 6], T[5, 7] = NAN, INF, -INF
    ids = labels((500,), 20, 2)
    Y = fk.fk_lookup(T.to(DEV), ids.to(DEV)).cpu()
    want = torch.where((ids >= 0)[:, None], T[ids.clamp(min=0).long()], torch.zeros((), dtype=T.dtype))
    assert torch.equal(Y.view(torch.int16)[~want.isnan()], want.view(torch.int16)[~want.isnan()])
    assert torch.equal(Y.isnan(), want.isnan())


def test_lookup_beyond_32_bit_offsets():
    """Rows of Y past 2^31 elements, and of T past 2^31 elements."""
    N, K, D = (1 << 20) + 3, 300, 2056
    T = torch.randn(K, D, generator=gen(3)).bfloat16().to(DEV)
    ids = labels((N,), K, 4).to(DEV)
    Y = fk.fk_lookup(T, ids)
    for at in (0, N // 2, N - 5):
        i = ids[at:at + 5].long()
        want = torch.where((i >= 0)[:, None], T[i.clamp(min=0)], torch.zeros((), dtype=T.dtype, device=DEV))
        assert torch.equal(Y[at:at + 5], want)
    back = torch.arange(N - 100, N, device=DEV, dtype=torch.int32)
    assert torch.equal(fk.fk_lookup(Y, back), Y[N - 100:])


# ---------------------------------------------------------------- gradient --
GRAD = [  # (B, N, K, D, offset, share of hot labels)
    (1, 1, 7, 128, 0, 0.0), (1, 2, 1, 8, 0, 0.0), (1, 33, 5, 64, 0, 0.0), (1, 1000, 50, 128, 0, 0.3), (1, 5000, 3, 128, 0, 0.9),
    (1, 3000, 700, 100, 0, 0.2), (1, 2000, 900, 1002, 0, 0.5), (1, 700, 40, 127, 0, 0.1), (1, 999, 10, 1, 0, 0.3),
    (1, 20000, 3000, 32, 0, 0.4), (4, 4096, 100, 128, 0, 0.2), (32, 4096, 200, 16, 0, 0.2), (7, 513, 19, 72, 0, 0.1),
    (1, 800, 30, 128, 1, 0.2), (1, 800, 30, 128, 2, 0.2), (1, 300, 20, 16384, 0, 0.3), (1, 100000, 70000, 8, 0, 0.1),
    (3, 8192, 2100, 24, 0, 0.0), (1, 70001, 40, 256, 0, 0.5), (1, 300, (1 << 22) - 1, 2, 0, 0.1),
]


def _grad_case(case, dt, none=0.1):
    B, N, K, D, by, hot = case
    dY = torch.randn(B, N, D, generator=gen(N + D)).to(TORCH_DT[dt])
    return dY, labels((B, N), K, N + K, none=none, hot=hot)


def _call_grad(dY, ids, K, by, scale, dT, **kw):
    dY, ids = offset(dY, by), ids.to(DEV)
    if dY.shape[0] == 1:
        fk.fk_lookup_grad(dY[0], ids[0], K, scale, dT=dT[0], **kw)
    else:
        fk.fk_lookup_grad(dY, ids, K, scale, dT=dT, **kw)
    fk.fk_sync()


@pytest.mark.parametrize("out", DTS)
@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("case", GRAD, ids=lambda c: "x".join(map(str, c)))
def test_lookup_grad(case, dt, out):
    B, N, K, D, by, _ = case
    dY, ids = _grad_case(case, dt)
    scale = 0.25
    dT, check = guarded((B, K, D), TORCH_DT[out], by)
    _call_grad(dY, ids, K, by, scale, dT)
    check()
    g, mag, cnt = ref.lookup_grad(dY, ids, K, scale)
    err = (dT.cpu().double() - g).abs()
    assert bool((err <= ref.lookup_grad_tol(g, mag, cnt, TORCH_DT[out])).all())
    assert bool((dT.cpu()[cnt == 0] == 0).all())


@pytest.mark.parametrize("out", DTS)
@pytest.mark.parametrize("case", [GRAD[i] for i in (0, 3, 5, 7, 10, 13, 18)], ids=lambda c: "x".join(map(str, c)))
def test_lookup_grad_accumulates(case, out):
    """Added to what dT holds; rows that no label names keep their bits."""
    B, N, K, D, by, _ = case
    dY, ids = _grad_case(case, "bf16")
    dT, check = guarded((B, K, D), TORCH_DT[out], by)
    dT.copy_(torch.randn(B, K, D, generator=gen(5)) * 2)
    old = dT.cpu().clone()
    _call_grad(dY, ids, K, by, 1.5, dT, accumulate=True)
    check()
    g, mag, cnt = ref.lookup_grad(dY, ids, K, 1.5)
    err = (dT.cpu().double() - (g + old.double())).abs()
    assert bool((err <= ref.lookup_grad_tol(g, mag, cnt, TORCH_DT[out], old.double())).all())
    assert torch.equal(dT.cpu()[cnt == 0], old[cnt == 0])


@pytest.mark.parametrize("N", [1, 5, 1000, 9000, 70000])
@pytest.mark.parametrize("what", ["one label", "none", "all but one none", "one each", "descending"])
def test_lookup_grad_of_uneven_labels(N, what):
    K, D = N + 3, 64
    ids = {"one label": torch.full((N,), K - 1), "none": torch.full((N,), -1), "one each": torch.arange(N),
           "descending": torch.arange(N).flip(0) // 3,
           "all but one none": torch.where(torch.arange(N) == N // 2, 2, -1)}[what].int()[None]
    dY = torch.randn(1, N, D, generator=gen(N)).half()
    dT, check = guarded((1, K, D), torch.float32)
    _call_grad(dY, ids, K, 0, 1.0, dT)
    check()
    g, mag, cnt = ref.lookup_grad(dY, ids, K, 1.0)
    assert bool(((dT.cpu().double() - g).abs() <= ref.lookup_grad_tol(g, mag, cnt, torch.float32)).all())


def test_lookup_grad_leaves_rows_without_a_label_unread():
    """NaN and infinities in rows whose label is -1 reach no sum."""
    dY = torch.randn(600, 128, generator=gen(8)).bfloat16()
    ids = labels((600,), 9, 9, none=0.3)
    clean = fk.fk_lookup_grad(dY.to(DEV), ids.to(DEV), 9)
    dY[ids < 0] = NAN
    dY[(ids < 0) & (torch.arange(600) % 2 == 0)] = INF
    assert torch.equal(fk.fk_lookup_grad(dY.to(DEV), ids.to(DEV), 9), clean)
    dY[0, 3], ids[0] = NAN, 4  # one that counts does
    got = fk.fk_lookup_grad(dY.to(DEV), ids.to(DEV), 9)
    assert bool(got[4, 3].isnan()) and int(got.isnan().sum()) == 1


def test_lookup_grad_is_the_same_on_every_run():
    dY = torch.randn(200000, 128, generator=gen(10)).bfloat16().to(DEV)
    ids = labels((200000,), 1000, 11, hot=0.2).to(DEV)
    first = fk.fk_lookup_grad(dY, ids, 1000)
    for _ in range(3):
        assert torch.equal(fk.fk_lookup_grad(dY, ids, 1000), first)


def test_lookup_grad_against_differences():
    """Differences of the 64-bit lookup along rows of T (the lookup is linear:
    they are its gradient up to rounding)."""
    g = gen(12)
    T, V = torch.randn(1, 6, 24, generator=g, dtype=torch.float64), torch.randn(1, 6, 24, generator=g, dtype=torch.float64)
    ids = labels((1, 90), 6, 13)
    dY = torch.randn(1, 90, 24, generator=g)
    diff = ((ref.lookup(T + V, ids, 0.5) - ref.lookup(T - V, ids, 0.5)) * dY.double()).sum() / 2
    got = fk.fk_lookup_grad(dY[0].to(DEV), ids[0].to(DEV), 6, 0.5).double().cpu()
    _, mag, cnt = ref.lookup_grad(dY, ids, 6, 0.5)
    tol = ((cnt[0][:, None] + 3) * ref.U * mag[0] * V[0].abs()).sum() + 1e-10
    assert abs(float((got * V[0]).sum() - diff)) <= float(tol)


@pytest.mark.parametrize("bad", [16, -2, 1 << 30, -(1 << 31)])
def test_labels_out_of_range_are_reported(bad):
    """Each call treats such a label as -1 and reports it once."""
    T = torch.randn(16, 16, device=DEV)
    ids = torch.tensor([1, bad, 2, -1], dtype=torch.int32, device=DEV)
    none = torch.tensor([1, -1, 2, -1], dtype=torch.int32, device=DEV)
    for call in (lambda i: fk.fk_lookup(T, i), lambda i: fk.fk_lookup_grad(T[:4], i, 16), lambda i: fk.fk_balance(T[:4], i)[1]):
        out = call(ids)
        with pytest.raises(fk.FKError) as e:
            fk.fk_sync()
        assert e.value.status == fk.FK_ERR_BAD_LABEL
        assert torch.equal(out, call(none))
        fk.fk_sync()  # cleared, and -1 is no error


# ----------------------------------------------------------------- balance --
BAL = [  # (B, N, E, M, offset of Z)
    (1, 1, 8, 2, 0), (1, 300, 8, 2, 0), (1, 3, 1, 1, 0), (1, 100, 2, 1, 0), (1, 1000, 64, 2, 0), (4, 257, 64, 8, 0),
    (1, 500, 60, 4, 0), (1, 400, 515, 1, 0), (2, 300, 1024, 2, 0), (1, 200, 1032, 3, 0), (1, 77, 1025, 1, 0), (1, 130, 4096, 6, 0),
    (1, 64, 8192, 64, 0), (1, 33, 8191, 1, 0), (1, 900, 128, 2, 1), (3, 200, 256, 2, 3), (300, 17, 16, 1, 0), (1, 40000, 32, 4, 0),
    (1, 30000, 7, 1, 0), (1, 2500, 288, 2, 0),
    # rows of whole 4-byte pieces: 16-bit logits in pairs
    (1, 300, 258, 2, 0), (1, 90, 1026, 1, 0), (1, 40, 8190, 2, 0), (2, 200, 256, 2, 2), (1, 500, 34, 3, 2), (3, 64, 516, 1, 2),
    # rows of several warps, some of which have one row more than others, or none
    (1, 79, 1025, 1, 0), (1, 3, 2049, 1, 0), (1, 75, 2050, 2, 0), (2, 33, 4097, 1, 0), (1, 1200, 1280, 1, 0), (1, 700, 2560, 2, 0),
]


def _bal_case(case, dt, seed=0):
    B, N, E, M, by = case
    g = gen(N + E + seed)
    Z = torch.randn(B, N, E, generator=g) * 2 + torch.randn(E, generator=g)
    mask = torch.rand(B, N, generator=g) < 0.85
    if E > 4:
        Z[..., 1] = -INF                       # a column switched off
        Z[..., 2] = torch.finfo(TORCH_DT[dt]).min if dt != "f16" else -60000.0   # and one by a large negative number
    if N > 8:
        Z[:, 4] = -INF                         # a row that leaves nothing
        Z[:, 5] = torch.finfo(TORCH_DT[dt]).min   # a row of the lowest value: even
        Z[:, 6, 0] = -INF
    ids = torch.randint(-1, E, (B, N, M), generator=g, dtype=torch.int32)
    Z = Z.to(TORCH_DT[dt])
    Z[~mask] = NAN                             # rows left out are not looked at
    return Z, ids, mask


def _call_bal(Z, ids, mask, by, coef, **kw):
    Zd = offset(Z, by)
    md = None if mask is None else mask.to(DEV)
    ids = ids.to(DEV)
    if ids.shape[2] == 1:
        ids = ids[..., 0].contiguous()
    if Z.shape[0] == 1:
        out = fk.fk_balance(Zd[0], ids[0], mask=None if md is None else md[0], coef=coef, **kw)
        out = [o[None] for o in out]
    else:
        out = fk.fk_balance(Zd, ids, mask=md, coef=coef, **kw)
    fk.fk_sync()
    return Zd, dict(zip(("loss", "counts", "tokens", "meanp", "lse"), out))


def _clean(Z, mask):
    """Masked rows hold NaN; the reference takes them out before its arithmetic."""
    return Z if mask is None else torch.where(mask[..., None], Z, torch.zeros((), dtype=Z.dtype))


def _check_bal(out, Z, r):
    loss, P, lse = ref.balance_tol(Z, r)
    assert torch.equal(out["counts"].cpu(), r["counts"]) and torch.equal(out["tokens"].cpu(), r["tokens"])
    got = out["lse"].double().cpu()
    assert torch.equal(got == INF, ~r["on"])
    fin = r["on"]
    assert bool(((got - r["lse"]).abs()[fin] <= lse[fin]).all())
    assert bool(((out["meanp"].double().cpu() - r["meanp"]).abs() <= P).all())
    assert bool(((out["loss"].double().cpu() - r["loss"]).abs() <= loss).all())


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("case", BAL, ids=lambda c: "x".join(map(str, c)))
def test_balance_and_its_gradient(case, dt):
    B, N, E, M, by = case
    Z, ids, mask = _bal_case(case, dt)
    coef = 0.7
    Zd, out = _call_bal(Z, ids, mask, by, coef)
    Zc = _clean(Z, mask)
    r = ref.balance(Zc, ids, mask, coef)
    _check_bal(out, Zc, r)
    gl = torch.linspace(0.5, 300.0, B)
    dZ, check = guarded((B, N, E), TORCH_DT[dt], by)
    args = [out[k] for k in ("counts", "tokens", "lse")]
    if B == 1:
        fk.fk_balance_grad(Zd[0], *[a[0] for a in args], M, coef=coef, gloss=gl[0].to(DEV), dZ=dZ[0])
    else:
        fk.fk_balance_grad(Zd, *args, M, coef=coef, gloss=gl.to(DEV), dZ=dZ)
    fk.fk_sync()
    check()
    want = ref.balance_grad(r, gl, coef)
    err = (dZ.double().cpu() - want).abs()
    assert bool((err <= ref.balance_grad_tol(Zc, r, gl, coef, TORCH_DT[dt])).all())
    assert bool((dZ.cpu()[~r["on"]] == 0).all())
    # in place, the same bits
    if B == 1:
        fk.fk_balance_grad(Zd[0], *[a[0] for a in args], M, coef=coef, gloss=gl[0].to(DEV), dZ=Zd[0])
    else:
        fk.fk_balance_grad(Zd, *args, M, coef=coef, gloss=gl.to(DEV), dZ=Zd)
    assert torch.equal(Zd, dZ)


@pytest.mark.parametrize("dt", DTS)
def test_balance_where_no_row_takes_part(dt):
    for Z, mask in ((torch.randn(2, 40, 24), torch.zeros(2, 40, dtype=torch.bool)), (torch.full((2, 40, 24), -INF), None),
                    (torch.zeros(2, 0, 24), None)):
        Z = Z.to(TORCH_DT[dt])
        N = Z.shape[1]
        ids = torch.zeros(2, N, 1, dtype=torch.int32)
        Zd, out = _call_bal(Z, ids, mask, 0, 1.0)
        for k in ("loss", "counts", "tokens", "meanp"):
            assert bool((out[k] == 0).all())
        assert bool((out["lse"] == INF).all())
        dZ = fk.fk_balance_grad(Zd, out["counts"], out["tokens"], out["lse"], 1)
        assert bool((dZ == 0).all())


def test_balance_mask_types_and_optional_results():
    Z, ids, mask = _bal_case((1, 200, 16, 2, 0), "f32")
    _, a = _call_bal(Z, ids, mask, 0, 1.0)
    _, b = _call_bal(Z, ids, mask.to(torch.uint8) * 3, 0, 1.0)  # any value but 0 takes part
    for k in a:
        assert torch.equal(a[k], b[k])
    loss, counts, tokens = (torch.empty(n, dtype=t, device=DEV) for n, t in ((1, torch.float32), (16, torch.int32), (1, torch.int32)))
    Zd, idd, md = Z.to(DEV), ids.to(DEV), mask.to(DEV)
    st = fk.lib.fk_balance(Zd.data_ptr(), 1, 200, 16, fk.FK_F32, idd.data_ptr(), 2, md.data_ptr(), 1.0, loss.data_ptr(),
                           counts.data_ptr(), tokens.data_ptr(), None, None, None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == fk.FK_OK
    assert torch.equal(loss, a["loss"]) and torch.equal(counts[None], a["counts"]) and torch.equal(tokens, a["tokens"])


@pytest.mark.parametrize("E", [8, 64, 515, 2048])
@pytest.mark.parametrize("value", [NAN, INF])
def test_balance_nan_and_inf_follow_the_formula(E, value):
    """A NaN or +inf logit of a row that takes part makes its lse, the loss and
    every mean NaN, and its own row of dZ; other rows of dZ stay finite."""
    Z = torch.randn(50, E, generator=gen(E)).to(DEV)
    ids = torch.zeros(50, dtype=torch.int32, device=DEV)
    Z[7] = -INF
    Z[7, E // 2] = value
    loss, counts, tokens, meanp, lse = fk.fk_balance(Z, ids)
    assert int(tokens) == 50 and int(counts[0]) == 50
    assert bool(loss.isnan()) and bool(meanp.isnan().all())
    assert bool(lse[7].isnan()) and int(lse.isnan().sum()) == 1
    dZ = fk.fk_balance_grad(Z, counts, tokens, lse, 1)
    assert bool(dZ[7].isnan().any()) and bool(dZ[torch.arange(50) != 7].isfinite().all())


def test_balance_is_the_same_on_every_run():
    g = gen(21)
    Z = torch.randn(50000, 96, generator=g).bfloat16().to(DEV)
    ids = torch.randint(0, 96, (50000, 2), generator=g, dtype=torch.int32).to(DEV)
    first = fk.fk_balance(Z, ids)
    for _ in range(3):
        for a, b in zip(first, fk.fk_balance(Z, ids)):
            assert torch.equal(a, b)


def test_balance_beyond_32_bit_offsets():
    N, E = (1 << 20) + 1, 2056
    Z = torch.zeros(N, E, dtype=torch.bfloat16, device=DEV)
    Z[-1, 5] = 20.0
    ids = torch.zeros(N, dtype=torch.int32, device=DEV)
    loss, counts, tokens, meanp, lse = fk.fk_balance(Z, ids)
    assert int(counts[0]) == N and int(tokens) == N
    import math
    want = 20 + math.log1p((E - 1) * math.exp(-20))
    assert abs(float(lse[-1]) - want) < 1e-5 and abs(float(lse[0]) - math.log(E)) < 1e-5
    assert abs(float(loss) - E * float(meanp[0])) < 1e-5
    dZ = fk.fk_balance_grad(Z, counts, tokens, lse, 1, gloss=torch.tensor(float(N), device=DEV))
    # f = (1, 0, ...): dZ = E p_e ([e = 0] - p_0); the last row's p_0 = exp(-lse)
    p0 = math.exp(-want)
    assert abs(float(dZ[-1, 0]) - E * p0 * (1 - p0)) <= 2 ** -8 * E * p0 * 1.01
    assert abs(float(dZ[-2, 0]) - (1 - 1 / E)) <= 2 ** -8 * 1.01


# ------------------------------------------------- streams, graphs, threads --
def test_other_streams_and_pointers():
    """On a side stream the result is the same, ordered after that stream's
    work; a stream of no device of the tensors is refused."""
    dY = torch.randn(5000, 128, generator=gen(30)).bfloat16().to(DEV)
    ids = labels((5000,), 70, 31).to(DEV)
    want = fk.fk_lookup_grad(dY, ids, 70)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        late = torch.empty_like(dY)
        torch.cuda._sleep(20_000_000)
        late.copy_(dY)
    got = fk.fk_lookup_grad(late, ids, 70, stream=s)
    raw = fk.fk_lookup_grad(late, ids, 70, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(raw, want)


def test_captured_and_replayed():
    """Two graphs of all four calls, replayed in turn on new inputs, with eager
    calls between; each graph has a workspace of its own."""
    N, K, D, E = 6000, 90, 128, 64

    def inputs(seed):
        g = gen(seed)
        return [t.to(DEV) for t in (torch.randn(K, D, generator=g).bfloat16(), labels((N,), K, seed),
                                    torch.randn(N, E, generator=g).bfloat16(),
                                    torch.randint(-1, E, (N, 2), generator=g, dtype=torch.int32))]

    def step(T, ids, Z, ch):
        Y = fk.fk_lookup(T, ids, 2.0)
        dT = fk.fk_lookup_grad(Y, ids, K, 2.0)
        loss, counts, tokens, meanp, lse = fk.fk_balance(Z, ch, coef=0.1)
        return Y, dT, loss, counts, tokens, meanp, lse, fk.fk_balance_grad(Z, counts, tokens, lse, 2, coef=0.1)

    step(*inputs(1))
    torch.cuda.synchronize()
    graphs = []
    for seed in (2, 3):
        static = inputs(seed)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(*static)
        graphs.append((graph, static, out))
    for round_ in range(3):
        for i, (graph, static, out) in enumerate(graphs):
            new = inputs(100 + 10 * round_ + i)
            want = [t.clone() for t in step(*new)]
            for a, b in zip(static, new):
                a.copy_(b)
            graph.replay()
            fk.fk_lookup_grad(torch.zeros(200000, D, dtype=torch.bfloat16, device=DEV), labels((200000,), K, 7).to(DEV), K)
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_capture_without_a_workspace_is_refused_by_the_library():
    dY = torch.randn(500, 64, device=DEV)
    ids = labels((500,), 9, 1).to(DEV)
    dT = torch.zeros(9, 64, device=DEV)
    fk.fk_lookup_grad(dY, ids, 9, dT=dT)
    want = dT.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st = fk.lib.fk_lookup_grad(dY.data_ptr(), 1, 500, 64, fk.FK_F32, ids.data_ptr(), 9, 1.0, dT.data_ptr(), fk.FK_F32, 0,
                                   None, 0, torch.cuda.current_stream().cuda_stream)
        assert st == fk.FK_ERR_UNSUPPORTED
        assert "workspace" in fk.lib.fk_last_error_message().decode()
        dT.add_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dT, want + 1.0)


def test_workspace_argument():
    dY = torch.randn(3000, 64, device=DEV)
    ids = labels((3000,), 50, 1).to(DEV)
    need = fk.lib.fk_lookup_grad_workspace(1, 3000, 64, fk.FK_F32, 50)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    want = fk.fk_lookup_grad(dY, ids, 50)
    assert torch.equal(fk.fk_lookup_grad(dY, ids, 50, workspace=ws[:need]), want)
    assert bool((ws[need:] == 0x5A).all())
    for bad in (ws[:need - 1], ws[1:need + 1]):
        with pytest.raises(fk.FKError) as e:
            fk.fk_lookup_grad(dY, ids, 50, workspace=bad)
        assert e.value.status == fk.FK_ERR_INVALID_ARG
    Z = torch.randn(3000, 40, device=DEV)
    need = fk.lib.fk_balance_workspace(1, 3000, 40, fk.FK_F32)
    ch = labels((3000,), 40, 2).to(DEV)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    for a, b in zip(fk.fk_balance(Z, ch), fk.fk_balance(Z, ch, workspace=ws[:need])):
        assert torch.equal(a, b)
    assert bool((ws[need:] == 0x5A).all())
    with pytest.raises(fk.FKError):
        fk.fk_balance(Z, ch, workspace=ws[:need - 1])


def test_calls_from_several_threads():
    """Threads that share a stream, and so the library's scratch, and threads
    with streams of their own."""
    cases = []
    for i in range(4):
        dY = torch.randn(9000 + 1000 * i, 128, generator=gen(i)).bfloat16().to(DEV)
        ids = labels((dY.shape[0],), 300, i).to(DEV)
        cases.append((dY, ids, fk.fk_lookup_grad(dY, ids, 300)))
    torch.cuda.synchronize()
    bad = []

    def work(i, own):
        dY, ids, want = cases[i]
        s = torch.cuda.Stream() if own else None
        for _ in range(20):
            got = fk.fk_lookup_grad(dY, ids, 300, stream=s)
            torch.cuda.synchronize()
            if not torch.equal(got, want):
                bad.append(i)
    for own in (False, True):
        ts = [threading.Thread(target=work, args=(i, own)) for i in range(4)]
        [t.start() for t in ts]
        [t.join() for t in ts]
    assert not bad


def test_scratch_allocation_failure():
    dY = torch.randn(5000, 64, device=DEV)
    ids = labels((5000,), 30, 3).to(DEV)
    want = fk.fk_lookup_grad(dY, ids, 30)
    torch.cuda.synchronize()
    fk.fk_release_workspace()
    fk.fk_debug_inject(fk.FK_INJECT_SCRATCH_ALLOC)
    dT = torch.full((30, 64), 5.0, device=DEV)
    with pytest.raises(fk.FKError) as e:
        fk.fk_lookup_grad(dY, ids, 30, dT=dT)
    assert e.value.status == fk.FK_ERR_OOM
    assert bool((dT == 5).all())
    assert torch.equal(fk.fk_lookup_grad(dY, ids, 30), want)


# ----------------------------------------------------------- used together --
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_a_codebook_in_training(dt):
    """One step as a model makes it: points to their two nearest rows
    (fk_assign_top2), the nearest rows looked up, the gradient of
    0.5 |Y - X|^2 back to the codebook, and the balance loss of the two
    choices on the points' scores with its gradient -- each against its
    64-bit definition on what the step before gave."""
    N, K, D = 5000, 48, 64
    g = gen(40)
    C = torch.randn(K, D, generator=g).to(TORCH_DT[dt]).to(DEV)
    X = (C.cpu().float()[torch.randint(0, K, (N,), generator=g)] + 0.4 * torch.randn(N, D, generator=g)).to(TORCH_DT[dt]).to(DEV)
    l1, l2, _, _ = fk.fk_assign_top2(X, C)
    Y = fk.fk_lookup(C, l1)
    assert torch.equal(Y, C[l1.long()])
    R = (Y.float() - X.float()).to(TORCH_DT[dt])
    dC = fk.fk_lookup_grad(R, l1, K)
    gr, mag, cnt = ref.lookup_grad(R.cpu()[None], l1.cpu()[None], K, 1.0)
    assert bool(((dC.double().cpu()[None] - gr).abs() <= ref.lookup_grad_tol(gr, mag, cnt, torch.float32)).all())
    Z = (X.float() @ C.float().T - 0.5 * C.float().square().sum(1)).to(TORCH_DT[dt])
    ch = torch.stack([l1, l2], 1).contiguous()
    Zd, out = _call_bal(Z.cpu()[None], ch.cpu()[None], None, 0, 0.01)
    r = ref.balance(Z.cpu()[None], ch.cpu()[None], None, 0.01)
    _check_bal(out, Z.cpu()[None], r)
    dZ = fk.fk_balance_grad(Z, out["counts"][0], out["tokens"][0], out["lse"][0], 2, coef=0.01)
    want, one = ref.balance_grad(r, torch.ones(1), 0.01), torch.ones(1)
    assert bool(((dZ.double().cpu()[None] - want).abs() <= ref.balance_grad_tol(Z.cpu()[None], r, one, 0.01, TORCH_DT[dt])).all())


def test_the_gradient_sums_are_the_updates():
    """fk_update's means are fk_lookup_grad's sums over the counts: two orders of the same fp32 sums."""
    N, K, D = 30000, 64, 128
    X = torch.randn(N, D, generator=gen(50)).bfloat16().to(DEV)
    lab = labels((N,), K, 51, none=0.0).to(DEV)
    C = torch.zeros(K, D, device=DEV)
    counts = torch.empty(K, dtype=torch.int32, device=DEV)
    fk.fk_update(X, lab, C, counts)
    S = fk.fk_lookup_grad(X, lab, K)
    fk.fk_sync()
    _, mag, cnt = ref.lookup_grad(X.cpu()[None], lab.cpu()[None], K, 1.0)
    assert torch.equal(counts.cpu().double(), cnt[0])
    tol = 2 * (cnt[0] + 3)[:, None] * ref.U * mag[0]
    assert bool(((C.double() * counts[:, None]).cpu() - S.double().cpu()).abs().le(tol).all())


def test_as_many_problems_as_there_may_be():
    """B = 65,535 problems of a few rows each."""
    B, N, K, D = 65535, 3, 2, 4
    T = torch.randn(B, K, D, generator=gen(60)).half()
    ids = labels((B, N), K, 61)
    Y = fk.fk_lookup(T.to(DEV), ids.to(DEV))
    assert torch.equal(Y.cpu().double(), ref.lookup(T, ids, 1.0))
    dT = fk.fk_lookup_grad(Y, ids.to(DEV), K)
    g, mag, cnt = ref.lookup_grad(Y.cpu(), ids, K, 1.0)
    assert bool(((dT.cpu().double() - g).abs() <= ref.lookup_grad_tol(g, mag, cnt, torch.float32)).all())
    Z = torch.randn(B, N, 4, generator=gen(62))
    ch = torch.randint(-1, 4, (B, N, 2), generator=gen(63), dtype=torch.int32)
    Zd, out = _call_bal(Z, ch, None, 0, 1.0)
    r = ref.balance(Z, ch, None, 1.0)
    _check_bal(out, Z, r)
    dZ = fk.fk_balance_grad(Zd, out["counts"], out["tokens"], out["lse"], 2)
    one = torch.ones(B)
    err = (dZ.double().cpu() - ref.balance_grad(r, one, 1.0)).abs()
    assert bool((err <= ref.balance_grad_tol(Z, r, one, 1.0, torch.float32)).all())


@pytest.mark.parametrize("N", [32768, 32769, 100000])
def test_lookup_grad_either_side_of_the_one_launch_sort(N):
    """The same labels and rows, sorted by one cluster (up to 32,768 rows) and by
    the kernels for more: rows behind the first 32,768 carry no label."""
    K, D = 5000, 32
    dY = torch.randn(N, D, generator=gen(70)).half()
    ids = labels((N,), K, 71, hot=0.1)
    ids[32768:] = -1
    a = fk.fk_lookup_grad(dY.to(DEV), ids.to(DEV), K)
    b = fk.fk_lookup_grad(dY[:32768].to(DEV).contiguous(), ids[:32768].to(DEV).contiguous(), K)
    _, mag, cnt = ref.lookup_grad(dY[None], ids[None], K, 1.0)
    # two orders of the same sums
    assert bool(((a.double() - b.double()).abs().cpu() <= 2 * (cnt[0][:, None] + 2) * ref.U * mag[0]).all())


@pytest.mark.parametrize("K", [1, 2, 510, 511, 512, 262142, 262143, 262144, (1 << 22) - 1])
def test_lookup_grad_at_the_digits_edges(K):
    """Key counts around the sorts' digit and pass borders, the largest labels among them."""
    N, D = 3000, 2
    dY = torch.randn(N, D, generator=gen(80))
    ids = labels((N,), K, 81)
    ids[:3] = K - 1
    dT = fk.fk_lookup_grad(dY.to(DEV), ids.to(DEV), K).cpu()
    fk.fk_sync()
    g, mag, cnt = ref.lookup_grad(dY[None], ids[None], K, 1.0)
    assert bool(((dT.double() - g[0]).abs() <= ref.lookup_grad_tol(g, mag, cnt, torch.float32)[0]).all())


@pytest.mark.parametrize("E", [2, 8, 64, 515, 1024, 2050])
def test_balance_of_certain_choices(E):
    """One column switched on, or far ahead of the rest: its probability is 1, its
    lse its logit and the gradient nothing, to the rounding of 2^x at 0 (4 u), of
    the sum's logarithm and of lse itself (u each)."""
    N = 200
    z = torch.linspace(-90.0, 90.0, N)
    for rest in (-INF, -1e4, -1e9, -1e30, -3e38):
        Z = torch.full((N, E), rest)
        Z[:, E // 2] = z
        Zd, ids = Z.to(DEV), torch.full((N,), E // 2, dtype=torch.int32, device=DEV)
        loss, counts, tokens, meanp, lse = fk.fk_balance(Zd, ids)
        tol = 16 * ref.U + 2 * ref.U * z.abs()
        assert bool(((lse.cpu() - z).abs() <= tol).all())
        assert abs(float(meanp[E // 2]) - 1) <= 16 * ref.U and abs(float(loss) - E) <= E * 20 * ref.U
        dZ = fk.fk_balance_grad(Zd, counts, tokens, lse, 1, gloss=torch.tensor(float(N), device=DEV)).cpu()
        # E p (1 - p): p is off by the error of lse and 6 u
        assert bool((dZ.abs().amax(1) <= 1.1 * E * (tol + 6 * ref.U)).all())
