"""fk_lookup_grad with large tables, whose zero fill runs beside the one-launch sort
(up to 32,768 labels) or is a kernel of its own beside it, and captured calls
of more labels than that, against sums in 64 bits."""
import pytest
import torch

import distance_argmin_flashassign_b200 as fk
from tests import balance_bounds as bb
from tests.codebook_ref import U, half_step, tiny
from tests.parity import TORCH_DT

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(N, K, D, dt, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dY = torch.randn(N, D, device=DEV, generator=g).to(TORCH_DT[dt])
    ids = torch.randint(0, K, (N,), device=DEV, generator=g, dtype=torch.int32)
    ids[torch.rand(N, device=DEV, generator=g) < 0.2] = K // 3
    ids[torch.rand(N, device=DEV, generator=g) < 0.1] = -1
    ids[0], ids[-1] = K - 1, 0
    return dY, ids


def check(dT, dY, ids, scale=0.5):
    """n additions in any order, the scale, the rounding to the output type."""
    K, D = dT.shape
    at = torch.where(ids >= 0, ids.long(), K)
    y = dY.double() * scale
    s = torch.zeros(K + 1, D, dtype=torch.float64, device=DEV).index_add_(0, at, y)[:K]
    mag = torch.zeros(K + 1, D, dtype=torch.float64, device=DEV).index_add_(0, at, y.abs())[:K]
    n = torch.bincount(at, minlength=K + 1)[:K, None]
    e = (n + 2) * U * mag
    h, t = half_step(dT.dtype), tiny(dT.dtype)
    assert bool(((dT.double() - s).abs() <= 1.001 * (e + h * (s.abs() + e) + t + (n + 2) * tiny(torch.float32))).all())
    assert bool((dT[n[:, 0] == 0] == 0).all())


def table(K, D, dt, by):
    """A table of NaN `by` elements behind a 256-byte border, between two guards."""
    n = K * D
    buf = torch.full((n + 256 + by,), 77.0, dtype=TORCH_DT[dt], device=DEV)
    v = buf[128 + by:128 + by + n].view(K, D)
    v.fill_(float("nan"))

    def stands():
        assert bool((buf[:128 + by] == 77).all()) and bool((buf[128 + by + n:] == 77).all())
    return v, stands


# tables filled by blocks of the sort's own launch, and (over 2^26 bytes) by a kernel beside it
BIG = [("f32", 32768, 256, 0), ("f32", 32769, 256, 0), ("f32", 70000, 130, 0), ("f32", 70000, 130, 1), ("bf16", 140000, 130, 0),
       ("bf16", 140000, 130, 1), ("f16", 600001, 33, 1), ("bf16", 131072, 2048, 0), ("f32", 65536, 256, 0), ("f32", 65537, 256, 0),
       ("f32", 140000, 130, 1), ("bf16", 270000, 130, 0), ("bf16", 270000, 130, 1), ("f16", 1200001, 33, 3)]


@pytest.mark.parametrize("N", [1, 700, 32768])
@pytest.mark.parametrize("out,K,D,by", BIG)
def test_tables_filled_beside_the_sort(out, K, D, by, N):
    """Every element of a table of NaN is written, between guards that stand; calls
    follow one another on one stream with other labels and no wait between."""
    sets = [make(N, K, D, "bf16", 10 * K + i) for i in range(3)]
    outs = [table(K, D, out, by) for _ in sets]
    for _ in range(2):
        for (dY, ids), (dT, _) in zip(sets, outs):
            fk.fk_lookup_grad(dY, ids, K, 0.5, dT=dT)
    fk.fk_sync()
    for (dY, ids), (dT, stands) in zip(sets, outs):
        check(dT, dY, ids)
        stands()


@pytest.mark.parametrize("N,K,D", [(5000, 70000, 130), (32768, 300000, 64), (5000, 140001, 130), (40000, 9000, 64), (300000, 70000, 16), (100, 50, 64)])
def test_captured_on_new_labels(N, K, D):
    """The sort with its fill beside it, and the sort for more labels behind a
    memset, replayed on labels and rows that change, with work before and
    behind the call in the graph and the same bits as eager calls."""
    dY, ids = make(N, K, D, "bf16", 1)
    fk.fk_lookup_grad(dY, ids, K, 0.5)
    torch.cuda.synchronize()
    new = [make(N, K, D, "bf16", 20 + i) for i in range(3)]
    want = [fk.fk_lookup_grad(y, i, K, 0.5) for y, i in new]
    src_y, src_i = torch.zeros_like(dY), torch.full_like(ids, -1)
    graph = torch.cuda.CUDAGraph()
    dT = torch.empty(K, D, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        dT.fill_(float("nan"))
        dY.copy_(src_y)
        ids.copy_(src_i)
        fk.fk_lookup_grad(dY, ids, K, 0.5, dT=dT)
        copy = dT.clone()
        fk.fk_lookup_grad(dY, ids, K, 0.5, dT=dT, accumulate=True)
    for _ in range(2):
        for (y, i), w in zip(new, want):
            src_y.copy_(y)
            src_i.copy_(i)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(copy, w)
            assert torch.equal(dT, w + w)
            check(copy, y, i)


def test_autograd_does_not_see_the_calls():
    """Results do not require a gradient even where inputs do; the gradient calls
    give what autograd gives for the plain operations."""
    N, K, D, E, M = 400, 30, 24, 12, 2
    g = torch.Generator(device=DEV).manual_seed(9)
    T = torch.randn(K, D, device=DEV, generator=g, requires_grad=True)
    Z = torch.randn(N, E, device=DEV, generator=g, requires_grad=True)
    ids = torch.randint(0, K, (N,), device=DEV, generator=g, dtype=torch.int32)
    ch = torch.randint(0, E, (N, M), device=DEV, generator=g, dtype=torch.int32)
    dY = torch.randn(N, D, device=DEV, generator=g)
    Y = fk.fk_lookup(T, ids, 1.5)
    loss, counts, tokens, meanp, lse = fk.fk_balance(Z, ch, coef=0.3)
    assert not any(t.requires_grad for t in (Y, loss, meanp, lse))
    T64, Z64 = T.detach().double().requires_grad_(), Z.detach().double().requires_grad_()
    (T64[ids.long()] * 1.5 * dY.double()).sum().backward()
    f = counts.double() / (M * N)
    (0.3 * E * (f * torch.softmax(Z64, 1).mean(0)).sum()).backward()
    dT = fk.fk_lookup_grad(dY, ids, K, 1.5)
    n = torch.bincount(ids, minlength=K)[:, None]
    mag = torch.zeros(K, D, device=DEV, dtype=torch.float64).index_add_(0, ids.long(), 1.5 * dY.double().abs())
    assert bool(((dT.double() - T64.grad).abs() <= 1.01 * (n + 3) * U * mag).all())
    dZ = fk.fk_balance_grad(Z, counts, tokens, lse, M, coef=0.3)
    r = bb.balance(Z.detach()[None], ch[None], None, 0.3)
    t = bb.grad_tol(r, torch.ones(1, device=DEV), 0.3, torch.float32)[0]
    assert bool(((dZ.double() - Z64.grad).abs() <= t).all())
