"""Codebook calls (fk_lookup, fk_lookup_grad, fk_balance, fk_balance_grad):
what they refuse, checked on the host without a GPU, and the formulas the GPU
tests hold them to, checked against differences."""
import ctypes

import pytest
import torch

import distance_argmin_flashassign_b200 as fk
from tests import codebook_ref as ref

P, Q = 4096, 8192  # addresses that are never read
INV, UNS = fk.FK_ERR_INVALID_ARG, fk.FK_ERR_UNSUPPORTED
NAN, INF = float("nan"), float("inf")


def _lookup(T=P, B=1, K=5, D=8, dt=1, ids=P, N=10, scale=1.0, Y=Q, dt_y=1):
    return fk.lib.fk_lookup(T, B, K, D, dt, ids, N, scale, Y, dt_y, None)


def _grad(dY=P, B=1, N=10, D=8, dt=1, ids=P, K=5, scale=1.0, dT=Q, dt_t=0, acc=0, ws=None, nws=0):
    return fk.lib.fk_lookup_grad(dY, B, N, D, dt, ids, K, scale, dT, dt_t, acc, ws, nws, None)


def _bal(Z=P, B=1, N=10, E=8, dt=1, ids=P, M=1, mask=None, coef=1.0, loss=Q, counts=Q, tokens=Q, meanp=None, lse=None):
    return fk.lib.fk_balance(Z, B, N, E, dt, ids, M, mask, coef, loss, counts, tokens, meanp, lse, None, 0, None)


def _bgrad(Z=P, B=1, N=10, E=8, dt=1, counts=P, tokens=P, lse=P, M=1, coef=1.0, gloss=None, dZ=Q):
    return fk.lib.fk_balance_grad(Z, B, N, E, dt, counts, tokens, lse, M, coef, gloss, dZ, None)


@pytest.mark.parametrize("kw,what", [
    (dict(B=0), "B"), (dict(B=65536), "B"), (dict(N=-1), "N"), (dict(N=1 << 31), "B*N"), (dict(B=2, N=1 << 30), "B*N"),
    (dict(D=0), "D"), (dict(D=16385), "D"), (dict(K=0), "K"), (dict(K=1 << 22), "B*K"), (dict(B=4, K=1 << 20), "B*K"),
    (dict(dt=3), "dtype"), (dict(scale=NAN), "scale"), (dict(scale=INF), "scale"),
], ids=str)
def test_lookup_and_its_gradient_refuse_bad_sizes(kw, what):
    for call in (_lookup, _grad):
        assert call(**kw) == INV
        assert what in fk.lib.fk_last_error_message().decode()
        assert fk.lib.fk_get_last_error() == INV


def test_lookup_refuses_bad_pointers_and_types():
    for kw in (dict(T=None), dict(ids=None), dict(Y=None), dict(dt_y=7)):
        assert _lookup(**kw) == INV
    for kw in (dict(dY=None), dict(ids=None), dict(dT=None), dict(dt_t=-1), dict(acc=2), dict(acc=-1)):
        assert _grad(**kw) == INV
    assert _lookup(N=0, T=None, ids=None, Y=None) == fk.FK_OK  # nothing to do, no device touched


@pytest.mark.parametrize("kw,what", [
    (dict(B=0), "B"), (dict(N=-1), "N"), (dict(N=1 << 31), "B*N"), (dict(E=0), "E"), (dict(E=8193), "E"), (dict(dt=9), "dtype"),
    (dict(M=0), "M"), (dict(M=65), "M"), (dict(N=1 << 26, M=32), "B*N*M"), (dict(coef=INF), "coef"),
    (dict(Z=None), "Z"), (dict(counts=None), "counts"), (dict(tokens=None), "tokens"),
], ids=str)
def test_balance_and_its_gradient_refuse_bad_arguments(kw, what):
    for call in (_bal, _bgrad):
        assert call(**kw) == INV
        assert what in fk.lib.fk_last_error_message().decode()


def test_balance_refuses_missing_arrays():
    assert _bal(ids=None) == INV and _bal(loss=None) == INV
    assert _bgrad(lse=None) == INV and _bgrad(dZ=None) == INV
    assert _bgrad(N=0) == fk.FK_OK


def test_workspace_sizes():
    n = fk.lib.fk_lookup_grad_workspace(1, 1000, 128, 1, 50)
    assert n > 0 and fk.lib.fk_lookup_grad_workspace(1, 100000, 128, 1, 50) > n
    assert fk.lib.fk_lookup_grad_workspace(1, 0, 128, 1, 50) == 0
    assert fk.lib.fk_lookup_grad_workspace(1, 10, 0, 1, 50) == INV
    assert fk.lib.fk_lookup_grad_workspace(1, 1 << 31, 8, 1, 50) == INV
    assert fk.lib.fk_balance_workspace(1, 1000, 64, 1) > 0
    assert fk.lib.fk_balance_workspace(1, 0, 64, 1) == 0
    assert fk.lib.fk_balance_workspace(1, 1000, 9000, 1) == INV
    # sizes beyond 32 bits
    assert fk.lib.fk_lookup_grad_workspace(1, (1 << 31) - 1, 64, 1, (1 << 22) - 1) > 4 * ((1 << 31) - 1)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
def test_no_device_is_an_error_not_a_crash():
    for st in (_lookup(), _grad(), _bal(), _bgrad()):
        assert st == fk.FK_ERR_CUDA
        assert fk.lib.fk_last_error_message()


def test_binding_refuses_what_the_library_cannot_see():
    T, ids = torch.zeros(5, 8), torch.zeros(10, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fk.fk_lookup(T, ids)
    with pytest.raises(ValueError, match="ids"):
        fk.fk_lookup(T, ids.long())
    with pytest.raises(ValueError, match="ids"):
        fk.fk_lookup(T, ids[::2])
    with pytest.raises(ValueError, match="T:"):
        fk.fk_lookup(T.t(), ids)
    with pytest.raises(TypeError):
        fk.fk_lookup(T.double(), ids)
    with pytest.raises(ValueError, match="ids"):
        fk.fk_lookup_grad(torch.zeros(9, 8), ids, 5)
    with pytest.raises(ValueError, match="accumulate"):
        fk.fk_lookup_grad(torch.zeros(10, 8), ids, 5, accumulate=True)
    Z = torch.zeros(10, 4)
    with pytest.raises(ValueError, match="ids"):
        fk.fk_balance(Z, ids[:9])
    with pytest.raises(ValueError, match="mask"):
        fk.fk_balance(Z, ids, mask=torch.ones(10))
    with pytest.raises(ValueError, match="Z"):
        fk.fk_balance(Z[:, ::2], ids)
    with pytest.raises(ValueError, match="CUDA"):
        fk.fk_balance(Z, ids)
    c, t, l = torch.zeros(4, dtype=torch.int32), torch.zeros((), dtype=torch.int32), torch.zeros(10)
    with pytest.raises(ValueError, match="lse"):
        fk.fk_balance_grad(Z, c, t, l[:9], 1)
    with pytest.raises(ValueError, match="gloss"):
        fk.fk_balance_grad(Z, c, t, l, 1, gloss=torch.zeros(2))


def test_balance_formula_against_differences():
    """dZ of the 64-bit formula against central differences of its loss, the
    counts held fixed (|second derivative| <= coef E, so the differences are
    good to h^2 and to 1e-16 / h)."""
    g = torch.Generator().manual_seed(1)
    Z = torch.randn(2, 9, 5, generator=g, dtype=torch.float64)
    ids = torch.randint(-1, 5, (2, 9, 2), generator=g, dtype=torch.int32)
    mask = torch.rand(2, 9, generator=g) < 0.8
    Z[0, 3, 1:4] = -INF
    gl = torch.tensor([2.0, -0.5])
    r = ref.balance(Z, ids, mask, 0.3)
    d = ref.balance_grad(r, gl, 0.3)
    h = 1e-5
    for at in [(0, 0, 0), (0, 3, 0), (0, 3, 2), (1, 8, 4), (1, 2, 3), (0, 7, 1)]:
        up, down = Z.clone(), Z.clone()
        up[at] += h
        down[at] -= h
        diff = (gl.double() * (ref.balance(up, ids, mask, 0.3)["loss"] - ref.balance(down, ids, mask, 0.3)["loss"])).sum() / (2 * h)
        assert abs(float(diff - d[at])) < 1e-8


def test_lookup_formula_is_its_gradients_adjoint():
    g = torch.Generator().manual_seed(2)
    T = torch.randn(2, 7, 3, generator=g, dtype=torch.float64)
    dY = torch.randn(2, 11, 3, generator=g, dtype=torch.float64)
    ids = torch.randint(-1, 7, (2, 11), generator=g, dtype=torch.int32)
    left = (ref.lookup(T, ids, 0.7) * dY).sum()
    right = (T * ref.lookup_grad(dY, ids, 7, 0.7)[0]).sum()
    assert abs(float(left - right)) < 1e-12
