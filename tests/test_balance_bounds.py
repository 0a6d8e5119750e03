"""The bounds that the balance kernels are held to (tests/balance_bounds.py),
checked on the host: they are tight, they reject wrong results, and their
definition agrees with the other one (tests/codebook_ref.py) and with
differences."""
import pytest
import torch

from tests import balance_bounds as bb
from tests import codebook_ref as ref
from tests.test_gpu_codebook import BAL, _bal_case, _clean

INF = float("inf")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", BAL, ids=lambda c: "x".join(map(str, c)))
def test_bounds_are_tight_and_reject_wrong_results(case, dt):
    if case[1] * case[2] > 1 << 20:
        case = (case[0], (1 << 20) // case[2]) + case[2:]
    Z, ids, mask = _bal_case(case, dt)
    coef, Z = 0.7, _clean(Z, mask)
    r = bb.balance(Z, ids, mask, coef)
    # the other definition, which takes exp(z - lse) and so needs |z| that 64 bits resolve
    near = torch.where((Z < -1e30).all(2, keepdim=True) & (Z > -INF).any(2, keepdim=True), torch.ones_like(Z), Z)
    new, old = bb.balance(near, ids, mask, coef), ref.balance(near, ids, mask, coef)
    for k in ("loss", "meanp", "lse"):
        assert torch.allclose(new[k], old[k], rtol=1e-11, atol=1e-14)
    assert torch.equal(new["counts"], old["counts"]) and torch.equal(new["tokens"], old["tokens"])
    loss, P, _ = bb.tol(r, coef)
    used = r["tokens"] > 0
    assert bool((loss <= 1e-3 * r["loss"] + 1e-30).all())
    assert bool((P <= 1e-3 * r["meanp"] + 1e-30).all())
    for wrong in (0.0, 0.99, 1.01):  # nothing written, one per cent off
        assert not bool(used.any()) or not bool((((r["meanp"] * wrong) - r["meanp"]).abs() <= P)[used].all())
        assert bool((((r["loss"] * wrong) - r["loss"]).abs() > loss)[r["loss"] > 0].all())
    # the gradient: within a few roundings of its type (and 1e-4 of the products it is a difference of)
    gl = torch.linspace(0.5, 300.0, case[0])
    g = bb.balance_grad(r, gl, coef)
    t = bb.grad_tol(r, gl, coef, Z.dtype)
    p, f = r["p"], r["f"][:, None, :]
    k = gl.double()[:, None, None] * coef * case[2] / r["tokens"].clamp(min=1)[:, None, None]
    tiny = torch.finfo(Z.dtype).smallest_normal * torch.finfo(Z.dtype).eps
    scale = k * p * (f + (f * p).sum(2, keepdim=True))
    h = torch.finfo(Z.dtype).eps / 2
    assert bool((t <= 1.1 * (1e-4 * scale + h * g.abs() + tiny) + 1e-30).all())


def test_gradient_of_a_row_far_from_zero_is_that_of_the_same_row_near_zero():
    """p depends on differences alone; a gradient made of exp(z - lse) with an lse
    rounded to fp32, as 1 in each column of a row of -1e9, is rejected."""
    Z = torch.tensor([-1e9, -3e38, 1e30, 0.0])[:, None].expand(-1, 8).contiguous()[None]
    ids = torch.tensor([0, 0, 0, 1], dtype=torch.int32)[None, :, None]
    r = bb.balance(Z, ids, None, 1.0)
    one = torch.ones(1)
    g, t = bb.balance_grad(r, one, 1.0), bb.grad_tol(r, one, 1.0, torch.float32)
    assert bool(((g - g[:, 3:]).abs() <= t).all())
    lse32 = r["lse"].float().double()
    r["p"] = torch.exp(Z.double() - lse32[..., None])
    bad = bb.balance_grad(r, one, 1.0)
    assert bool(((bad - g).abs() > t)[0, :3].all()) and bool(((bad - g).abs() <= t)[0, 3].all())


def test_spreads_cover_every_number_of_columns():
    for size in (2, 4):
        s = bb.spreads(size)
        assert len(s) == (51 if size == 2 else 38)
        for (VL, P, logg), cols in s.items():
            assert VL * P <= 32 and all((P << logg) * VL >= E for E in cols)
