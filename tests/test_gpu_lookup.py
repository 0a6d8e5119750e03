"""fk_lookup of rows of one to some lanes, many steps a warp: bit-equal to the fp32
product with one rounding."""
import pytest
import torch

import distance_argmin_flashassign_b200 as fk
from tests.parity import TORCH_DT

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 15, 16, 17, 24, 30, 32, 33, 48, 100])
def test_narrow_rows(D, dt, out):
    """From one row to several steps of every warp, of one problem and of three,
    with labels that name nothing, at aligned pointers and others."""
    g = torch.Generator(device=DEV).manual_seed(D)
    K, scale = 500, 0.7
    s32 = torch.tensor(scale, device=DEV)  # fp32
    for B, N, by in ((1, 1, 0), (1, 31, 0), (3, 257, 0), (1, 400003, 0), (1, 5000, 1), (2, 200001, 0)):
        T = torch.empty(B * K * D + by, device=DEV, dtype=TORCH_DT[dt])[by:].view(B, K, D)
        T.copy_(torch.randn(B, K, D, device=DEV, generator=g))
        ids = torch.randint(0, K, (B, N), device=DEV, generator=g, dtype=torch.int32)
        ids[torch.rand(B, N, device=DEV, generator=g) < 0.1] = -1
        buf = torch.full((B * N * D + by + 64,), 77.0, device=DEV, dtype=TORCH_DT[out])
        Y = buf[by:by + B * N * D].view(B, N, D)
        fk.fk_lookup(T, ids, scale, Y=Y)
        fk.fk_sync()
        rows = (T.float() * s32).to(TORCH_DT[out]).view(B * K, D)
        at = (ids.clamp(min=0) + K * torch.arange(B, device=DEV)[:, None]).view(-1).long()
        want = torch.where((ids.view(-1) >= 0)[:, None], rows[at], torch.zeros((), device=DEV, dtype=TORCH_DT[out]))
        assert torch.equal(Y.view(B * N, D), want)
        assert bool((buf[:by] == 77).all()) and bool((buf[by + B * N * D:] == 77).all())
