"""nvfp4_gated_backward has three kernels, for rows on 16 bytes, for rows off them and
for narrow ones: the same operations in the same order, so the same bits."""
import pytest
import torch

import w4a4_gemm_nvfp4_b200 as nv
from test_gpu_gated import random_checkpoint

pytestmark = pytest.mark.gpu


def at(M, cols, pitch, start):
    flat = torch.zeros(M * pitch + 16, dtype=torch.bfloat16, device="cuda")
    return flat.as_strided((M, cols), (pitch, 1), start)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("N", [8, 40, 64, 248, 256, 264, 1000])
def test_the_same_bits_at_any_alignment(act, N):
    M = max(8, 300000 // N)  # enough values to meet every rounding
    ck, _, _ = random_checkpoint(M, N, act, N)
    ck.scales.mul_(4)  # |g| to 30: open, closed and everything between
    dh = torch.randn(M, N, generator=torch.Generator().manual_seed(N)).to(torch.bfloat16).cuda()
    ref, href = nv.gated_backward(dh, ck, recompute=True)
    for pad, start in ((3, 0), (8, 1), (1, 5)):
        dv, out, h = at(M, N, N + pad, start), at(M, 2 * N, 2 * N + pad, start), at(M, N, N + pad, start)
        dv.copy_(dh)
        nv.gated_backward(dv, ck, out=out, h_out=h)
        assert torch.equal(out[:, :N], ref[:, :N]) and torch.equal(out[:, N:], ref[:, N:]) and torch.equal(h, href)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_a_column_does_not_depend_on_how_many_there_are(act):
    """The first columns of a wide matrix alone: 41 of 1001, in the narrow kernel."""
    M, N, n = 4000, 1001, 41
    ck, _, _ = random_checkpoint(M, N, act, 1)
    dh = torch.randn(M, N, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    ref, href = nv.gated_backward(dh, ck, recompute=True)
    part = nv.GatedCheckpoint(ck.codes[:, :, :64].contiguous(), ck.scales[:, :, :2].contiguous(), M, n, act)
    dgu, h = nv.gated_backward(dh[:, :n], part, recompute=True)
    assert torch.equal(dgu[:, :n], ref[:, :n]) and torch.equal(dgu[:, n:], ref[:, N:N + n]) and torch.equal(h, href[:, :n])
