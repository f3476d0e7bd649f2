"""The checkpoint's scales of a row go through shared memory when a row's blocks are a
multiple of four (three warps hand theirs to a fourth) and straight to memory when they
are not.  The same products either way: the same scales, over many tiles of a CTA pair,
so that every slot is used again and again."""
import pytest
import torch

import w4a4_gemm_nvfp4_b200 as nv

pytestmark = pytest.mark.gpu


def operand(rows, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, K, generator=g, device="cuda") * torch.rand(rows, 1, generator=g, device="cuda") * 4
    return nv.quantize(x.to(torch.bfloat16))


def with_rows(q, rows):
    """The first rows of an operand (its scale atoms hold 128)."""
    codes, scales = q.codes[:rows].contiguous(), q.scales[:nv.nvfp4_scales_bytes(rows, q.K)].clone()
    return nv.NVFP4Tensor(codes, scales, q.global_scale, None, rows, q.K)


@pytest.mark.parametrize("shape", [(1300, 12800, 64), (2304, 16384, 64), (2113, 12928, 128), (1025, 16256, 320),
                                   (4096, 9600, 512)], ids=lambda s: "x".join(map(str, s)))
def test_both_ways_give_the_same_scales(shape):
    M, N, K = shape
    assert N % 128 == 0
    a, big_g, big_u = operand(M, K, 1), operand(N + 32, K, 2), operand(N + 32, K, 3)
    ref_h, ref = nv.gemm_gated(a, big_g, big_u, checkpoint=True)  # one block more: not a multiple of four
    wg, wu = with_rows(big_g, N), with_rows(big_u, N)
    ws = torch.zeros(64, dtype=torch.uint8, device="cuda")
    for i in range(20):
        h, ck = nv.gemm_gated(a, wg, wu, checkpoint=True, workspace=ws if i == 0 else None)
        assert i or nv.device_status(ws) == nv.OK
        assert torch.equal(ck.scales, ref.scales[:, :, :N // 32])
        assert torch.equal(ck.codes, ref.codes[:, :, :N]) and torch.equal(h, ref_h[:, :N])


def test_many_calls_back_to_back():
    """Each starts while the one before it ends; each leaves the barriers' state to
    nobody."""
    M, N, K = 520, 20480, 64
    a, wg, wu = operand(M, K, 4), operand(N, K, 5), operand(N, K, 6)
    _, ref = nv.gemm_gated(a, wg, wu, checkpoint=True)
    kept = [nv.gemm_gated(a, wg, wu, checkpoint=True)[1] for _ in range(30)]
    torch.cuda.synchronize()
    assert all(torch.equal(k.scales, ref.scales) and torch.equal(k.codes, ref.codes) for k in kept)


@pytest.mark.parametrize("shape", [(1300, 9600, 256), (1300, 9632, 64), (300, 2304, 256), (2048, 14336, 128)],
                         ids=lambda s: "x".join(map(str, s)))
def test_codes_and_scales_are_those_of_the_products(shape):
    """From the products as nvfp4_gemm writes them, bit for bit and in every kernel
    (small and wide tiles, outputs on and off 16 bytes): the scale rounded up, the code
    one rounding of the exact v * fl(1 / s)."""
    M, N, K = shape
    a, wg, wu = operand(M, K, 1), operand(N, K, 2), operand(N, K, 3)
    for pitch in (N, N + 1):
        _, ck = nv.gemm_gated(a, wg, wu, checkpoint=True,
                              out=torch.zeros(M, pitch, dtype=torch.bfloat16, device="cuda")[:, :N])
        for i, w in enumerate((wg, wu)):
            v = nv.gemm(a, w, out_dtype=torch.float32).view(M, N // 32, 32)
            t = (v.abs().amax(-1) / 127.0).clamp(min=2.0 ** -100)
            s = ((t.view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32)
            q = torch.round(v.double() * (1.0 / s).double()[..., None])
            assert torch.equal(ck.scales[i].float(), s)
            assert torch.equal(ck.codes[i][:, :N], q.view(M, N).to(torch.int8))
