"""The activation far from zero, in each kernel that computes it.

act(g) = g sigma(z).  In binary32 -z log2(e) is off by at most four roundings (its
constants, g^2, the cubic, the product), so the exponential by |z| 2^-22 and its own
2^-22, the sum by 2^-24, the reciprocal by 2^-23, the products with g and u by 2^-24
each: |z| 2^-22 + 2^-21 of the value together.  sigma below 2^-126 counts as 0: past z =
-126 ln(2) = -87.34 act is 0 where it is g e^z, off by less than |g| 2^-126, and act' is
0 where it is sigma (1 + g z' (1 - sigma)), off by less than (1 + |g| z') 2^-126.

The reference takes sigma as 1 / (1 + e^-z) in binary64: (1 + tanh(z / 2)) / 2 has no
digit left below 2^-53."""
import numpy as np
import pytest
import torch

import oracle
import w4a4_gemm_nvfp4_b200 as nv
from test_gpu_gated import zgrad
from test_gpu_gemv import HALF, upload

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -126
EDGE = 126 * np.log(2.0)


def z_of(g, act):
    return g if act == "silu" else np.sqrt(8 / np.pi) * (g + 0.044715 * g ** 3)


def sigma64(z):
    return 1 / (1 + np.exp(-np.clip(z, -700.0, 700.0)))


def check(h, g, u, act, half, closes=True):
    """h against act(g) u; where sigma is below 2^-126 it is 0."""
    z = z_of(g, act)
    ref = g * sigma64(z) * u
    tol = np.abs(ref) * (np.abs(np.maximum(z, -90.0)) * 2.0 ** -22 + 2.0 ** -21 + half) + np.where(
        z < -EDGE + 1e-4, np.abs(g * u) * TINY, 0.0)
    assert np.all(np.abs(h - ref) <= tol)
    closed = z < -EDGE - 1e-4
    assert np.all(h[closed] == 0) and closed.any() == closes and np.all(h[(z > -EDGE + 1e-4) & (g != 0)] != 0)


def gates(act):
    """bf16 gates whose z runs to -100 and beyond, the last binades closely."""
    far = np.linspace(-95, -80, 241) if act == "silu" else np.linspace(-10.8, -9.8, 129)
    g = np.concatenate([far, np.linspace(-80 if act == "silu" else -9.8, 95, 300), [-3e38, 3e30, 1e-30, -1e-30]])
    return torch.from_numpy(g).to(torch.bfloat16)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gemv_gated(act):
    g = gates(act)
    w = []
    for k in (0, 1):  # gate is column 0, up column 1
        codes = torch.zeros(3, 32, dtype=torch.uint8)
        codes[:, 0] = (0x02, 0x20)[k]
        w.append(nv.NVFP4Tensor(codes.cuda(), torch.full((nv.nvfp4_scales_bytes(3, 64),), 0x38, dtype=torch.uint8).cuda(),
                                torch.ones(1, device="cuda"), None, 3, 64))
    x = torch.zeros(len(g), 64, dtype=torch.bfloat16)
    x[:, 0] = g
    x[:, 1] = torch.where(g.abs() > 1e6, g * 0.5, torch.ones_like(g) * 1.5)  # (one scale holds both)
    h = torch.cat([nv.gemv_gated(r.cuda(), *w, act, out_dtype=torch.float32) for r in x.split(16)])
    sure = x[:, 0].abs() > 1e-20
    gd, ud = x[sure, 0].double().numpy(), x[sure, 1].double().numpy()
    hd = h[sure.cuda()].double().cpu().numpy()
    assert np.array_equal(hd[:, 0], hd[:, 1]) and np.array_equal(hd[:, 0], hd[:, 2])
    fits = np.abs(gd * ud) < 1e38
    check(hd[fits, 0], gd[fits], ud[fits], act, 0.0)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("N", [96, 160, 4800])
def test_gemm_gated(act, N):
    """Every product is one weight: gates from -96 to 96 (silu) or -12 to 12 in steps of
    the E2M1 grid times 16 scales, ups of 1.5."""
    M, K = 64, 64
    one = np.full((M, K // 16), 0x38, np.uint8)
    ca = np.zeros((M, K // 2), np.uint8)
    ca[:, 0] = 0x22  # A is 1 at k = 0 and k = 1
    cg, cu = np.zeros((N, K // 2), np.uint8), np.zeros((N, K // 2), np.uint8)
    n = np.arange(N)
    cg[:, 0] = n % 16          # weight of k = 0
    cu[:, 0] = 0x30            # 1.5 at k = 1
    sg = np.full((N, K // 16), 0x38, np.uint8)
    sg[:, 0] = 0x70 + (n // 16) % 9  # 128 .. 256
    og, ou = (cg, sg, 16 / 256 if act == "silu" else 2 / 256), (cu, np.full((N, K // 16), 0x38, np.uint8), 1.0)
    h = nv.gemm_gated(upload((ca, one, 1.0)), upload(og), upload(ou), act, out_dtype=torch.float32)
    g = oracle.dequantize(*og)[:, 0][None].repeat(M, 0)
    check(h.double().cpu().numpy(), g, np.full_like(g, 1.5), act, 0.0,
          closes=N > 128)  # (the largest of the scales)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("N", [128, 320, 321, 41])
def test_gated_backward(act, N):
    """Gates to -127 (silu) and -12.7, through the kernels of aligned, of unaligned and
    of narrow rows."""
    M = 6
    blocks = -(-N // 32)
    codes = torch.zeros(2, M, blocks * 32, dtype=torch.int8)
    r = torch.Generator().manual_seed(N)
    codes[0] = torch.randint(-127, 128, codes[0].shape, generator=r).to(torch.int8)
    codes[0, 0] = torch.arange(blocks * 32).remainder(40).sub(127).to(torch.int8)
    codes[1] = 3
    scales = torch.full((2, M, blocks), 0.5, dtype=torch.bfloat16)
    scales[0] = 1.0 if act == "silu" else 0.1
    dh = torch.full((M, N), 2.0, dtype=torch.bfloat16)
    dgu, h = nv.gated_backward(dh.cuda(), nv.GatedCheckpoint(codes.cuda(), scales.cuda(), M, N, act), recompute=True)
    g = (codes[0].double() * scales[0].double().repeat_interleave(32, 1))[:, :N].numpy()
    u = np.full_like(g, 1.5)
    z = z_of(g, act)
    s, zg = sigma64(z), zgrad(g, act)
    dg = 2.0 * u * s * (1 + g * sigma64(-z) * zg)
    half = HALF[torch.bfloat16] * (1 + 2.0 ** -6)
    got = dgu.double().cpu().numpy()
    check(h.double().cpu().numpy(), g, u, act, half)
    check(got[:, N:], g, np.full_like(g, 2.0), act, half)
    # of sigma's error; 1 - sigma is off by 2^-23 where sigma is near 1
    tol = 3.0 * (1 + np.abs(g) * zg) * (s * (np.abs(z) * 2.0 ** -22 + 2.0 ** -20) + TINY) + half * np.abs(dg)
    assert np.all(np.abs(got[:, :N] - dg) <= tol)
