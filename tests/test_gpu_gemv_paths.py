"""Every way in which nvfp4_gemv and nvfp4_gemv_gated split a call: one CTA or a
cluster of 2, 4 or 8 for a row tile, x staged whole or in pieces, one or two column
tiles of tokens, four or two units of weights in flight, one wave of CTAs or more.

The reference is the product in binary64 of the same operands, decoded here.

Bound.  A unit is 256 k of a row tile: at most 16 tensor-core additions from zero,
each off by at most 2^-22 of the magnitudes that it adds, so 16 * 2^-22 of the unit's
sum |x w|, and of the whole sum over all units.  What follows is rounded to nearest
in binary32, half a step (2^-24 of a partial sum, and so of sum |x w|) each: a warp
joins at most one unit per step of a piece, the 16 warps' partials are added, then
the pieces, then the CTAs of a cluster; a unit's two chains and the tensor scale are
two more.  Together (16 * 2^-22 + J * 2^-24) sum |x w| with J = steps of a piece + 16
+ pieces + CTAs + 2.  The result is rounded once to its type.  On sums of small whole
numbers nothing rounds at all."""
import numpy as np
import pytest
import torch

import w4a4_gemm_nvfp4_b200 as nv
from test_gpu_gemv import HALF, gate64, gated_tolerance

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]

# (weights, M, N, K)
SHAPES = [
    # one CTA for a row tile: x whole, four and two units in flight; several waves
    (1, 3, 300, 512), (1, 8, 600, 4096), (1, 16, 600, 2048), (2, 5, 100, 256), (2, 16, 600, 1536),
    (2, 16, 100000, 512),
    # x in pieces
    (1, 12, 1184, 10240), (1, 16, 40000, 4096), (1, 16, 151936, 4096), (2, 12, 9600, 8192), (2, 16, 12288, 8192),
    (1, 8, 60000, 12288), (2, 8, 60000, 8192),
    # clusters of two
    (1, 8, 600, 6144), (1, 8, 600, 8192), (2, 16, 600, 2560), (2, 16, 2500, 5120), (2, 8, 600, 4608),
    (1, 8, 600, 16384), (1, 16, 5120, 17408), (1, 2, 600, 65536), (2, 2, 600, 65536), (2, 16, 14336, 8192),
    (2, 8, 600, 16384),
    # of four
    (1, 8, 300, 2048), (1, 16, 300, 8192), (1, 16, 300, 65536), (2, 2, 300, 131072), (2, 16, 300, 4608),
    (2, 16, 300, 16384), (2, 9, 23, 1088),
    # of eight
    (1, 8, 16, 2048), (1, 16, 16, 16384), (1, 16, 40, 131072), (1, 8, 16, 65536), (2, 8, 16, 32768), (2, 16, 40, 131072),
    (2, 9, 30, 2112),
]
SIZES = [pytest.param(s, id=("gated " if s[0] == 2 else "") + "x".join(map(str, s[1:]))) for s in SHAPES]


def path(plan, weights, M, sms):
    return weights, 1 if M <= 8 else 2, plan["ranks"], plan["pieces"] > 1, plan["depth"], plan["grid"] > sms


def test_the_sizes_take_every_path():
    """Every form of the kernel that a call on 148 SMs can take, by weights, column
    tiles of tokens, CTAs for a row tile, pieces of x and units in flight."""
    sms = 148
    taken = {path(nv.testing_gemv_plan(M, N, K, w, sms), w, M, sms) for w, M, N, K in SHAPES}
    for w in (1, 2):
        for ranks in (1, 2, 4, 8):
            for pieces in (False, True):
                assert any(t[0] == w and t[2:4] == (ranks, pieces) for t in taken), (w, ranks, pieces)
                assert any(t[1] == 1 and t[2:4] == (ranks, pieces) for t in taken), (ranks, pieces)
                assert any(t[1] == 2 and t[2:4] == (ranks, pieces) for t in taken), (ranks, pieces)
            assert {d for t in taken for d in [t[4]] if t[0] == w and t[2] == ranks} == {2, 4}, (w, ranks)
        assert any(t[0] == w and t[5] for t in taken)


def test_plan_refuses_what_the_call_refuses():
    for bad in ((0, 64, 64), (17, 64, 64), (1, 0, 64), (1, 64, 96), (1, 64, 0), (1, (1 << 30) + 1, 64)):
        with pytest.raises(ValueError):
            nv.testing_gemv_plan(*bad)


def bound(M, N, K, weights, sms=148):
    p = nv.testing_gemv_plan(M, N, K, weights, sms)
    joins = p["piece_steps"] + 16 + p["pieces"] + p["ranks"] + 2
    return 16 * 2.0 ** -22 + joins * 2.0 ** -24


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[2] * s[3] < 1 << 24][:24], ids=str)
def test_the_bound_sees_what_a_wrong_path_would_lose(shape):
    """A sum without one unit of 256 k, or without one MMA of 16 k, is off by more
    than the bound in most outputs, the largest K included.  Of `width` normal
    products the loss has deviation sqrt(width), and sum |x w| is 2 K / pi: an output
    hides it with P(|z| < bound * 2 K / (pi sqrt(width))), at K = 131072, where the
    bound is 6.4e-6, 3 % for 256 k and 11 % for 16."""
    w, M, N, K = shape
    N = min(N, 64)
    g = torch.Generator().manual_seed(K + N)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).double()
    dense = torch.randn(N, K, generator=g).double()
    tol = bound(*shape[1:], w) * (x.abs() @ dense.abs().T)
    for width, share in ((min(256, K), 0.9), (16, 0.75)):
        at = (K // width // 2) * width
        lost = x[:, at:at + width] @ dense[:, at:at + width].T
        assert float((lost.abs() > tol).double().mean()) > share, width


def random_weight(N, K, seed, whole):
    """(operand on the GPU, its rows in binary64 without the tensor scale by a function
    of a range): any codes; any finite scales, or all ones.  Scales of rows past N
    are NaN: no result may depend on them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if whole:
        scales = torch.full((N, K // 16), 0x38, device="cuda", dtype=torch.uint8)
    else:
        scales = torch.randint(0, 0x7F, (N, K // 16), generator=g, device="cuda", dtype=torch.uint8)
    padded = torch.full(((N + 127) // 128 * 128, K // 16), 0x7F, device="cuda", dtype=torch.uint8)
    padded[:N] = scales
    swizzled = padded.view(-1, 4, 32, K // 64, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    op = nv.NVFP4Tensor(codes, swizzled, torch.ones(1, device="cuda"), None, N, K)
    values = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64, device="cuda")

    def rows(lo, hi):
        c = codes[lo:hi].int()
        v = torch.stack([values[c & 15], values[c >> 4]], -1).view(hi - lo, K // 16, 16)
        return (v * scales[lo:hi].view(torch.float8_e4m3fn).double()[..., None]).view(hi - lo, K)

    return op, rows


def product(x, op, rows):
    """x W^T with the tensor scale, and sum |x w|, in binary64."""
    N, K = op.rows, op.K
    xd = x.double()
    y, guard = (torch.empty(x.shape[0], N, dtype=torch.float64, device="cuda") for _ in range(2))
    step = max(1, (1 << 26) // K)
    for lo in range(0, N, step):
        w = rows(lo, min(N, lo + step))
        y[:, lo:lo + step] = xd @ w.T
        guard[:, lo:lo + step] = xd.abs() @ w.abs().T
    alpha = float(op.global_scale)
    return y * alpha, guard * abs(alpha)


def close(got, ref, tol):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist())


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SIZES)
def test_small_whole_numbers(shape):
    """Nothing rounds: gemv is exact, and the gated form is the activation of exact
    products."""
    weights, M, N, K = shape
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    x = torch.randint(-3, 4, (M, K), generator=g, device="cuda").to(torch.bfloat16)
    ops = [random_weight(N, K, N + K + i, whole=True) for i in range(weights)]
    if weights == 1:
        ref, guard = product(x, *ops[0])
        assert float(guard.max()) < 2 ** 22  # (halves: below 2^23 of them)
        assert torch.equal(nv.gemv(x, ops[0][0], out_dtype=torch.float32).double(), ref)
        return
    for op, _ in ops:  # products of a few units
        op.global_scale.fill_(2.0 ** -round(np.log2(6.5 * K ** 0.5)))
    (gate, gg), (up, ug) = (product(x, *o) for o in ops)
    assert max(float(v.max()) for v in (gg, ug)) / float(ops[0][0].global_scale) < 2 ** 22
    gate, up = gate.cpu().numpy(), up.cpu().numpy()
    for act in ("silu", "gelu"):
        h = nv.gemv_gated(x, ops[0][0], ops[1][0], act, out_dtype=torch.float32).double().cpu().numpy()
        ref = gate64(gate, act) * up
        tol = gated_tolerance(gate, 0.0, up, 0.0, act) + 2.0 ** -22 * np.abs(ref)
        assert np.all(np.abs(h - ref) <= tol), float(np.max(np.abs(h - ref) / np.maximum(tol, 1e-300)))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SIZES)
def test_any_codes_and_scales(shape):
    weights, M, N, K = shape
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    ops = [random_weight(N, K, N + K + i, whole=False) for i in range(weights)]
    unit = bound(M, N, K, weights, sms())
    for op, _ in ops:
        op.global_scale.fill_(float(np.float32(2e-3 / K ** 0.5)))
    prods = [product(x, *o) for o in ops]
    for dtype in (torch.float32, torch.bfloat16):
        half = HALF[dtype] * (1 + 2.0 ** -6)
        if weights == 1:
            ref, guard = prods[0]
            close(nv.gemv(x, ops[0][0], out_dtype=dtype), ref, unit * guard + half * ref.abs())
            continue
        (gate, gg), (up, ug) = ((p.cpu().numpy(), q.cpu().numpy()) for p, q in prods)
        h = nv.gemv_gated(x, ops[0][0], ops[1][0], "gelu", out_dtype=dtype).double().cpu().numpy()
        ref = gate64(gate, "gelu") * up
        tol = gated_tolerance(gate, unit * gg, up, unit * ug, "gelu") + (half + 2.0 ** -22) * np.abs(ref)
        assert np.all(np.abs(h - ref) <= tol), float(np.max(np.abs(h - ref) / tol))
