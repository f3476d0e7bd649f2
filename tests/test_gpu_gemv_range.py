"""The range of x in nvfp4_gemv and nvfp4_gemv_gated.  Each 256 elements of a row
(from column 0 on) are held in f16 on the scale that takes the largest finite one
into [2^14, 2^15): exactly where they are at least 2^-31 of it, else rounded to the
nearest multiple of f16's least subnormal, 2^-24, which is off by at most 2^-25 on that
scale and so by 2^-39 of the largest, whatever the weights of the larger ones are.
Against unit rows a call gives back what it holds, bit for bit."""
import numpy as np
import pytest
import torch

import w4a4_gemm_nvfp4_b200 as nv
from test_gpu_gemv import gate64
from test_gpu_gemv_paths import bound, close, product, random_weight, sms

GROUP = 256


def groups(x):
    """x [M, K] in binary64 as [M, groups, 256], zeros behind the last column."""
    M, K = x.shape
    p = torch.zeros(M, (K + GROUP - 1) // GROUP * GROUP, dtype=torch.float64)
    p[:, :K] = x.double().cpu()
    return p.view(M, -1, GROUP)


def largest(x):
    p = groups(x)
    return torch.where(torch.isfinite(p), p.abs(), 0.0).amax(-1, keepdim=True)


def held(x):
    """x as the call holds it (finite rows), in binary64."""
    M, K = x.shape
    e = torch.frexp(largest(x))[1] - 1  # the largest is in [2^e, 2^(e + 1))
    k = torch.clamp(14 - e, max=126)
    f16 = torch.ldexp(groups(x), k).to(torch.float16).double()
    return torch.ldexp(f16, -k).view(M, -1)[:, :K]


def identity(K, N=None):
    """Weight row n is 1 at k = n % K and 0 elsewhere."""
    N = K if N is None else N
    codes = torch.zeros(N, K // 2, dtype=torch.uint8)
    n = torch.arange(N)
    k = n % K
    codes[n, k // 2] = torch.where(k % 2 == 0, 0x02, 0x20).to(torch.uint8)
    scales = torch.full((nv.nvfp4_scales_bytes(N, K),), 0x38, dtype=torch.uint8)
    return nv.NVFP4Tensor(codes.cuda(), scales.cuda(), torch.ones(1, device="cuda"), None, N, K)


def spread(M, K, seed, lo=-133, hi=127):
    """bf16 values of every exponent from lo to hi, in any order."""
    g = torch.Generator().manual_seed(seed)
    e = torch.randint(lo, hi + 1, (M, K), generator=g)
    m = torch.randint(0, 128, (M, K), generator=g).double() / 128 + 1
    sign = torch.randint(0, 2, (M, K), generator=g) * 2 - 1
    x = (sign * torch.ldexp(m, e)).to(torch.bfloat16)
    assert bool(torch.isfinite(x).all())
    return x


@pytest.mark.parametrize("lo,hi", [(-133, 127), (-133, -100), (-31, 0), (60, 127), (-133, -126)])
def test_what_is_held(lo, hi):
    """The statement above, of the model that the calls are compared with."""
    x = spread(5, 700, 1, lo, hi)
    x[2], x[3, 300] = 0.0, 0.0
    h, p, top = groups(held(x)), groups(x), largest(x)
    off = (h - p).abs()
    assert bool((off <= 2.0 ** -39 * top).all())
    assert bool((off[(p.abs() >= 2.0 ** -31 * top)] == 0).all())
    if hi - lo <= 31 or hi <= -100:  # (below 2^-96 f16 on that scale reaches the least bf16)
        assert not off.any()


@pytest.mark.gpu
@pytest.mark.parametrize("small", [-24, -31, -32, -38, -39, -40, -41, -60, -133])
def test_a_small_element_beside_a_large_one_that_meets_a_zero(small):
    K = 64
    x = torch.zeros(1, K, dtype=torch.bfloat16)
    x[0, 0], x[0, 1] = 1.0, 1.0078125 * 2.0 ** small
    codes = torch.zeros(2, K // 2, dtype=torch.uint8)
    codes[0, 0], codes[1, 0] = 0x30, 0x02  # 0 and 1.5; 1 and 0
    w = nv.NVFP4Tensor(codes.cuda(), torch.full((nv.nvfp4_scales_bytes(2, K),), 0x38, dtype=torch.uint8).cuda(),
                       torch.ones(1, device="cuda"), None, 2, K)
    y = nv.gemv(x.cuda(), w, out_dtype=torch.float32)[0].double().cpu()
    assert y[1] == 1.0 and y[0] == 1.5 * held(x)[0, 1]
    assert abs(float(y[0]) - 1.5 * float(x[0, 1])) <= (0.0 if small >= -31 else 1.5 * 2.0 ** -39)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 64), (3, 128), (8, 512), (16, 1024), (9, 2112), (16, 16384), (16, 65536), (2, 131072)],
                         ids=lambda s: "x".join(map(str, s)))
def test_the_identity_gives_back_what_is_held(shape):
    """Spread over the whole range of the type: with x whole, in clusters and in
    pieces."""
    M, K = shape
    x = spread(M, K, seed=K)
    x[0, 5] = 0.0
    for N in (K,) if K <= 2112 else (16, 300):
        y = nv.gemv(x.cuda(), identity(K, N), out_dtype=torch.float32).double().cpu()
        assert torch.equal(y, held(x)[:, torch.arange(N) % K])


@pytest.mark.gpu
@pytest.mark.parametrize("lo,hi", [(-31, 0), (96, 127), (-133, -102)])
def test_the_identity_gives_back_x_within_the_range_that_is_exact(lo, hi):
    x = spread(11, 640, 3, lo, hi)
    assert torch.equal(nv.gemv(x.cuda(), identity(640), out_dtype=torch.float32).cpu(), x.float())


@pytest.mark.gpu
def test_the_identity_in_pieces_without_a_cluster():
    M, N, K = 12, 1184, 10240
    assert nv.testing_gemv_plan(M, N, K, 1, sms())["ranks"] == 1 or sms() != 148
    x = spread(M, K, seed=1)
    y = nv.gemv(x.cuda(), identity(K, N), out_dtype=torch.float32).double().cpu()
    assert torch.equal(y, held(x)[:, torch.arange(N) % K])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 100, 512), (16, 333, 5120), (8, 64, 16384), (16, 300, 16384), (9, 600, 17408)],
                         ids=lambda s: "x".join(map(str, s)))
def test_spread_rows_against_any_weights(shape):
    """The bound of the sum on what is held, and what holding it loses beside x."""
    M, N, K = shape
    x = spread(M, K, seed=N, lo=-60, hi=10)
    x[:, : K // 2] = (x[:, : K // 2].double() * 2.0 ** -60).to(torch.bfloat16)
    op, rows = random_weight(N, K, N, whole=False)
    ref, guard = product(held(x).cuda(), op, rows)
    half = 2.0 ** -24 * ref.abs()
    y = nv.gemv(x.cuda(), op, out_dtype=torch.float32)
    close(y, ref, bound(M, N, K, 1, sms()) * guard + half)
    w = groups(rows(0, N)).abs().sum(-1)
    lost = (2.0 ** -39 * largest(x)[..., 0] @ w.T).cuda()
    ref, guard = product(x.cuda(), op, rows)
    close(y, ref, bound(M, N, K, 1, sms()) * (guard + lost) + lost + half * (1 + 2.0 ** -20))


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_form(act):
    """Gate from large elements, up from elements 2^-25 of them, in the same row."""
    M, N, K = 11, 200, 640
    g = torch.Generator().manual_seed(3)
    x = torch.randint(8, 16, (M, K), generator=g).double() * (torch.randint(0, 2, (M, K), generator=g) * 2 - 1)
    x[:, 1::2] *= 2.0 ** -25
    x = x.to(torch.bfloat16)
    assert torch.equal(held(x), x.double())
    (wg, rg), (wu, ru) = random_weight(N, K, 1, whole=True), random_weight(N, K, 2, whole=True)
    wg.codes &= 0x0F  # even k only
    wu.codes &= 0xF0  # odd k only
    wg.global_scale.fill_(0.005)
    xc = x.cuda()
    (gate, gg), (up, ug) = product(xc, wg, rg), product(xc, wu, ru)
    assert float(up.abs().max()) < 2.0 ** -12 and float(ug.min()) > 0
    h = nv.gemv_gated(xc, wg, wu, act, out_dtype=torch.float32).double().cpu().numpy()
    unit = bound(M, N, K, 2, sms())
    gate, gg, up, ug = (t.cpu().numpy() for t in (gate, gg, up, ug))
    ref = gate64(gate, act) * up
    a = np.abs(gate64(gate, act))
    da = 1.13 * unit * gg + a * (16 * 2.0 ** -24 + 90 * 2.0 ** -22)
    tol = da * np.abs(up) + (a + da) * unit * ug + 2.0 ** -22 * np.abs(ref)
    assert np.all(np.abs(h - ref) <= tol)


@pytest.mark.gpu
def test_infinities_and_nan_beside_small_elements():
    """They show where they are, the finite ones keep the scale of the largest finite
    one, and the other rows of the call are untouched."""
    K = 256
    x = spread(5, K, seed=2, lo=-120, hi=100)
    finite = held(x)
    x[1, 7], x[2, 9], x[3, 11] = float("inf"), float("-inf"), float("nan")
    y = nv.gemv(x.cuda(), identity(K), out_dtype=torch.float32).double().cpu()
    assert torch.equal(y[0], finite[0]) and torch.equal(y[4], finite[4])
    assert y[1, 7] == float("inf") and y[2, 9] == float("-inf") and torch.isnan(y[3]).all()
    for m, k in ((1, 7), (2, 9)):  # 0 * Inf everywhere else
        assert torch.isnan(y[m, torch.arange(K) != k]).all()
