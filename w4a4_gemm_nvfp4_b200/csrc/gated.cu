// gated.cu -- backward pass of the gated feed-forward block's first half from
// 8-bit checkpoints of its two products:
//
//   h = act(g) u;   dg = dh u act'(g),   du = dh act(g),
//   act(g) = g sigma(z),  act'(g) = sigma + g sigma (1 - sigma) z'(g)
//
// with g = s_g q_g and u = s_u q_u read from the checkpoint (one bf16 scale s
// for 32 columns of a row).  dg and du go side by side into one [rows, 2 cols]
// matrix: the operand of both gradient GEMMs, dX = [dg|du] [Wg; Wu] and
// d[Wg; Wu] = [dg|du]^T X.  h, which the down-projection's weight gradient
// needs, can be written again in the same pass instead of being kept.
//
// Nothing is used twice, so the kernel is bound by HBM: 2 + 2 (1 + 1/16) bytes
// in and 4 (6 with h) out per element (8192 x 14336: 159 us, 91 % of a copy's
// rate, 190 us and 95 % with h).  About 20 operations an element in packed
// binary32 hide behind that; results are rounded once, to bf16.  Rows off 16-byte
// alignment are put together in registers and bound by issue: 8192 x 14333 takes
// 199 us, 232 with h.
#include <cuda_bf16.h>

#include <algorithm>

#include "block_step.cuh"  // packed pairs (f2)
#include "common.cuh"
#include "gated.cuh"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

struct BackwardParams {
  const uint16_t* dh;
  int64_t ldd;
  const int8_t* codes;     // [2][rows][32 blocks]
  const uint16_t* scales;  // bf16 [2][rows][blocks]
  uint16_t* dgu;
  int64_t ldg;
  uint16_t* h;             // or null
  int64_t ldh;
  int64_t rows;
  int cols, blocks;
  uint32_t chunks;         // groups of columns in a row, one per thread (or warp)
  uint32_t step_chunks;    // the grid's stride in (rows, chunks)
  int64_t step_rows;
};

__device__ __forceinline__ float bf16_to_f32(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// g^2 in z' of GELU stays finite: past |g| = 16 the factor 1 - sigma (or sigma) is
// an exact zero, and that times an infinite z' would be NaN instead of 0.
constexpr float kSquareCap = 1.0e18f;

__device__ __forceinline__ float code_value(uint32_t word, int i) {
  return static_cast<float>(static_cast<int8_t>(word >> (8 * i)));
}

// dg, du and h of a pair of columns, in packed binary32: every kernel's, so that they
// agree bit for bit.  The activation is a constant (a branch on it for each pair:
// 8192 x 14333 220 us against 199, with GELU and h 267 against 256).
template <int ACT>
__device__ __forceinline__ void gate2(const f2& d, const f2& g, const f2& u, f2& vg, f2& vu, f2& vh) {
  const f2 one = make_f2(1.0f, 1.0f);
  const auto sigma = [&](const f2& t) {  // t = -z log2(e)
    const f2 e = add2(make_f2(ex2_approx(t.a()), ex2_approx(t.b())), one);
    return make_f2(rcp_approx(e.a()), rcp_approx(e.b()));
  };
  const auto less = [&](const f2& s) { return fma2(s, make_f2(-1.0f, -1.0f), one); };  // 1 - sigma
  // act' = sigma + g sigma (1 - sigma) z', the last product and the sum in one rounding,
  // said so: left to the compiler it was one in one kernel and two in another
  f2 s, a, slope;
  if constexpr (ACT == NVFP4_ACT_SILU) {
    s = sigma(mul2(g, make_f2(-kLog2e, -kLog2e)));
    a = mul2(g, s);
    slope = fma2(a, less(s), s);
  } else {
    f2 gg = mul2(g, g);
    gg = make_f2(fminf(gg.a(), kSquareCap), fminf(gg.b(), kSquareCap));
    s = sigma(mul2(g, fma2(gg, make_f2(kGeluT3, kGeluT3), make_f2(kGeluT1, kGeluT1))));
    a = mul2(g, s);
    slope = fma2(mul2(a, less(s)),
                 fma2(gg, make_f2(3.0f * kGelu2C * kGeluCubic, 3.0f * kGelu2C * kGeluCubic), make_f2(kGelu2C, kGelu2C)), s);
  }
  // u act'(g) first: dh u alone may leave the range that the gradient is in
  vg = mul2(d, mul2(u, slope));
  vu = mul2(d, a);
  vh = mul2(a, u);
}

// Eight columns: dh as four words, the codes and scales of g and u.
struct Eight {
  uint32_t dh[4];
  uint2 gq, uq;
  float gs, us;
};

// dg, du and h of eight columns in packed binary32, rounded to bf16: four words
// each.
template <int ACT>
__device__ __forceinline__ void gate8(const Eight& c, uint32_t* dg, uint32_t* du, uint32_t* h) {
  const f2 gs = make_f2(c.gs, c.gs), us = make_f2(c.us, c.us);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t gw = i < 2 ? c.gq.x : c.gq.y, uw = i < 2 ? c.uq.x : c.uq.y;
    const int b = 2 * (i & 1);
    const f2 d = make_f2(__uint_as_float(c.dh[i] << 16), __uint_as_float(c.dh[i] & 0xFFFF0000u));
    const f2 g = mul2(gs, make_f2(code_value(gw, b), code_value(gw, b + 1)));
    const f2 u = mul2(us, make_f2(code_value(uw, b), code_value(uw, b + 1)));
    f2 vg, vu, vh;
    gate2<ACT>(d, g, u, vg, vu, vh);
    dg[i] = pack2(vg.a(), vg.b());
    du[i] = pack2(vu.a(), vu.b());
    h[i] = pack2(vh.a(), vh.b());
  }
}

// Every row of dh, dgu and h starts on 16 bytes and 8 divides the columns: 8
// columns per thread, two such chunks in flight.
template <int ACT>
__global__ void __launch_bounds__(kThreads) gated_backward_kernel(const BackwardParams p) {
  pdl_launch_dependents();
  pdl_wait();  // the launch overlaps the previous kernel's tail
  const int64_t pitch = static_cast<int64_t>(p.blocks) * kCkptBlock;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  int64_t row = first / p.chunks;
  uint32_t chunk = static_cast<uint32_t>(first - row * p.chunks);
  auto advance = [&] {
    row += p.step_rows;
    chunk += p.step_chunks;
    if (chunk >= p.chunks) chunk -= p.chunks, ++row;
  };
  auto load = [&](Eight& c) {
    const uint32_t col = chunk * 8;
    const int64_t ur = p.rows + row;
    const uint4 d = __ldg(reinterpret_cast<const uint4*>(p.dh + row * p.ldd + col));
    c.dh[0] = d.x, c.dh[1] = d.y, c.dh[2] = d.z, c.dh[3] = d.w;
    c.gq = __ldg(reinterpret_cast<const uint2*>(p.codes + row * pitch + col));
    c.uq = __ldg(reinterpret_cast<const uint2*>(p.codes + ur * pitch + col));
    c.gs = bf16_to_f32(p.scales[row * p.blocks + col / kCkptBlock]);
    c.us = bf16_to_f32(p.scales[ur * p.blocks + col / kCkptBlock]);
  };
  auto finish = [&](const Eight& c, int64_t r, uint32_t ch) {
    uint32_t dg[4], du[4], h[4];
    gate8<ACT>(c, dg, du, h);
    uint16_t* g = p.dgu + r * p.ldg + ch * 8;
    *reinterpret_cast<uint4*>(g) = make_uint4(dg[0], dg[1], dg[2], dg[3]);
    *reinterpret_cast<uint4*>(g + p.cols) = make_uint4(du[0], du[1], du[2], du[3]);
    if (p.h) *reinterpret_cast<uint4*>(p.h + r * p.ldh + ch * 8) = make_uint4(h[0], h[1], h[2], h[3]);
  };
  while (row < p.rows) {
    Eight a, b;
    const int64_t row_a = row;
    const uint32_t chunk_a = chunk;
    load(a);
    advance();
    const bool two = row < p.rows;
    if (two) load(b);
    finish(a, row_a, chunk_a);
    if (two) {
      finish(b, row, chunk);
      advance();
    }
  }
}

// One column per thread: narrow matrices at any alignment.
template <int ACT>
__global__ void __launch_bounds__(kThreads) gated_backward_narrow_kernel(const BackwardParams p) {
  pdl_launch_dependents();
  pdl_wait();  // the launch overlaps the previous kernel's tail
  const int64_t pitch = static_cast<int64_t>(p.blocks) * kCkptBlock;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  int64_t row = first / p.chunks;
  uint32_t col = static_cast<uint32_t>(first - row * p.chunks);
  while (row < p.rows) {
    const int64_t ur = p.rows + row;
    const f2 gs = make_f2(bf16_to_f32(p.scales[row * p.blocks + col / kCkptBlock]), 0.0f);
    const f2 us = make_f2(bf16_to_f32(p.scales[ur * p.blocks + col / kCkptBlock]), 0.0f);
    f2 vg, vu, vh;
    gate2<ACT>(make_f2(bf16_to_f32(p.dh[row * p.ldd + col]), 0.0f), mul2(gs, make_f2(p.codes[row * pitch + col], 0.0f)),
               mul2(us, make_f2(p.codes[ur * pitch + col], 0.0f)), vg, vu, vh);
    uint16_t* out = p.dgu + row * p.ldg + col;
    out[0] = static_cast<uint16_t>(pack2(vg.a(), 0.0f));
    out[p.cols] = static_cast<uint16_t>(pack2(vu.a(), 0.0f));
    if (p.h) p.h[row * p.ldh + col] = static_cast<uint16_t>(pack2(vh.a(), 0.0f));
    row += p.step_rows;
    col += p.step_chunks;
    if (col >= p.chunks) col -= p.chunks, ++row;
  }
}

// ---- rows at any alignment: a warp takes 256 columns of a row, 8 per lane.
// The codes are aligned whatever the row; a row of dh, dgu or h that starts
// off a 16-byte boundary is still moved in aligned 16-byte vectors, each lane's
// put together from its own 8 values and its neighbour's.  Segments step by 248
// columns: lane 0 computes the 8 values before lane 1's again, so that every
// vector but a row's first and last is stored whole.
constexpr int kSegStep = 248;

// Values a .. a + 7 of the 16 in (lo, hi), 0 <= a <= 7.
__device__ __forceinline__ void take8(const uint32_t* lo, const uint32_t* hi, uint32_t a, uint32_t* out) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = lo[i], w[4 + i] = hi[i];
  if (a & 4) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (a & 2) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = a & 1 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
}

// Columns c .. c + 7 of a row (c may be negative or run past the row: zeros), c
// on a 16-byte boundary.
__device__ __forceinline__ void load_vector(const uint16_t* row, int c, int cols, uint32_t* v) {
  if (c >= 0 && c + 8 <= cols) {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(row + c));
    v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int lo = c + 2 * i, hi = lo + 1;
      v[i] = (lo >= 0 && lo < cols ? row[lo] : 0u) | ((hi >= 0 && hi < cols ? row[hi] : 0u) << 16);
    }
  }
}

// This lane's columns col .. col + 7 of a row; the whole warp calls it.  inside:
// the warp's columns and 8 on either side lie in the row.
__device__ __forceinline__ void load_row8(const uint16_t* row, int col, int cols, uint32_t lane, bool inside, uint32_t* v) {
  const uint32_t a = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row + col) >> 1) & 7u;  // the same in every lane
  const int c = col - static_cast<int>(a);
  auto load = [&](int at, uint32_t* to) {
    if (inside) {
      const uint4 r = __ldg(reinterpret_cast<const uint4*>(row + at));
      to[0] = r.x, to[1] = r.y, to[2] = r.z, to[3] = r.w;
    } else {
      load_vector(row, at, cols, to);
    }
  };
  uint32_t own[4];
  load(c, own);
  if (a == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = own[i];
    return;
  }
  uint32_t next[4], after[4] = {};
  if (lane == 31) load(c + 8, after);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    next[i] = __shfl_down_sync(0xffffffffu, own[i], 1);
    if (lane == 31) next[i] = after[i];
  }
  take8(own, next, a, v);
}

// Stores the 8 values of every lane but the first, together with those of its
// left neighbour that share its vector.
__device__ __forceinline__ void store_row8(uint16_t* row, int col, int cols, uint32_t lane, bool inside,
                                           const uint32_t* v) {
  const uint32_t b = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row + col) >> 1) & 7u;
  const int c = col - static_cast<int>(b);
  uint32_t out[4];
  if (b == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = v[i];
  } else {
    uint32_t prev[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) prev[i] = __shfl_up_sync(0xffffffffu, v[i], 1);
    take8(prev, v, 8 - b, out);
  }
  if (lane == 0) return;
  if (inside || (c >= 0 && c + 8 <= cols)) {
    *reinterpret_cast<uint4*>(row + c) = make_uint4(out[0], out[1], out[2], out[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i >= 0 && c + i < cols) row[c + i] = static_cast<uint16_t>(out[i / 2] >> (16 * (i & 1)));
  }
}

template <int ACT>
__global__ void __launch_bounds__(kThreads) gated_backward_rows_kernel(const BackwardParams p) {
  pdl_launch_dependents();
  pdl_wait();  // the launch overlaps the previous kernel's tail
  const uint32_t lane = threadIdx.x & 31;
  const int64_t pitch = static_cast<int64_t>(p.blocks) * kCkptBlock;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  int64_t row = first / p.chunks;
  uint32_t seg = static_cast<uint32_t>(first - row * p.chunks);
  while (row < p.rows) {
    const int begin = static_cast<int>(seg) * kSegStep - 8, col = begin + static_cast<int>(lane) * 8;
    const bool inside = begin >= 8 && begin + 264 <= p.cols;
    Eight c;
    c.gq = c.uq = make_uint2(0, 0);
    c.gs = c.us = 0.0f;
    if (inside || (col >= 0 && col < pitch)) {
      c.gq = __ldg(reinterpret_cast<const uint2*>(p.codes + row * pitch + col));
      c.uq = __ldg(reinterpret_cast<const uint2*>(p.codes + (p.rows + row) * pitch + col));
      c.gs = bf16_to_f32(p.scales[row * p.blocks + col / kCkptBlock]);
      c.us = bf16_to_f32(p.scales[(p.rows + row) * p.blocks + col / kCkptBlock]);
    }
    load_row8(p.dh + row * p.ldd, col, p.cols, lane, inside, c.dh);
    uint32_t dg[4], du[4], h[4];
    gate8<ACT>(c, dg, du, h);
    uint16_t* out = p.dgu + row * p.ldg;
    store_row8(out, col, p.cols, lane, inside, dg);
    store_row8(out + p.cols, col, p.cols, lane, inside, du);
    if (p.h) store_row8(p.h + row * p.ldh, col, p.cols, lane, inside, h);
    row += p.step_rows;
    seg += p.step_chunks;
    if (seg >= p.chunks) seg -= p.chunks, ++row;
  }
}

// Chunks of `width` columns, `per_cta` of them for a CTA at a time.  Up to 32 CTAs
// per SM: a few waves even out what each of them meets in HBM (8192 x 14336 with
// h, when they were compared: 221 us with 8, 205 with 16, 193 with 32, 225 with one
// chunk or two per thread).
unsigned spread(BackwardParams& p, int sms, int64_t cols, int width, int per_cta) {
  p.chunks = static_cast<uint32_t>((cols + width - 1) / width);
  const int64_t total = p.rows * p.chunks;
  const int64_t grid = std::min<int64_t>((total + per_cta - 1) / per_cta, static_cast<int64_t>(sms) * 32);
  const int64_t stride = grid * per_cta;
  p.step_rows = stride / p.chunks;
  p.step_chunks = static_cast<uint32_t>(stride % p.chunks);
  return static_cast<unsigned>(grid);
}

// N: columns; wide: every row on 16 bytes and 8 divides N.  256 columns are a
// warp's segment in the rows kernel; below that most of its lanes would idle
// (8192 x 130: 9.4 us against 6.9, 8192 x 999: 26.9 against 31.6).
template <int ACT>
cudaError_t launch_backward(BackwardParams& p, bool wide, int sms, cudaStream_t s) {
  if (wide) {
    const unsigned grid = spread(p, sms, p.cols, 8, kThreads);
    return launch_kernel(gated_backward_kernel<ACT>, dim3(grid), dim3(kThreads), 0, s, true, p);
  }
  if (p.cols >= 256) {
    // (a row's last vector may start up to 7 columns early)
    const unsigned grid = spread(p, sms, static_cast<int64_t>(p.cols) + 7, kSegStep, kThreads / 32);
    return launch_kernel(gated_backward_rows_kernel<ACT>, dim3(grid), dim3(kThreads), 0, s, true, p);
  }
  const unsigned grid = spread(p, sms, p.cols, 1, kThreads);
  return launch_kernel(gated_backward_narrow_kernel<ACT>, dim3(grid), dim3(kThreads), 0, s, true, p);
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

size_t nvfp4_checkpoint_codes_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return 2 * static_cast<size_t>(rows) * static_cast<size_t>((cols + kCkptBlock - 1) / kCkptBlock * kCkptBlock);
}

size_t nvfp4_checkpoint_scales_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return 4 * static_cast<size_t>(rows) * static_cast<size_t>((cols + kCkptBlock - 1) / kCkptBlock);
}

nvfp4_status nvfp4_gated_backward(const void* dh, int64_t ldd, const void* ckpt_codes, const void* ckpt_scales,
                                  int64_t M, int64_t N, int act, void* dgu, int64_t ldg, void* h, int64_t ldh,
                                  void* stream) {
  const char* fn = "nvfp4_gated_backward";
  if (!dh || !ckpt_codes || !ckpt_scales || !dgu) return set_error(NVFP4_ERR_INVALID_ARG, "%s: null pointer argument", fn);
  if (M < 1 || N < 1 || M > (1ll << 30) || N > (1ll << 30))
    return set_error(NVFP4_ERR_INVALID_ARG, "%s: need 1 <= M, N <= 2^30 (M=%lld N=%lld)", fn, (long long)M, (long long)N);
  if (ldd < N || ldg < 2 * N || (h && ldh < N) || ldd > (int64_t{1} << 40) || ldg > (int64_t{1} << 40) ||
      (h && ldh > (int64_t{1} << 40)))
    return set_error(NVFP4_ERR_INVALID_ARG, "%s: need N <= ldd, 2 N <= ldg, N <= ldh, none above 2^40", fn);
  if (act != NVFP4_ACT_SILU && act != NVFP4_ACT_GELU)
    return set_error(NVFP4_ERR_INVALID_ARG, "%s: unknown act %d", fn, act);
  if (!aligned16(ckpt_codes) || ((reinterpret_cast<uintptr_t>(ckpt_scales) | reinterpret_cast<uintptr_t>(dh) |
                                  reinterpret_cast<uintptr_t>(dgu) | reinterpret_cast<uintptr_t>(h)) & 1u))
    return set_error(NVFP4_ERR_INVALID_ARG, "%s: misaligned buffer", fn);
  int sms = 0;
  nvfp4_status st = check_device(nullptr, &sms);
  if (st != NVFP4_OK) return st;
  BackwardParams p = {};
  p.dh = static_cast<const uint16_t*>(dh);
  p.ldd = ldd;
  p.codes = static_cast<const int8_t*>(ckpt_codes);
  p.scales = static_cast<const uint16_t*>(ckpt_scales);
  p.dgu = static_cast<uint16_t*>(dgu);
  p.ldg = ldg;
  p.h = static_cast<uint16_t*>(h);
  p.ldh = ldh;
  p.rows = M;
  p.cols = static_cast<int>(N);
  p.blocks = static_cast<int>((N + kCkptBlock - 1) / kCkptBlock);
  const bool wide = N % 8 == 0 && aligned16(dh) && aligned16(dgu) && ldd % 8 == 0 && ldg % 8 == 0 &&
                    (!h || (aligned16(h) && ldh % 8 == 0));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = act == NVFP4_ACT_SILU ? launch_backward<NVFP4_ACT_SILU>(p, wide, sms, s)
                                              : launch_backward<NVFP4_ACT_GELU>(p, wide, sms, s);
  if (e != cudaSuccess) return cuda_status(e, "gated_backward_kernel launch");
  return NVFP4_OK;
}

}  // extern "C"
