// gemv.cu -- a few bf16 rows against NVFP4 weights (decode):
//
//   y[m, n] = alpha_W * sum_k x[m, k] * s[n, k/16] * q[n, k],   1 <= m <= 16
//
// and the gated form act(x Wg^T) * (x Wu^T), both products in one kernel.
//
// The weight is read once and nothing else is large, so the kernel is bound by
// HBM: (1/2 + 1/16) bytes a weight.  One byte holds two weights, so what has
// to stay below the memory time is the work to decode them.  Per 8 weights of
// a lane: four cvt.f16x2.e2m1x2, four f16x2 products with the block's scale,
// one mma.m16n8k16.  q * s has at most 2 + 4 significant bits and lies between
// 2^-10 and 2688, so the f16 weights are exact; the products with x are exact
// in the tensor core and are summed in binary32.  (Decoding to bf16 has no
// conversion instruction; with shifts and masks it measured half the rate of
// the conversion, 12.4 against 24.6 T weights/s, too near the 11.7 T that HBM
// delivers.)
//
// x is bf16 and the MMA wants f16: each 256 k of a token are scaled by the power
// of two that takes their largest finite |x| into [2^14, 2^15).  That is exact
// for every element of at least 2^-31 of that largest one; smaller ones are
// rounded to multiples of f16's least subnormal, 2^-24, off by at most half of it
// and so by 2^-39 of the largest.  That is 2^-15 of what a binary32 sum with the
// largest in it rounds, but where the larger ones' weights are zero or cancel it
// is what the small ones are known to.  Held exactly, by going over the weights
// again with the rest of the rounding where a CTA has one, every call pays (16 x
// 17408 x 5120 18.9 -> 20.0 us, 16 x 5120 x 17408 31.9 -> 34.3, 1 x 256 x 512 2.7 ->
// 2.9), and twice its time where a closed GELU gate (g below -5.5) is in a row.
// Inf and NaN pass through and act as in a binary32 sum.
//
// Mapping.  An MMA tile is 16 weight rows x 16 k.  A lane (g, t) of the MMA
// holds rows g and g + 8; the order of k inside a tile is free as long as x
// agrees, so lane t takes 64 consecutive k (32 bytes of codes, one 4-byte word
// of 4 scales) of a 256-wide step, and a row's part of a step is a whole
// 128-byte line.  The 16 rows are 4 consecutive ones in each of the four 32-row
// groups of a 128-row scale atom: their scale words are 64 contiguous bytes.
//
// Split.  A CTA of 16 warps owns a run of row tiles.  Its (tile, step) units
// are cut into 16 equal runs, one per warp; each warp copies its units into its
// own ring in shared memory, four (or two) ahead, so there is no barrier in the
// stream.  A warp leaves one partial 16 x m tile per row tile that it touched
// in shared memory, and after one barrier the partials of a tile are summed in
// warp order: no atomics, the same result every time.  Where there are more SMs
// than row tiles, or x is too large for one CTA, a cluster shares the tiles, each
// CTA with a part of K, and their sums are added in the order of the CTAs.
//
// Measured (device time, weights from HBM): 1 x 14336 x 4096 9.4 us (3.5 TB/s;
// about 3 us of it launch, x and the last sum), the gated form 15.7 us (4.2
// TB/s), 5 x 12283 x 5120 13 us (3 us of it x), gated 16 x 17408 x 5120 28.7 us
// (3.5 TB/s; there the stream takes 22 us, 15 with its loads alone and 18 with its
// arithmetic alone, 380 warp instructions for a unit of 16 x 256 weights, 286 with one
// column tile of tokens), 16 x 5120 x 17408 32 us (half of it x, in four pieces).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "block_step.cuh"  // packed pairs (f2)
#include "common.cuh"
#include "gated.cuh"
#include "nvfp4_testing.h"

namespace nvfp4 {
namespace {

constexpr int kMaxTokens = 16;
constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kStepK = 256;                   // k per step: 4 lanes x 64
constexpr uint32_t kGroupBytes = 144;         // 64 staged k of a token and padding
constexpr uint32_t kZeroBytes = 640;          // zeros that lanes without a token read
constexpr uint32_t kUnitBytes = 2048 + 256;   // 16 rows x 256 k: codes and scales
constexpr uint32_t kRedPitch = 20;            // floats per token of a partial tile: 16, and conflict-free stores
constexpr uint32_t kSmemLimit = 232448 - 1024;

// Bytes of a staged token: 64 more than a multiple of 128.
__host__ __device__ constexpr uint32_t token_bytes(uint32_t steps) {
  return (steps * 4 * kGroupBytes + 63) / 128 * 128 + 64;
}

struct GemvParams {
  const uint16_t* x;      // bf16 [M, K]
  int64_t ldx;
  const uint8_t* codes[2];
  const uint8_t* scales[2];
  const float* alpha[2];
  void* y;
  int64_t ldy;
  int M, N;
  uint32_t kgroups;       // K / 64
  uint32_t share, share_rest;  // row tiles of a CTA; the first share_rest CTAs have one more
  uint32_t all_steps;     // 256-wide steps of K
  uint32_t ranks;         // CTAs that share row tiles, each with a part of K: 1, or a cluster of 2, 4 or 8
  uint32_t rank_log;      // log2 of that
  uint32_t piece_steps;   // steps of x staged at a time
  uint32_t slots;         // partial tiles per warp
  uint32_t off_ring, off_red, off_acc, off_scale;
  int act, out_fp32, x_vec;
};

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The 8 codes of a word as four f16 pairs, k ascending.
__device__ __forceinline__ void decode8(uint32_t w, uint32_t* h) {
  asm("{\n\t.reg .b8 x0, x1, x2, x3;\n\t"
      "mov.b32 {x0, x1, x2, x3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, x0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, x1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, x2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, x3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Four E4M3 scales as f16 pairs, each scale in both halves.
__device__ __forceinline__ void decode_scales(uint32_t w, uint32_t* s) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  s[0] = __byte_perm(lo, lo, 0x1010);
  s[1] = __byte_perm(lo, lo, 0x3232);
  s[2] = __byte_perm(hi, hi, 0x1010);
  s[3] = __byte_perm(hi, hi, 0x3232);
}

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^k brings a largest finite |x| with the bf16 bits mx into [2^14, 2^15): k =
// 14 - exponent, at most 126 (then every |x| is below 2^-112 and the f16 values
// are still exact).
__device__ __forceinline__ int x_shift(int mx) { return min(141 - (mx >> 7), 126); }

// Two bf16 values times (f, f), a power of two, as f16.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, f2 f) {
  const f2 v = mul2(make_f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)), f);
  const __half2 h = __floats2half2_rn(v.a(), v.b());
  return *reinterpret_cast<const uint32_t*>(&h);
}

// V * S = U units cut into kWarps runs [w U / kWarps, (w + 1) U / kWarps): lane w
// keeps warp w's.
struct WarpRuns {
  uint32_t begin, end, first;  // first: the first virtual tile of the run
  __device__ __forceinline__ WarpRuns(uint32_t lane, uint32_t S, uint32_t U)
      : begin(lane < kWarps ? lane * U / kWarps : U), end(lane < kWarps ? (lane + 1) * U / kWarps : U), first(begin / S) {}
  // Outputs of virtual tile vt, summed over the warps in their order: v[q] is
  // MMA row lane % 16 of token 8 n + 2 q + lane / 16.  All lanes of a warp call
  // it with the same vt and n.
  __device__ __forceinline__ void sum(const float* red, uint32_t slots, uint32_t M, uint32_t vt, uint32_t S, uint32_t n,
                                      uint32_t lane, float* v) const {
    const uint32_t lo = vt * S;
    uint32_t at[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      at[q] = min(8 * n + 2 * q + (lane >> 4), M - 1) * kRedPitch + (lane & 15);
      v[q] = 0.0f;
    }
    for (uint32_t left = __ballot_sync(0xffffffffu, begin < end && begin < lo + S && end > lo); left; left &= left - 1) {
      const uint32_t w = __ffs(left) - 1;
      const float* tile = red + (w * slots + vt - __shfl_sync(0xffffffffu, first, w)) * (M * kRedPitch);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (8 * n + 2 * q < M) v[q] += tile[at[q]];
    }
  }
};

// First weight row of tile `tile` for MMA row 0; MMA row i is row
// base + (i & 3) + 32 * (i >> 2).
__device__ __forceinline__ uint32_t tile_base(uint32_t tile) { return (tile >> 3) * 128u + (tile & 7u) * 4u; }

// d = a * b
__device__ __forceinline__ void mma_f16_first(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of this thread's groups are in flight.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Largest finite |x| of 8 bf16 values, as bf16 bits.
__device__ __forceinline__ uint32_t finite_max8(const uint4& r) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t v = __vmaxu2(__vmaxu2(r.x & m, r.y & m), __vmaxu2(r.z & m, r.w & m));
  uint32_t mx = max(v & 0xFFFFu, v >> 16);
  if (mx >= 0x7F80u) {  // an Inf or NaN among them
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    mx = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = w[j] & 0x7FFFu, hi = (w[j] >> 16) & 0x7FFFu;
      if (lo < 0x7F80u) mx = max(mx, lo);
      if (hi < 0x7F80u) mx = max(mx, hi);
    }
  }
  return mx;
}

// NT: MMA column tiles (8 tokens each); GATED: two weights, one output; D:
// units in flight per warp.
// R: 1 CTA or a cluster of 2 for a row tile, 0: a cluster of any size (as constants
// they save a few percent: gated 1 x 14336 x 4096 15.8 us against 16.2).
template <int NT, bool GATED, int D, int R>
__global__ void __launch_bounds__(kThreads, 1) gemv_kernel(const GemvParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr uint32_t MATS = GATED ? 2 : 1;
  const uint32_t xs = smem_u32(smem);
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t g = lane >> 2, t = lane & 3;
  const uint32_t M = static_cast<uint32_t>(p.M), N = static_cast<uint32_t>(p.N);
  const uint32_t ranks = R ? R : p.ranks, rank_log = R == 0 ? p.rank_log : R == 2;
  const uint32_t rank = ranks > 1 ? cluster_ctarank() : 0, group = blockIdx.x >> rank_log;
  // the row tiles of this CTA (or of its cluster), dealt out evenly
  const uint32_t t0 = group * p.share + min(group, p.share_rest);
  const uint32_t V = (p.share + (group < p.share_rest ? 1 : 0)) * MATS;  // virtual tiles: (row tile, weight)
  // and its steps of K
  const uint32_t s_begin = (rank * p.all_steps) >> rank_log, s_end = ((rank + 1) * p.all_steps) >> rank_log;
  const uint32_t tile_floats = M * kRedPitch;
  float* red = reinterpret_cast<float*>(smem + p.off_red);    // [warp][slot][token][kRedPitch]
  float* acc = reinterpret_cast<float*>(smem + p.off_acc);    // [virtual tile][token][16], several pieces only
  float* xscale = reinterpret_cast<float*>(smem + p.off_scale);  // [step][kMaxTokens]: what a unit's sum is times
  const bool pieces = p.off_acc != p.off_scale;
  // launched as a programmatic dependent: the launch overlaps the previous
  // kernel's tail, and no global memory is touched before that has finished
  pdl_launch_dependents();
  pdl_wait();
  const float alpha0 = __ldg(p.alpha[0]), alpha1 = __ldg(p.alpha[1]);
  if (pieces)
    for (uint32_t i = threadIdx.x; i < V * 16 * M; i += kThreads) acc[i] = 0.0f;

  const int64_t row_bytes = static_cast<int64_t>(p.kgroups) * 32;
  const uint32_t ring = p.off_ring + warp * (D * kUnitBytes);
  uint32_t U = 0, S = 1;
  for (uint32_t sb = s_begin; sb < s_end; sb += p.piece_steps) {
    S = min(p.piece_steps, s_end - sb);
    U = V * S;
    const uint32_t ub = warp * U / kWarps, ue = (warp + 1) * U / kWarps;
    const uint32_t first_v = ub / S;
    const uint32_t tok_bytes = token_bytes(S);

    // ---- stage x as f16, scaled per token and step.  A step of a token is 32
    // chunks of 16 bytes, one per lane; a warp copies, measures and converts
    // the same run of steps.  A group of 64 k takes 128 bytes and 16 of padding,
    // and a token 64 bytes more than a multiple of 128, so that the 8 lanes of a
    // load phase below (2 tokens, 4 groups) hit 8 bank groups.
    const uint32_t xb = warp * M * S / kWarps, xe = (warp + 1) * M * S / kWarps;
    const uint32_t xm0 = xb / S, xs0 = xb - xm0 * S;
    const uint32_t lane_at = kZeroBytes + lane * 16 + (lane >> 3) * 16;
    if (threadIdx.x < kZeroBytes / 4) reinterpret_cast<uint32_t*>(smem)[threadIdx.x] = 0;
    for (uint32_t j = xb, m = xm0, st = xs0; j < xe; ++j) {
      const uint32_t k = (sb + st) * kStepK + lane * 8;
      const bool real = k < p.kgroups * 64;
      const uint16_t* src = p.x + m * p.ldx + k;
      const uint32_t at = lane_at + m * tok_bytes + st * (4 * kGroupBytes);
      if (p.x_vec) {
        cp_async16(xs + at, real ? src : p.x, real);
      } else {
        uint4 r = make_uint4(0, 0, 0, 0);
        if (real) {
          r.x = src[0] | (static_cast<uint32_t>(src[1]) << 16);
          r.y = src[2] | (static_cast<uint32_t>(src[3]) << 16);
          r.z = src[4] | (static_cast<uint32_t>(src[5]) << 16);
          r.w = src[6] | (static_cast<uint32_t>(src[7]) << 16);
        }
        *reinterpret_cast<uint4*>(smem + at) = r;
      }
      if (++st == S) st = 0, ++m;
    }
    cp_async_commit();

    // ---- the first weights are on their way while x is measured and converted.
    // A unit: 16 rows x 128 bytes of codes, chunk c of row r at chunk c ^ (r & 7),
    // then 16 chunks of scales ([4 groups of 64 k][4 rows][4 row groups x 4]).
    // Loads never leave the operands: rows past N read row N - 1 and are not
    // stored, k past K is filled with zeros.
    const uint32_t lr = lane >> 3, lc = lane & 7;
    uint32_t nv = first_v, ns = ub - first_v * S;
    const uint8_t *pc, *ps;        // the tile being loaded: this lane's first row and chunk, its scale chunk
    int64_t up1, up2, up3;         // to its other rows
    auto open_tile = [&] {
      const uint32_t mat = GATED ? (nv & 1u) : 0u;
      const uint32_t base = tile_base(t0 + (GATED ? (nv >> 1) : nv));
      const uint32_t r0 = min(base + lr, N - 1);
      pc = p.codes[mat] + r0 * row_bytes + lc * 16;
      up1 = (min(base + lr + 32, N - 1) - r0) * row_bytes;
      up2 = (min(base + lr + 64, N - 1) - r0) * row_bytes;
      up3 = (min(base + lr + 96, N - 1) - r0) * row_bytes;
      ps = p.scales[mat] + (static_cast<int64_t>(base >> 7) * p.kgroups + ((lane >> 2) & 3)) * 512 +
           ((base & 31) + (lane & 3)) * 16;
    };
    const uint32_t dst = xs + ring + lr * 128;
    const uint32_t sw0 = (lc ^ lr) << 4, sw1 = (lc ^ (lr + 4)) << 4;
    uint32_t load_at = 0;
    auto load_next = [&] {
      const uint32_t kg = (sb + ns) * 4;
      const uint32_t d = dst + load_at, ds = xs + ring + load_at + 2048 + lane * 16;
      if (kg + 4 <= p.kgroups) {
        const uint8_t* c = pc + kg * 32;
        cp_async16(d + sw0, c);
        cp_async16(d + 512 + sw1, c + up1);
        cp_async16(d + 1024 + sw0, c + up2);
        cp_async16(d + 1536 + sw1, c + up3);
        if (lane < 16) cp_async16(ds, ps + kg * 512);
      } else {
        const bool real = kg * 2 + lc < p.kgroups * 2;  // 16-byte chunks of a row
        const uint8_t* c = real ? pc + kg * 32 : p.codes[0];
        cp_async16(d + sw0, c, real);
        cp_async16(d + 512 + sw1, real ? c + up1 : c, real);
        cp_async16(d + 1024 + sw0, real ? c + up2 : c, real);
        cp_async16(d + 1536 + sw1, real ? c + up3 : c, real);
        const bool sreal = kg + (lane >> 2) < p.kgroups;
        if (lane < 16) cp_async16(ds, sreal ? ps + kg * 512 : p.scales[0], sreal);
      }
      load_at = load_at + kUnitBytes == D * kUnitBytes ? 0 : load_at + kUnitBytes;
      if (++ns == S) {
        ns = 0;
        if (++nv < V) open_tile();
      }
    };
    uint32_t v = first_v, s = ns;  // unit being computed
    if (ub < ue) open_tile();
#pragma unroll
    for (uint32_t k = 0; k < D; ++k) {
      if (ub + k < ue) load_next();
      cp_async_commit();
    }

    cp_async_wait<D>();  // this thread's part of x
    auto convert = [&](const uint4& r, uint32_t m, uint32_t st) {
      const int k = x_shift(static_cast<int>(__reduce_max_sync(0xffffffffu, finite_max8(r))));
      const float one = __int_as_float((k + 127) << 23);
      const f2 f = make_f2(one, one);
      if (lane == 0) xscale[st * kMaxTokens + m] = __int_as_float((127 - k) << 23);
      return make_uint4(bf16x2_to_f16x2(r.x, f), bf16x2_to_f16x2(r.y, f), bf16x2_to_f16x2(r.z, f),
                        bf16x2_to_f16x2(r.w, f));
    };
    for (uint32_t j = xb, m = xm0, st = xs0; j < xe; j += 2) {  // two at a time: independent chains
      const uint32_t m1 = st + 1 == S ? m + 1 : m, st1 = st + 1 == S ? 0 : st + 1;
      uint4* at0 = reinterpret_cast<uint4*>(smem + lane_at + m * tok_bytes + st * (4 * kGroupBytes));
      uint4* at1 = reinterpret_cast<uint4*>(smem + lane_at + m1 * tok_bytes + st1 * (4 * kGroupBytes));
      if (j + 1 < xe) {
        const uint4 r0 = *at0, r1 = *at1;
        const uint4 h0 = convert(r0, m, st), h1 = convert(r1, m1, st1);
        *at0 = h0;
        *at1 = h1;
      } else {
        *at0 = convert(*at0, m, st);
      }
      m = st1 + 1 == S ? m1 + 1 : m1;
      st = st1 + 1 == S ? 0 : st1 + 1;
    }
    __syncthreads();

    // ---- stream the weights
    float sum[NT][4];
    auto clear = [&] {
#pragma unroll
      for (int n = 0; n < NT; ++n) sum[n][0] = sum[n][1] = sum[n][2] = sum[n][3] = 0.0f;
    };
    // this lane's tokens in the staged x; a lane without one reads zeros
    uint32_t xa[NT], xstep[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool real = g + 8 * n < M;
      xa[n] = (real ? kZeroBytes + (g + 8 * n) * tok_bytes : (g & 1) * 64) + t * kGroupBytes;
      xstep[n] = real ? 4 * kGroupBytes : 0;
    }
    // The tensor core truncates what it adds, so a chain of additions drifts:
    // a unit is summed from zero (two chains of 8 MMAs for one column tile),
    // taken times its step's power of two and added to the tile's sum in
    // binary32, rounded to nearest.
    constexpr int CH = NT == 1 ? 2 : 1;
    const uint32_t row_at = ring + g * 128, ch0 = ((2 * t) ^ g) << 4, ch1 = ((2 * t + 1) ^ g) << 4;
    const uint32_t sc_at = ring + 2048 + t * 64 + (g & 3) * 16 + (g >> 2) * 4;
    uint32_t use_at = 0;
    auto compute_unit = [&] {
      const uint8_t* w = smem + row_at + use_at;
      const uint8_t* sc = smem + sc_at + use_at;
      uint32_t sca[4], scb[4], at[NT];
      decode_scales(*reinterpret_cast<const uint32_t*>(sc), sca);
      decode_scales(*reinterpret_cast<const uint32_t*>(sc + 8), scb);
      float d[CH][NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) at[n] = xa[n] + s * xstep[n];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint4 wa = *reinterpret_cast<const uint4*>(w + (half ? ch1 : ch0));
        const uint4 wb = *reinterpret_cast<const uint4*>(w + 1024 + (half ? ch1 : ch0));
        const uint32_t ca[4] = {wa.x, wa.y, wa.z, wa.w}, cb[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 xv[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) xv[n] = *reinterpret_cast<const uint4*>(smem + at[n] + (half * 4 + j) * 16);
          uint32_t ha[4], hb[4];
          decode8(ca[j], ha);
          decode8(cb[j], hb);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            ha[q] = hmul2(ha[q], sca[half * 2 + j / 2]);
            hb[q] = hmul2(hb[q], scb[half * 2 + j / 2]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const bool fresh = half == 0 && j == 0;
            if (fresh) mma_f16_first(d[0][n], ha[0], hb[0], ha[1], hb[1], xv[n].x, xv[n].y);
            else mma_f16(d[0][n], ha[0], hb[0], ha[1], hb[1], xv[n].x, xv[n].y);
            if (fresh && CH == 2) mma_f16_first(d[CH - 1][n], ha[2], hb[2], ha[3], hb[3], xv[n].z, xv[n].w);
            else mma_f16(d[CH - 1][n], ha[2], hb[2], ha[3], hb[3], xv[n].z, xv[n].w);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 f = *reinterpret_cast<const float2*>(xscale + s * kMaxTokens + 8 * n + 2 * t);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          sum[n][q] = fmaf(CH == 2 ? d[0][n][q] + d[CH - 1][n][q] : d[0][n][q], q & 1 ? f.y : f.x, sum[n][q]);
      }
      use_at = use_at + kUnitBytes == D * kUnitBytes ? 0 : use_at + kUnitBytes;
    };
    // this warp's partial of virtual tile v
    auto flush = [&] {
      float* to = red + (warp * p.slots + (v - first_v)) * tile_floats;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t m = 8 * n + 2 * t + j;
          if (m < M) {
            to[m * kRedPitch + g] = sum[n][j];
            to[m * kRedPitch + g + 8] = sum[n][2 + j];
          }
        }
      clear();
    };
    clear();
    for (uint32_t i = ub; i < ue; ++i) {
      cp_async_wait<D - 1>();
      __syncwarp();  // every lane's part of the unit has landed
      compute_unit();
      __syncwarp();  // and is read before it is overwritten
      if (i + D < ue) load_next();
      cp_async_commit();
      if (++s == S || i + 1 == ue) {
        flush();
        if (s == S) {
          s = 0;
          ++v;
        }
      }
    }
    if (!pieces) break;
    __syncthreads();
    const WarpRuns runs(lane, S, U);
    for (uint32_t item = warp; item < V * NT; item += kWarps) {
      const uint32_t vt = item / NT, n = item % NT;
      float v[4];
      runs.sum(red, p.slots, M, vt, S, n, lane, v);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t m = 8 * n + 2 * q + (lane >> 4);
        if (m < M) acc[(vt * M + m) * 16 + (lane & 15)] += v[q];
      }
    }
    __syncthreads();
  }

  // ---- sum the warps' partials of each tile in warp order, then a cluster's CTAs'
  // in theirs; row tile i is finished by CTA i % ranks.  A warp takes 8 tokens of a
  // row tile at a time.
  if (ranks == 1) __syncthreads();
  else cluster_sync_all();  // all are done with their x
  const WarpRuns runs(lane, S, U);
  auto local_sum = [&](uint32_t vt, uint32_t n, float* v) {
    if (!pieces) {
      runs.sum(red, p.slots, M, vt, S, n, lane, v);
      return;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = acc[(vt * M + min(8 * n + 2 * q + (lane >> 4), M - 1)) * 16 + (lane & 15)];
  };
  const uint32_t row_tiles = V / MATS;
  // the other CTAs' sums of this one's tiles, over the staged x: [tile / ranks][CTA]
  const float* other = reinterpret_cast<const float*>(smem);
  const uint32_t others = ranks - 1;
  auto other_at = [&](uint32_t slot, uint32_t from, uint32_t mat, uint32_t m) {
    return (((slot * others + from) * MATS + mat) * M + m) * 16 + (lane & 15);
  };
  if constexpr (R != 1) {
    const uint32_t rounds = (row_tiles + others) >> rank_log;
    for (uint32_t item = warp; item < rounds * others * NT; item += kWarps) {
      const uint32_t n = item % NT, k = item / NT, slot = others > 1 ? k / others : k, r = k - slot * others;
      const uint32_t to_rank = r < rank ? r : r + 1, tile = (slot << rank_log) + to_rank;
      if (tile >= row_tiles) continue;
      const uint32_t to = map_to_rank(xs, to_rank), from = rank < to_rank ? rank : rank - 1;
#pragma unroll
      for (uint32_t mat = 0; mat < MATS; ++mat) {
        float v[4];
        local_sum(tile * MATS + mat, n, v);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t m = 8 * n + 2 * q + (lane >> 4);
          if (m < M) st_cluster_f32(to + 4 * other_at(slot, from, mat, m), v[q]);
        }
      }
    }
    cluster_sync_all();
  }
  const uint32_t mine = row_tiles > rank ? (row_tiles - rank + others) >> rank_log : 0;
  for (uint32_t item = warp; item < mine * NT; item += kWarps) {
    const uint32_t i = item / NT, n = item % NT, tile = (i << rank_log) + rank;
    float v[MATS][4];
#pragma unroll
    for (uint32_t mat = 0; mat < MATS; ++mat) {
      local_sum(tile * MATS + mat, n, v[mat]);
      if constexpr (R != 1) {  // in the order of the CTAs, this one's in its place
        float t[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) t[q] = rank == 0 ? v[mat][q] : 0.0f;
        for (uint32_t r = 0; r < others; ++r) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            t[q] += other[other_at(i, r, mat, min(8 * n + 2 * q + (lane >> 4), M - 1))];
            if (r + 1 == rank) t[q] += v[mat][q];
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) v[mat][q] = t[q];
      }
    }
    const uint32_t row = tile_base(t0 + tile) + (lane & 3) + 32 * ((lane & 15) >> 2);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t m = 8 * n + 2 * q + (lane >> 4);
      if (m >= M || row >= N) continue;
      float y = v[0][q] * alpha0;
      if (GATED) y = act_mul(y, v[MATS - 1][q] * alpha1, p.act);
      const int64_t at = static_cast<int64_t>(m) * p.ldy + row;
      if (p.out_fp32) static_cast<float*>(p.y)[at] = y;
      else static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(y);
    }
  }
}

struct GemvPlan {
  uint32_t grid = 0, ranks = 1, depth = 0, piece_steps = 0, slots = 0;
  uint32_t off_ring = 0, off_red = 0, off_acc = 0, off_scale = 0, smem = 0;
};

// Shared memory of a CTA that holds `share` row tiles and `steps` steps of K,
// staging `piece` of them at a time; false when it does not fit.
bool lay_out(GemvPlan& g, uint64_t share, uint64_t steps, uint64_t piece, uint64_t M, uint64_t mats) {
  const uint64_t V = share * mats;
  if (V * piece >= (1u << 24)) return false;  // 32-bit unit arithmetic in the kernel
  // a warp's run of ceil(V S / warps) units, begun anywhere, touches at most
  // ceil(V / warps) + 1 tiles, whatever S is
  const uint64_t slots = std::min(V, (V + kWarps - 1) / kWarps + 1);
  uint64_t x = kZeroBytes + M * token_bytes(static_cast<uint32_t>(piece));
  if (g.ranks > 1)  // the other CTAs' sums take its place
    x = std::max(x, (share + g.ranks - 1) / g.ranks * (g.ranks - 1) * mats * 16 * M * 4);
  x = (x + 127) / 128 * 128;
  const uint64_t ring = kWarps * g.depth * kUnitBytes, red = kWarps * slots * M * kRedPitch * 4;
  const uint64_t acc = steps > piece ? V * 16 * M * 4 : 0;
  const uint64_t total = x + ring + red + acc + piece * kMaxTokens * 4;
  g.piece_steps = static_cast<uint32_t>(piece);
  g.slots = static_cast<uint32_t>(slots);
  g.off_ring = static_cast<uint32_t>(x);
  g.off_red = static_cast<uint32_t>(x + ring);
  g.off_acc = static_cast<uint32_t>(x + ring + red);
  g.off_scale = static_cast<uint32_t>(x + ring + red + acc);
  g.smem = static_cast<uint32_t>(total);
  return total <= kSmemLimit;
}

// CTAs that share a row tile where there are SMs to spare.  A step of K costs a CTA
// about 0.04 us a weight and 0.025 us a token; the cluster itself 1.4 us (4 or 8
// CTAs) to 2.5 us (two).  us, one CTA (or what x needs) against a cluster: 16 x 64 x
// 8192 12.0 and 6.3 (8), 16 x 256 x 8192 12.2 and 7.4 (4), 1 x 256 x 8192 5.6 and 5.1
// (4), gated 1 x 1184 x 16384 12.9 and 11.4 (2); where the rule says no: 1 x 512 x
// 4096 4.6 and 4.9 (4), gated 8 x 1024 x 4096 7.6 and 8.6 (2).
uint32_t cluster_size(uint32_t tiles, uint32_t steps, uint32_t M, uint32_t mats, uint32_t sms) {
  const uint64_t work = static_cast<uint64_t>(steps) * (8 * mats + 5 * M);  // in 5 ns
  // (how many CTAs in clusters of that size run at once: those of 8 and 4 leave SMs
  // of their GPCs empty, and a second wave costs more than it gives)
  auto room = [&](uint32_t r) { return r == 8 ? sms / 2 : r == 4 ? sms * 7 / 8 : sms; };
  for (uint32_t r = 8; r > 1; r /= 2)
    if (static_cast<uint64_t>(tiles) * r <= room(r) && r <= steps) return work * (r - 1) / r > (r > 2 ? 280 : 500) ? r : 1;
  return 1;
}

// One CTA per SM with the whole x staged and four units in flight per warp;
// where that does not fit, two in flight; then clusters of two CTAs (or of what
// cluster_size says) with a part of K each; then x in pieces, and more CTAs with
// fewer tiles each.
GemvPlan plan_gemv(uint32_t tiles, uint32_t steps, uint32_t M, uint32_t mats, uint32_t sms) {
  GemvPlan g;
  const uint32_t first = cluster_size(tiles, steps, M, mats, sms);
  for (uint32_t waves = 1;; waves *= 2) {
    for (uint32_t n = 1; n <= steps; ++n) {
      bool more = false;
      for (uint32_t ranks = first; ranks <= std::max(first, 2u) && ranks <= steps; ranks *= 2) {
        const uint32_t groups = static_cast<uint32_t>(std::min<uint64_t>(tiles, static_cast<uint64_t>(std::max(1u, sms / ranks)) * waves));
        const uint32_t part = (steps + ranks - 1) / ranks, piece = (part + n - 1) / n;
        more = more || piece > 1;
        g.ranks = ranks;
        for (g.depth = 4; g.depth >= 2; g.depth -= 2)
          if (lay_out(g, (tiles + groups - 1) / groups, part, piece, M, mats)) {
            g.grid = groups * ranks;
            return g;
          }
      }
      if (!more) break;
    }
    if (static_cast<uint64_t>(sms) * waves >= static_cast<uint64_t>(tiles) * 2) break;
  }
  g.grid = 0;
  return g;
}

// Row tiles of N weight rows: 8 for each 128 rows, in the last 128 those that hold a row.
uint32_t row_tiles(int64_t N) { return static_cast<uint32_t>(N / 128 * 8 + std::min<int64_t>(8, (N % 128 + 3) / 4)); }

template <int NT, bool GATED, int D, int R>
cudaError_t launch_gemv(int dev, const GemvPlan& plan, cudaStream_t s, const GemvParams& p) {
  static PerContextCache<int> attr;
  int done = 0;
  const cudaError_t e = per_context(attr, dev, [](int* v) {
    *v = 1;
    return cudaFuncSetAttribute(gemv_kernel<NT, GATED, D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kSmemLimit));
  }, &done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = plan.smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = plan.ranks;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = plan.ranks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, gemv_kernel<NT, GATED, D, R>, p);
}

template <int NT, bool GATED, int D>
cudaError_t launch_gemv(int dev, const GemvPlan& plan, cudaStream_t s, const GemvParams& p) {
  if (plan.ranks == 1) return launch_gemv<NT, GATED, D, 1>(dev, plan, s, p);
  if (plan.ranks == 2) return launch_gemv<NT, GATED, D, 2>(dev, plan, s, p);
  return launch_gemv<NT, GATED, D, 0>(dev, plan, s, p);
}

template <int NT, bool GATED>
cudaError_t launch_gemv(int dev, const GemvPlan& plan, cudaStream_t s, const GemvParams& p) {
  return plan.depth == 4 ? launch_gemv<NT, GATED, 4>(dev, plan, s, p) : launch_gemv<NT, GATED, 2>(dev, plan, s, p);
}

nvfp4_status gemv_impl(const char* fn, const void* x, int64_t M, int64_t K, int64_t ldx, int mats,
                       const void* const* codes, const void* const* scales, const float* const* alpha, int64_t N,
                       int act, void* y, int64_t ldy, int out_dtype, void* stream) {
  if (!x || !y) return set_error(NVFP4_ERR_INVALID_ARG, "%s: null pointer argument", fn);
  for (int i = 0; i < mats; ++i)
    if (!codes[i] || !scales[i] || !alpha[i]) return set_error(NVFP4_ERR_INVALID_ARG, "%s: null pointer argument", fn);
  if (M < 1 || M > kMaxTokens)
    return set_error(NVFP4_ERR_INVALID_ARG, "%s: need 1 <= M <= %d (M=%lld); quantize more rows and use a GEMM", fn,
                     kMaxTokens, (long long)M);
  if (N < 1 || N > (1ll << 30) || K < 64 || K % 64 != 0 || K > (1ll << 24))
    return set_error(NVFP4_ERR_INVALID_ARG,
                     "%s: need 1 <= N <= 2^30 and K a positive multiple of 64 up to 2^24 (N=%lld K=%lld)", fn,
                     (long long)N, (long long)K);
  if (ldx < K || ldx > (int64_t{1} << 40)) return set_error(NVFP4_ERR_INVALID_ARG, "%s: need K <= ldx <= 2^40", fn);
  if (ldy < N || ldy > (int64_t{1} << 40)) return set_error(NVFP4_ERR_INVALID_ARG, "%s: need N <= ldy <= 2^40", fn);
  if (out_dtype != NVFP4_OUT_BF16 && out_dtype != NVFP4_OUT_FP32)
    return set_error(NVFP4_ERR_INVALID_ARG, "%s: unknown out_dtype %d", fn, out_dtype);
  if (mats == 2 && act != NVFP4_ACT_SILU && act != NVFP4_ACT_GELU)
    return set_error(NVFP4_ERR_INVALID_ARG, "%s: unknown act %d", fn, act);
  for (int i = 0; i < mats; ++i)
    if (!aligned16(codes[i]) || !aligned16(scales[i]) || (reinterpret_cast<uintptr_t>(alpha[i]) & 3u))
      return set_error(NVFP4_ERR_INVALID_ARG, "%s: misaligned buffer", fn);
  if ((reinterpret_cast<uintptr_t>(x) & 1u) ||
      (reinterpret_cast<uintptr_t>(y) & (out_dtype == NVFP4_OUT_FP32 ? 3u : 1u)))
    return set_error(NVFP4_ERR_INVALID_ARG, "%s: misaligned buffer", fn);
  int dev = 0, sms = 0;
  nvfp4_status st = check_device(&dev, &sms);
  if (st != NVFP4_OK) return st;

  GemvParams p = {};
  p.x = static_cast<const uint16_t*>(x);
  p.ldx = ldx;
  for (int i = 0; i < 2; ++i) {
    const int j = std::min(i, mats - 1);
    p.codes[i] = static_cast<const uint8_t*>(codes[j]);
    p.scales[i] = static_cast<const uint8_t*>(scales[j]);
    p.alpha[i] = alpha[j];
  }
  p.y = y;
  p.ldy = ldy;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.kgroups = static_cast<uint32_t>(K / 64);
  p.act = act;
  p.out_fp32 = out_dtype == NVFP4_OUT_FP32;
  p.x_vec = aligned16(x) && ldx % 8 == 0;
  const uint32_t tiles = row_tiles(N);
  p.all_steps = static_cast<uint32_t>((K + kStepK - 1) / kStepK);
  const GemvPlan plan = plan_gemv(tiles, p.all_steps, static_cast<uint32_t>(M), static_cast<uint32_t>(mats),
                                  static_cast<uint32_t>(sms));
  if (!plan.grid) return set_error(NVFP4_ERR_INVALID_ARG, "%s: shape does not fit", fn);
  const uint32_t groups = plan.grid / plan.ranks;
  p.share = tiles / groups;
  p.share_rest = tiles % groups;
  p.ranks = plan.ranks;
  while ((1u << p.rank_log) < p.ranks) ++p.rank_log;
  p.off_ring = plan.off_ring;
  p.piece_steps = plan.piece_steps;
  p.slots = plan.slots;
  p.off_red = plan.off_red;
  p.off_acc = plan.off_acc;
  p.off_scale = plan.off_scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (mats == 1) e = M <= 8 ? launch_gemv<1, false>(dev, plan, s, p) : launch_gemv<2, false>(dev, plan, s, p);
  else e = M <= 8 ? launch_gemv<1, true>(dev, plan, s, p) : launch_gemv<2, true>(dev, plan, s, p);
  if (e != cudaSuccess) return cuda_status(e, "gemv_kernel launch");
  return NVFP4_OK;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

int nvfp4_testing_gemv_plan(int64_t M, int64_t N, int64_t K, int weights, int sms, int plan[5]) {
  if (M < 1 || M > kMaxTokens || N < 1 || N > (1ll << 30) || K < 64 || K % 64 != 0 || K > (1ll << 24) || weights < 1 ||
      weights > 2 || sms < 1)
    return 0;
  const uint32_t steps = static_cast<uint32_t>((K + kStepK - 1) / kStepK);
  const GemvPlan g = plan_gemv(row_tiles(N), steps, static_cast<uint32_t>(M), static_cast<uint32_t>(weights),
                               static_cast<uint32_t>(sms));
  const uint32_t part = (steps + g.ranks - 1) / g.ranks;
  plan[0] = static_cast<int>(g.grid);
  plan[1] = static_cast<int>(g.ranks);
  plan[2] = static_cast<int>(g.piece_steps);
  plan[3] = static_cast<int>((part + g.piece_steps - 1) / g.piece_steps);
  plan[4] = static_cast<int>(g.depth);
  return g.grid > 0;
}

nvfp4_status nvfp4_gemv(const void* x, int64_t M, int64_t K, int64_t ldx, const void* w_codes, const void* w_scales,
                        const float* w_global, int64_t N, void* y, int64_t ldy, int out_dtype, void* stream) {
  return gemv_impl("nvfp4_gemv", x, M, K, ldx, 1, &w_codes, &w_scales, &w_global, N, 0, y, ldy, out_dtype, stream);
}

nvfp4_status nvfp4_gemv_gated(const void* x, int64_t M, int64_t K, int64_t ldx, const void* gate_codes,
                              const void* gate_scales, const float* gate_global, const void* up_codes,
                              const void* up_scales, const float* up_global, int64_t N, int act, void* h, int64_t ldh,
                              int out_dtype, void* stream) {
  const void* codes[2] = {gate_codes, up_codes};
  const void* scales[2] = {gate_scales, up_scales};
  const float* alpha[2] = {gate_global, up_global};
  return gemv_impl("nvfp4_gemv_gated", x, M, K, ldx, 2, codes, scales, alpha, N, act, h, ldh, out_dtype, stream);
}

}  // extern "C"
