// fp8_block_kernel.cuh -- appending K/V to the FP8 cache that attention reads in place (sm_100a).
//
// The cache holds e4m3 codes and, for every block of 16 tokens of a page and every head, one
// power-of-two scale for K and one for V (e8m0: the byte b stands for 2^(b - 127)):
//   value = code * 2^(b - 127).
// For a block whose largest finite magnitude is a, the scale is the smallest power of two with
// a / scale <= 448, its exponent kept in [-100, 119]; code = e4m3(x / scale), rounded to nearest
// even, saturated at 448; a value that is not finite is stored as NaN and does not count for a.
// With a power of two the division is exact, so the code's rounding is the only one, and a row
// that stays while its block's scale grows is shifted exactly (but for values that fall under
// e4m3's smallest normal, 2^-6 of the scale).
//
// Blocks are 16 tokens because page sizes are multiples of 16: a block never crosses a page, and
// a tile of 128 keys holds 8 whole blocks.  Chunks are not multiples of 16 long, so an append may
// start or end inside a block.  The block's other live rows -- logical tokens below the end of
// the wavefront -- are kept: decoded, counted for the new scale and coded again.  Rows past the end
// are dead, hold anything, and are left as they were.
//
// Two warps per (block, head, tensor), 8 rows each: the rows sit in registers as fp32 (D/16 lanes per
// row, as in the bf16 pass), so the block is read once; the scale is two warp reductions and a
// barrier away.  A CTA takes one block's heads; the 16 tokens' cos and sin wait in shared memory for
// all of them, and each head's values are asked for while the one before is worked on.  Heads of K and
// of V alternate, and at any time half the warp pairs work on K, so that arithmetic (K) and plain
// copying (V) share the SM.
//
// On 23 400 tokens of 12 heads of 128, 3 axes: 50.6 us, 216 MB, 4.3 TB/s (one chunk of 4680: 10.0 us);
// 51.4 with all K before all V,
// 65 with one warp for all 16 rows (64 values a lane).  Bound by how loads and arithmetic overlap: the
// issue slots are at 41 % and HBM at 0.65 of a copy.  Neither more warps (3 CTAs an SM: 53.1) nor
// more heads asked for ahead (2 through shared memory 53.1, 3 54.9, 5 62.9) nor 4 warps to a block
// (55.7) did better.
#pragma once

#include <cuda_fp8.h>

#include "norm_rope_kernel.cuh"

namespace wfk {

constexpr int kFp8BlockTokens = 16;
constexpr int kFp8AppendPairs = kNormRopeThreads / 64;     // warp pairs of a CTA
constexpr int kFp8AppendCtas = 2;                          // per SM, at least
constexpr int kScaleExpMin = -100, kScaleExpMax = 119;

struct Fp8BlockAppendParams {
  RowSet set[2];              // K (normed and turned) and V; dst unused
  uint8_t* codes[2];          // pools [pages * page_size][H][D]
  uint8_t* scale[2];          // [pages * page_size / 16][H]
  NormRope rule;
  int weight_per_head;
  int token0, tokens, live;   // appended: [token0, token0 + tokens); live: [0, live)
  int H, page_size, num_pages;
  int items;                  // (head, tensor) rows per CTA: 2 H or a multiple of 4
  const int* pt_row;
  int* status;
};

// 4 e4m3 codes (code i in byte i) of 4 values already divided by the scale.
__device__ __forceinline__ uint32_t encode4(float4 x) {
  uint32_t c;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(c)
      : "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w));
  return c;
}

// The largest of m >= 0, |a| and |b|; NaN when one of them is.
__device__ __forceinline__ float max_abs(float m, float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

__device__ __forceinline__ float4 decode4(uint32_t c, float scale) {
  const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
      static_cast<__nv_fp8x2_storage_t>(c & 0xFFFFu), __NV_E4M3)));
  const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
      static_cast<__nv_fp8x2_storage_t>(c >> 16), __NV_E4M3)));
  return make_float4(a.x * scale, a.y * scale, b.x * scale, b.y * scale);
}

// Exponent of the smallest power of two that brings a >= 0 (finite) to 448 = 1.75 2^8 or less.
__device__ __forceinline__ int scale_exponent(float a) {
  const uint32_t b = __float_as_uint(a);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(kScaleExpMin, min(kScaleExpMax, e));      // a subnormal or zero a: the least
}

__device__ __forceinline__ float exp2_int(int e) {     // 2^e, e in [-126, 127]
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// grid: (blocks of 16 tokens, runs of p.items (head, tensor) rows).
template <int D, int kMode>
__global__ void __launch_bounds__(kNormRopeThreads, kFp8AppendCtas)
    wf_fp8_block_append_kernel(const __grid_constant__ Fp8BlockAppendParams p) {
  constexpr int LPR = D / 16, RPS = 32 / LPR, STEPS = kFp8BlockTokens / 2 / RPS;
  constexpr int MAXP = D / 2;                        // pairs
  // (cos, cos, sin, sin) of two pairs of the block's tokens; a row is padded by one float4 so that
  // the rows of a warp step start on different banks
  constexpr int CSP = MAXP / 2 + 1;
  __shared__ float4 angles[kMode != kRopeNone ? kFp8BlockTokens * CSP : 1];
  __shared__ float stage_all[kMode == kRopeSplitPartial ? kNormRopeThreads * 16 : 1];
  __shared__ float tops[2][kFp8AppendPairs][2];
  wait_for_previous();
  launch_next();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* const stage = stage_all + (kMode == kRopeSplitPartial ? warp * 512 : 0);
  const int sub = lane % LPR;
  const int pair = warp >> 1, half = warp & 1;
  const int r0 = half * 8 + lane / LPR;              // this lane's row of step i: r0 + i RPS
  const int blk = p.token0 / kFp8BlockTokens + static_cast<int>(blockIdx.x);
  const int tok0 = blk * kFp8BlockTokens;
  // rows of the block: new ones [n0, n1), others live below n_live
  const int n0 = max(p.token0 - tok0, 0);
  const int n1 = min(p.token0 + p.tokens - tok0, kFp8BlockTokens);
  const int n_live = min(p.live - tok0, kFp8BlockTokens);
  const bool keeps = n0 > 0 || n1 < n_live;          // live rows that stay
  const int hh0 = static_cast<int>(blockIdx.y) * p.items;
  const int hh1 = min(hh0 + p.items, 2 * p.H);

  uint4 lo[STEPS], hi[STEPS];
  const bool whole = n1 - n0 == kFp8BlockTokens;
  // The CTA's rows alternate between K and V, for every second round of the pairs the other way round.
  const auto which_of = [&](int hh) { return (hh ^ (hh >> 2)) & 1; };
  const auto load = [&](int hh) {
    const int which = which_of(hh), h = hh >> 1;
    const RowSet& s = p.set[which];
    const __nv_bfloat16* src =
        s.src + static_cast<int64_t>(tok0 + r0 - p.token0) * s.stride + (h * D + 8 * sub);
#pragma unroll
    for (int i = 0; i < STEPS; ++i, src += RPS * s.stride) {
      const int r = r0 + i * RPS;
      if (whole || (r >= n0 && r < n1)) {
        lo[i] = *reinterpret_cast<const uint4*>(src);
        hi[i] = *reinterpret_cast<const uint4*>(src + D / 2);
      } else {
        lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
      }
    }
  };
  if (hh0 + pair < hh1) load(hh0 + pair);
  const int pg = p.pt_row[tok0 / p.page_size];
  if (pg < 0 || pg >= p.num_pages) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, 5 /* WF_ERR_PAGE_OOB */);
    return;
  }
  if (kMode != kRopeNone) {
    // a block with a position off the table is left as it was: its codes and scale belong together
    bool bad = false;
    // split partial: slots by pair; else by what the lanes turn, slots past the pairs stay as they are
    constexpr int per_row = MAXP / 2;
    for (int i = threadIdx.x; i < kFp8BlockTokens * per_row; i += kNormRopeThreads) {
      const int r = i / per_row, j = i - r * per_row;
      float4 cs = make_float4(1.f, 1.f, 0.f, 0.f);
      if (2 * j < p.rule.pairs && r >= n0 && r < n1) {
        int pos[3];
        if (load_positions(p.rule, tok0 + r - p.token0, pos)) cs = load_pairs(p.rule, pos, 2 * j);
        else bad = true;
      }
      angles[r * CSP + j] = cs;
    }
    if (__syncthreads_or(bad)) {
      if (threadIdx.x == 0) atomicCAS(p.status, 0, 9 /* WF_ERR_POSITION */);
      return;
    }
  }
  const int64_t prow = static_cast<int64_t>(pg) * p.page_size + tok0 % p.page_size;
  const int64_t cstep = static_cast<int64_t>(p.H) * D * RPS;       // from step to step
  const int64_t code0 = (prow + r0) * p.H * D + 8 * sub;
  const int64_t scale0 = prow / kFp8BlockTokens * p.H;
  int turn = 0;
#pragma unroll 1
  for (int hh = hh0 + pair; hh < hh1; hh += kFp8AppendPairs, turn ^= 1) {
    const int which = which_of(hh), h = hh >> 1;
    uint8_t* const codes = p.codes[which] + code0 + h * D;
    uint8_t* const scale = p.scale[which] + scale0 + h;
    Row x[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) unpack_row<kMode>(lo[i], hi[i], x[i]);
    if (hh + kFp8AppendPairs < hh1) load(hh + kFp8AppendPairs);
    if (which == 0 && (kMode != kRopeNone || p.rule.norm)) {
      Row w;
      load_weight<D, kMode>(p.set[0].weight, p.weight_per_head ? static_cast<int64_t>(h) * D : 0,
                            sub, w);
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const float4* row = angles + (r0 + i * RPS) * CSP;
        const auto at = [&](int j) {
          if (kMode != kRopeSplitPartial) return row[lane_pair<D, kMode>(sub, j, MAXP) / 2];
          const int pr = lane_pair<D, kMode>(sub, j, p.rule.pairs);
          return pr >= 0 ? row[pr / 2] : make_float4(1.f, 1.f, 0.f, 0.f);
        };
        // a row that is not new is zeros here, and a norm's rsqrt(0 + eps) may be infinite: the
        // row is replaced below
        norm_rope_row<D, kMode>(x[i], p.rule, sub, w, at, stage);
      }
    }
    if (!whole) {                                    // a block at an end of the append
      const float old_scale =
          keeps ? __uint_as_float(static_cast<uint32_t>(*scale) << 23) : 0.f;
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int r = r0 + i * RPS;
        if (r >= n0 && r < n1) continue;
        uint2 c0 = make_uint2(0, 0), c1 = c0;
        if (r < n_live) {
          c0 = *reinterpret_cast<const uint2*>(codes + i * cstep);
          c1 = *reinterpret_cast<const uint2*>(codes + i * cstep + D / 2);
        }
        set_channels4<kMode>(x[i], 0, decode4(c0.x, old_scale));
        set_channels4<kMode>(x[i], 1, decode4(c0.y, old_scale));
        set_channels4<kMode>(x[i], 2, decode4(c1.x, old_scale));
        set_channels4<kMode>(x[i], 3, decode4(c1.y, old_scale));
      }
    }
    float top = 0.f;                                 // NaN or infinite when a value is
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        top = max_abs(top, x[i].u[j].x, x[i].u[j].y);
        top = max_abs(top, x[i].v[j].x, x[i].v[j].y);
      }
    // magnitudes order as their bit patterns, infinity above all and NaN above that
    uint32_t wtop = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
    if (wtop >= 0x7F800000u) {
      top = 0.f;
      auto clean = [&](float& v) {
        const float m = fabsf(v);
        if (m < INFINITY) top = fmaxf(top, m);
        else v = __uint_as_float(0x7FFFFFFFu);
      };
#pragma unroll
      for (int i = 0; i < STEPS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          clean(x[i].u[j].x);
          clean(x[i].u[j].y);
          clean(x[i].v[j].x);
          clean(x[i].v[j].y);
        }
      wtop = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
    }
    if (lane == 0) tops[turn][pair][half] = __uint_as_float(wtop);
    // the pair's barrier; the other buffer is next turn's, so this one is not overwritten before the
    // pair has met again
    asm volatile("bar.sync %0, 64;" ::"r"(1 + pair) : "memory");
    top = fmaxf(tops[turn][pair][0], tops[turn][pair][1]);
    const int e = scale_exponent(top);
    const float inv = exp2_int(-e);
    const float2 inv2 = make_float2(inv, inv);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int r = r0 + i * RPS;
      if (whole || r < n1 || r < n_live) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[i].u[j] = __fmul2_rn(x[i].u[j], inv2);
          x[i].v[j] = __fmul2_rn(x[i].v[j], inv2);
        }
        *reinterpret_cast<uint2*>(codes + i * cstep) =
            make_uint2(encode4(channels4<kMode>(x[i], 0)), encode4(channels4<kMode>(x[i], 1)));
        *reinterpret_cast<uint2*>(codes + i * cstep + D / 2) =
            make_uint2(encode4(channels4<kMode>(x[i], 2)), encode4(channels4<kMode>(x[i], 3)));
      }
    }
    if (half == 0 && lane == 0) *scale = static_cast<uint8_t>(e + 127);
  }
}

}  // namespace wfk
