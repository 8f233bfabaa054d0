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
// One warp per (block, head, tensor): the 16 rows sit in registers as fp32 (D/16 lanes per row, as
// in the bf16 pass), so the block is read once and its scale is one warp reduction away.  A CTA
// takes one block's heads; the 16 tokens' cos and sin wait in shared memory for all of them.
#pragma once

#include <cuda_fp8.h>

#include "norm_rope_kernel.cuh"

namespace wfk {

constexpr int kFp8BlockTokens = 16;
constexpr int kScaleExpMin = -100, kScaleExpMax = 119;

struct Fp8BlockAppendParams {
  RowSet set[2];              // K (normed and turned) and V; dst unused
  uint8_t* codes[2];          // pools [pages * page_size][H][D]
  uint8_t* scale[2];          // [pages * page_size / 16][H]
  NormRope rule;
  int weight_per_head;
  int token0, tokens, live;   // appended: [token0, token0 + tokens); live: [0, live)
  int H, page_size, num_pages;
  int items;                  // (head, tensor) rows per CTA
  const int* pt_row;
  int* status;
};

// 4 e4m3 codes (code i in byte i) of 4 values already divided by the scale.
__device__ __forceinline__ uint32_t encode4(const float* x) {
  const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
  return (a & 0xFFFFu) | (b << 16);
}

__device__ __forceinline__ void decode4(uint32_t c, float scale, float* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((c >> (16 * i)) & 0xFFFFu), __NV_E4M3));
    const float2 f = __half22float2(h);
    x[2 * i] = f.x * scale;
    x[2 * i + 1] = f.y * scale;
  }
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

// grid: (blocks of 16 tokens, runs of p.items (head, tensor) rows; K rows first).
template <int D, int kMode>
__global__ void __launch_bounds__(kNormRopeThreads, 2)
    wf_fp8_block_append_kernel(const __grid_constant__ Fp8BlockAppendParams p) {
  constexpr int LPR = D / 16, RPS = 32 / LPR, STEPS = kFp8BlockTokens / RPS;
  constexpr int MAXP = D / 2;                        // pairs
  // cos, sin of the block's tokens, as float4 (two pairs); a row is padded by one float4 so that
  // the rows of a warp step start on different banks
  constexpr int CSP = MAXP / 2 + 1;
  __shared__ float4 angles[kMode != kRopeNone ? kFp8BlockTokens * CSP : 1];
  __shared__ float stage_all[kMode == kRopeSplitPartial ? kNormRopeThreads * 16 : 1];
  float* const stage = stage_all + (kMode == kRopeSplitPartial ? (threadIdx.x >> 5) * 512 : 0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % LPR, rsub = lane / LPR;
  const int blk = p.token0 / kFp8BlockTokens + static_cast<int>(blockIdx.x);
  const int tok0 = blk * kFp8BlockTokens;
  // rows of the block: new ones [n0, n1), others live below n_live
  const int n0 = max(p.token0 - tok0, 0);
  const int n1 = min(p.token0 + p.tokens - tok0, kFp8BlockTokens);
  const int n_live = min(p.live - tok0, kFp8BlockTokens);
  const bool keeps = n0 > 0 || n1 < n_live;          // live rows that stay
  const int pg = __ldg(p.pt_row + tok0 / p.page_size);
  if (pg < 0 || pg >= p.num_pages) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, 5 /* WF_ERR_PAGE_OOB */);
    return;
  }
  if (kMode != kRopeNone) {
    // a block with a position off the table is left as it was: its codes and scale belong together
    bool bad = false;
    const int per_row = p.rule.pairs / 2;
    for (int i = threadIdx.x; i < kFp8BlockTokens * per_row; i += kNormRopeThreads) {
      const int r = i / per_row, j = i - r * per_row;
      float4 cs = make_float4(1.f, 0.f, 1.f, 0.f);
      if (r >= n0 && r < n1) {
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
  const int64_t cstep = static_cast<int64_t>(p.H) * D;
  const int hh0 = static_cast<int>(blockIdx.y) * p.items;
  const int hh1 = min(hh0 + p.items, 2 * p.H);
  for (int hh = hh0 + warp; hh < hh1; hh += kNormRopeThreads / 32) {
    const int which = hh >= p.H ? 1 : 0, h = hh - which * p.H;
    uint8_t* const codes = p.codes[which] + (prow * p.H + h) * D + 8 * sub;
    uint8_t* const scale = p.scale[which] + prow / kFp8BlockTokens * p.H + h;
    const RowSet& s = p.set[which];
    uint4 lo[STEPS], hi[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int r = i * RPS + rsub;
      lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
      if (r >= n0 && r < n1) {
        const __nv_bfloat16* src = s.src + static_cast<int64_t>(tok0 + r - p.token0) * s.stride +
                                   static_cast<int64_t>(h) * D + 8 * sub;
        lo[i] = *reinterpret_cast<const uint4*>(src);
        hi[i] = *reinterpret_cast<const uint4*>(src + D / 2);
      }
    }
    uint4 wl = make_uint4(kOnes, kOnes, kOnes, kOnes), wh = wl;
    if (s.weight != nullptr) {
      const __nv_bfloat16* wp = s.weight + (p.weight_per_head ? h * D : 0) + 8 * sub;
      wl = __ldg(reinterpret_cast<const uint4*>(wp));
      wh = __ldg(reinterpret_cast<const uint4*>(wp + D / 2));
    }
    float x[STEPS][16];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      unpack8(lo[i], x[i]);
      unpack8(hi[i], x[i] + 8);
    }
    if (which == 0 && (kMode != kRopeNone || p.rule.norm)) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        LaneAngles<kMode> a;
        const float4* row = angles + (i * RPS + rsub) * CSP;
#pragma unroll
        for (int j = 0; j < LaneAngles<kMode>::N; ++j) {
          const int pr = lane_pair<D, kMode>(sub, j, p.rule.pairs);
          a.cs[j] = pr >= 0 ? row[pr / 2] : make_float4(1.f, 0.f, 1.f, 0.f);
        }
        // a row that is not new is zeros here; without a norm it stays zeros, and a norm's
        // rsqrt(0 + eps) may be infinite: it is replaced, or not stored, below
        norm_rope_row<D, kMode>(x[i], p.rule, sub, wl, wh, a, stage);
      }
    }
    if (n0 > 0 || n1 < kFp8BlockTokens) {            // a block at an end of the append
      const float old_scale =
          keeps ? __uint_as_float(static_cast<uint32_t>(*scale) << 23) : 0.f;
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int r = i * RPS + rsub;
        if (r >= n0 && r < n1) continue;
#pragma unroll
        for (int j = 0; j < 16; ++j) x[i][j] = 0.f;
        if (r < n_live) {
          const uint2 c0 = *reinterpret_cast<const uint2*>(codes + r * cstep);
          const uint2 c1 = *reinterpret_cast<const uint2*>(codes + r * cstep + D / 2);
          decode4(c0.x, old_scale, x[i]);
          decode4(c0.y, old_scale, x[i] + 4);
          decode4(c1.x, old_scale, x[i] + 8);
          decode4(c1.y, old_scale, x[i] + 12);
        }
      }
    }
    float top = 0.f;
    float2 odd = make_float2(0.f, 0.f);              // NaN once a value is not finite
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        top = max3(top, fabsf(x[i][j]), fabsf(x[i][j + 1]));
        odd = __ffma2_rn(make_float2(x[i][j], x[i][j + 1]), make_float2(0.f, 0.f), odd);
      }
    if (__any_sync(0xffffffffu, isnan(odd.x + odd.y))) {
      top = 0.f;
#pragma unroll
      for (int i = 0; i < STEPS; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float m = fabsf(x[i][j]);
          if (m < INFINITY) top = fmaxf(top, m);
          else x[i][j] = __uint_as_float(0x7FFFFFFFu);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = scale_exponent(top);
    const float inv = exp2_int(-e);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int r = i * RPS + rsub;
      if (r < n1 || r < n_live) {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[i][j] *= inv;
        *reinterpret_cast<uint2*>(codes + r * cstep) = make_uint2(encode4(x[i]), encode4(x[i] + 4));
        *reinterpret_cast<uint2*>(codes + r * cstep + D / 2) =
            make_uint2(encode4(x[i] + 8), encode4(x[i] + 12));
      }
    }
    if (lane == 0) *scale = static_cast<uint8_t>(e + 127);
  }
}

}  // namespace wfk
