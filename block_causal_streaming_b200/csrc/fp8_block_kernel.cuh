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
// One warp per (block, head, tensor): the 16 rows sit in registers as fp32 (D/8 lanes per row,
// as in the bf16 pass), so the block is read once and its scale is one warp reduction away.
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

template <int D, int kMode>
__global__ void __launch_bounds__(kNormRopeThreads)
    wf_fp8_block_append_kernel(const __grid_constant__ Fp8BlockAppendParams p) {
  constexpr int LPR = D / 8, RPS = 32 / LPR, STEPS = kFp8BlockTokens / RPS;
  const int lane = threadIdx.x & 31;
  const int sub = lane % LPR, rsub = lane / LPR;
  const int b0 = p.token0 / kFp8BlockTokens;
  const int nb = (p.token0 + p.tokens - 1) / kFp8BlockTokens - b0 + 1;
  const int64_t items = static_cast<int64_t>(nb) * 2 * p.H;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kNormRopeThreads / 32);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kNormRopeThreads / 32) +
                    (threadIdx.x >> 5);
       it < items; it += warps) {
    // heads fastest: the warps of a block share the tokens' cos and sin in L1
    const int blk = b0 + static_cast<int>(it / (2 * p.H));
    const int hh = static_cast<int>(it % (2 * p.H));
    const int which = hh >= p.H ? 1 : 0, h = hh - which * p.H;
    const int tok0 = blk * kFp8BlockTokens;
    const int pg = __ldg(p.pt_row + tok0 / p.page_size);
    if (pg < 0 || pg >= p.num_pages) {
      if (lane == 0) atomicCAS(p.status, 0, 5 /* WF_ERR_PAGE_OOB */);
      continue;
    }
    const int64_t prow = static_cast<int64_t>(pg) * p.page_size + tok0 % p.page_size;
    uint8_t* const codes = p.codes[which] + (prow * p.H + h) * D + 4 * sub;
    uint8_t* const scale = p.scale[which] + prow / kFp8BlockTokens * p.H + h;
    const RowSet& s = p.set[which];
    const int64_t cstep = static_cast<int64_t>(p.H) * D;

    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    if (s.weight != nullptr) {
      const __nv_bfloat16* wp = s.weight + (p.weight_per_head ? h * D : 0) + 4 * sub;
      unpack4(__ldg(reinterpret_cast<const uint2*>(wp)), w);
      unpack4(__ldg(reinterpret_cast<const uint2*>(wp + D / 2)), w + 4);
    }
    // rows of the block: new ones [n0, n1), others live below `live`
    const int n0 = max(p.token0 - tok0, 0);
    const int n1 = min(p.token0 + p.tokens - tok0, kFp8BlockTokens);
    const int n_live = min(p.live - tok0, kFp8BlockTokens);
    float old_scale = 0.f;
    if (n0 > 0 || n1 < n_live) old_scale = __uint_as_float(static_cast<uint32_t>(*scale) << 23);

    float x[STEPS][8];
    bool skip = false;                       // a new row has a position off the table
    if (kMode != kRopeNone && which == 1) {
      for (int i = lane; i < (n1 - n0) * p.rule.num_axes; i += 32) {
        const int at = __ldg(p.rule.positions +
                             static_cast<int64_t>(tok0 + n0 - p.token0) * p.rule.num_axes + i);
        skip |= at < 0 || at >= p.rule.table_rows;
      }
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int r = i * RPS + rsub;
      const bool fresh = r >= n0 && r < n1;
      uint2 lo = make_uint2(0, 0), hi = make_uint2(0, 0);
      if (fresh) {
        const __nv_bfloat16* src = s.src + static_cast<int64_t>(tok0 + r - p.token0) * s.stride +
                                   static_cast<int64_t>(h) * D + 4 * sub;
        lo = *reinterpret_cast<const uint2*>(src);
        hi = *reinterpret_cast<const uint2*>(src + D / 2);
      }
      unpack4(lo, x[i]);
      unpack4(hi, x[i] + 4);
      if (!fresh && r < n_live) {
        decode4(*reinterpret_cast<const uint32_t*>(codes + r * cstep), old_scale, x[i]);
        decode4(*reinterpret_cast<const uint32_t*>(codes + r * cstep + D / 2), old_scale,
                x[i] + 4);
      }
    }
    if (which == 0 && (kMode != kRopeNone || p.rule.norm)) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int r = i * RPS + rsub;
        const bool fresh = r >= n0 && r < n1;
        LaneAngles<kMode> a;
        if (fresh) {
          skip |= !load_angles<D, kMode>(p.rule, tok0 + r - p.token0, sub, a);
        } else {
#pragma unroll
          for (int j = 0; j < LaneAngles<kMode>::N; ++j) a.cs[j] = make_float2(1.f, 0.f);
        }
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[i][j];
        norm_rope_row<D, kMode>(y, p.rule, sub, w, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] = fresh ? y[j] : x[i][j];
      }
    }
    // a block with such a row is left as it was: its codes and scale belong together
    if (kMode != kRopeNone && __any_sync(0xffffffffu, skip)) {
      if (lane == 0) atomicCAS(p.status, 0, 9 /* WF_ERR_POSITION */);
      continue;
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float m = fabsf(x[i][j]);
        const bool finite = m < INFINITY;              // false for NaN
        if (!finite) x[i][j] = __uint_as_float(0x7FFFFFFFu);
        top = fmaxf(top, finite ? m : 0.f);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = scale_exponent(top);
    const float inv = exp2_int(-e);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int r = i * RPS + rsub;
      if (r < n1 || r < n_live) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[i][j] * inv;
        *reinterpret_cast<uint32_t*>(codes + r * cstep) = encode4(y);
        *reinterpret_cast<uint32_t*>(codes + r * cstep + D / 2) = encode4(y + 4);
      }
    }
    if (lane == 0) *scale = static_cast<uint8_t>(e + 127);
  }
}

}  // namespace wfk
