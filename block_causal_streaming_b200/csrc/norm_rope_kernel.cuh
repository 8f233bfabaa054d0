// norm_rope_kernel.cuh -- norms of queries and keys for each head with the position rotation in
// the same pass, alone or on the way into the bf16 pages (sm_100a).
//
// For one (token, head) row x of D values:
//   y = x * rsqrt(mean(x^2) + eps) * w          (without a norm: y = x)
//   pair i < pairs turns by the angle of the token's position along the pair's axis:
//     (y_a, y_b) <- (y_a cos - y_b sin, y_a sin + y_b cos)
//   with (a, b) = (2i, 2i + 1) (interleaved) or (i, pairs + i); channels from 2 pairs on stay.
// Everything between the bf16 load and the one rounding of the result is fp32.  cos and sin come
// from the caller's table (fp32, [position][pair]), so far positions keep the caller's accuracy.
//
// Row layout.  D / 8 lanes share a row; lane `sub` holds channels [4 sub, 4 sub + 4) and
// [D/2 + 4 sub, ... + 4).  Interleaved pairs and the halves of a full split rotation then both sit
// inside one lane; only a partial split rotation (2 pairs < D) exchanges values between lanes.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace wfk {

constexpr int kNormRopeThreads = 256;

// How the pairs of a row are laid out.
enum RopeMode { kRopeNone = 0, kRopeInterleaved = 1, kRopeSplit = 2, kRopeSplitPartial = 3 };

struct NormRope {
  const float2* table;        // [table_rows][pairs] (cos, sin)
  const int* positions;       // [tokens][num_axes]
  int table_rows, pairs, num_axes;
  int axis1, axis2;           // first pair of axis 1 and of axis 2 (`pairs` when there is none)
  int norm;
  float eps;
};

// cos and sin of the pairs a lane turns, for one token.  N: 4 pairs, or 8 in kRopeSplitPartial
// (both groups of a lane may belong to different pairs).
template <int kMode>
struct LaneAngles {
  static constexpr int N = kMode == kRopeSplitPartial ? 8 : 4;
  float2 cs[N];
};

// Pair of slot j of a lane (j < 4: the low group, j >= 4: the high group), -1: not turned.
template <int D, int kMode>
__device__ __forceinline__ int lane_pair(int sub, int j, int pairs) {
  if (kMode == kRopeInterleaved) {
    const int i = j < 2 ? 2 * sub + j : D / 4 + 2 * sub + (j - 2);   // j: pair slot 0..3
    return i < pairs ? i : -1;
  }
  if (kMode == kRopeSplit) return 4 * sub + j;                       // j: pair slot 0..3
  const int ch = (j < 4 ? 4 * sub + j : D / 2 + 4 * sub + (j - 4));  // channel
  return ch < pairs ? ch : ch < 2 * pairs ? ch - pairs : -1;
}

// False when a position of token t lies outside the table (the caller skips the token).
template <int D, int kMode>
__device__ __forceinline__ bool load_angles(const NormRope& r, int64_t t, int sub,
                                            LaneAngles<kMode>& a) {
  if (kMode == kRopeNone) return true;
  int pos[3] = {0, 0, 0};
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (i < r.num_axes) {
      pos[i] = __ldg(r.positions + t * r.num_axes + i);
      ok = ok && pos[i] >= 0 && pos[i] < r.table_rows;
    }
  }
  if (!ok) return false;
#pragma unroll
  for (int j = 0; j < LaneAngles<kMode>::N; ++j) {
    const int p = lane_pair<D, kMode>(sub, j, r.pairs);
    a.cs[j] = make_float2(1.f, 0.f);
    if (p >= 0) {
      const int at = p >= r.axis2 ? pos[2] : p >= r.axis1 ? pos[1] : pos[0];
      a.cs[j] = __ldg(r.table + static_cast<int64_t>(at) * r.pairs + p);
    }
  }
  return true;
}

// Sum over the LPR adjacent lanes of a row (every lane of the warp takes part).
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void unpack4(uint2 w, float* x) {
  x[0] = __uint_as_float(w.x << 16);
  x[1] = __uint_as_float(w.x & 0xFFFF0000u);
  x[2] = __uint_as_float(w.y << 16);
  x[3] = __uint_as_float(w.y & 0xFFFF0000u);
}

// Norm and rotation of one row held by D/8 lanes.  Every lane of the warp calls it.
template <int D, int kMode>
__device__ __forceinline__ void norm_rope_row(float (&x)[8], const NormRope& r, int sub,
                                              const float (&w)[8], const LaneAngles<kMode>& a) {
  constexpr int LPR = D / 8;
  if (r.norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    const float inv = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + r.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
  }
  if (kMode == kRopeInterleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float u = x[2 * j], v = x[2 * j + 1];
      x[2 * j] = u * a.cs[j].x - v * a.cs[j].y;
      x[2 * j + 1] = u * a.cs[j].y + v * a.cs[j].x;
    }
  } else if (kMode == kRopeSplit) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float u = x[j], v = x[4 + j];
      x[j] = u * a.cs[j].x - v * a.cs[j].y;
      x[4 + j] = u * a.cs[j].y + v * a.cs[j].x;
    }
  } else if (kMode == kRopeSplitPartial) {
    // 4-channel groups: group g < G turns with group g + G (G = pairs / 4 < LPR).  The low slot
    // of lane `sub` is group `sub`, the high slot group LPR + sub.
    const int G = r.pairs / 4;
    const int lane = threadIdx.x & 31, base = lane - sub;
    const bool first = sub < G;                               // low slot leads a pair
    const bool low2 = sub >= G && sub < 2 * G;                // low slot follows one
    const bool high2 = LPR + sub < 2 * G;                     // high slot follows one
    const int partner = first ? sub + G : sub - G;            // group the low slot turns with
    const int src = base + ((first ? partner % LPR : low2 ? partner : sub));
    const int src_high = base + (high2 ? LPR + sub - G : sub);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float from_low = __shfl_sync(0xffffffffu, x[j], src);
      const float from_high = __shfl_sync(0xffffffffu, x[4 + j], src);
      const float for_high = __shfl_sync(0xffffffffu, x[j], src_high);
      const float other = first && partner >= LPR ? from_high : from_low;
      const float c = a.cs[j].x, s = a.cs[j].y;
      const float c2 = a.cs[4 + j].x, s2 = a.cs[4 + j].y;
      const float lo = x[j], hi = x[4 + j];
      x[j] = first ? lo * c - other * s : low2 ? other * s + lo * c : lo;
      x[4 + j] = high2 ? for_high * s2 + hi * c2 : hi;
    }
  }
}

// The rows of one tensor: [tokens] rows of `heads` x D values, `stride` values from token to token.
struct RowSet {
  const __nv_bfloat16* src;
  int64_t stride;
  __nv_bfloat16* dst;           // [tokens][heads][D], or the pool [pages * page_size][heads][D]
  const __nv_bfloat16* weight;  // [D] or [heads][D]; null: ones
  int heads;
};

struct NormRopeParams {
  RowSet set[2];        // queries and keys, or (append) keys and values
  NormRope rule;
  int weight_per_head;
  int tokens;
  int chunk;            // rows (heads of both sets together) per work item
  int items_per_token;
  int* status;
  // append only: token i of the call is logical token token0 + i
  const int* pt_row;
  int token0, page_size, num_pages;
};

// One warp per (token, run of `chunk` heads); a warp step covers 32 / (D/8) heads, so the token's
// cos and sin are read once and kept in registers while the heads go by.  kAppend: rows go to
// their page, and set 1 (values) is copied bit for bit.
template <int D, int kMode, bool kAppend>
__global__ void __launch_bounds__(kNormRopeThreads)
    wf_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int LPR = D / 8, RPS = 32 / LPR;      // lanes per row, rows per warp step
  const int lane = threadIdx.x & 31;
  const int sub = lane % LPR, rsub = lane / LPR;
  const int rows = p.set[0].heads + p.set[1].heads;
  const int64_t items = static_cast<int64_t>(p.tokens) * p.items_per_token;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kNormRopeThreads / 32);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kNormRopeThreads / 32) +
                    (threadIdx.x >> 5);
       it < items; it += warps) {
    const int64_t t = it / p.items_per_token;
    const int r0 = static_cast<int>(it - t * p.items_per_token) * p.chunk;
    const int r1 = min(r0 + p.chunk, rows);
    int64_t row = t;                              // destination row of the token
    if (kAppend) {
      const int tok = p.token0 + static_cast<int>(t);
      const int pg = __ldg(p.pt_row + tok / p.page_size);
      if (pg < 0 || pg >= p.num_pages) {
        if (lane == 0) atomicCAS(p.status, 0, 5 /* WF_ERR_PAGE_OOB */);
        continue;
      }
      row = static_cast<int64_t>(pg) * p.page_size + tok % p.page_size;
    }
    LaneAngles<kMode> a;
    if (!load_angles<D, kMode>(p.rule, t, sub, a)) {   // the same answer in every lane
      if (lane == 0) atomicCAS(p.status, 0, 9 /* WF_ERR_POSITION */);
      continue;
    }
    for (int rb = r0; rb < r1; rb += RPS) {
      const int r = rb + rsub;
      const bool in = r < r1;
      const bool second = in && r >= p.set[0].heads;
      const RowSet& s = p.set[second ? 1 : 0];
      const int h = second ? r - p.set[0].heads : r;
      const __nv_bfloat16* src = s.src + t * s.stride + static_cast<int64_t>(h) * D + 4 * sub;
      uint2 lo = make_uint2(0, 0), hi = make_uint2(0, 0);
      if (in) {
        lo = *reinterpret_cast<const uint2*>(src);
        hi = *reinterpret_cast<const uint2*>(src + D / 2);
      }
      float x[8], w[8];
      unpack4(lo, x);
      unpack4(hi, x + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.f;
      if (in && s.weight != nullptr) {
        const __nv_bfloat16* wp = s.weight + (p.weight_per_head ? h * D : 0) + 4 * sub;
        unpack4(__ldg(reinterpret_cast<const uint2*>(wp)), w);
        unpack4(__ldg(reinterpret_cast<const uint2*>(wp + D / 2)), w + 4);
      }
      norm_rope_row<D, kMode>(x, p.rule, sub, w, a);
      if (!in) continue;
      if (!(kAppend && second)) {
        lo = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        hi = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
      }
      __nv_bfloat16* dst = s.dst + (row * s.heads + h) * D + 4 * sub;
      *reinterpret_cast<uint2*>(dst) = lo;
      *reinterpret_cast<uint2*>(dst + D / 2) = hi;
    }
  }
}

}  // namespace wfk
