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
// Row layout.  D / 16 lanes share a row; lane `sub` holds channels [8 sub, 8 sub + 8) and
// [D/2 + 8 sub, ... + 8), two 16-byte loads.  Interleaved pairs and the halves of a full split
// rotation then both sit inside one lane; only a partial split rotation (2 pairs < D) exchanges
// values between lanes, through shared memory.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "sm100.cuh"

namespace wfk {

constexpr int kNormRopeThreads = 256;

// How the pairs of a row are laid out.
enum RopeMode { kRopeNone = 0, kRopeInterleaved = 1, kRopeSplit = 2, kRopeSplitPartial = 3 };

struct NormRope {
  const float2* table;        // [table_rows][pairs] (cos, sin), 16-byte aligned, pairs % 4 == 0
  const int* positions;       // [tokens][num_axes]
  int table_rows, pairs, num_axes;
  int axis1, axis2;           // first pair of axis 1 and of axis 2 (`pairs` when there is none)
  int norm;
  float eps;
};

// cos and sin of the pairs a lane turns, two pairs to a float4: 8 pairs, or one for each of the 16
// channels in kRopeSplitPartial (the halves of a lane may belong to different pairs).
template <int kMode>
struct LaneAngles {
  static constexpr int N = kMode == kRopeNone ? 0 : kMode == kRopeSplitPartial ? 8 : 4;
  float4 cs[N > 0 ? N : 1];
};

// First pair of slot j (two pairs) of a lane, -1 when these are not turned.  In kRopeSplitPartial a
// slot is two neighbouring channels; pairs % 4 == 0 keeps both on one side of every border.
template <int D, int kMode>
__device__ __forceinline__ int lane_pair(int sub, int j, int pairs) {
  if (kMode == kRopeInterleaved) {
    const int i = j < 2 ? 4 * sub + 2 * j : D / 4 + 4 * sub + 2 * (j - 2);
    return i < pairs ? i : -1;
  }
  if (kMode == kRopeSplit) return 8 * sub + 2 * j;
  const int ch = j < 4 ? 8 * sub + 2 * j : D / 2 + 8 * sub + 2 * (j - 4);
  return ch < pairs ? ch : ch < 2 * pairs ? ch - pairs : -1;
}

// A token's position along each axis; false when one lies outside the table.
__device__ __forceinline__ bool load_positions(const NormRope& r, int64_t t, int (&pos)[3]) {
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    pos[i] = 0;
    if (i < r.num_axes) {
      pos[i] = __ldg(r.positions + t * r.num_axes + i);
      ok = ok && pos[i] >= 0 && pos[i] < r.table_rows;
    }
  }
  return ok;
}

// (cos, sin) of pairs i and i + 1 (i even) at a position inside the table.
__device__ __forceinline__ float4 load_pairs(const NormRope& r, const int (&pos)[3], int i) {
  const int a = i >= r.axis2 ? pos[2] : i >= r.axis1 ? pos[1] : pos[0];
  const int b = i + 1 >= r.axis2 ? pos[2] : i + 1 >= r.axis1 ? pos[1] : pos[0];
  const float2* at = r.table + static_cast<int64_t>(a) * r.pairs + i;
  if (a == b) return __ldg(reinterpret_cast<const float4*>(at));
  const float2 x = __ldg(at), y = __ldg(r.table + static_cast<int64_t>(b) * r.pairs + i + 1);
  return make_float4(x.x, x.y, y.x, y.y);
}

template <int D, int kMode>
__device__ __forceinline__ void load_angles(const NormRope& r, const int (&pos)[3], int sub,
                                            LaneAngles<kMode>& a) {
#pragma unroll
  for (int j = 0; j < LaneAngles<kMode>::N; ++j) {
    const int p = lane_pair<D, kMode>(sub, j, r.pairs);
    a.cs[j] = p >= 0 ? load_pairs(r, pos, p) : make_float4(1.f, 0.f, 1.f, 0.f);
  }
}

// Sum over the LPR adjacent lanes of a row (every lane of the warp takes part).
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void unpack2(uint32_t w, float* x) {
  x[0] = __uint_as_float(w << 16);
  x[1] = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void unpack8(uint4 w, float* x) {
  unpack2(w.x, x);
  unpack2(w.y, x + 2);
  unpack2(w.z, x + 4);
  unpack2(w.w, x + 6);
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// Norm and rotation of one row held by D/16 lanes: x[0..7] the low channels, x[8..15] the high.
// wl, wh: the row's weights, 8 bf16 each.  Every lane of the warp calls it; `stage` is the warp's
// 32 x 16 floats of shared memory, used in kRopeSplitPartial.
template <int D, int kMode>
__device__ __forceinline__ void norm_rope_row(float (&x)[16], const NormRope& r, int sub,
                                              uint4 wl, uint4 wh, const LaneAngles<kMode>& a,
                                              float* stage) {
  constexpr int LPR = D / 16;
  if (r.norm) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s0 = fmaf(x[i], x[i], s0);
      s1 = fmaf(x[8 + i], x[8 + i], s1);
    }
    const float inv = rsqrtf(row_sum<LPR>(s0 + s1) * (1.f / D) + r.eps);
    float w[8];
    unpack8(wl, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
    unpack8(wh, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[8 + i] = x[8 + i] * inv * w[i];
  }
  if (kMode == kRopeInterleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 cs = a.cs[j / 2];
      const float c = j & 1 ? cs.z : cs.x, s = j & 1 ? cs.w : cs.y;
      const float u = x[2 * j], v = x[2 * j + 1];
      x[2 * j] = u * c - v * s;
      x[2 * j + 1] = u * s + v * c;
    }
  } else if (kMode == kRopeSplit) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 cs = a.cs[j / 2];
      const float c = j & 1 ? cs.z : cs.x, s = j & 1 ? cs.w : cs.y;
      const float u = x[j], v = x[8 + j];
      x[j] = u * c - v * s;
      x[8 + j] = u * s + v * c;
    }
  } else if (kMode == kRopeSplitPartial) {
    float* const row = stage + ((threadIdx.x & 31) / LPR) * D;
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        *reinterpret_cast<float4*>(row + h * (D / 2) + 8 * sub + i) =
            make_float4(x[8 * h + i], x[8 * h + i + 1], x[8 * h + i + 2], x[8 * h + i + 3]);
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 8; i += 4) {       // 4 channels: pairs % 4 == 0 keeps them together
        const int ch = h * (D / 2) + 8 * sub + i;
        if (ch < 2 * r.pairs) {
          const bool lead = ch < r.pairs;
          const float4 o = *reinterpret_cast<const float4*>(row + (lead ? ch + r.pairs
                                                                        : ch - r.pairs));
          const float other[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 cs = a.cs[4 * h + (i + k) / 2];
            const float c = k & 1 ? cs.z : cs.x, s = k & 1 ? cs.w : cs.y;
            float& v = x[8 * h + i + k];
            v = lead ? v * c - other[k] * s : other[k] * s + v * c;
          }
        }
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

constexpr uint32_t kOnes = 0x3F803F80u;           // two bf16 ones
constexpr int kNormRopeBatch = 3;                 // warp steps whose loads are in flight together

// One warp per (token, run of `chunk` heads); a warp step covers 32 / (D/16) heads, so the token's
// cos and sin are read once and kept in registers while the heads go by.  kAppend: rows go to
// their page, and set 1 (values) is copied bit for bit.
//
// Bound by HBM: 4 D bytes for each row, and the table from L2.  On 23 400 tokens of 12 + 12 heads of
// 128 (288 MB): see the launch's rule for `chunk`; with 8-byte loads, one step at a time, this took
// 79 us (3.6 TB/s).
template <int D, int kMode, bool kAppend>
__global__ void __launch_bounds__(kNormRopeThreads)
    wf_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int LPR = D / 16, RPS = 32 / LPR, B = kNormRopeBatch;   // lanes per row, rows per step
  __shared__ float stage_all[kMode == kRopeSplitPartial ? kNormRopeThreads * 16 : 1];
  const int lane = threadIdx.x & 31;
  float* const stage = stage_all + (kMode == kRopeSplitPartial ? (threadIdx.x >> 5) * 512 : 0);
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
    if (kMode != kRopeNone) {
      int pos[3];
      if (!load_positions(p.rule, t, pos)) {      // the same answer in every lane
        if (lane == 0) atomicCAS(p.status, 0, 9 /* WF_ERR_POSITION */);
        continue;
      }
      load_angles<D, kMode>(p.rule, pos, sub, a);
    }
    for (int rb = r0; rb < r1; rb += B * RPS) {
      uint4 lo[B], hi[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int r = rb + b * RPS + rsub;
        lo[b] = hi[b] = make_uint4(0, 0, 0, 0);
        if (r < r1) {
          const bool second = r >= p.set[0].heads;
          const RowSet& s = p.set[second ? 1 : 0];
          const int h = second ? r - p.set[0].heads : r;
          const __nv_bfloat16* src = s.src + t * s.stride + static_cast<int64_t>(h) * D + 8 * sub;
          lo[b] = *reinterpret_cast<const uint4*>(src);
          hi[b] = *reinterpret_cast<const uint4*>(src + D / 2);
        }
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if (rb + b * RPS >= r1) break;            // the whole warp
        const int r = rb + b * RPS + rsub;
        const bool in = r < r1;
        const bool second = in && r >= p.set[0].heads;
        const RowSet& s = p.set[second ? 1 : 0];
        const int h = second ? r - p.set[0].heads : r;
        uint4 wl = make_uint4(kOnes, kOnes, kOnes, kOnes), wh = wl;
        if (in && s.weight != nullptr) {
          const __nv_bfloat16* wp = s.weight + (p.weight_per_head ? h * D : 0) + 8 * sub;
          wl = __ldg(reinterpret_cast<const uint4*>(wp));
          wh = __ldg(reinterpret_cast<const uint4*>(wp + D / 2));
        }
        float x[16];
        unpack8(lo[b], x);
        unpack8(hi[b], x + 8);
        norm_rope_row<D, kMode>(x, p.rule, sub, wl, wh, a, stage);
        if (!in) continue;
        __nv_bfloat16* dst = s.dst + (row * s.heads + h) * D + 8 * sub;
        const bool copy = kAppend && second;
        *reinterpret_cast<uint4*>(dst) = copy ? lo[b] : pack8(x);
        *reinterpret_cast<uint4*>(dst + D / 2) = copy ? hi[b] : pack8(x + 8);
      }
    }
  }
}

}  // namespace wfk
