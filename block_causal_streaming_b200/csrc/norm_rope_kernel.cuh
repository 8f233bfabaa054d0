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

// How the pairs of a row are laid out, and whether all of its channels are turned.
enum RopeMode {
  kRopeNone = 0,
  kRopeInterleaved = 1,
  kRopeSplit = 2,
  kRopeSplitPartial = 3,
  kRopeInterleavedPartial = 4
};
template <int kMode>
constexpr bool kInterleaved = kMode == kRopeInterleaved || kMode == kRopeInterleavedPartial;

struct NormRope {
  const float2* table;        // [table_rows][pairs] (cos, sin), 16-byte aligned, pairs % 4 == 0
  const int* positions;       // [tokens][num_axes]
  int table_rows, pairs, num_axes;
  int axis1, axis2;           // first pair of axis 1 and of axis 2 (`pairs` when there is none)
  int norm;
  float eps;
};

// A lane's 16 channels as eight packed pairs of floats, so that norm and rotation run two values to
// an instruction.  Interleaved: u[i], v[i] are the first and second channels of pairs 2i and 2i + 1;
// else u the low channels and v the high ones, in order (a full split rotation turns u with v).
struct Row {
  float2 u[4], v[4];
};

// cos and sin of what a lane turns, (cos, cos, sin, sin) of two pairs a slot: the pairs 2i and 2i + 1
// of u[i], v[i], or in kRopeSplitPartial, where the channels of a lane may belong to different
// pairs, those of its channels 2i and 2i + 1.
template <int kMode>
struct LaneAngles {
  float4 p[kMode == kRopeNone ? 1 : kMode == kRopeSplitPartial ? 8 : 4];
  __device__ __forceinline__ float4 operator()(int j) const { return p[j]; }
};
template <int kMode>
constexpr int kAngleSlots = kMode == kRopeNone ? 0 : kMode == kRopeSplitPartial ? 8 : 4;

// First pair of slot j (two pairs) of a lane, -1 when these are not turned.  In kRopeSplitPartial a
// slot is two neighbouring channels; pairs % 4 == 0 keeps both on one side of every border.
template <int D, int kMode>
__device__ __forceinline__ int lane_pair(int sub, int j, int pairs) {
  if (kInterleaved<kMode>) {
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
      pos[i] = r.positions[t * r.num_axes + i];
      ok = ok && pos[i] >= 0 && pos[i] < r.table_rows;
    }
  }
  return ok;
}

// (cos, cos, sin, sin) of pairs i and i + 1 (i even) at a position inside the table.
__device__ __forceinline__ float4 load_pairs(const NormRope& r, const int (&pos)[3], int i) {
  const int a = i >= r.axis2 ? pos[2] : i >= r.axis1 ? pos[1] : pos[0];
  const int b = i + 1 >= r.axis2 ? pos[2] : i + 1 >= r.axis1 ? pos[1] : pos[0];
  const float2* at = r.table + static_cast<int64_t>(a) * r.pairs + i;
  if (a == b) {
    const float4 x = *reinterpret_cast<const float4*>(at);
    return make_float4(x.x, x.z, x.y, x.w);
  }
  const float2 x = *at, y = r.table[static_cast<int64_t>(b) * r.pairs + i + 1];
  return make_float4(x.x, y.x, x.y, y.y);
}

template <int D, int kMode>
__device__ __forceinline__ void load_angles(const NormRope& r, const int (&pos)[3], int sub,
                                            LaneAngles<kMode>& a) {
#pragma unroll
  for (int j = 0; j < kAngleSlots<kMode>; ++j) {
    const int p = lane_pair<D, kMode>(sub, j, r.pairs);
    a.p[j] = p >= 0 ? load_pairs(r, pos, p) : make_float4(1.f, 1.f, 0.f, 0.f);
  }
}

// Sum over the LPR adjacent lanes of a row (every lane of the warp takes part).
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) {
  return __uint_as_float(w & 0xFFFF0000u);
}

// 16 bf16 channels (low 8, high 8) <-> a lane's row.
template <int kMode>
__device__ __forceinline__ void unpack_row(uint4 lo, uint4 hi, Row& x) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kInterleaved<kMode>) {
      x.u[i] = make_float2(bf16_low(w[2 * i]), bf16_low(w[2 * i + 1]));
      x.v[i] = make_float2(bf16_high(w[2 * i]), bf16_high(w[2 * i + 1]));
    } else {
      x.u[i] = make_float2(bf16_low(w[i]), bf16_high(w[i]));
      x.v[i] = make_float2(bf16_low(w[4 + i]), bf16_high(w[4 + i]));
    }
  }
}
// Channels 4 i .. 4 i + 3 of a lane's 16, in order (the high 8 from i = 2 on).
template <int kMode>
__device__ __forceinline__ float4 channels4(const Row& x, int i) {
  if (kInterleaved<kMode>) return make_float4(x.u[i].x, x.v[i].x, x.u[i].y, x.v[i].y);
  return i < 2 ? make_float4(x.u[2 * i].x, x.u[2 * i].y, x.u[2 * i + 1].x, x.u[2 * i + 1].y)
               : make_float4(x.v[2 * i - 4].x, x.v[2 * i - 4].y, x.v[2 * i - 3].x,
                             x.v[2 * i - 3].y);
}
template <int kMode>
__device__ __forceinline__ void set_channels4(Row& x, int i, float4 c) {
  if (kInterleaved<kMode>) {
    x.u[i] = make_float2(c.x, c.z);
    x.v[i] = make_float2(c.y, c.w);
  } else if (i < 2) {
    x.u[2 * i] = make_float2(c.x, c.y);
    x.u[2 * i + 1] = make_float2(c.z, c.w);
  } else {
    x.v[2 * i - 4] = make_float2(c.x, c.y);
    x.v[2 * i - 3] = make_float2(c.z, c.w);
  }
}
template <int kMode>
__device__ __forceinline__ uint4 pack_channels8(const Row& x, int half) {
  const float4 a = channels4<kMode>(x, 2 * half), b = channels4<kMode>(x, 2 * half + 1);
  return make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y),
                    pack_bf16x2(b.z, b.w));
}

// Norm and rotation of one row held by D/16 lanes; w: the row's weights, angles(j): slot j's cos and
// sin.  Every lane of the warp calls it; `stage` is the warp's 32 x 16 floats of shared memory, used in
// kRopeSplitPartial.  The weights come before the norm's factor: a product of two bf16 values is exact
// in fp32, so that is one rounding less (192 of 216 million normed and turned keys in another code than
// float64's in the FP8 cache, against 224, at the same speed; with a correctly rounded reciprocal square
// root 177, and queries and keys take 3 % longer).
template <int D, int kMode, typename Angles>
__device__ __forceinline__ void norm_rope_row(Row& x, const NormRope& r, int sub, const Row& w,
                                              const Angles& angles, float* stage) {
  constexpr int LPR = D / 16;
  if (r.norm) {
    float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s0 = __ffma2_rn(x.u[i], x.u[i], s0);
      s1 = __ffma2_rn(x.v[i], x.v[i], s1);
    }
    s0 = __fadd2_rn(s0, s1);
    const float inv = rsqrtf(row_sum<LPR>(s0.x + s0.y) * (1.f / D) + r.eps);
    const float2 inv2 = make_float2(inv, inv);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x.u[i] = __fmul2_rn(__fmul2_rn(x.u[i], w.u[i]), inv2);
      x.v[i] = __fmul2_rn(__fmul2_rn(x.v[i], w.v[i]), inv2);
    }
  }
  if constexpr (kInterleaved<kMode> || kMode == kRopeSplit) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // Channels that are not turned stay: under an angle of 0 an infinity would reach the other channel
      // of its pair.  (A mode of its own: asked of rows that are turned whole, 61.8 us against 52.8.)
      if (kMode == kRopeInterleavedPartial && lane_pair<D, kMode>(sub, i, r.pairs) < 0) continue;
      const float4 p = angles(i);
      const float2 c = make_float2(p.x, p.y), s = make_float2(p.z, p.w);
      const float2 u = x.u[i], v = x.v[i];
      x.u[i] = __ffma2_rn(v, make_float2(-p.z, -p.w), __fmul2_rn(u, c));
      x.v[i] = __ffma2_rn(u, s, __fmul2_rn(v, c));
    }
  } else if constexpr (kMode == kRopeSplitPartial) {
    float* const row = stage + ((threadIdx.x & 31) / LPR) * D;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(row + (i / 2) * (D / 2) + 8 * sub + 4 * (i & 1)) =
          channels4<kMode>(x, i);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {            // 4 channels: pairs % 4 == 0 keeps them together
      const int ch = (i / 2) * (D / 2) + 8 * sub + 4 * (i & 1);
      if (ch < 2 * r.pairs) {
        const bool lead = ch < r.pairs;
        const float4 o = *reinterpret_cast<const float4*>(row + (lead ? ch + r.pairs
                                                                      : ch - r.pairs));
        const float4 p = angles(2 * i), q = angles(2 * i + 1);
        float4 y = channels4<kMode>(x, i);
        const float sgn = lead ? -1.f : 1.f;
        y.x = y.x * p.x + sgn * (o.x * p.z);
        y.y = y.y * p.y + sgn * (o.y * p.w);
        y.z = y.z * q.x + sgn * (o.z * q.z);
        y.w = y.w * q.y + sgn * (o.w * q.w);
        set_channels4<kMode>(x, i, y);
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
  int chunk;            // warp steps (of both sets together) per work item
  int items_per_token;
  int* status;
  // append only: token i of the call is logical token token0 + i
  const int* pt_row;
  int token0, page_size, num_pages;
};

constexpr uint32_t kOnes = 0x3F803F80u;           // two bf16 ones
// Warp steps whose loads are in flight together, and CTAs per SM at least.  23 400 tokens of 12 + 12
// heads of 128: 3 steps at 3 CTAs 52.7 us, 2 steps 56.6, 4 steps 59.6; 3 steps at 2 CTAs 56.4.
constexpr int kNormRopeBatch = 3;
constexpr int kNormRopeCtas = 3;

// A lane's weights of one head (ones without a weight).
template <int D, int kMode>
__device__ __forceinline__ void load_weight(const __nv_bfloat16* weight, int64_t at, int sub,
                                            Row& w) {
  uint4 lo = make_uint4(kOnes, kOnes, kOnes, kOnes), hi = lo;
  if (weight != nullptr) {
    lo = *reinterpret_cast<const uint4*>(weight + at + 8 * sub);
    hi = *reinterpret_cast<const uint4*>(weight + at + 8 * sub + D / 2);
  }
  unpack_row<kMode>(lo, hi, w);
}

// One warp per (token, run of `chunk` warp steps); a step covers 32 / (D/16) heads of one tensor,
// the first tensor's steps before the second's, so the token's cos and sin and a tensor's weights
// are read once and kept in registers while the heads go by.  kAppend: rows go to their page, and
// set 1 (values) is copied bit for bit.
//
// Bound by HBM: 4 D bytes for each row, and the table from L2.  23 400 tokens, 12 + 12 heads of 128 with
// three axes: 52.5 us in a graph, 5.5 TB/s (0.84 of a copy), 55-57 call after call (0.77-0.80); the same into
// pages, 52.3 and 53-55.  With 8-byte loads 79 us; with single floats instead of packed pairs 57 (issue
// slots two thirds full).
template <int D, int kMode, bool kAppend>
__global__ void __launch_bounds__(kNormRopeThreads, kNormRopeCtas)
    wf_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int LPR = D / 16, RPS = 32 / LPR, B = kNormRopeBatch;   // lanes per row, rows per step
  __shared__ float stage_all[kMode == kRopeSplitPartial ? kNormRopeThreads * 16 : 1];
  wait_for_previous();
  launch_next();
  const int lane = threadIdx.x & 31;
  float* const stage = stage_all + (kMode == kRopeSplitPartial ? (threadIdx.x >> 5) * 512 : 0);
  const int sub = lane % LPR, rsub = lane / LPR;
  const int steps0 = (p.set[0].heads + RPS - 1) / RPS;
  const int steps = steps0 + (p.set[1].heads + RPS - 1) / RPS;
  const int64_t items = static_cast<int64_t>(p.tokens) * p.items_per_token;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kNormRopeThreads / 32);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kNormRopeThreads / 32) +
                    (threadIdx.x >> 5);
       it < items; it += warps) {
    const int64_t t = it / p.items_per_token;
    const int st0 = static_cast<int>(it - t * p.items_per_token) * p.chunk;
    const int st1 = min(st0 + p.chunk, steps);
    // the first heads' values, the token's page and its positions are asked for together
    uint4 lo[B], hi[B];
    const auto load = [&](const RowSet& s, int hb, int h1) {
      const __nv_bfloat16* const src = s.src + t * s.stride + 8 * sub;
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int h = hb + b * RPS + rsub;
        lo[b] = hi[b] = make_uint4(0, 0, 0, 0);
        if (h < h1) {
          lo[b] = *reinterpret_cast<const uint4*>(src + h * D);
          hi[b] = *reinterpret_cast<const uint4*>(src + h * D + D / 2);
        }
      }
    };
    const int first = st0 < steps0 ? 0 : 1;
    const auto begin = [&](int which) { return max(st0 - (which ? steps0 : 0), 0) * RPS; };
    const auto end = [&](int which) {
      return min((st1 - (which ? steps0 : 0)) * RPS, p.set[which].heads);
    };
    load(p.set[first], begin(first), end(first));
    int64_t row = t;                              // destination row of the token
    if (kAppend) {
      const int tok = p.token0 + static_cast<int>(t);
      const int pg = p.pt_row[tok / p.page_size];
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
#pragma unroll 1
    for (int which = first; which < 2; ++which) {
      const RowSet& s = p.set[which];
      const int h0 = begin(which), h1 = end(which);
      if (h0 >= h1) continue;
      __nv_bfloat16* const dst = s.dst + row * s.heads * D + 8 * sub;
      const bool copy = kAppend && which == 1;
      Row w;
      if (!copy) load_weight<D, kMode>(s.weight, 0, sub, w);
      for (int hb = h0; hb < h1; hb += B * RPS) {
        if (which != first || hb != h0) load(s, hb, h1);
#pragma unroll
        for (int b = 0; b < B; ++b) {
          if (hb + b * RPS >= h1) break;          // the whole warp
          const int h = hb + b * RPS + rsub;
          if (!copy) {
            if (p.weight_per_head && h < h1)
              load_weight<D, kMode>(s.weight, static_cast<int64_t>(h) * D, sub, w);
            Row x;
            unpack_row<kMode>(lo[b], hi[b], x);
            norm_rope_row<D, kMode>(x, p.rule, sub, w, a, stage);
            lo[b] = pack_channels8<kMode>(x, 0);
            hi[b] = pack_channels8<kMode>(x, 1);
          }
          if (h < h1) {
            *reinterpret_cast<uint4*>(dst + h * D) = lo[b];
            *reinterpret_cast<uint4*>(dst + h * D + D / 2) = hi[b];
          }
        }
      }
    }
  }
}

}  // namespace wfk
