// attn_fp8_few_kernel.cuh -- attention straight over the FP8 cache for few query rows (sm_100a).
//
// With few rows the time is the cache's bytes: every code of the visible prefix is read once per
// K/V head and used for all query heads that share it.  So rows and shared heads are packed: row m
// of a tile is (query row, query head of the group), 16 rows to a tile (the M of the matrix
// instruction), and the work is spread over the keys.
//
// A warp takes one block of 16 keys at a time, straight from global memory into registers, in an
// order chosen so that no code has to move between lanes:
//   S = Q K^T   lane (g, t) (g = lane / 4, t = lane % 4) holds channels {16 t ..} and {64 + 16 t ..}
//               of keys g and g + 8; a k step takes four of them, and Q's fragments are laid out in
//               the same channel order.
//   O += P V    lane (g, t) holds channels [D/8 g, D/8 (g + 1)) of the four keys whose logits it
//               computed (2t, 2t + 1, 8 + 2t, 9 + 2t), so P is the accumulator of S as it stands;
//               bytes of two keys are interleaved and widened together.
// e4m3 widens exactly to f16, so codes go to the tensor core without their scale: the key scale is
// multiplied into the logits (fp32).  Q goes to f16 under a power of two for each row that brings
// its largest magnitude to [2^14, 2^15): exact for values down to 2^-32 of it.  The weights carry
// the value scale: w = p 2^15 2^(e_v - E) with E the largest value exponent the warp has met, so
// w <= 2^15, rounded to f16 (2^-11 of its value; what falls under f16's range is below 2^-39 of the
// largest value's weight).  Maxima, sums and outputs are fp32.
//
// A tile never spans query segments, so all its rows see the same keys: blocks past the limit are
// not read, and keys past it in the last block get weight 0 and zeroed values, whatever their
// bytes are.  The warps' results are joined in shared memory, the parts of a split key range by the
// merge kernel.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>
#include <type_traits>

#include "sm100.cuh"

namespace wfk {

constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewSegs = 64;

struct AttnFewParams {
  const __nv_bfloat16* q;        // [T_q][Hq][D]
  const uint8_t* k_codes;        // [pages * page_size][Hk][D]
  const uint8_t* v_codes;
  const uint8_t* k_scale;        // [pages * page_size / 16][Hk]
  const uint8_t* v_scale;
  const int* page_table;
  __nv_bfloat16* out;            // [T_q][Hq][D]
  float* lse;                    // [Hq][T_q] or null
  float* part_o;                 // [splits][T_q][Hq][D] when splits > 1
  float* part_lse;               // [splits][Hq][T_q]
  int* status;
  int T_q, Hq, Hk, group, page_size, num_pages, splits, tiles;
  float sl2;                     // scale * log2(e)
  int nseg;
  int seg_tile_end[kFewSegs];    // tiles of the segments up to and including i
  int seg_row_end[kFewSegs];
  int seg_kv[kFewSegs];
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two e4m3 codes -> two f16 (code of the low byte in the low half), exact.
__device__ __forceinline__ uint32_t widen2(uint32_t c) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(h)
      : "r"(c));
  return h;
}
__device__ __forceinline__ uint32_t widen2_high(uint32_t c) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(h)
      : "r"(c));
  return h;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Codes are read once by a tile: keep them out of L1.
template <typename T>
__device__ __forceinline__ T load_codes(const uint8_t* p);
template <>
__device__ __forceinline__ uint4 load_codes<uint4>(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
template <>
__device__ __forceinline__ uint2 load_codes<uint2>(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p));
  return v;
}

__device__ __forceinline__ float pow2f(int e) {     // 2^e, e clamped to the normal range
  return __uint_as_float(static_cast<uint32_t>(min(max(e, -126), 127) + 127) << 23);
}

// MT tiles of 16 packed rows for each block.
template <int D, int MT>
struct FewSmem {
  static constexpr int STEPS = D / 16;
  static constexpr int OPITCH = D + 4;                       // floats per joined output row
  static constexpr uint32_t Q_OFF = 0;                       // fragments [MT][STEPS][32] x 16 B
  static constexpr uint32_t QF_OFF = Q_OFF + MT * STEPS * 512u;      // row factors [MT * 16]
  static constexpr uint32_t M_OFF = QF_OFF + MT * 64u;       // per warp and row: max, sum
  static constexpr uint32_t L_OFF = M_OFF + kFewWarps * MT * 64u;
  static constexpr uint32_t O_OFF = L_OFF + kFewWarps * MT * 64u;    // [warps][MT * 16][OPITCH]
  static constexpr uint32_t BYTES = O_OFF + kFewWarps * MT * 16u * OPITCH * 4u;
};

template <int D, int MT>
__global__ void __launch_bounds__(kFewThreads, MT == 1 ? 2 : 1)
    wf_attn_fp8_few_kernel(const __grid_constant__ AttnFewParams p) {
  using L = FewSmem<D, MT>;
  constexpr int STEPS = L::STEPS, R = MT * 16;
  constexpr int KV = D / 64;                     // 16-byte pieces of a key a lane holds
  constexpr int VW = D / 32;                     // words of a value row a lane holds (D/8 codes)
  extern __shared__ __align__(16) uint8_t few_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  // tile fastest, then head, then part of the keys: tiles that read the same keys run together
  const int tile = static_cast<int>(blockIdx.x) % p.tiles;
  const int rest = static_cast<int>(blockIdx.x) / p.tiles;
  const int head = rest % p.Hk, split = rest / p.Hk;
  int seg = 0;
  while (tile >= p.seg_tile_end[seg]) ++seg;
  const int seg_row0 = seg > 0 ? p.seg_row_end[seg - 1] : 0;
  const int tile0 = seg > 0 ? p.seg_tile_end[seg - 1] : 0;
  const int m_total = (p.seg_row_end[seg] - seg_row0) * p.group;   // packed rows of the segment
  const int m0 = (tile - tile0) * R;
  const int n = p.seg_kv[seg];
  const int blocks = (n + 15) / 16;
  const int lo = static_cast<int>(static_cast<int64_t>(split) * blocks / p.splits);
  const int hi = static_cast<int>(static_cast<int64_t>(split + 1) * blocks / p.splits);

  // ---- Q to f16 fragments
  uint4* const qfrag = reinterpret_cast<uint4*>(few_smem + L::Q_OFF);
  float* const qfac = reinterpret_cast<float*>(few_smem + L::QF_OFF);
  for (int m = warp; m < R; m += kFewWarps) {
    constexpr int PER = D / 32;                  // channels per lane
    float x[PER];
    const int mm = m0 + m;
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = 0.f;
    if (mm < m_total) {
      const int row = seg_row0 + mm / p.group, h = head * p.group + mm % p.group;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          p.q + (static_cast<int64_t>(row) * p.Hq + h) * D + lane * PER);
#pragma unroll
      for (int i = 0; i < PER / 2; ++i) {
        const uint32_t w = __ldg(src + i);
        x[2 * i] = __uint_as_float(w << 16);
        x[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
      }
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    const int up = top > 0.f ? min(14 - e, 126) : 0;
    const float f = pow2f(up);
    if (lane == 0) qfac[m] = pow2f(-up) * p.sl2;
    // channels c, c + 1 of row m: fragment word of step (c / 64) 4 + (c % 16) / 4
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
      const int c = lane * PER + i;
      const int s = (c / 64) * 4 + (c % 16) / 4, tt = (c % 64) / 16;
      const int word = ((c & 2) ? 2 : 0) + ((m & 8) ? 1 : 0);
      reinterpret_cast<uint32_t*>(qfrag + ((m / 16) * STEPS + s) * 32 + (m & 7) * 4 + tt)[word] =
          pack_f16x2(x[i] * f, x[i + 1] * f);
    }
  }
  __syncthreads();

  float rf[MT][2], mx[MT][2], sum[MT][2], o[MT][D / 8][4];
#pragma unroll
  for (int a = 0; a < MT; ++a) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      rf[a][i] = qfac[a * 16 + g + 8 * i];
      mx[a][i] = -INFINITY;
      sum[a][i] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[a][j][i] = 0.f;
  }
  int E = -200;                                  // largest value exponent met
  const int64_t row_bytes = static_cast<int64_t>(p.Hk) * D;

  // Block `lo + warp + i kFewWarps` for iteration i; lane i % 32 looks up its page and scales, 32
  // iterations at a time.
  const int iters = hi - lo > warp ? (hi - lo - warp + kFewWarps - 1) / kFewWarps : 0;
  int64_t my_row = 0;
  int my_ks = 127, my_vs = 127;
  auto look_up = [&](int i0) {
    const int i = i0 + lane;
    if (i < iters) {
      const int tok = (lo + warp + i * kFewWarps) * 16;
      const int idx = tok / p.page_size;
      int pg = __ldg(p.page_table + idx);
      if (pg < 0 || pg >= p.num_pages) {
        atomicCAS(p.status, 0, 5 /* WF_ERR_PAGE_OOB */);
        pg = 0;
      }
      my_row = static_cast<int64_t>(pg) * p.page_size + (tok - idx * p.page_size);
      const int64_t at = my_row / 16 * p.Hk + head;
      my_ks = __ldg(p.k_scale + at);
      my_vs = __ldg(p.v_scale + at);
    }
  };
  using VecV = typename std::conditional<D == 128, uint4, uint2>::type;
  uint4 kc[2][KV];
  VecV vc[4];
  auto load_k = [&](int64_t row) {
    const uint8_t* src = p.k_codes + (row + g) * row_bytes + static_cast<int64_t>(head) * D + 16 * t;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < KV; ++c)
        kc[i][c] = load_codes<uint4>(src + 8 * i * row_bytes + 64 * c);
  };
  auto load_v = [&](int64_t row) {
    const uint8_t* src = p.v_codes + (row + 2 * t) * row_bytes + static_cast<int64_t>(head) * D +
                         (D / 8) * g;
    vc[0] = load_codes<VecV>(src);
    vc[1] = load_codes<VecV>(src + row_bytes);
    vc[2] = load_codes<VecV>(src + 8 * row_bytes);
    vc[3] = load_codes<VecV>(src + 9 * row_bytes);
  };
  if (iters > 0) {
    look_up(0);
    const int64_t r0 = __shfl_sync(0xffffffffu, my_row, 0);
    load_k(r0);
    load_v(r0);
  }
  for (int i = 0; i < iters; ++i) {
    const int ks = __shfl_sync(0xffffffffu, my_ks, i & 31);
    const int vs = __shfl_sync(0xffffffffu, my_vs, i & 31) - 127;
    const int key0 = (lo + warp + i * kFewWarps) * 16;
    const int left = n - key0;                    // visible keys of the block
    // S: 16 rows x 16 keys per tile
    float s[MT][2][4];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[a][j][c] = 0.f;
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
      uint32_t b[2][2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 q4 = kc[j][st / 4];
        const uint32_t w = st % 4 == 0 ? q4.x : st % 4 == 1 ? q4.y : st % 4 == 2 ? q4.z : q4.w;
        b[j][0] = widen2(w);
        b[j][1] = widen2_high(w);
      }
#pragma unroll
      for (int a = 0; a < MT; ++a) {
        const uint4 f = qfrag[(a * STEPS + st) * 32 + lane];
        const uint32_t fa[4] = {f.x, f.y, f.z, f.w};
        mma_f16(s[a][0], fa, b[0][0], b[0][1]);
        mma_f16(s[a][1], fa, b[1][0], b[1][1]);
      }
    }
    // the next block's keys are on their way while this one's weights are computed
    int64_t next = 0;
    if (i + 1 < iters) {
      if (((i + 1) & 31) == 0) look_up(i + 1);
      next = __shfl_sync(0xffffffffu, my_row, (i + 1) & 31);
      load_k(next);
    }
    const float kf = __uint_as_float(static_cast<uint32_t>(ks) << 23);
    const int e_old = E;
    E = max(E, vs);
    const float wf = pow2f(15 + vs - E);          // weight factor of this block
    const float ef = pow2f(e_old - E);            // what the outputs so far shrink by
    uint32_t pa[MT][4];
#pragma unroll
    for (int a = 0; a < MT; ++a) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float x[4] = {s[a][0][2 * r], s[a][0][2 * r + 1], s[a][1][2 * r], s[a][1][2 * r + 1]};
        const float f = rf[a][r] * kf;
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] *= f;
        if (left < 16) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (2 * t + (c & 1) + 8 * (c >> 1) >= left) x[c] = -INFINITY;
        }
        float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float m_new = fmaxf(mx[a][r], top);
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = ex2_approx(mx[a][r] - ref);     // 0 at the first block
        mx[a][r] = m_new;
        float w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = ex2_approx(x[c] - ref);
        sum[a][r] = sum[a][r] * alpha + ((w[0] + w[1]) + (w[2] + w[3]));
        const float shrink = alpha * ef;
        if (__any_sync(0xffffffffu, shrink != 1.f)) {
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            o[a][j][2 * r] *= shrink;
            o[a][j][2 * r + 1] *= shrink;
          }
        }
        pa[a][r] = pack_f16x2(w[0] * wf, w[1] * wf);
        pa[a][2 + r] = pack_f16x2(w[2] * wf, w[3] * wf);
      }
    }
    if (left < 16) {                              // values past the limit may be anything
      const VecV zero = {};
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (2 * t + (c & 1) + 8 * (c >> 1) >= left) vc[c] = zero;
    }
    // O += P V: 4 channels of a lane's run at a time
#pragma unroll
    for (int wd = 0; wd < VW; ++wd) {
      uint32_t v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = reinterpret_cast<const uint32_t*>(&vc[c])[wd];
      const uint32_t a01 = __byte_perm(v[0], v[1], 0x5140), a23 = __byte_perm(v[0], v[1], 0x7362);
      const uint32_t b01 = __byte_perm(v[2], v[3], 0x5140), b23 = __byte_perm(v[2], v[3], 0x7362);
      const uint32_t f0[4] = {widen2(a01), widen2_high(a01), widen2(a23), widen2_high(a23)};
      const uint32_t f1[4] = {widen2(b01), widen2_high(b01), widen2(b23), widen2_high(b23)};
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int a = 0; a < MT; ++a) mma_f16(o[a][4 * wd + c], pa[a], f0[c], f1[c]);
    }
    if (i + 1 < iters) load_v(next);
  }

  // ---- join the warps
  float* const sm_m = reinterpret_cast<float*>(few_smem + L::M_OFF);
  float* const sm_l = reinterpret_cast<float*>(few_smem + L::L_OFF);
  float* const sm_o = reinterpret_cast<float*>(few_smem + L::O_OFF);
  const float unscale = pow2f(E - 15);
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float l = sum[a][r];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      const int m = a * 16 + g + 8 * r;
      if (t == 0) {
        sm_m[warp * R + m] = mx[a][r];
        sm_l[warp * R + m] = l;
      }
      float* dst = sm_o + (warp * R + m) * L::OPITCH + (D / 4) * t;
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int j = 0; j < D / 8; j += 4)
          *reinterpret_cast<float4*>(dst + (D / 8) * half + j) =
              make_float4(o[a][j][2 * r + half] * unscale, o[a][j + 1][2 * r + half] * unscale,
                          o[a][j + 2][2 * r + half] * unscale, o[a][j + 3][2 * r + half] * unscale);
    }
  __syncthreads();
  constexpr int PER = D / 32;
  for (int m = warp; m < R && m0 + m < m_total; m += kFewWarps) {
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) top = fmaxf(top, sm_m[w * R + m]);
    const float ref = top == -INFINITY ? 0.f : top;
    float l = 0.f, acc[PER];
#pragma unroll
    for (int c = 0; c < PER; ++c) acc[c] = 0.f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      const float wt = ex2_approx(sm_m[w * R + m] - ref);
      l += wt * sm_l[w * R + m];
#pragma unroll
      for (int c = 0; c < PER; ++c)
        acc[c] = fmaf(wt, sm_o[(w * R + m) * L::OPITCH + lane * PER + c], acc[c]);
    }
    // a row that sees no key (of this part): 0, log-sum-exp -inf; a NaN sum stays NaN
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float lse = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718056f;
    const int row = seg_row0 + (m0 + m) / p.group, h = head * p.group + (m0 + m) % p.group;
    const int64_t orow = static_cast<int64_t>(row) * p.Hq + h;
    if (p.splits > 1) {
      float* dst = p.part_o + (static_cast<int64_t>(split) * p.T_q * p.Hq + orow) * D + lane * PER;
#pragma unroll
      for (int c = 0; c < PER; ++c) dst[c] = acc[c] * inv;
      if (lane == 0)
        p.part_lse[(static_cast<int64_t>(split) * p.Hq + h) * p.T_q + row] = lse;
    } else {
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + orow * D + lane * PER);
#pragma unroll
      for (int c = 0; c < PER / 2; ++c)
        dst[c] = pack_bf16x2(acc[2 * c] * inv, acc[2 * c + 1] * inv);
      if (lane == 0 && p.lse != nullptr) p.lse[static_cast<int64_t>(h) * p.T_q + row] = lse;
    }
  }
}

}  // namespace wfk
