// attn_fp8_few_kernel.cuh -- attention straight over the FP8 cache for few query rows (sm_100a).
//
// With few rows the time is the cache's bytes: every code of the visible prefix is read once per
// K/V head and used for all query heads that share it.  So rows and shared heads are packed: row m
// of a tile is (query row, query head of the group), 8 rows to a column tile of the matrix
// instructions, whose 16 rows are keys (S^T = K Q^T) and then channels (O^T = V^T P^T); and the work
// is spread over the keys.
//
// A warp takes one block of 16 keys at a time.  Its codes come by TMA into the warp's own ring of
// slots in shared memory, refilled by the warp itself as soon as a slot is read, so no warp waits
// for another.  The order of channels and keys over the lanes is chosen so that no code has to move
// between lanes:
//   S^T = K Q^T    lane (g, t) (g = lane / 4, t = lane % 4) holds channels {16 t ..} and {64 + 16 t ..}
//                  of keys g and g + 8; a k step takes four of them, and Q's fragments are laid out
//                  in the same channel order;
//   O^T += V^T P^T lane (g, t) holds channels [D/8 g, D/8 (g + 1)) of keys 2t, 2t + 1, 8 + 2t, 9 + 2t;
//                  bytes of two keys are interleaved and widened together, and P^T is the
//                  accumulator of S^T rounded to f16 and transposed (one instruction for 8 keys).
// e4m3 widens exactly to f16, so codes go to the tensor core without their scale: the key scale is
// multiplied into the logits (fp32).  Q goes to f16 under a power of two for each row that brings
// its largest magnitude to [2^14, 2^15): exact for values down to 2^-32 of it.  The weights carry
// the value scale: w = p 2^13 2^(e_v - E) with E the largest value exponent the warp has met and p
// against a reference that trails the maximum by at most 2^2, so w <= 2^15, rounded to f16: 2^-11
// of its value, steps of 2^-37 of the largest value's weight below.  (A trailing reference costs a
// vote for 16 keys; the maximum itself three exchanges a row.)  Maxima, sums and outputs are fp32.
//
// A tile never spans query segments, so all its rows see the same keys: blocks past the limit are
// not read, and keys past it in the last block get weight 0 and zeroed values, whatever their
// bytes are.  The warps' results are joined in shared memory, the parts of a split key range by
// wf_join_kernel.
//
// One row is bound by HBM.  One token, 40 heads x 51 480 keys (527 MB): 88-92 us, 5.8-6.0 TB/s, 0.88-0.91
// of a copy.  One token of 32 heads on 8 x 37 441 keys (77 MB): 20 us in a graph, 3.8 TB/s; of these about
// 12 are the bytes, the rest the first page-table and scale look-ups, the last blocks and the join.  More
// rows are bound by latency: a warp has one block of 16 keys in work at a time, and above 16 rows an SM
// has 8 warps: 12 heads x 37 440 keys, 1 row 25.6 us, 8 rows 27.5, 16 rows 35.4, 32 rows 49.5.  On the way
// there: codes straight to registers 38 us (130 with 40 heads), one TMA ring for a CTA 29 (109), a ring
// for each warp 28 (111), keys as the rows of the products instead of query rows, so that no shuffle
// is needed between them, 23 (93), launches over the tail of the kernel before 21 (89).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>
#include <type_traits>

#include "sm100.cuh"

namespace wfk {

constexpr int kFewWarps = 8;
constexpr int kFewThreads = kFewWarps * 32;
constexpr int kFewSegs = 64;

struct AttnFewParams {
  CUtensorMap tm_k;  // e4m3 (D, Hk, num_pages * page_size), box (D, 1, box_rows = 16), D-byte swizzle
  CUtensorMap tm_v;
  const __nv_bfloat16* q;        // [T_q][Hq][D]
  const uint8_t* k_scale;        // [pages * page_size / 16][Hk]
  const uint8_t* v_scale;
  const int* page_table;
  __nv_bfloat16* out;            // [T_q][Hq][D]
  float* lse;                    // [Hq][T_q] or null
  float* part_o;                 // [splits][T_q][Hq][D] when splits > 1
  float* part_lse;               // [splits][Hq][T_q]
  int* status;
  unsigned* grid_abort;
  unsigned launch_id;
  int T_q, Hq, Hk, group, page_size, num_pages, total_rows, box_rows, splits, tiles;
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

// Offset of 16-byte piece c of row r in a tile of D-byte rows under the D-byte swizzle.
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return D == 128 ? static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) * 16))
                  : static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) * 16));
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// Transpose of an 8 x 8 matrix of 16-bit values, two of a row to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ float pow2f(int e) {     // 2^e, e clamped to the normal range
  return __uint_as_float(static_cast<uint32_t>(min(max(e, -126), 127) + 127) << 23);
}

// Pool row of logical token `tok`; a page outside the pool is recorded and read as page 0.
template <typename P>
__device__ __forceinline__ int fp8_row(const P& p, int tok) {
  const int idx = tok / p.page_size;
  int pg = p.page_table[idx];
  if (pg < 0 || pg >= p.num_pages) {
    atomicCAS(p.status, 0, 5 /* WF_ERR_PAGE_OOB */);
    pg = 0;
  }
  return pg * p.page_size + (tok - idx * p.page_size);
}

// Wait on a phase with only a timeout: used to drain loads before shared memory is released.
__device__ __forceinline__ bool few_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_test(bar, parity))
    if (globaltimer_ns() - t0 > 200000000ull) return false;
  return true;
}

// NT column tiles of 8 packed rows.
template <int D, int NT>
struct FewSmem {
  static constexpr int STEPS = D / 16;
  static constexpr int CTAS = NT <= 2 ? 2 : 1;               // per SM
  // slots of a warp: 96 KB for the CTA where two share an SM, 160 KB where the accumulators leave
  // room for one
  static constexpr uint32_t CTILE = 16 * D;                  // K or V codes of a block
  static constexpr int NS = (CTAS == 2 ? 96 : 160) * 1024 / (kFewWarps * 2 * CTILE);
  static constexpr int OPITCH = D + 4;                       // floats per joined output row
  static constexpr uint32_t RING_OFF = 0;                    // [warps][NS][K, V]
  static constexpr uint32_t O_OFF = 0;                       // joined outputs, after the ring's use
  static constexpr uint32_t RING = kFewWarps * NS * 2 * CTILE;
  static constexpr uint32_t Q_OFF = RING_OFF + RING;         // fragments [NT][STEPS][32] x 8 B
  static constexpr uint32_t QF_OFF = Q_OFF + NT * STEPS * 256u;      // row factors [NT * 8]
  static constexpr uint32_t M_OFF = QF_OFF + NT * 32u;       // per warp and row: max, sum
  static constexpr uint32_t L_OFF = M_OFF + kFewWarps * NT * 32u;
  static constexpr uint32_t BAR_OFF = L_OFF + kFewWarps * NT * 32u;  // [warps][NS]
  static constexpr uint32_t MISC_OFF = BAR_OFF + 8u * kFewWarps * NS;
  static constexpr uint32_t E_OFF = MISC_OFF + 16u;          // exponents of the warps' outputs
  static constexpr uint32_t BYTES = E_OFF + kFewWarps * 4u;
  static constexpr uint32_t ALLOC = BYTES + 1024;            // slack for 1024-byte alignment
  static_assert(kFewWarps * NT * 8u * OPITCH * 4u <= RING, "outputs fit the ring");
  static_assert(ALLOC <= (CTAS == 2 ? 113u : 227u) * 1024u, "shared memory per CTA");
};

template <int D, int NT>
__global__ void __launch_bounds__(kFewThreads, FewSmem<D, NT>::CTAS)
    wf_attn_fp8_few_kernel(const __grid_constant__ AttnFewParams p) {
  using L = FewSmem<D, NT>;
  constexpr int STEPS = L::STEPS, R = NT * 8, NS = L::NS;
  constexpr int VW = D / 32;                     // words of a value row a lane holds (D/8 codes)
  constexpr float kShiftBits = 13.f;             // weights: at most 2^(13 + 2)
  extern __shared__ uint8_t few_raw[];
  const uint32_t base = (smem_u32(few_raw) + 1023u) & ~1023u;
  uint8_t* const few_smem = few_raw + (base - smem_u32(few_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  auto full = [&](int i) -> uint32_t { return base + L::BAR_OFF + 8u * (warp * NS + i); };
  const uint32_t ring = base + L::RING_OFF + warp * (NS * 2 * L::CTILE);
  volatile int* const cta_abort = reinterpret_cast<volatile int*>(few_smem + L::MISC_OFF);
  const WaitCtx w8{cta_abort, p.grid_abort, p.status, p.launch_id, 6 /* WF_ERR_TIMEOUT */,
                   2000000000ull};

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
  // this part's blocks of 16 keys; the warp's are lo + warp + 8 j, j < nk
  const int blocks = (n + 15) / 16;
  const int lo = static_cast<int>(static_cast<int64_t>(split) * blocks / p.splits) + warp;
  const int hi = static_cast<int>(static_cast<int64_t>(split + 1) * blocks / p.splits);
  const int nk = hi > lo ? (hi - lo + kFewWarps - 1) / kFewWarps : 0;
  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(full(i), 1);
    mbar_init_fence();
  }
  wait_for_previous();
  launch_next();
  if (threadIdx.x == 0) {
    *cta_abort = (*reinterpret_cast<volatile unsigned*>(p.grid_abort) == p.launch_id) ? 1 : 0;
    // (a captured launch keeps its id: a replay after a wait ran out says so again)
    if (*cta_abort) atomicCAS(p.status, 0, 6 /* WF_ERR_TIMEOUT */);
  }
  // lane j % 32 looks up the pool row and the scales of block j, 32 blocks at a time
  int my_row = 0, my_ks = 127, my_vs = 127;
  auto look_up = [&](int j0) {
    if (j0 + lane < nk) {
      my_row = fp8_row(p, (lo + (j0 + lane) * kFewWarps) * 16);
      const int64_t at = static_cast<int64_t>(my_row / 16) * p.Hk + head;
      my_ks = p.k_scale[at];
      my_vs = p.v_scale[at];
    }
  };
  // bring block j, at pool row `row`, into its slot (which every lane has left)
  auto issue = [&](int j, int row) {
    if (lane == 0) {
      const int st = j % NS;
      const uint32_t at = ring + st * 2 * L::CTILE;
      mbar_arrive_expect_tx(full(st), 2 * L::CTILE);
      tma_load_3d(at, &p.tm_k, 0, head, row, full(st));
      tma_load_3d(at + L::CTILE, &p.tm_v, 0, head, row, full(st));
    }
  };
  __syncthreads();
  const bool skip = *cta_abort != 0;
  int issued = 0;
  if (!skip) {
    look_up(0);
    for (; issued < NS && issued < nk; ++issued)
      issue(issued, __shfl_sync(0xffffffffu, my_row, issued));
  }

  // ---- Q to f16 fragments
  uint2* const qfrag = reinterpret_cast<uint2*>(few_smem + L::Q_OFF);
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
        const uint32_t w = src[i];
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
    // An infinite value makes its row NaN: as a logit of -inf for every key it would look like a row
    // that sees none.
    const float f = top < INFINITY ? pow2f(up) : __uint_as_float(0x7FFFFFFFu);
    if (lane == 0) qfac[m] = pow2f(-up) * p.sl2;
    // channels c, c + 1 of row m: fragment of step (c / 64) 4 + (c % 16) / 4
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
      const int c = lane * PER + i;
      const int s = (c / 64) * 4 + (c % 16) / 4, tt = (c % 64) / 16;
      reinterpret_cast<uint32_t*>(qfrag + ((m / 8) * STEPS + s) * 32 + (m & 7) * 4 + tt)[(c & 2) / 2] =
          pack_f16x2(x[i] * f, x[i + 1] * f);
    }
  }
  __syncthreads();

  // rows 2t and 2t + 1 of each column tile are this lane's
  float rf[NT][2], mx[NT][2], sum[NT][2], o[NT][D / 16][4];
#pragma unroll
  for (int a = 0; a < NT; ++a) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      rf[a][i] = qfac[a * 8 + 2 * t + i];
      mx[a][i] = -INFINITY;
      sum[a][i] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[a][j][i] = 0.f;
  }
  int E = -200;                                  // largest value exponent met

  bool ok = !skip;
  int ahead_row = my_row;                         // rows of the 32 blocks that `issued` is among
  for (int j = 0; j < nk && ok; ++j) {
    if (j > 0 && (j & 31) == 0) look_up(j);
    const int ks = __shfl_sync(0xffffffffu, my_ks, j & 31);
    const int vs = __shfl_sync(0xffffffffu, my_vs, j & 31) - 127;
    const int st = j % NS;
    const int left = n - (lo + j * kFewWarps) * 16;              // visible keys of the block
    ok = __all_sync(0xffffffffu, mbar_wait(full(st), (j / NS) & 1, w8));
    if (!ok) break;
    const uint32_t kt = ring + st * 2 * L::CTILE, vt = kt + L::CTILE;
    uint4 kc[2][D / 64];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        kc[i][c] = ld_shared_v4(kt + swz<D>(g + 8 * i, t + 4 * c));
    // S^T: 16 keys x 8 rows per column tile, in two chains of k steps
    float s[NT][2][4];
#pragma unroll
    for (int a = 0; a < NT; ++a)
#pragma unroll
      for (int c = 0; c < 8; ++c) s[a][c / 4][c % 4] = 0.f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const uint4 k0 = kc[0][i / 4], k1 = kc[1][i / 4];
      const uint32_t w0 = i % 4 == 0 ? k0.x : i % 4 == 1 ? k0.y : i % 4 == 2 ? k0.z : k0.w;
      const uint32_t w1 = i % 4 == 0 ? k1.x : i % 4 == 1 ? k1.y : i % 4 == 2 ? k1.z : k1.w;
      const uint32_t ka[4] = {widen2(w0), widen2(w1), widen2_high(w0), widen2_high(w1)};
#pragma unroll
      for (int a = 0; a < NT; ++a) {
        const uint2 f = qfrag[(a * STEPS + i) * 32 + lane];
        mma_f16(s[a][i & 1], ka, f.x, f.y);
      }
    }
    const float kf = __uint_as_float(static_cast<uint32_t>(ks) << 23);
    const int e_old = E;
    E = max(E, vs);
    const float wf = pow2f(vs - E);               // what this block's weights shrink by
    float x[NT][4];                               // (key g, rows 2t, 2t + 1), (key g + 8, ..)
    bool grows = false;
#pragma unroll
    for (int a = 0; a < NT; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        x[a][c] = (s[a][0][c] + s[a][1][c]) * (rf[a][c & 1] * kf);
        if (left < 16 && g + 8 * (c >> 1) >= left) x[a][c] = -INFINITY;
        grows |= x[a][c] > mx[a][c & 1] + 2.f;
      }
    if (__any_sync(0xffffffffu, grows || E != e_old)) {
      // move the references to the maxima, and what was summed under the old ones with them
      const float ef = pow2f(e_old - E);
#pragma unroll
      for (int a = 0; a < NT; ++a) {
        float shrink[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float top = fmaxf(x[a][r], x[a][2 + r]);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const float m_new = fmaxf(mx[a][r], top);
          const float alpha = m_new == -INFINITY ? 1.f : ex2_approx(mx[a][r] - m_new);
          mx[a][r] = m_new;
          sum[a][r] *= alpha;
          shrink[r] = alpha * ef;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[a][j][c] *= shrink[c & 1];
      }
    }
    uint32_t pb[NT][2];
#pragma unroll
    for (int a = 0; a < NT; ++a) {
      float w[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float ref = mx[a][c & 1] == -INFINITY ? 0.f : mx[a][c & 1] - kShiftBits;
        w[c] = ex2_approx(x[a][c] - ref);
        sum[a][c & 1] += w[c];
      }
      pb[a][0] = transpose8(pack_f16x2(w[0] * wf, w[1] * wf));
      pb[a][1] = transpose8(pack_f16x2(w[2] * wf, w[3] * wf));
    }
    // this lane's run of channels of its four keys; the slot is free once they are read
    uint32_t vc[4][VW];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int r = 2 * t + (c & 1) + 8 * (c >> 1);
      if (D == 128) {
        const uint4 x = ld_shared_v4(vt + swz<D>(r, g));
        vc[c][0] = x.x;
        vc[c][1] = x.y;
        vc[c][VW - 2] = x.z;
        vc[c][VW - 1] = x.w;
      } else {
        const uint2 x = ld_shared_v2(vt + swz<D>(r, g / 2) + (g & 1) * 8);
        vc[c][0] = x.x;
        vc[c][1] = x.y;
      }
      if (r >= left) {                            // values past the limit may be anything
#pragma unroll
        for (int i = 0; i < VW; ++i) vc[c][i] = 0u;
      }
    }
    __syncwarp();
    if (issued < nk) {
      if ((issued & 31) == 0) {                   // the next 32 rows
        if (issued + lane < nk) ahead_row = fp8_row(p, (lo + (issued + lane) * kFewWarps) * 16);
      }
      issue(issued, __shfl_sync(0xffffffffu, ahead_row, issued & 31));
      ++issued;
    }
    // O^T += V^T P^T: 16 channels to a step, slot g of them channel 2 j of lane g's run, slot g + 8
    // channel 2 j + 1
#pragma unroll
    for (int wd = 0; wd < VW; ++wd) {
      const uint32_t a01 = __byte_perm(vc[0][wd], vc[1][wd], 0x5140);
      const uint32_t a23 = __byte_perm(vc[0][wd], vc[1][wd], 0x7362);
      const uint32_t b01 = __byte_perm(vc[2][wd], vc[3][wd], 0x5140);
      const uint32_t b23 = __byte_perm(vc[2][wd], vc[3][wd], 0x7362);
      const uint32_t v0[4] = {widen2(a01), widen2_high(a01), widen2(b01), widen2_high(b01)};
      const uint32_t v1[4] = {widen2(a23), widen2_high(a23), widen2(b23), widen2_high(b23)};
#pragma unroll
      for (int a = 0; a < NT; ++a) {
        mma_f16(o[a][2 * wd], v0, pb[a][0], pb[a][1]);
        mma_f16(o[a][2 * wd + 1], v1, pb[a][0], pb[a][1]);
      }
    }
  }

  // Every load was waited for, unless a wait ran out: then they are given time to land.
  if (!ok && lane == 0)
    for (int r = 0; r < NS && r < issued; ++r) {
      const int jl = issued - 1 - r;
      few_drain(full(jl % NS), (jl / NS) & 1);
    }
  // The ring is done with.  One warp's lost wait is the CTA's: it writes nothing (the parts of other
  // CTAs, and what a join makes of missing ones, are undefined after a timeout).
  if (!__syncthreads_and(ok)) return;
  // ---- join the warps
  float* const sm_m = reinterpret_cast<float*>(few_smem + L::M_OFF);
  float* const sm_l = reinterpret_cast<float*>(few_smem + L::L_OFF);
  float* const sm_o = reinterpret_cast<float*>(few_smem + L::O_OFF);
  int* const sm_e = reinterpret_cast<int*>(few_smem + L::E_OFF);
  if (lane == 0) sm_e[warp] = E;
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float l = sum[a][r];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      const int m = a * 8 + 2 * t + r;
      if (g == 0) {
        sm_m[warp * R + m] = mx[a][r];
        sm_l[warp * R + m] = l;
      }
      float* dst = sm_o + (warp * R + m) * L::OPITCH + (D / 8) * g;
#pragma unroll
      for (int j = 0; j < D / 16; j += 2)
        *reinterpret_cast<float4*>(dst + 2 * j) =
            make_float4(o[a][j][r], o[a][j][2 + r], o[a][j + 1][r], o[a][j + 1][2 + r]);
    }
  __syncthreads();
  constexpr int PER = D / 32;
  // outputs stand for o 2^E; sums and outputs share the factor 2^13.  2^E is multiplied in after the
  // division, so that values near the largest that fp32 holds do not overflow in the sum.
  int e_max = sm_e[0];
#pragma unroll
  for (int w = 1; w < kFewWarps; ++w) e_max = max(e_max, sm_e[w]);
  const float size = pow2f(e_max);
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
      const float wo = wt * pow2f(sm_e[w] - e_max);
#pragma unroll
      for (int c = 0; c < PER; ++c)
        acc[c] = fmaf(wo, sm_o[(w * R + m) * L::OPITCH + lane * PER + c], acc[c]);
    }
    // a row that sees no key (of this part): 0, log-sum-exp -inf; a NaN sum stays NaN
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float lse = l == 0.f ? -INFINITY : (top - kShiftBits + log2f(l)) * 0.69314718056f;
    const int row = seg_row0 + (m0 + m) / p.group, h = head * p.group + (m0 + m) % p.group;
    const int64_t orow = static_cast<int64_t>(row) * p.Hq + h;
    if (p.splits > 1) {
      float* dst = p.part_o + (static_cast<int64_t>(split) * p.T_q * p.Hq + orow) * D + lane * PER;
#pragma unroll
      for (int c = 0; c < PER; ++c) dst[c] = acc[c] * inv * size;
      if (lane == 0)
        p.part_lse[(static_cast<int64_t>(split) * p.Hq + h) * p.T_q + row] = lse;
    } else {
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + orow * D + lane * PER);
#pragma unroll
      for (int c = 0; c < PER / 2; ++c)
        dst[c] = pack_bf16x2(acc[2 * c] * inv * size, acc[2 * c + 1] * inv * size);
      if (lane == 0 && p.lse != nullptr) p.lse[static_cast<int64_t>(h) * p.T_q + row] = lse;
    }
  }
}

// Joins the parts of a split key range when rows are few and parts many: one block per (row, head),
//   lse = log sum_s exp(lse_s),  out = sum_s exp(lse_s - lse) O_s,
// eight warps over the parts.  (The merge kernel of the many-row path runs a warp per row over its
// parts one after the other: 18 us for 32 rows of 37 parts, against 3 here.)
constexpr int kJoinThreads = 256;
constexpr int kMaxJoin = 256;                       // parts
// Parts are summed with weights made smaller by this power of two, so that the sum of the most parts
// stays in range whatever the values.
constexpr float kJoinDown = 1.f / kMaxJoin, kJoinUp = kMaxJoin;

template <int D>
__global__ void __launch_bounds__(kJoinThreads)
    wf_join_kernel(const float* part_o, const float* part_lse, int splits, int T_q, int Hq,
                   __nv_bfloat16* out, float* lse) {
  constexpr int PER = D / 32;
  __shared__ float wt[kMaxJoin], red[kJoinThreads / 32], acc_s[kJoinThreads / 32][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int row = static_cast<int>(blockIdx.x) / Hq, h = static_cast<int>(blockIdx.x) % Hq;
  wait_for_previous();
  launch_next();
  const float ls = tid < splits
                       ? part_lse[(static_cast<int64_t>(tid) * Hq + h) * T_q + row] : -INFINITY;
  float top = ls;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) red[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kJoinThreads / 32; ++i) top = fmaxf(top, red[i]);
  const float ref = top == -INFINITY ? 0.f : top;
  const float w = expf(ls - ref);
  if (tid < splits) wt[tid] = w * kJoinDown;
  float sum = w;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncthreads();
  if (lane == 0) red[warp] = sum;
  float acc[PER];
#pragma unroll
  for (int c = 0; c < PER; ++c) acc[c] = 0.f;
  const float* src = part_o + (static_cast<int64_t>(row) * Hq + h) * D + lane * PER;
  const int64_t step = static_cast<int64_t>(T_q) * Hq * D;
#pragma unroll 8
  for (int s = warp; s < splits; s += kJoinThreads / 32) {
    float x[PER];
    if (PER == 4) {
      const float4 v = *reinterpret_cast<const float4*>(src + s * step);
      x[0] = v.x, x[1] = v.y, x[PER - 2] = v.z, x[PER - 1] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(src + s * step);
      x[0] = v.x, x[1] = v.y;
    }
#pragma unroll
    for (int c = 0; c < PER; ++c) acc[c] = fmaf(wt[s], x[c], acc[c]);
  }
#pragma unroll
  for (int c = 0; c < PER; ++c) acc_s[warp][lane * PER + c] = acc[c];
  __syncthreads();
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinThreads / 32; ++i) total += red[i];
  if (tid < D) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinThreads / 32; ++i) v += acc_s[i][tid];
    out[(static_cast<int64_t>(row) * Hq + h) * D + tid] =
        __float2bfloat16_rn(total == 0.f ? 0.f : v / total * kJoinUp);
  }
  if (tid == 0 && lse != nullptr)
    lse[static_cast<int64_t>(h) * T_q + row] = total == 0.f ? -INFINITY : ref + logf(total);
}

}  // namespace wfk
