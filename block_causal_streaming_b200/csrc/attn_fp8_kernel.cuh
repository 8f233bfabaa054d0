// attn_fp8_kernel.cuh -- attention straight over the FP8 cache for many query rows (sm_100a,
// tcgen05 + TMEM + TMA).
//
// The block-causal attention kernel's design (two 128-row Q tiles per CTA share every K/V tile,
// one S buffer the tiles take turns in, P in its own TMEM columns, QK^T and P.V issued by two
// threads) on keys and values that arrive as e4m3 codes, 16 KB a tile instead of 32:
//   - QK^T runs on the codes as they are (kind::f8f6f4).  A bf16 query value has 8 significant bits
//     and e4m3 has 4, so each row is split once into two e4m3 rows, hi + lo, under a power of two
//     for the row; S = hi K^T + lo K^T is the exact product for values down to 2^-10 of the row's
//     largest (and within 2^-18 of that largest below), at the time of one bf16 product.  The other
//     way, K to bf16 in shared memory, would double the converters' work and take 16 KB a tile more.
//   - The key scale of each 16 keys multiplies its 16 columns of S, inside the multiply-add that
//     subtracts the maximum; the maximum is taken over the 8 blocks' scaled maxima.
//   - Values go to f16 (exact) in shared memory, by four converter warps: 16 codes a step, times
//     2^(e_v - E + 7), E the largest value exponent of this CTA's keys (read up front; one byte for
//     16 keys).  What a block with a small scale loses lies below 2^-40 of the largest value.
//     f16 rather than bf16: one instruction widens two codes, and the weights keep 11 bits.
//   - Weights are f16, p 2^13 against a reference that trails the maximum by at most 2^2, so
//     p 2^13 <= 2^15: 11 bits down to 2^-27 of the largest weight, then steps of 2^-37 of it.
//     The row sum adds the weights before rounding, two at a time (so lse is good to fp32; a sum
//     of the rounded ones is off by 2^-12 / sqrt(keys)).  (A reference that may trail by 2^8, as where weights
//     are bf16, would leave f16 no room: steps of 2^-31, seen where blocks' values differ by 2^20.)
//
// A unit is one K/V head and up to 256 packed rows of ONE query segment; packed row m is query row
// m / group, head m % group of the K/V head's group, so heads that share keys share the tiles too.
// With one limit per unit nothing a row may not see is ever multiplied with a weight of 0 (0 x NaN):
// tiles past the limit are not read, the last tile's columns past it get weight 0 and its values
// are zeroed.
//
// One CTA an SM works through a list of pieces, a piece being a unit or a run of its key tiles: whole
// units first, unit k G + i to CTA i, then an even share of the tiles of the units that are left, cut
// wherever the share ends.  Pieces of a cut unit go to a workspace and are joined by a second
// launch.  So the SMs end together whatever the number of units (228 units of equal length on 148
// SMs: 1.54 units each, where whole units take 2 turns and uniform parts 4 to 5 percent of joining
// and 10 of idle SMs), and loads run ahead from one piece into the next.
//
// Bound by the chain that passes one S buffer between two Q tiles, no pipe in it full: MUFU 63 %, tensor
// pipe 61 %, issue slots 51 % (one chunk, counters); a pair of Q tiles takes 3240 cycles for a key tile,
// of which either pipe is busy for about 2048.  In long runs by the power limit too.  12 heads of 128: the
// 5-chunk wavefront (23 400 rows, up to 32 760 keys, 3.36 TFLOP) 3.00-3.12 ms call after call, 0.65 of a
// cuBLAS bf16 product (2.8 for the fastest single ones; the bf16 kernel takes 2.99 in the same loop); one
// chunk of 4680 rows against 37 440 keys 0.98-1.0 ms call after call, 860-910 us for a few; 12 heads of 64
// 763 us.  With no more than 128 packed rows a unit has one Q tile, half the softmax warps idle and the
// chain is serial: 128 rows of 12 heads 56 us (DRAM 17), MUFU and tensor pipe under 30 %.
// Steps on the way (the wavefront unless said otherwise): row sums with packed adds 3.50 -> 3.11 ms;
// pieces instead of uniform parts, one chunk 1000 -> 854 us; loops that fit the instruction cache
// (compact waits, one piece loop for the eight warps that are not softmax) were worth a factor 1.7.
//
// Warp roles (512 threads): 0-3, 4-7 softmax of Q tile 0, 1 (thread = row; they also split Q);
// 8 TMA of K, key scales; 9 issues QK^T; 10 issues P.V; 11 TMA of V codes; 12-15 convert V.  Rings
// and barrier phases run on over the pieces: `it` counts key tiles, and what belongs to one Q tile is
// counted for it alone, since a unit's last 128 rows may be missing.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cfloat>

#include "attn_fp8_few_kernel.cuh"
#include "attn_kernel.cuh"
#include "fp8_block_kernel.cuh"

namespace wfk {

constexpr int kFp8AttnThreads = 512;
constexpr int kFp8LaunchRegs = 128;          // 65536 / 512
constexpr int kFp8RegSoftmax = 200, kFp8RegOther = 2 * kFp8LaunchRegs - kFp8RegSoftmax;
static_assert(kFp8RegSoftmax % 8 == 0 && kFp8RegOther % 8 == 0 && kFp8RegOther >= 24,
              "setmaxnreg counts are multiples of 8");
static_assert(256 * kFp8RegSoftmax + 256 * kFp8RegOther <= 512 * kFp8LaunchRegs,
              "split exceeds the launch");

constexpr float kTrail = 2.f, kShift = 15.f - kTrail;   // weights: at most 2^15

constexpr int kFp8MaxCtas = 160;             // CTAs of a launch (one an SM)
constexpr int kUnitTileRows = 2 * kBM;       // packed rows of a unit

// The units of a launch: row blocks of the segments (most keys first), heads in groups; those that
// see no key come last and apart.
struct Fp8Units {
  int Hk, group, head_group;                 // head_group: K/V heads per dispatch group
  int pairs;                                 // row blocks that see keys
  int seg_pair_end[kFewSegs];                // row blocks up to and including segment i
  int seg_row0[kFewSegs];
  int seg_rows[kFewSegs];
  int seg_kv[kFewSegs];
};

struct UnitAt {
  int seg, m0, head;
};
__host__ __device__ __forceinline__ UnitAt unit_at(const Fp8Units& u, int unit) {
  const int per_group = u.pairs * u.head_group;
  const int hgrp = unit / per_group, in_group = unit - hgrp * per_group;
  const int block = in_group / u.head_group;
  UnitAt r;
  r.head = hgrp * u.head_group + in_group % u.head_group;
  r.seg = 0;
  while (block >= u.seg_pair_end[r.seg]) ++r.seg;
  r.m0 = (block - (r.seg > 0 ? u.seg_pair_end[r.seg - 1] : 0)) * kUnitTileRows;
  return r;
}

struct AttnFp8Params {
  CUtensorMap tm_k;  // e4m3 (D, Hk, num_pages * page_size), box (D, 1, box_rows), D-byte swizzle
  CUtensorMap tm_v;
  const __nv_bfloat16* q;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  const int* page_table;
  __nv_bfloat16* out;
  float* lse;
  float* part_o;                     // [slots][D / 4][256 packed rows][4], a slot for each part of a
                                     // cut unit: a thread's row is one of 256, so writes run along rows
  float* part_lse;                   // [slots][256]
  int* status;
  unsigned* grid_abort;
  unsigned launch_id;
  int T_q, Hq, Hk, page_size, num_pages, total_rows, box_rows;
  float sl2;                         // scale * log2(e)
  Fp8Units units;
  int n_whole;                       // the first n_whole units that see keys go out whole
  int n_blank;                       // units that see none
  // share of CTA i in the tiles of units n_whole ..: from tile share_tile[i] of unit share_unit[i],
  // share_tiles[i] of them; its parts of units go to the slots from share_slot[i] on
  int share_unit[kFp8MaxCtas];
  int share_tile[kFp8MaxCtas];
  int share_tiles[kFp8MaxCtas];
  int share_slot[kFp8MaxCtas];
};
static_assert(sizeof(AttnFp8Params) <= 4096, "kernel parameters");

// A piece of work, the same in every warp of the CTA.
struct Piece {
  int seg, m0, head, nq;             // nq: Q tiles with rows
  int n_max, kb, nk;                 // keys the rows see; tiles [kb, kb + nk) of them
  int m_total;                       // packed rows of the segment
  int slot;                          // workspace slot of a part, -1: whole
};
struct PieceList {
  int unit, share_unit, share_tile, share_left, slot, blank;
  __device__ __forceinline__ explicit PieceList(const AttnFp8Params& p) {
    const int i = static_cast<int>(blockIdx.x);
    unit = i;
    share_unit = p.share_unit[i];
    share_tile = p.share_tile[i];
    share_left = p.share_tiles[i];
    slot = p.share_slot[i];
    blank = i;
  }
  __device__ __forceinline__ bool next(const AttnFp8Params& p, Piece* w) {
    const Fp8Units& u = p.units;
    int at = unit, first = 0, len = -1;                // len < 0: to the end
    w->slot = -1;
    if (unit < p.n_whole) {
      unit += static_cast<int>(gridDim.x);
    } else if (share_left > 0) {
      at = share_unit++;
      first = share_tile;
      len = share_left;
      share_tile = 0;
    } else if (blank < p.n_blank) {
      const int block = u.pairs + blank / p.Hk;        // segments that see nothing: the last ones
      w->head = blank % p.Hk;
      blank += static_cast<int>(gridDim.x);
      int seg = 0;
      while (block >= u.seg_pair_end[seg]) ++seg;
      w->seg = seg;
      w->m0 = (block - (seg > 0 ? u.seg_pair_end[seg - 1] : 0)) * kUnitTileRows;
      w->m_total = u.seg_rows[seg] * u.group;
      w->nq = w->m0 + kBM < w->m_total ? 2 : 1;
      w->n_max = w->kb = w->nk = 0;
      return true;
    } else {
      return false;
    }
    const UnitAt r = unit_at(u, at);
    w->seg = r.seg;
    w->m0 = r.m0;
    w->head = r.head;
    w->m_total = u.seg_rows[r.seg] * u.group;
    w->nq = r.m0 + kBM < w->m_total ? 2 : 1;
    w->n_max = u.seg_kv[r.seg];
    const int tiles = (w->n_max + kBN - 1) / kBN;
    w->kb = first;
    w->nk = len < 0 ? tiles : min(tiles - first, len);
    if (len >= 0) {
      share_left -= w->nk;
      if (w->nk < tiles) w->slot = slot++;
    }
    return true;
  }
};

template <int D>
struct AttnFp8Smem {
  static constexpr int BN = kBN;
  static constexpr int DH = D / 64;                       // 128-byte halves of an f16 value row
  static constexpr int NK = D == 128 ? 4 : 6;             // K slots
  static constexpr int NC = D == 128 ? 2 : 4;             // V code slots
  static constexpr int NV = D == 128 ? 2 : 4;             // V f16 slots
  static constexpr uint32_t QTERM = kBM * D;              // one e4m3 term of a Q tile
  static constexpr uint32_t CTILE = BN * D;               // a tile of codes
  static constexpr uint32_t VHALF = BN * 128u;
  static constexpr uint32_t VTILE = DH * VHALF;           // a tile of f16 values
  static constexpr uint32_t Q_OFF = 0;                    // [2 tiles][hi, lo]
  static constexpr uint32_t K_OFF = Q_OFF + 4 * QTERM;
  static constexpr uint32_t C_OFF = K_OFF + NK * CTILE;
  static constexpr uint32_t V_OFF = C_OFF + NC * CTILE;
  static constexpr uint32_t KS_OFF = V_OFF + NV * VTILE;  // key scales [2 NK][8] floats
  static constexpr uint32_t BAR_OFF = KS_OFF + 2 * NK * 32;
  static constexpr int B_Q = 0, B_KF = 2, B_KE = B_KF + NK, B_CF = B_KE + NK, B_CE = B_CF + NC,
                       B_VF = B_CE + NC, B_VE = B_VF + NV, B_S = B_VE + NV, B_P = B_S + 2,
                       B_O = B_P + 2, B_SF = B_O + 2, B_DRAIN = B_SF + 1, B_EX = B_DRAIN + 2,
                       B_EM = B_EX + 1, NBAR = B_EM + 8;
  // Exponents E of the last 8 pieces.  A softmax reads its piece's before it hands over its last P,
  // and the conversion of V is at most NV tiles ahead of P.V and so NV + 1 pieces ahead of that.
  static constexpr int NE = 8;
  static_assert(NV + 1 < NE, "exponents kept");
  static constexpr uint32_t MISC_OFF = BAR_OFF + NBAR * 8;   // tmem base, abort flag
  static constexpr uint32_t EM_OFF = MISC_OFF + 8;           // E [NE], the warps' maxima [2][4]
  static constexpr uint32_t BYTES = EM_OFF + NE * 4 + 32;
  static constexpr uint32_t ALLOC = BYTES + 1024;         // slack for 1024-byte alignment
  static_assert(ALLOC <= 227u * 1024u, "shared memory per CTA exceeds 227 KB");
};

// Shared-memory matrix descriptor of a K-major tile of D-byte rows under the D-byte swizzle.
template <int D>
__device__ __forceinline__ uint64_t smem_desc_codes(uint32_t start) {
  if (D == 128) return smem_desc_sw128(start, 16, 1024);
  uint64_t d = 0;                                         // 64-byte swizzle: 8 rows are 512 bytes
  d |= static_cast<uint64_t>((start >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(1u) << 16;
  d |= static_cast<uint64_t>(512u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(4u) << 61;
  return d;
}

// Instruction descriptor for kind::f16 with f16 A/B, B MN-major, and fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_f16_f32_bmn(int M, int N) {
  return (1u << 4) | (1u << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ void st_shared_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z,
                                             uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t a) {
  const uint4 v = ld_shared_v4(a);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                     __uint_as_float(v.w));
}

// Bounded wait of this kernel: false once it has run for 2 s or another warp of the CTA has given up.
// It only reports; the caller leaves its loops and raises the CTA's flag and the status at the end of
// its role.  (The kernel has about twenty waits: with the whole of the general wait's slow path at
// each of them its loops no longer fit the instruction cache.)
__device__ __forceinline__ bool fp8_wait(uint32_t bar, uint32_t parity, volatile int* cta_abort) {
  uint64_t t0 = 0;
  for (uint32_t i = 0; !mbar_try(bar, parity);) {
    if ((++i & 255u) != 0) continue;
    const uint64_t now = globaltimer_ns();
    if (i == 256u) t0 = now;
    if (*cta_abort != 0 || now - t0 > kWaitTimeoutNs) return false;
  }
  return true;
}

template <int D>
__global__ void __launch_bounds__(kFp8AttnThreads, 1)
    wf_attn_fp8_kernel(const __grid_constant__ AttnFp8Params p) {
  using L = AttnFp8Smem<D>;
  constexpr int BN = L::BN, NK = L::NK, NC = L::NC, NV = L::NV;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + L::MISC_OFF);
  volatile int* const cta_abort = reinterpret_cast<volatile int*>(base_ptr + L::MISC_OFF + 4);
  int* const emax_slot = reinterpret_cast<int*>(base_ptr + L::EM_OFF);
  auto bar = [&](int i) -> uint32_t { return base + L::BAR_OFF + 8u * static_cast<uint32_t>(i); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::NBAR; ++i) {
      uint32_t count = 1;
      if (i < L::B_KF) count = 128u;
      else if (i >= L::B_CE && i < L::B_VE) count = 128u;       // V codes read, V f16 written
      else if (i >= L::B_S && i < L::B_P) count = 2u;           // commit and the issuer itself
      else if (i >= L::B_P && i < L::B_O) count = 128u;
      else if (i == L::B_SF || i == L::B_EX) count = 4u;
      mbar_init(bar(i), count);
    }
    mbar_init_fence();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  wait_for_previous();
  launch_next();
  if (threadIdx.x == 0) {
    *cta_abort = (*reinterpret_cast<volatile unsigned*>(p.grid_abort) == p.launch_id) ? 1 : 0;
    // (a captured launch keeps its id: a replay after a wait ran out says so again)
    if (*cta_abort) atomicCAS(p.status, 0, 6 /* WF_ERR_TIMEOUT */);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool skip = *cta_abort != 0;
  const WaitCtx w{cta_abort, p.grid_abort, p.status, p.launch_id, 6 /* WF_ERR_TIMEOUT */,
                  kWaitTimeoutNs};

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFp8RegSoftmax) : "memory");
    const int q = warp >> 2, wq = warp & 3;
    PieceList list(p);
    Piece pc;
    int done = 0;                      // tiles this Q tile has been through, over all pieces
    int tiles = 0, n_piece = 0;        // tiles and pieces with keys of the CTA
    bool ok = !skip;
    while (ok && list.next(p, &pc)) {
      const int nk = pc.nk;
      const int it = tiles, piece = n_piece;
      tiles += nk;
      n_piece += nk > 0;
      if (q >= pc.nq) continue;
      // ------------------------------------------------------------------ softmax warpgroups
      const int row = wq * 32 + lane;                       // row within the Q tile == TMEM lane
      const int m = pc.m0 + q * kBM + row;                  // packed row
      const bool live = m < pc.m_total;
      const int64_t qrow = p.units.seg_row0[pc.seg] + m / p.units.group;
      const int qhead = pc.head * p.units.group + m % p.units.group;
      const int64_t orow = qrow * p.Hq + qhead;
      float sl2 = 0.f;
      if (nk > 0) {
        // split this row into hi + lo e4m3 under 2^-e, and store both K-major
        uint4 x[D / 8];
        const uint4* src = reinterpret_cast<const uint4*>(p.q + orow * D);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) x[c] = live ? src[c] : make_uint4(0, 0, 0, 0);
        uint32_t mw = 0;                                    // largest |x|, as a bit pattern
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          mw = __vmaxu2(mw, x[c].x & 0x7FFF7FFFu);
          mw = __vmaxu2(mw, x[c].y & 0x7FFF7FFFu);
          mw = __vmaxu2(mw, x[c].z & 0x7FFF7FFFu);
          mw = __vmaxu2(mw, x[c].w & 0x7FFF7FFFu);
        }
        const uint32_t top = max(mw & 0xFFFFu, mw >> 16);   // an infinite value makes its row NaN
        const int e = scale_exponent(__uint_as_float(top << 16));
        const float f = top < 0x7F80u ? exp2_int(-e) : __uint_as_float(0x7FFFFFFFu);
        sl2 = p.sl2 * exp2_int(e);
        const uint32_t hi_t = base + L::Q_OFF + 2 * q * L::QTERM, lo_t = hi_t + L::QTERM;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t hw[4], lw[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {                     // 4 values: two words of bf16
            const uint4 v = x[2 * c + (i >> 1)];
            const uint32_t w0 = (i & 1) ? v.z : v.x, w1 = (i & 1) ? v.w : v.y;
            float4 y = make_float4(bf16_low(w0) * f, bf16_high(w0) * f, bf16_low(w1) * f,
                                   bf16_high(w1) * f);
            hw[i] = encode4(y);
            const float4 back = decode4(hw[i], 1.f);
            lw[i] = encode4(make_float4(y.x - back.x, y.y - back.y, y.z - back.z, y.w - back.w));
          }
          st_shared_v4(hi_t + swz<D>(row, c), hw[0], hw[1], hw[2], hw[3]);
          st_shared_v4(lo_t + swz<D>(row, c), lw[0], lw[1], lw[2], lw[3]);
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(L::B_Q + q));
      }
      const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
      const uint32_t tS = tmem + lane_off;                               // the shared S buffer
      const uint32_t tP = tmem + lane_off + 128u + static_cast<uint32_t>(q * 64);
      const uint32_t tO = tmem + lane_off + 256u + static_cast<uint32_t>(q * D);
      float m2 = -INFINITY;   // running reference of the base-2 logits
      float l = 0.f;          // running sum of exp2(t - m2 + kShift)
      int e_v = 0;            // E of the piece
      for (int j = 0; j < nk; ++j) {
        ok = __all_sync(0xffffffffu, fp8_wait(bar(L::B_S + q), (done + j) & 1, cta_abort));
        if (!ok) break;
        tc_fence_after();
        float s[BN];
        {
          uint32_t r[BN];
#pragma unroll
          for (int c = 0; c < BN / 32; ++c)
            tmem_ld32(tS + 32u * c, *reinterpret_cast<uint32_t(*)[32]>(&r[32 * c]));
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::B_SF));
#pragma unroll
          for (int c = 0; c < BN; ++c) s[c] = __uint_as_float(r[c]);
        }
        // logit factor of each block of 16 keys; kept positive so a masked column stays -inf
        const uint32_t ks = base + L::KS_OFF + static_cast<uint32_t>((it + j) % (2 * NK)) * 32u;
        const float4 ka = ld_shared_f4(ks), kc = ld_shared_f4(ks + 16);
        float f[8] = {ka.x, ka.y, ka.z, ka.w, kc.x, kc.y, kc.z, kc.w};
#pragma unroll
        for (int b = 0; b < 8; ++b) f[b] = fmaxf(f[b] * sl2, FLT_MIN);
        const int lim = pc.n_max - (pc.kb + j) * BN;        // visible columns of this tile
        if (lim < BN) {
#pragma unroll
          for (int c = 0; c < BN; ++c) s[c] = (c < lim) ? s[c] : -INFINITY;
        }
        float bm[8];
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const float* t = s + 16 * b;
          const float u = max3(t[0], t[1], t[2]), v = max3(t[3], t[4], t[5]);
          const float x = max3(t[6], t[7], t[8]), y = max3(t[9], t[10], t[11]);
          bm[b] = max3(max3(u, v, x), max3(y, t[12], t[13]), fmaxf(t[14], t[15])) * f[b];
        }
        const float tmax = max3(max3(bm[0], bm[1], bm[2]), max3(bm[3], bm[4], bm[5]),
                                fmaxf(bm[6], bm[7]));
        // the reference moves only when the maximum exceeds it by more than 2^kTrail
        const bool need = tmax > m2 + kTrail;
        float alpha = 1.f;
        if (need) {
          alpha = ex2_approx(m2 - tmax);                    // 0 on the first visible tile
          m2 = tmax;
        }
        const float mref = m2 == -INFINITY ? 0.f : m2 - kShift;
        const float2 negm = make_float2(-mref, -mref);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                         make_float2(0.f, 0.f)};
        uint32_t pk[BN / 2];
#pragma unroll
        for (int i = 0; i < BN / 2; ++i) {
          const float2 x = __ffma2_rn(make_float2(s[2 * i], s[2 * i + 1]),
                                      make_float2(f[i / 8], f[i / 8]), negm);
          const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
          pk[i] = pack_f16x2(e.x, e.y);
          acc[i & 3] = __fadd2_rn(acc[i & 3], e);
        }
        if (j > 0) {
          ok = __all_sync(0xffffffffu, fp8_wait(bar(L::B_O + q), (done + j - 1) & 1, cta_abort));
          if (!ok) break;
          tc_fence_after();
          if (__any_sync(0xffffffffu, need)) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t r[32];
              tmem_ld32(tO + 32u * c, r);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i)
                r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
              tmem_st32(tO + 32u * c, r);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < BN / 64; ++h)
          tmem_st32(tP + 32u * h, *reinterpret_cast<uint32_t(*)[32]>(&pk[32 * h]));
        {
          const float2 t = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
          l = l * alpha + (t.x + t.y);
        }
        if (j == nk - 1) {                                  // see NE
          ok = __all_sync(0xffffffffu, fp8_wait(bar(L::B_EM + piece % L::NE),
                                                 (piece / L::NE) & 1, cta_abort));
          if (!ok) break;
          e_v = emax_slot[piece % L::NE];
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(L::B_P + q));
      }
      // ------------------------------------------------------------------------- epilogue
      float inv = 0.f;
      if (nk > 0) {
        if (ok)
          ok = __all_sync(0xffffffffu, fp8_wait(bar(L::B_O + q), (done + nk - 1) & 1, cta_abort));
        tc_fence_after();
        if (ok) inv = l == 0.f ? 0.f : pow2f(e_v - 7) / l;
      }
      done += nk;
      if (ok) {
        // O / l: bf16 into `out`, or fp32 into the workspace for a part; 0 and -inf for rows that
        // see no key (of the part)
        const bool part = pc.slot >= 0;
        const int64_t prow = static_cast<int64_t>(pc.slot) * kUnitTileRows + q * kBM + row;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[32];
          if (nk > 0) {
            tmem_ld32(tO + 32u * c, r);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = 0u;
          }
          if (live && part) {
            float4* dst = reinterpret_cast<float4*>(p.part_o) +
                          (static_cast<int64_t>(pc.slot) * (D / 4) + 8 * c) * kUnitTileRows +
                          q * kBM + row;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i * kUnitTileRows] = make_float4(
                  __uint_as_float(r[4 * i]) * inv, __uint_as_float(r[4 * i + 1]) * inv,
                  __uint_as_float(r[4 * i + 2]) * inv, __uint_as_float(r[4 * i + 3]) * inv);
          } else if (live) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              pk[i] = pack_bf16x2(__uint_as_float(r[2 * i]) * inv,
                                  __uint_as_float(r[2 * i + 1]) * inv);
            uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D + 32 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
          }
        }
        const float lse = l == 0.f ? -INFINITY : (m2 - kShift + __log2f(l)) * 0.69314718056f;
        if (live && part) p.part_lse[prow] = lse;
        else if (live && p.lse != nullptr) p.lse[static_cast<int64_t>(qhead) * p.T_q + qrow] = lse;
      }
    }
    if (!ok && !skip) raise_abort(w);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFp8RegOther) : "memory");
    // One loop over the pieces for all of these warps (it is inlined where it stands).  `it` counts key
    // tiles over all pieces.
    const bool producer = warp == 8 || warp == 11, issuer = warp == 9 || warp == 10;
    bool ok = !skip && !(issuer && lane != 0);
    int it = 0;
    // TMA producers: K (with the key scales) or V codes
    const bool is_k = warp == 8;
    const CUtensorMap* const map = is_k ? &p.tm_k : &p.tm_v;
    const int ns = is_k ? NK : NC;
    const int bf = is_k ? L::B_KF : L::B_CF, be = is_k ? L::B_KE : L::B_CE;
    if (producer && lane == 0) tma_prefetch_desc(map);
    // V to f16: pieces so far, and the row of a tile this thread converts
    int piece = 0;
    const int key = threadIdx.x - 384;
    // issuers: S-free phases consumed (nothing to wait for before the first S), pieces each Q tile has
    // been part of, tiles Q tile 1 has been through (Q tile 0: all of them)
    int sf = -1, n_q0 = 0, n_q1 = 0, n_p1 = 0;

    PieceList list(p);
    Piece pc;
    while (ok && list.next(p, &pc)) {
      const int nk = pc.nk;
      if (nk == 0) continue;
      if (producer) {
        const int R = p.box_rows, nb = BN / R;             // page boxes per tile (<= BN / 16)
        auto box_row = [&](int t, int b) -> int {          // past the pool (zeros) beyond n_max
          const int tok = (pc.kb + t) * BN + b * R;
          if (b >= nb || t >= nk || tok >= pc.n_max) return p.total_rows;
          return fp8_row(p, tok);
        };
        // key scale of block `lane` of a tile (lanes 0..7)
        auto key_scale = [&](int t) -> float {
          const int tok = (pc.kb + t) * BN + lane * 16;
          if (!is_k || lane >= 8 || t >= nk || tok >= pc.n_max) return 1.f;
          const int r = fp8_row(p, tok);
          const uint32_t b = p.k_scale[static_cast<int64_t>(r / 16) * p.Hk + pc.head];
          return __uint_as_float(b << 23);
        };
        int coord = box_row(0, lane);                      // looked up one tile ahead
        float ks = key_scale(0);
#pragma unroll 1
        for (int j = 0; j < nk; ++j, ++it) {
          const int slot = it % ns;
          ok = fp8_wait(bar(be + slot), ((it / ns) & 1) ^ 1, cta_abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (is_k && lane < 8) {
            // Scales of tile `it` go to slot it mod 2 NK, last read for tile it - 2 NK.  This tile's
            // K slot was freed by QK^T of tile it - NK, issued after a softmax had read S of the tile
            // before that one; a Q tile that is not part of those tiles' units holds P.V, and with
            // it the other Q tile's next but one softmax, until it is done with its own last tile.
            *reinterpret_cast<float*>(base_ptr + L::KS_OFF + (it % (2 * NK)) * 32 + lane * 4) = ks;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(bar(bf + slot), L::CTILE);
          __syncwarp();
          if (lane < nb)                                   // a box a lane
            tma_load_3d(base + (is_k ? L::K_OFF : L::C_OFF) + slot * L::CTILE +
                            static_cast<uint32_t>(lane * R * D),
                        map, 0, pc.head, coord, bar(bf + slot));
          __syncwarp();
          if (j + 1 < nk) {
            coord = box_row(j + 1, lane);
            ks = key_scale(j + 1);
          }
        }
      } else if (warp >= 12) {
        const int first = pc.kb * BN, last = min((pc.kb + nk) * BN, pc.n_max);
        auto exponent = [&](int tok) -> int {              // value scale of a token's block, biased
          return p.v_scale[static_cast<int64_t>(fp8_row(p, tok) / 16) * p.Hk + pc.head];
        };
        // exponent of this thread's row of a tile, looked up a tile ahead; -1: nothing to see there
        auto row_exponent = [&](int t) -> int {
          const int tok = (pc.kb + t) * BN + key / 16 * 16;
          return t >= nk || tok >= pc.n_max ? -1 : exponent(tok);
        };
        int e_next = row_exponent(0);
        // the largest value exponent of this piece's keys
        int emax = 0;
#pragma unroll 1
        for (int tok = first + 16 * key; tok < last; tok += 16 * 128) emax = max(emax, exponent(tok));
        emax = __reduce_max_sync(0xffffffffu, emax);
        // One word per warp, in turn for even and odd pieces: a warp is at most one phase ahead.
        // (An mbarrier and no bar.sync: a warp whose wait runs out must not leave others waiting.)
        int* const em = emax_slot + L::NE + 4 * (piece & 1);
        if (lane == 0) {
          em[warp - 12] = emax;
          mbar_arrive(bar(L::B_EX));
        }
        ok = __all_sync(0xffffffffu, fp8_wait(bar(L::B_EX), piece & 1, cta_abort));
        if (!ok) break;
        emax = max(max(em[0], em[1]), max(em[2], em[3])) - 127;
        if (key == 0) {
          emax_slot[piece % L::NE] = emax;
          mbar_arrive(bar(L::B_EM + piece % L::NE));
        }
        ++piece;
#pragma unroll 1
        for (int j = 0; j < nk; ++j, ++it) {
          // 2^(e_v - E + 7) as two f16, 0 below their range
          const int e = e_next - 127 - emax + 7;
          uint32_t f = e_next < 0 ? 0u : e >= -14 ? static_cast<uint32_t>(e + 15) << 10
                       : e >= -24 ? 1u << (e + 24) : 0u;
          f |= f << 16;
          e_next = row_exponent(j + 1);
          const int cs = it % NC, vs = it % NV;
          ok = fp8_wait(bar(L::B_CF + cs), (it / NC) & 1, cta_abort) &&
               fp8_wait(bar(L::B_VE + vs), ((it / NV) & 1) ^ 1, cta_abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t src = base + L::C_OFF + cs * L::CTILE;
          const uint32_t dst = base + L::V_OFF + vs * L::VTILE;
          // zeros past the limit, whatever the bytes
          const uint32_t seen = (pc.kb + j) * BN + key < pc.n_max ? 0xFFFFFFFFu : 0u;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint4 v = ld_shared_v4(src + swz<D>(key, c));
            const uint32_t in[4] = {v.x & seen, v.y & seen, v.z & seen, v.w & seen};
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              o[2 * i] = mul_f16x2(widen2(in[i]), f);
              o[2 * i + 1] = mul_f16x2(widen2_high(in[i]), f);
            }
            // f16 channels 16 c .. 16 c + 15: pieces 2 c and 2 c + 1 of the 128-byte halves
            const uint32_t half = dst + static_cast<uint32_t>(c / 4) * L::VHALF;
            const int c2 = (c % 4) * 2;
            st_shared_v4(half + swz<128>(key, c2), o[0], o[1], o[2], o[3]);
            st_shared_v4(half + swz<128>(key, c2 + 1), o[4], o[5], o[6], o[7]);
          }
          fence_proxy_async_smem();
          mbar_arrive(bar(L::B_VF + vs));
          mbar_arrive(bar(L::B_CE + cs));
        }
      } else if (warp == 9) {
        // S(j, q) = (hi_q + lo_q) K_j^T: 2 D/32 steps of 32 channels into the shared S columns
        constexpr uint32_t idesc = idesc_e4m3_f32(kBM, BN);
        ok = fp8_wait(bar(L::B_Q), (n_q0++) & 1, cta_abort);
        if (ok && pc.nq > 1) ok = fp8_wait(bar(L::B_Q + 1), (n_q1++) & 1, cta_abort);
#pragma unroll 1
        for (int j = 0; ok && j < nk; ++j, ++it) {
          const uint64_t dk =
              smem_desc_codes<D>(base + L::K_OFF + static_cast<uint32_t>(it % NK) * L::CTILE);
          ok = fp8_wait(bar(L::B_KF + it % NK), (it / NK) & 1, cta_abort);
#pragma unroll 1
          for (int q = 0; ok && q < pc.nq; ++q) {
            if (sf >= 0) ok = fp8_wait(bar(L::B_SF), sf & 1, cta_abort);
            ++sf;
            if (!ok) break;
            tc_fence_after();
            const uint64_t dq = smem_desc_codes<D>(base + L::Q_OFF + 2u * q * L::QTERM);
#pragma unroll
            for (int kk = 0; kk < 2 * (D / 32); ++kk)
              umma_ss_f8(tmem, dq + ((kk / (D / 32) * L::QTERM + kk % (D / 32) * 32) >> 4),
                         dk + ((kk % (D / 32) * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
            umma_commit(bar(L::B_S + q));
            // a second, plain arrival: it hands on what this thread saw with K_j, the key scales
            mbar_arrive(bar(L::B_S + q));
          }
          if (ok) umma_commit(bar(L::B_KE + it % NK));               // K_j free
        }
      } else {
        // O_q += P_q(j) V_j
        constexpr uint32_t idesc = idesc_f16_f32_bmn(kBM, D);
#pragma unroll 1
        for (int j = 0; ok && j < nk; ++j, ++it) {
          const uint64_t dv = smem_desc_sw128(
              base + L::V_OFF + static_cast<uint32_t>(it % NV) * L::VTILE, L::VHALF, 1024);
          ok = fp8_wait(bar(L::B_VF + it % NV), (it / NV) & 1, cta_abort);
#pragma unroll 1
          for (int q = 0; ok && q < pc.nq; ++q) {
            ok = fp8_wait(bar(L::B_P + q), (q ? n_p1++ : it) & 1, cta_abort);
            if (!ok) break;
            tc_fence_after();
            const uint32_t pa = tmem + 128u + static_cast<uint32_t>(q * 64);
            const uint32_t od = tmem + 256u + static_cast<uint32_t>(q * D);
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
              umma_ts(od, pa + 8u * kk, dv + ((kk * 2048u) >> 4), idesc,
                      (j > 0 || kk > 0) ? 1u : 0u);
            umma_commit(bar(L::B_O + q));
          }
          if (ok) umma_commit(bar(L::B_VE + it % NV));               // V_j free
        }
      }
    }
    if (!ok && !skip && !(issuer && lane != 0)) raise_abort(w);
    if (producer && lane == 0) {
      // every load this warp issued must land before shared memory is released
      for (int r = 0; r < ns && r < it; ++r) {
        const int jl = it - 1 - r;
        mbar_wait_drain(bar(bf + jl % ns), (jl / ns) & 1);
      }
    }
    if (issuer && lane == 0) {
      // every MMA this thread issued must complete before TMEM is released
      umma_commit(bar(L::B_DRAIN + (warp - 9)));
      mbar_wait_drain(bar(L::B_DRAIN + (warp - 9)), 0);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of the units that were cut: out = sum_s exp(lse_s - lse) O_s.  A block takes
// kPieceJoinRows packed rows of a cut unit, a thread 4 channels of a row, rows fastest (the parts lie
// that way).  The parts of a cut unit lie in consecutive slots.
struct Fp8JoinParams {
  Fp8Units units;
  const float* part_o;
  const float* part_lse;
  __nv_bfloat16* out;
  float* lse;
  int T_q, Hq;
  int unit[kFp8MaxCtas];
  int slot[kFp8MaxCtas];     // of the unit's first part
  int parts[kFp8MaxCtas];
};

constexpr int kPieceJoinRows = 8;

template <int D>
__global__ void __launch_bounds__(kPieceJoinRows * D / 4)
    wf_piece_join_kernel(const __grid_constant__ Fp8JoinParams p) {
  constexpr int R = kPieceJoinRows, THREADS = R * D / 4;
  __shared__ float wt[kFp8MaxCtas][R];       // log-sum-exps of every part and row
  const int parts = p.parts[blockIdx.x];
  const int64_t slot0 = p.slot[blockIdx.x];
  const int tr = threadIdx.x % R, c = threadIdx.x / R;
  const int r0 = static_cast<int>(blockIdx.y) * R;
  const UnitAt at = unit_at(p.units, p.unit[blockIdx.x]);
  const int m = at.m0 + r0 + tr;
  if (at.m0 + r0 >= p.units.seg_rows[at.seg] * p.units.group) return;     // the whole block
  wait_for_previous();
  launch_next();
  for (int i = threadIdx.x; i < parts * R; i += THREADS)
    wt[i / R][i % R] = p.part_lse[(slot0 + i / R) * kUnitTileRows + r0 + i % R];
  const float4* o = reinterpret_cast<const float4*>(p.part_o) +
                    (slot0 * (D / 4) + c) * kUnitTileRows + r0 + tr;
  __syncthreads();
  if (m >= p.units.seg_rows[at.seg] * p.units.group) return;
  float top = -INFINITY;
  for (int s = 0; s < parts; ++s) top = fmaxf(top, wt[s][tr]);
  const float ref = top == -INFINITY ? 0.f : top;
  float total = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < parts; s0 += 8) {    // eight parts' values in flight
    float4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (s0 + i < parts) x[i] = o[static_cast<int64_t>(s0 + i) * (D / 4) * kUnitTileRows];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (s0 + i >= parts) break;
      const float w = expf(wt[s0 + i][tr] - ref);
      const float d = w * kJoinDown;
      total += w;
      acc.x = fmaf(d, x[i].x, acc.x);
      acc.y = fmaf(d, x[i].y, acc.y);
      acc.z = fmaf(d, x[i].z, acc.z);
      acc.w = fmaf(d, x[i].w, acc.w);
    }
  }
  static_assert(kFp8MaxCtas <= kMaxJoin, "parts of a unit");
  const float inv = total == 0.f ? 0.f : kJoinUp / total;
  const int64_t row = p.units.seg_row0[at.seg] + m / p.units.group;
  const int h = at.head * p.units.group + m % p.units.group;
  *reinterpret_cast<uint2*>(p.out + (row * p.Hq + h) * D + 4 * c) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (c == 0 && p.lse != nullptr)
    p.lse[static_cast<int64_t>(h) * p.T_q + row] = total == 0.f ? -INFINITY : ref + logf(total);
}

}  // namespace wfk
