// Dense attend over the paged cache: every new token attends to every key of
// its sequence (the layers of the model that select no blocks), split over the
// cache's length and joined.
//
// Definition.  Query token i of sequence s sits at position p = T - Q + i; with
// x_t = sm_scale <q, k_t> over the keys t <= p of the row's KV head,
//   m = max x_t, l = sum e^(x_t - m), out = (sum e^(x_t - m) v_t) / l, lse = m + ln l
// in one pass: a running (m, l, O) per row, rescaled when m grows, and partial
// results (m_i, l_i, O_i) joined by M = max m_i, l = sum e^(m_i - M) l_i and the
// same weights on O_i.  A row that sees no key has l = 0: out 0, lse -inf.
//
// Bound: HBM.  A key is read once for all the columns (query token, head) of
// its group: 8 flop a byte at 4 columns over FP8, far below the tensor rate, so
// the design is a stream of K / V tiles with as much in flight as fits.
//
// Split.  A unit is SK keys of one (sequence, group); the units of the batch,
// in (sequence, group, position) order, are cut into equal contiguous runs, one
// per CTA (one CTA an SM), whatever the lengths are: the lengths stay on the
// device and every CTA does the same work to within a unit.  A run crosses
// (sequence, group) borders; a segment it holds whole is written out at once,
// a cut one leaves its partial in the workspace (at most two a CTA), joined by
// the combine kernel.  No atomics: the result does not depend on timing.
//
// A CTA has one producer warp, which walks the run, publishes each segment's
// facts and query rows in one of two slots and streams the tiles through a
// ring of stages (tensor copies, mbarriers), and two groups of four consumer
// warps that take alternate units.  In a group the warps divide the unit as NT
// tiles of 16 columns x key ranges.
//
// Tensor-core mapping (mma.sync: 4 to 64 columns are far too few for a 128-row
// tile), queries as the 16 rows, so that P leaves the softmax in the layout in
// which it enters the second product, with no exchange between lanes:
//   S[col][key] = Q[col][:] . K[key][:]     (A = Q, B = K)
//   O[col][d]  += sum_key P[col][key] V[key][d]  (A = P, B = V)
//   FP8    K enters e4m3 MMAs as it is, a bf16 query as e4m3 hi + lo terms after
//          a power-of-two row scale (exact to 2^-10 of the row's 448); with up
//          to 8 columns the lo terms are the tile's rows 8 to 15 and cost
//          nothing.  V becomes f16 (exact) and P x vscale f16 (11 bits).
//   NVFP4  K and V become f16 in registers (e2m1 x e4m3 fits 6 bits: exact).
//   BF16   as it is; P enters as bf16 hi + lo terms (16 bits; with up to 8
//          columns again in the rows 8 to 15), since one bf16 term alone would
//          add an error as large as the output's own rounding.
// P is scaled by 2^14 where it becomes f16, l with it, so that f16's range
// reaches 2^-28 of the row's largest weight before it loses bits.
//
// A masked key's logit is replaced, not multiplied; in units that hold masked
// keys V is masked in registers too, so NaN or infinity in rows past the end of a
// sequence, or in a later token's row, reaches no output (0 x inf is NaN).
#pragma once

#include "msa_device.cuh"
#include "msa_internal.h"

namespace msa {

constexpr int kDenseGroups = 2;   // consumer groups, alternate units
constexpr int kDenseWpg = 4;      // warps a group
constexpr int kDenseWarps = kDenseGroups * kDenseWpg;
constexpr int kDenseConsumers = 32 * kDenseWarps;
constexpr int kDenseThreads = kDenseConsumers + 32;
constexpr float kDensePShift = 14.f;  // log2 of the scale of P (f16 formats)

template <int FMT>
struct DenseTraits;
template <>
struct DenseTraits<FMT_FP8> {
  static constexpr int SK = 128, TILE = 128 * 128, SC = 512;  // keys, bytes of a K or V tile, of its scales
};
template <>
struct DenseTraits<FMT_BF16> {
  static constexpr int SK = 64, TILE = 64 * 256, SC = 0;
};
template <>
struct DenseTraits<FMT_NVFP4> {
  static constexpr int SK = 128, TILE = 128 * 64, SC = 1024;
};

// What the producer publishes for one segment (the CTA's part of one sequence and group).
struct DenseFacts {
  int32_t s, g, cg;       // sequence, KV head, group of columns
  int32_t T;              // sequence length
  int32_t k0, n;          // first unit of the segment within the sequence, units; n = -1: no more segments
  int32_t part;           // partial slot, or -1: the segment is whole
  int32_t pad;
};

// NT: tiles of 16 query columns; R8: NT = 1 and at most 8 columns.
template <int FMT, int NT, bool R8>
struct DenseLayout {
  using T = DenseTraits<FMT>;
  static constexpr int ROWS = R8 ? 8 : 16 * NT;  // columns (query rows) of a unit
  static constexpr int TR = R8 ? 8 : 16;         // of one warp
  static constexpr size_t STAGE = 2 * (size_t)T::TILE;  // K tile, V tile
  static constexpr size_t SCALES = 2 * (size_t)T::SC;   // their scales, in a region of their own
  static constexpr int DCH = R8 ? 64 : 32;       // output dims a merge pass takes
  static constexpr int MROW = DCH + 4;           // padded row of the merge area
  static constexpr size_t MERGE_BYTES = (size_t)kDenseWarps * TR * MROW * 4;
  static constexpr size_t ML_BYTES = (size_t)kDenseWarps * TR * 8;
  static constexpr int QROW = 272;               // a query row, padded (conflict-free reads)
  static constexpr size_t QSLOT = (size_t)ROWS * QROW;
  static constexpr size_t FIXED = MERGE_BYTES + ML_BYTES + 2 * QSLOT + 2 * sizeof(DenseFacts) + 512;
  // Ring stages: an even number, so that a stage always belongs to the same
  // consumer group and the group sees every phase of its barriers.
  static constexpr int NST = (int)((227 * 1024 - 1024 - FIXED) / (STAGE + SCALES)) / 2 * 2;
  static constexpr size_t SC = STAGE * NST;
  static constexpr size_t MERGE = SC + SCALES * NST;
  static constexpr size_t ML = MERGE + MERGE_BYTES;
  static constexpr size_t Q = ML + ML_BYTES;
  static constexpr size_t FACTS = Q + 2 * QSLOT;
  static constexpr size_t BARS = FACTS + 2 * sizeof(DenseFacts);
  static constexpr size_t TOTAL = BARS + 8 * (2 * NST + 4) + 4 * NST + 16;
  static constexpr size_t SMEM = TOTAL + 1024;
  static_assert(SMEM <= 227 * 1024 && NST >= 4 && NST <= 16 && NST % kDenseGroups == 0, "stages");
  static_assert(STAGE % 1024 == 0 && MERGE_BYTES % 16 == 0 && ML_BYTES % 16 == 0 && QSLOT % 16 == 0, "alignment");
};

namespace dense {

__device__ __forceinline__ uint32_t swz128(uint32_t base, int row, int chunk) {
  return base + row * 128 + ((chunk ^ (row & 7)) << 4);
}
// 64-byte rows under the 64-byte swizzle
__device__ __forceinline__ uint32_t swz64(uint32_t base, int row, int chunk) {
  return base + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {  // the low two codes
  uint32_t h;
  asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo; }" : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t w) {  // the high two
  uint32_t h;
  asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, hi; }" : "=r"(h) : "r"(w));
  return h;
}
// the four bytes of packed e2m1 codes of w as four f16 pairs (low nibble first)
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{ .reg .b8 b0, b1, b2, b3; mov.b32 {b0, b1, b2, b3}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, b0; cvt.rn.f16x2.e2m1x2 %1, b1; cvt.rn.f16x2.e2m1x2 %2, b2; cvt.rn.f16x2.e2m1x2 %3, b3; }"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float2 lds_f2(const float* p) { return *reinterpret_cast<const float2*>(p); }

__device__ __forceinline__ bool is_dead(const int* flag) { return *reinterpret_cast<const volatile int*>(flag) != 0; }
__device__ __forceinline__ void set_dead(int* flag, DeviceStatus* st, int detail) {
  if (!is_dead(flag)) raise_flag(st, FLAG_TIMEOUT, detail);
  *reinterpret_cast<volatile int*>(flag) = 1;
}
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, const int* dead) {
  if (is_dead(dead)) return false;
  return mbar_wait_warp(bar, parity);
}

// Units of a sequence of length T (0: malformed or empty).
template <int SK>
__device__ __forceinline__ int units_of(int T, int max_nb) {
  return (T < 1 || T > max_nb * kBlock) ? 0 : (T + SK - 1) / SK;
}

__device__ __forceinline__ long warp_sum(long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ long warp_scan(long v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// ---------------------------------------------------------------- the producer warp

template <int FMT, int NT, bool R8>
__device__ void producer(const CUtensorMap* tmk, const CUtensorMap* tmv, const DenseParams& p, uint8_t* base,
                         uint64_t* full, uint64_t* empty, uint64_t* ifull, uint64_t* iempty, int* dead,
                         DenseFacts* facts, int* stage_ok, int lane) {
  using TR = DenseTraits<FMT>;
  using LY = DenseLayout<FMT, NT, R8>;
  constexpr int NST = LY::NST;
  const int S = p.S, max_nb = p.max_nb;
  const long GC = (long)p.G * p.CG;
  // units in all, then the run of this CTA: [u0, u1)
  long total = 0;
#pragma unroll 4
  for (int s = lane; s < S; s += 32) total += units_of<TR::SK>(__ldg(p.seq_lens + s), max_nb);
  total = warp_sum(total) * GC;
  const long grid = total < (long)gridDim.x ? total : (long)gridDim.x;
  const long c = blockIdx.x;
  long u0 = 0, u1 = 0;
  if (c < grid) {
    u0 = c * total / grid;
    u1 = (c + 1) * total / grid;
  }
  // the sequence that holds u0: sb units (x GC) come before it
  int s = 0;
  long sb = 0;
  if (u1 > u0) {
    for (int s0 = 0; s0 < S; s0 += 32) {
      const long mine = s0 + lane < S ? GC * units_of<TR::SK>(__ldg(p.seq_lens + s0 + lane), max_nb) : 0;
      const long incl = warp_scan(mine, lane);
      const uint32_t over = __ballot_sync(0xffffffffu, sb + incl > u0);
      if (over) {
        const int l = __ffs(over) - 1;
        s = s0 + l;
        sb += __shfl_sync(0xffffffffu, incl - mine, l);
        break;
      }
      sb += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  // what the combine reads: the segment the run begins in, and whether it began before
  long u = u0;
  int bi = 0, ii = 0;
  bool ok = true;
  bool first = true;
  if (u1 <= u0 && lane == 0) p.info[c] = make_int2(-1, 0);
#pragma unroll 1
  while (u < u1 && ok) {
    const int T = __ldg(p.seq_lens + s);
    const int un = units_of<TR::SK>(T, max_nb);
    if (un == 0) {  // an empty sequence holds no units
      ++s;
      continue;
    }
    const long in_s = u - sb;
    const int gc = (int)(in_s / un), k0 = (int)(in_s - (long)gc * un);
    const long left = u1 - u;
    const int n = left < (long)(un - k0) ? (int)left : un - k0;
    const int g = gc / p.CG, cg = gc - g * p.CG;
    const bool cut_start = k0 > 0, cut_end = k0 + n < un;
    const int sg = (int)((long)s * GC + gc);
    if (first && lane == 0) p.info[c] = make_int2(sg, cut_start ? 1 : 0);
    first = false;
    // publish the segment and its query rows
    const int slot = ii & 1, use = ii >> 1;
    if (use > 0 && !ring_wait(&iempty[slot], (uint32_t)((use - 1) & 1), dead)) {
      set_dead(dead, p.status, sg);
      ok = false;
      break;
    }
    const int qrow_bytes = p.q_fp8 ? 128 : 256;
    const int c0 = cg * LY::ROWS;
    const int nrows = p.cols - c0 < LY::ROWS ? p.cols - c0 : LY::ROWS;
    if (lane == 0) {
      DenseFacts& f = facts[slot];
      f.s = s;
      f.g = g;
      f.cg = cg;
      f.T = T;
      f.k0 = k0;
      f.n = n;
      f.part = (cut_start || cut_end) ? (int)(2 * c + (cut_start ? 0 : 1)) : -1;
      fence_proxy_async();
      mbar_expect_tx(&ifull[slot], (uint32_t)(nrows * qrow_bytes));
    }
    __syncwarp();
    for (int row = lane; row < nrows; row += 32) {
      const int col = c0 + row, i = col / p.r, h = col - i * p.r;
      const size_t src = ((size_t)s * p.Q + i) * ((size_t)p.G * p.r) + (size_t)g * p.r + h;
      bulk_g2s(base + LY::Q + (size_t)slot * LY::QSLOT + (size_t)row * LY::QROW,
               static_cast<const uint8_t*>(p.q) + src * qrow_bytes, (uint32_t)qrow_bytes, &ifull[slot]);
    }
    ++ii;
    // its tiles, 32 block-table entries at a time
    const int32_t* row = p.block_table + (size_t)s * max_nb;
    constexpr int UPB = kBlock / TR::SK;  // units a block
    int b_have = -1, phys = -1;           // entries [b_have, b_have + 32) one per lane
#pragma unroll 1
    for (int k = k0; k < k0 + n; ++k) {
      const int b = k / UPB, half = k - b * UPB;
      if (b_have < 0 || b >= b_have + 32) {
        b_have = b;
        const int mine = b + lane;
        phys = -1;
        if (mine * UPB < k0 + n) {
          const int ph = __ldg(row + mine);
          if (ph < 0 || ph >= p.num_blocks) raise_flag(p.status, FLAG_BAD_BLOCK, ph);
          else phys = ph;
        }
      }
      const int ph = __shfl_sync(0xffffffffu, phys, b - b_have);
      const int st = bi % NST, ub = bi / NST;
      if (ub > 0 && !ring_wait(&empty[st], (uint32_t)((ub - 1) & 1), dead)) {
        set_dead(dead, p.status, sg);
        ok = false;
        break;
      }
      if (lane == 0) {
        stage_ok[st] = ph >= 0 ? 1 : 0;
        if (ph >= 0) {
          uint8_t* stg = base + (size_t)st * LY::STAGE;
          const size_t tile = (size_t)ph * p.G + g;
          const int y = (int)(tile * kBlock) + half * TR::SK;
          fence_proxy_async();
          mbar_expect_tx(&full[st], (uint32_t)(LY::STAGE + LY::SCALES));
          if constexpr (FMT == FMT_BF16) {
            tma_load_2d(stg, tmk, 0, y, &full[st]);
            tma_load_2d(stg + TR::SK * 128, tmk, 64, y, &full[st]);
            tma_load_2d(stg + TR::TILE, tmv, 0, y, &full[st]);
            tma_load_2d(stg + TR::TILE + TR::SK * 128, tmv, 64, y, &full[st]);
          } else {
            tma_load_2d(stg, tmk, 0, y, &full[st]);
            tma_load_2d(stg + TR::TILE, tmv, 0, y, &full[st]);
            uint8_t* sc = base + LY::SC + (size_t)st * LY::SCALES;
            bulk_g2s(sc, p.k_sc + tile * TR::SC, TR::SC, &full[st]);
            bulk_g2s(sc + TR::SC, p.v_sc + tile * TR::SC, TR::SC, &full[st]);
          }
        } else {
          mbar_arrive(&full[st]);  // a rejected block: an empty phase keeps the ring in step
        }
      }
      ++bi;
    }
    u += n;
    if (u >= sb + (long)un * GC) {
      sb += (long)un * GC;
      ++s;
    }
  }
  if (ok) {
    const int slot = ii & 1, use = ii >> 1;
    if (use > 0 && !ring_wait(&iempty[slot], (uint32_t)((use - 1) & 1), dead)) {
      set_dead(dead, p.status, -1);
    } else if (lane == 0) {
      facts[slot].n = -1;
      mbar_arrive(&ifull[slot]);
    }
    ++ii;
  }
  // before exiting, let the last copy into every stage and slot land (immediate
  // in a healthy run: the consumers waited for all of them)
  if (lane == 0) {
    for (int st = 0; st < NST; ++st) {
      const int uses = bi > st ? (bi - 1 - st) / NST + 1 : 0;
      if (uses > 0) mbar_wait(&full[st], (uint32_t)((uses - 1) & 1), 2000);
    }
    for (int sl = 0; sl < 2; ++sl) {
      const int uses = ii > sl ? (ii - 1 - sl) / 2 + 1 : 0;
      if (uses > 0) mbar_wait(&ifull[sl], (uint32_t)((uses - 1) & 1), 2000);
    }
  }
}

// ---------------------------------------------------------------- consumer pieces

// The A fragments of a warp's 16 query columns (rows g8 and g8 + 8 of the
// tile) from the raw query rows in shared memory, and the factor of each row's
// logits (log2 domain).
//   FP8    a[0]: hi terms (R8: rows 8-15 the lo terms of columns 0-7), a[1]: lo
//   16-bit a[0][ks]: k slots of lane j as in slot_dim()
template <int FMT>
struct QRegs {
  static constexpr int KS = FMT == FMT_FP8 ? 4 : 8;
};

template <int FMT>
__device__ __forceinline__ int slot_dim(int ks, int hi, int j) {  // first dim of k slots 2j (hi = 0) or 2j + 8
  if constexpr (FMT == FMT_FP8) return 32 * ks + 16 * hi + 4 * j;
  else if constexpr (FMT == FMT_BF16) return 16 * ks + 8 * hi + 2 * j;
  else return 32 * j + 4 * ks + 2 * hi;  // NVFP4: a lane's 32 consecutive dims
}

__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// qs: the rows of the segment's columns, QROW bytes apart.
template <int FMT, bool R8, int SP, int QROW>
__device__ __forceinline__ void load_q(const uint8_t* qs, int row0, int nrows, bool q_fp8, float q_scale, float cst,
                                       int lane, uint32_t (&a)[SP][QRegs<FMT>::KS][4], float (&colf)[2]) {
  constexpr int KS = QRegs<FMT>::KS;
  constexpr int W = FMT == FMT_FP8 ? 2 : 1;  // words of two elements a (k step, half) takes
  const int g8 = lane >> 2, j = lane & 3;
#pragma unroll
  for (int rr = 0; rr < (R8 ? 1 : 2); ++rr) {
    const int row = row0 + g8 + 8 * rr;
    const bool have = row < nrows;
    const uint8_t* src = qs + (size_t)row * QROW;
    if (q_fp8) {
      // E4M3 codes: as they are, or widened exactly
      colf[rr] = q_scale * cst;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
          const int d = slot_dim<FMT>(ks, hi, j);
          uint32_t w = 0;
          if constexpr (FMT == FMT_FP8) {
            if (have) w = *reinterpret_cast<const uint32_t*>(src + d);
          } else {
            const uint32_t c2 = have ? *reinterpret_cast<const uint16_t*>(src + d) : 0u;
            if constexpr (FMT == FMT_BF16) {
              const float2 v = e4m3x2_to_float2((uint16_t)c2);
              w = pack_bf16x2(v.x, v.y);
            } else {
              w = e4m3x2_to_f16x2(c2);
            }
          }
          a[0][ks][rr + 2 * hi] = w;
          if constexpr (R8) a[0][ks][1 + 2 * hi] = 0u;
          else if constexpr (SP == 2) a[1][ks][rr + 2 * hi] = 0u;
        }
      continue;
    }
    uint32_t raw[KS][2][W];
    float amax = 0.f;
    bool bad = false;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        const uint8_t* at = src + 2 * slot_dim<FMT>(ks, hi, j);
        if constexpr (FMT == FMT_FP8) {
          const uint2 w = have ? *reinterpret_cast<const uint2*>(at) : make_uint2(0u, 0u);
          raw[ks][hi][0] = w.x;
          raw[ks][hi][W - 1] = w.y;
        } else {
          raw[ks][hi][0] = have ? *reinterpret_cast<const uint32_t*>(at) : 0u;
        }
        if constexpr (FMT != FMT_BF16) {
#pragma unroll
          for (int t = 0; t < W; ++t) {
            const float2 v = bf16x2_to_float2(raw[ks][hi][t] & 0x7fff7fffu);
            amax = fmaxf(amax, fmaxf(v.x, v.y));
            bad |= !(v.x <= 3.4e38f) || !(v.y <= 3.4e38f);
          }
        }
      }
    float ps = 1.f, back = 1.f;
    if constexpr (FMT != FMT_BF16) {
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      bad = ((__ballot_sync(0xffffffffu, bad) >> (4 * g8)) & 0xfu) != 0;
      int e = pow2_fit(amax, FMT == FMT_FP8 ? 448.f : 16384.f);
      e = e < -126 ? -126 : (e > 126 ? 126 : e);
      ps = pow2i(e);
      back = pow2i(-e);
    }
    // a query row that is not finite has no finite logits; the reduced formats would hide that
    colf[rr] = bad ? __int_as_float(0x7fc00000) : back * cst;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        uint32_t h = 0, l = 0;
        if constexpr (FMT == FMT_FP8) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float2 x = bf16x2_to_float2(raw[ks][hi][t]);
            const uint16_t hw = pack_e4m3x2(x.x * ps, x.y * ps);
            const float2 hv = e4m3x2_to_float2(hw);
            h |= (uint32_t)hw << (16 * t);
            l |= (uint32_t)pack_e4m3x2(x.x * ps - hv.x, x.y * ps - hv.y) << (16 * t);
          }
        } else if constexpr (FMT == FMT_BF16) {
          h = raw[ks][hi][0];
        } else {
          const float2 x = bf16x2_to_float2(raw[ks][hi][0]);
          h = pack_f16x2(x.x * ps, x.y * ps);
        }
        a[0][ks][rr + 2 * hi] = h;
        if constexpr (R8) a[0][ks][1 + 2 * hi] = l;
        else if constexpr (SP == 2) a[1][ks][rr + 2 * hi] = l;
      }
  }
  if constexpr (R8) colf[1] = 0.f;
}

// S of KC keys from key row kb of the tile.
template <int FMT, bool R8, int SP, bool NVR, int KC>
__device__ __forceinline__ void logits(const uint8_t* stg, const uint8_t* sc, int kb, int lane,
                                       const uint32_t (&a)[SP][QRegs<FMT>::KS][4], float (&sacc)[KC / 8][4]) {
  using TR = DenseTraits<FMT>;
  const uint32_t kt = smem_u32(stg);
#pragma unroll
  for (int t = 0; t < KC / 8; ++t) {
    sacc[t][0] = sacc[t][1] = sacc[t][2] = sacc[t][3] = 0.f;
    if constexpr (FMT == FMT_FP8) {
      const int row = kb + 8 * t + (lane & 7);
#pragma unroll
      for (int kp = 0; kp < 2; ++kp) {
        uint32_t b[4];
        ldmatrix_x4(b, swz128(kt, row, 4 * kp + (lane >> 3)));
        mma_e4m3_k32(sacc[t], a[0][2 * kp], b[0], b[1]);
        mma_e4m3_k32(sacc[t], a[0][2 * kp + 1], b[2], b[3]);
        if constexpr (SP == 2) {
          mma_e4m3_k32(sacc[t], a[1][2 * kp], b[0], b[1]);
          mma_e4m3_k32(sacc[t], a[1][2 * kp + 1], b[2], b[3]);
        }
      }
    } else if constexpr (FMT == FMT_BF16) {
      const int row = kb + 8 * t + (lane & 7);
      float s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kp = 0; kp < 4; ++kp) {
        uint32_t b[4];
        ldmatrix_x4(b, swz128(kt + (kp >> 1) * (TR::SK * 128), row, 4 * (kp & 1) + (lane >> 3)));
        mma_bf16_k16(sacc[t], a[0][2 * kp], b[0], b[1]);
        mma_bf16_k16(s2, a[0][2 * kp + 1], b[2], b[3]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sacc[t][e] += s2[e];
    } else {
      const int g8 = lane >> 2, j = lane & 3;
      const int row = kb + 8 * t + g8;
      uint4 w;
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                   : "r"(swz64(kt, row, j)));
      const uint32_t s2 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(sc + row * 8 + 2 * j));
      const uint32_t sA = __byte_perm(s2, s2, 0x1010), sB = __byte_perm(s2, s2, 0x3232);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // 8 dims: two k steps
        uint32_t h[4];
        e2m1x8_to_f16(ww[q], h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[i] = hmul2(h[i], q < 2 ? sA : sB);
          if constexpr (NVR) h[i] = e4m3_round_f16x2(h[i]);
        }
        mma_f16_k16(sacc[t], a[0][2 * q], h[0], h[1]);
        mma_f16_k16(sacc[t], a[0][2 * q + 1], h[2], h[3]);
      }
    }
  }
}

// One accumulator tile += A B.  MASK: only the rows that are kept (0 x NaN is NaN
// in every row of a product).
template <int FMT, bool R8, bool MASK>
__device__ __forceinline__ void mma_rows(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool keep0,
                                         bool keep1) {
  if constexpr (!MASK) {
    if constexpr (FMT == FMT_BF16) mma_bf16_k16(d, a, b0, b1);
    else mma_f16_k16(d, a, b0, b1);
  } else {
    float t[4] = {d[0], d[1], d[2], d[3]};
    if constexpr (FMT == FMT_BF16) mma_bf16_k16(t, a, b0, b1);
    else mma_f16_k16(t, a, b0, b1);
    d[0] = keep0 ? t[0] : d[0];
    d[1] = keep0 ? t[1] : d[1];
    d[2] = (R8 ? keep0 : keep1) ? t[2] : d[2];
    d[3] = (R8 ? keep0 : keep1) ? t[3] : d[3];
  }
}

// O += P V over 16 keys from key row kb; pa (and pl, the lo terms of bf16) are
// P's A fragments.  MASK: V of the keys beyond row klim of the tile counts as 0,
// and only the lane's rows g8 (keep0) and g8 + 8 (keep1) are added to.
template <int FMT, bool R8, bool NVR, bool MASK>
__device__ __forceinline__ void pv16(const uint8_t* stg, const uint8_t* vs, int kb, int klim, int lane, const uint32_t (&pa)[4],
                                     const uint32_t (&pl)[4], float (&o)[16][4], bool keep0, bool keep1) {
  using TR = DenseTraits<FMT>;
  const uint32_t vt = smem_u32(stg + TR::TILE);
  const int j = lane & 3;
  const int mrow = kb + (lane & 7) + ((lane >> 3) & 1) * 8, mch = lane >> 4;
  uint32_t m0 = 0xffffffffu, m1 = 0xffffffffu;  // keys 2j, 2j + 1 and 2j + 8, 2j + 9 of the step
  if constexpr (MASK) {
    const int k = kb + 2 * j;
    m0 = (k <= klim ? 0xffffu : 0u) | (k + 1 <= klim ? 0xffff0000u : 0u);
    m1 = (k + 8 <= klim ? 0xffffu : 0u) | (k + 9 <= klim ? 0xffff0000u : 0u);
  }
  if constexpr (FMT == FMT_FP8) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t r[4];
      ldmatrix_x4_trans(r, swz128(vt, mrow, 2 * c + mch));
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t x0 = __byte_perm(r[2 * q], 0u, 0x3120), x1 = __byte_perm(r[2 * q + 1], 0u, 0x3120);
        uint32_t b0 = e4m3x2_to_f16x2(x0), b1 = e4m3x2_to_f16x2(x1);
        uint32_t d0 = e4m3x2_hi_to_f16x2(x0), d1 = e4m3x2_hi_to_f16x2(x1);
        if constexpr (MASK) {
          b0 &= m0;
          d0 &= m0;
          b1 &= m1;
          d1 &= m1;
        }
        mma_rows<FMT, R8, MASK>(o[2 * (2 * c + q)], pa, b0, b1, keep0, keep1);
        mma_rows<FMT, R8, MASK>(o[2 * (2 * c + q) + 1], pa, d0, d1, keep0, keep1);
      }
    }
  } else if constexpr (FMT == FMT_BF16) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint32_t r[4];
      ldmatrix_x4_trans(r, swz128(vt + (c >> 2) * (TR::SK * 128), mrow, 2 * (c & 3) + mch));
      if constexpr (MASK) {
        r[0] &= m0;
        r[1] &= m1;
        r[2] &= m0;
        r[3] &= m1;
      }
      mma_rows<FMT, R8, MASK>(o[2 * c], pa, r[0], r[1], keep0, keep1);
      mma_rows<FMT, R8, MASK>(o[2 * c + 1], pa, r[2], r[3], keep0, keep1);
      if constexpr (!R8) {
        mma_rows<FMT, R8, MASK>(o[2 * c], pl, r[0], r[1], keep0, keep1);
        mma_rows<FMT, R8, MASK>(o[2 * c + 1], pl, r[2], r[3], keep0, keep1);
      }
    }
  } else {
    // the scales of this lane's keys (2j, 2j + 1, 2j + 8, 2j + 9), of the groups 2c + (g8 >> 2)
    const uint8_t* sf = vs + (kb + 2 * j) * 8;
    const int sh = (lane >> 4) * 8;
    uint2 w[4];
    w[0] = *reinterpret_cast<const uint2*>(sf);
    w[1] = *reinterpret_cast<const uint2*>(sf + 8);
    w[2] = *reinterpret_cast<const uint2*>(sf + 64);
    w[3] = *reinterpret_cast<const uint2*>(sf + 72);
    uint32_t sc[2][4];  // [key half][c]: (scale of key 2j, scale of key 2j + 1)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t lo0 = w[2 * h].x >> sh, lo1 = w[2 * h + 1].x >> sh;
      const uint32_t hi0 = w[2 * h].y >> sh, hi1 = w[2 * h + 1].y >> sh;
      const uint32_t a = __byte_perm(lo0, lo1, 0x6240), b = __byte_perm(hi0, hi1, 0x6240);
      sc[h][0] = e4m3x2_to_f16x2(a);
      sc[h][1] = e4m3x2_hi_to_f16x2(a);
      sc[h][2] = e4m3x2_to_f16x2(b);
      sc[h][3] = e4m3x2_hi_to_f16x2(b);
      if constexpr (MASK) {  // e2m1 codes are finite: a scale of zero masks the key
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[h][c] &= h ? m1 : m0;
      }
    }
#pragma unroll
    for (int cp = 0; cp < 2; ++cp) {
      uint32_t r[4];
      ldmatrix_x4_trans(r, swz64(vt, mrow, 2 * cp + mch));
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int c = 2 * cp + q;
        uint32_t bb[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t x[4];  // key 2j: dims 0,1 / 2,3; key 2j + 1: dims 0,1 / 2,3
          e2m1x8_to_f16(r[2 * q + h], x);
          bb[h][0] = hmul2(__byte_perm(x[0], x[2], 0x5410), sc[h][c]);
          bb[h][1] = hmul2(__byte_perm(x[0], x[2], 0x7632), sc[h][c]);
          bb[h][2] = hmul2(__byte_perm(x[1], x[3], 0x5410), sc[h][c]);
          bb[h][3] = hmul2(__byte_perm(x[1], x[3], 0x7632), sc[h][c]);
          if constexpr (NVR) {
#pragma unroll
            for (int i = 0; i < 4; ++i) bb[h][i] = e4m3_round_f16x2(bb[h][i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_rows<FMT, R8, MASK>(o[4 * c + i], pa, bb[0][i], bb[1][i], keep0, keep1);
      }
    }
  }
}

// Whether V of any key in tile rows [r0, r1) is not finite (whole warp).
template <int FMT>
__device__ __forceinline__ bool v_not_finite(const uint8_t* stg, const uint8_t* vs, int r0, int r1, int lane) {
  using TR = DenseTraits<FMT>;
  bool bad = false;
  for (int row = r0; row < r1; ++row) {
    if constexpr (FMT == FMT_FP8) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(stg + TR::TILE + row * 128 + 4 * lane);
#pragma unroll
      for (int i = 0; i < 4; ++i) bad |= ((w >> (8 * i)) & 0x7fu) == 0x7fu;
    } else if constexpr (FMT == FMT_BF16) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(stg + TR::TILE + half * (TR::SK * 128) + row * 128 + 4 * lane);
        bad |= (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
      }
    } else {
      if (lane < 8) bad |= (vs[row * 8 + lane] & 0x7fu) == 0x7fu;
    }
  }
  return __any_sync(0xffffffffu, bad);
}

// The first of the consecutive dims that o[t][0..3] of lane j belong to is
//   FP8    16 (t / 2) + 4j + (t & 1) + 2e   BF16  8 t + 2j + e   NVFP4  32 (t / 4) + 8j + (t & 3) + 4e
// for the accumulator columns e = 0, 1.
template <int FMT>
__device__ __forceinline__ int out_dim(int t, int e, int j) {
  if constexpr (FMT == FMT_FP8) return 16 * (t >> 1) + 4 * j + (t & 1) + 2 * e;
  else if constexpr (FMT == FMT_BF16) return 8 * t + 2 * j + e;
  else return 32 * (t >> 2) + 8 * j + (t & 3) + 4 * e;
}

template <int FMT, int NT, bool R8, int SP, bool NVR>
__device__ void consumer(const DenseParams& p, uint8_t* base, uint64_t* full, uint64_t* empty, uint64_t* ifull,
                         uint64_t* iempty, int* dead, const DenseFacts* facts, const int* stage_ok, int warp, int lane) {
  using TR = DenseTraits<FMT>;
  using LY = DenseLayout<FMT, NT, R8>;
  constexpr int NST = LY::NST;
  constexpr int KGW = kDenseWpg / NT;          // warps of a group that share a column tile
  constexpr int KW = TR::SK / KGW;             // keys of a warp in a unit
  constexpr int KC = KW < 32 ? KW : 32;        // keys a softmax step takes
  constexpr int NR = R8 ? 1 : 2;               // rows of a lane
  constexpr bool F16P = FMT != FMT_BF16;
  const int grp = warp / kDenseWpg, sub = warp % kDenseWpg;
  const int ct = sub / KGW, kw = (sub % KGW) * KW;
  const int tid = warp * 32 + lane;
  const int g8 = lane >> 2, j = lane & 3;
  const int H = p.G * p.r;
  float* mo = reinterpret_cast<float*>(base + LY::MERGE);   // [warps][TR rows][MROW]
  float* ml = reinterpret_cast<float*>(base + LY::ML);      // [warps][TR rows][2]
  int bi = 0;
#pragma unroll 1
  for (int ii = 0;; ++ii) {
    const int slot = ii & 1;
    const bool got = ring_wait(&ifull[slot], (uint32_t)((ii >> 1) & 1), dead);
    if (!got) set_dead(dead, p.status, ii);
    if (named_bar_or(1, kDenseConsumers, !got)) break;  // every consumer warp leaves together
    const DenseFacts f = facts[slot];
    if (f.n < 0) break;
    const int c0 = f.cg * LY::ROWS;
    const int nrows = p.cols - c0 < LY::ROWS ? p.cols - c0 : LY::ROWS;
    uint32_t aq[SP][QRegs<FMT>::KS][4];
    float colf[2];
    load_q<FMT, R8, SP, LY::QROW>(base + LY::Q + (size_t)slot * LY::QSLOT, 16 * ct, nrows, p.q_fp8 != 0, p.q_scale, p.col_const,
                        lane, aq, colf);
    __syncwarp();
    if (lane == 0) mbar_arrive(&iempty[slot]);

    int qi[2], qlim[2];
    float m_run[2], l_run[2];
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const int row = 16 * ct + g8 + 8 * rr;
      qi[rr] = (c0 + row) / p.r;
      qlim[rr] = row < nrows ? f.T - p.Q + qi[rr] : -1;
      m_run[rr] = -INFINITY;
      l_run[rr] = 0.f;
    }
    float o[16][4];
#pragma unroll
    for (int t = 0; t < 16; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    int ev = 0;           // FP8: P carries vscale x 2^ev
    bool ev_set = false;
    const int lim0 = f.T - p.Q;  // every row sees the keys up to here

#pragma unroll 1
    for (int k = f.k0; k < f.k0 + f.n; ++k, ++bi) {
      if ((bi & (kDenseGroups - 1)) != grp) continue;
      const int st = bi % NST;
      const bool have = ring_wait(&full[st], (uint32_t)((bi / NST) & 1), dead);
      if (!have) set_dead(dead, p.status, f.s);
      const uint8_t* stg = base + (size_t)st * LY::STAGE;
      const uint8_t* ksc = base + LY::SC + (size_t)st * LY::SCALES;  // scales of K, then of V
      const uint8_t* vsb = ksc + TR::SC;
      if (have && stage_ok[st]) {
#pragma unroll 1
        for (int kb = kw; kb < kw + KW; kb += KC) {
          const int key0 = k * TR::SK + kb;  // position of the step's first key
          if (key0 >= f.T) break;
          float sacc[KC / 8][4];
          logits<FMT, R8, SP, NVR, KC>(stg, ksc, kb, lane, aq, sacc);
          const bool masked = key0 + KC - 1 > lim0;
          // ---- scale and mask, the row's new maximum
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int t = 0; t < KC / 8; ++t) {
            float2 ks = make_float2(1.f, 1.f);
            if constexpr (FMT == FMT_FP8)
              ks = lds_f2(reinterpret_cast<const float*>(ksc) + kb + 8 * t + 2 * j);
            if constexpr (R8 && FMT == FMT_FP8) {  // hi + lo terms
              sacc[t][0] += sacc[t][2];
              sacc[t][1] += sacc[t][3];
            }
#pragma unroll
            for (int rr = 0; rr < NR; ++rr) {
              float x0 = sacc[t][2 * rr] * (ks.x * colf[rr]), x1 = sacc[t][2 * rr + 1] * (ks.y * colf[rr]);
              if (masked) {
                const int key = key0 + 8 * t + 2 * j;
                x0 = key <= qlim[rr] ? x0 : -INFINITY;
                x1 = key + 1 <= qlim[rr] ? x1 : -INFINITY;
              }
              sacc[t][2 * rr] = x0;
              sacc[t][2 * rr + 1] = x1;
              mx[rr] = fmaxf(mx[rr], fmaxf(x0, x1));
            }
          }
          float msub[2], alpha[2];
          bool grew = false;
#pragma unroll
          for (int rr = 0; rr < NR; ++rr) {
            mx[rr] = fmaxf(mx[rr], __shfl_xor_sync(0xffffffffu, mx[rr], 1));
            mx[rr] = fmaxf(mx[rr], __shfl_xor_sync(0xffffffffu, mx[rr], 2));
            const float mnew = fmaxf(m_run[rr], mx[rr]);
            msub[rr] = mnew == -INFINITY ? 0.f : mnew;
            alpha[rr] = ex2(m_run[rr] - msub[rr]);
            grew |= mnew != m_run[rr];
            m_run[rr] = mnew;
            if constexpr (F16P) msub[rr] -= kDensePShift;
          }
          // ---- FP8: the power of two that keeps P x vscale in f16's range
          float resc = 1.f;
          const float* vsc = reinterpret_cast<const float*>(vsb) + kb;
          float fe = 1.f;
          if constexpr (FMT == FMT_FP8) {
            float vm = 0.f;
            if (lane < KC && key0 + lane < f.T) vm = fabsf(vsc[lane]);
            vm = vm <= 3.0e38f ? vm : 0.f;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, s));
            const float cur = vm * pow2i(ev);
            if (!ev_set || cur > 2.f || cur < 0.00390625f) {
              if (vm > 0.f) {
                const int be = (int)(__float_as_uint(vm) >> 23) - 127;  // vm in [2^be, 2^(be + 1))
                int en = -3 - be;                                      // vm x 2^en in [1/8, 1/4)
                en = en < -126 ? -126 : (en > 120 ? 120 : en);
                if (ev_set) {
                  const int de = en - ev < -126 ? -126 : (en - ev > 126 ? 126 : en - ev);
                  resc = pow2i(de);
                  grew = true;
                }
                ev = en;
                ev_set = true;
              }
            }
            fe = pow2i(ev);
          }
          if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int rr = 0; rr < NR; ++rr) {
              l_run[rr] *= alpha[rr];
              const float w = alpha[rr] * resc;
#pragma unroll
              for (int t = 0; t < 16; ++t) {
                o[t][2 * rr] *= w;
                o[t][2 * rr + 1] *= w;
                if constexpr (R8 && FMT == FMT_BF16) {  // the lo terms' rows belong to the same column
                  o[t][2] *= w;
                  o[t][3] *= w;
                }
              }
            }
          }
          // ---- P, its row sums, and P's fragments: keys 2j, 2j + 1 of tile t
          uint32_t ph[KC / 8][2], plo[KC / 8][2];
#pragma unroll
          for (int t = 0; t < KC / 8; ++t) {
            float2 vs = make_float2(fe, fe);
            if constexpr (FMT == FMT_FP8) {
              const float2 v = lds_f2(vsc + 8 * t + 2 * j);
              vs.x *= v.x;
              vs.y *= v.y;
              if (masked) {  // the scale of a row that holds no key may be anything
                const int key = key0 + 8 * t + 2 * j;
                vs.x = key < f.T ? vs.x : 0.f;
                vs.y = key + 1 < f.T ? vs.y : 0.f;
              }
            }
#pragma unroll
            for (int rr = 0; rr < NR; ++rr) {
              float p0 = ex2(sacc[t][2 * rr] - msub[rr]), p1 = ex2(sacc[t][2 * rr + 1] - msub[rr]);
              l_run[rr] += p0 + p1;
              if constexpr (FMT == FMT_FP8) {
                if (masked) {  // a masked weight stays 0 beside a scale that is not finite
                  p0 = p0 == 0.f ? 0.f : p0 * vs.x;
                  p1 = p1 == 0.f ? 0.f : p1 * vs.y;
                } else {
                  p0 *= vs.x;
                  p1 *= vs.y;
                }
              }
              if constexpr (F16P) {
                ph[t][rr] = pack_f16x2(p0, p1);
                plo[t][rr] = 0u;
              } else {
                const uint32_t h = pack_bf16x2(p0, p1);
                ph[t][rr] = h;
                plo[t][rr] = pack_bf16x2(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xffff0000u));
              }
            }
          }
          // ---- O += P V
#define MSA_DENSE_PV(MASK, KLIM, KEEP0, KEEP1)                                               \
  _Pragma("unroll") for (int h = 0; h < KC / 16; ++h) {                                      \
    /* R8: rows 8 to 15 hold the lo terms of rows 0 to 7 */                                  \
    const uint32_t pa[4] = {ph[2 * h][0], R8 ? plo[2 * h][0] : ph[2 * h][NR - 1],            \
                            ph[2 * h + 1][0], R8 ? plo[2 * h + 1][0] : ph[2 * h + 1][NR - 1]}; \
    const uint32_t pl[4] = {plo[2 * h][0], plo[2 * h][NR - 1], plo[2 * h + 1][0], plo[2 * h + 1][NR - 1]}; \
    pv16<FMT, R8, NVR, MASK>(stg, vsb, kb + 16 * h, KLIM, lane, pa, pl, o, KEEP0, KEEP1);    \
  }
          if (!masked) {
            MSA_DENSE_PV(false, 0, true, true)
          } else {
            // tile rows up to the last key of the sequence; with several new tokens a
            // row between lim0 and there is seen by some of them only
            const int klast = f.T - 1 - k * TR::SK;
            int r0 = lim0 + 1 - k * TR::SK, r1 = klast + 1;
            r0 = r0 < kb ? kb : r0;
            r1 = r1 > kb + KC ? kb + KC : r1;
            if (p.Q == 1 || !v_not_finite<FMT>(stg, vsb, r0, r1, lane)) {
              MSA_DENSE_PV(true, klast, true, true)
            } else {
              // a later token's V is not finite: each token by itself, up to its own position
#pragma unroll 1
              for (int i = 0; i < p.Q; ++i) {
                MSA_DENSE_PV(true, klast - (p.Q - 1 - i), qi[0] == i, qi[1] == i)
              }
            }
          }
#undef MSA_DENSE_PV
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // ---------------- the segment's result: the warps of a column tile hold different keys
#pragma unroll
    for (int rr = 0; rr < NR; ++rr) {
      l_run[rr] += __shfl_xor_sync(0xffffffffu, l_run[rr], 1);
      l_run[rr] += __shfl_xor_sync(0xffffffffu, l_run[rr], 2);
      if (j == 0) {
        ml[(warp * LY::TR + g8 + 8 * rr) * 2] = m_run[rr];
        ml[(warp * LY::TR + g8 + 8 * rr) * 2 + 1] = l_run[rr];
      }
    }
    const float osc = FMT == FMT_FP8 ? pow2i(-ev) : (FMT == FMT_NVFP4 ? p.v_global : 1.f);
    const bool whole = f.part < 0;
    constexpr int D4 = LY::DCH / 4;
#pragma unroll
    for (int pass = 0; pass < 128 / LY::DCH; ++pass) {
      // the dims of accumulators [pass * 16 / passes, ...) are consecutive from pass * DCH
#pragma unroll
      for (int tt = 0; tt < 16 * LY::DCH / 128; ++tt) {
        const int t = pass * (16 * LY::DCH / 128) + tt;
#pragma unroll
        for (int rr = 0; rr < NR; ++rr)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = o[t][2 * rr + e];
            if constexpr (R8 && FMT == FMT_BF16) v += o[t][2 + e];
            mo[(warp * LY::TR + g8 + 8 * rr) * LY::MROW + out_dim<FMT>(t, e, j) - pass * LY::DCH] = v * osc;
          }
      }
      named_bar_sync(1, kDenseConsumers);
#pragma unroll 1
      for (int x = tid; x < LY::ROWS * D4; x += kDenseConsumers) {
        const int row = x / D4, d = 4 * (x - row * D4);
        if (row >= nrows) continue;
        const int tile = R8 ? 0 : row >> 4, tr = R8 ? row : row & 15;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kDenseGroups * KGW; ++w) {
          const int src = (w / KGW) * kDenseWpg + tile * KGW + w % KGW;
          M = fmaxf(M, ml[(src * LY::TR + tr) * 2]);
        }
        const float ms = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kDenseGroups * KGW; ++w) {
          const int src = (w / KGW) * kDenseWpg + tile * KGW + w % KGW;
          const float2 v = lds_f2(ml + (src * LY::TR + tr) * 2);
          const float fw = ex2(v.x - ms);
          L += fw * v.y;
          const float4 ov = *reinterpret_cast<const float4*>(mo + (src * LY::TR + tr) * LY::MROW + d);
          acc.x += fw * ov.x;
          acc.y += fw * ov.y;
          acc.z += fw * ov.z;
          acc.w += fw * ov.w;
        }
        const int dim = pass * LY::DCH + d;
        if (whole) {
          const float inv = L == 0.f ? 0.f : 1.f / L;
          const int col = c0 + row, i = col / p.r, h = col - i * p.r;
          const size_t orow = ((size_t)f.s * p.Q + i) * H + (size_t)f.g * p.r + h;
          uint2 pk;
          pk.x = pack_bf16x2(acc.x * inv, acc.y * inv);
          pk.y = pack_bf16x2(acc.z * inv, acc.w * inv);
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + orow * kDim + dim) = pk;
          if (dim == 0 && p.lse)
            p.lse[orow] = L == 0.f ? -INFINITY : (M - (F16P ? kDensePShift : 0.f) + log2f(L)) * 0.69314718055994531f;
        } else {
          *reinterpret_cast<float4*>(p.part_o + ((size_t)f.part * LY::ROWS + row) * kDim + dim) = acc;
          if (dim == 0) p.part_ml[(size_t)f.part * LY::ROWS + row] = make_float2(M, L);
        }
      }
      named_bar_sync(1, kDenseConsumers);  // the merge area is free again
    }
  }
}

// 9 warps a CTA, one CTA an SM: up to 224 registers a thread.
template <int FMT, int NT, bool R8, int SP, bool NVR>
__global__ void __launch_bounds__(kDenseThreads, 1)
    dense_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const DenseParams p) {
  using LY = DenseLayout<FMT, NT, R8>;
  constexpr int NST = LY::NST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(base + LY::BARS);
  uint64_t* empty = full + NST;
  uint64_t* ifull = empty + NST;
  uint64_t* iempty = ifull + 2;
  int* stage_ok = reinterpret_cast<int*>(iempty + 2);
  int* dead = stage_ok + NST;
  DenseFacts* facts = reinterpret_cast<DenseFacts*>(base + LY::FACTS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int st = 0; st < NST; ++st) {
      mbar_init(&full[st], 1);
      mbar_init(&empty[st], kDenseWpg);
    }
    for (int sl = 0; sl < 2; ++sl) {
      mbar_init(&ifull[sl], 1);
      mbar_init(&iempty[sl], kDenseWarps);
    }
    *dead = 0;
    fence_mbar_init();
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
  }
  __syncthreads();
  pdl_launch_dependents();  // the combine's CTAs may take their place as soon as this grid's leave room
  if (warp == kDenseWarps) {
    producer<FMT, NT, R8>(&tmk, &tmv, p, base, full, empty, ifull, iempty, dead, facts, stage_ok, lane);
  } else {
    // sequences without keys (and malformed ones) have no units: their rows here
    for (int s = blockIdx.x + warp * gridDim.x; s < p.S; s += gridDim.x * kDenseWarps) {
      const int T = __ldg(p.seq_lens + s);
      if (T >= 1 && T <= p.max_nb * kBlock) continue;
      if (T != 0 && lane == 0) raise_flag(p.status, FLAG_BAD_SEQLEN, T);
      const long rows = (long)p.Q * p.G * p.r;
      uint2* orow = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + (size_t)s * rows * kDim);
      for (long x = lane; x < rows * 32; x += 32) orow[x] = make_uint2(0u, 0u);
      if (p.lse)
        for (long x = lane; x < rows; x += 32) p.lse[(size_t)s * rows + x] = -INFINITY;
    }
    consumer<FMT, NT, R8, SP, NVR>(p, base, full, empty, ifull, iempty, dead, facts, stage_ok, warp, lane);
  }
}

template <int FMT, int NT, bool R8, int SP, bool NVR>
cudaError_t launch_one(const CUtensorMap* tk, const CUtensorMap* tv, const DenseParams& p, int num_sms, cudaStream_t st) {
  constexpr size_t smem = DenseLayout<FMT, NT, R8>::SMEM;
  auto kern = dense_kernel<FMT, NT, R8, SP, NVR>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)num_sms, kDenseThreads, smem, st>>>(*tk, *tv, p);
  return cudaGetLastError();
}

}  // namespace dense
}  // namespace msa
