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
// Split.  A unit is SK keys of one (sequence, group of heads); the units of the
// batch, in (sequence, group, position) order, are cut into equal contiguous
// runs, one per team, whatever the lengths are: the lengths stay on the device
// and every team does the same work to within a unit.  A run crosses (sequence,
// group) borders; a segment it holds whole is written out at once, a cut one
// leaves its partial in the workspace (at most two a run), joined by the
// combine kernel.  No atomics: the result does not depend on timing.
//
// A team is one producer warp and four consumer warps with a ring of their own;
// a CTA (one an SM) holds two or three, so that one team's segment ends (the
// join of its warps, the output) pass behind the others' work.  The producer
// walks the run, publishes each segment's facts and query rows in one of two
// slots and streams the tiles through the ring (tensor copies, mbarriers).  The
// consumers divide a unit as NCG groups of 8 NN columns x key ranges; a warp takes
// up to 32 columns, so that the tile it has converted serves them all.
//
// Tensor-core mapping (mma.sync: up to 64 columns are too few for a 128-row
// tile).  The queries are the rows of the first product and the columns of the
// second, so that P leaves the softmax in the lanes and order in which it enters
// the second product, with no exchange between lanes, and with up to 8 columns
// the output takes 32 registers and no MMA works on empty columns:
//   S[col][key]   = Q[col][:] . K[key][:]             (A = Q, B = K)
//   O^T[d][col]  += sum_key V[key][d] P[col][key]     (A = V^T, B = P)
//   FP8    K and V become f16 (exact); a bf16 query f16 after a power-of-two row
//          scale (11 bits, exact to 2^-25 of 16,384 below it), P x vscale f16 (below).
//          K as it is, against the query's two e4m3 terms (e4m3 k32 MMAs), takes
//          as long with 4 columns (4 x 524,288 tokens: 330 us both ways) and
//          longer with more: 105 us against 97 with 16 columns (16 x 32,768), 222
//          against 133 with 32 (8 x 65,536).
//   NVFP4  K and V become f16 in registers (e2m1 x e4m3 fits 6 bits: exact).
//   BF16   as it is; P enters as bf16 hi + lo terms (16 bits), since one bf16
//          term alone would add an error near the output's own rounding.
//
// The running maximum is lazy: m moves only when a logit passes it by 2^8, so
// that the output is rescaled a few times a segment and the lanes of a row need
// not agree on a maximum at every step (one vote instead).  NVFP4's P is scaled by
// 2^7 where it becomes f16, l with it: at most 2^15, and 2^-21 of the row's
// reference weight before f16 loses bits.
//
// FP8's P enters with V's scale in it, and scales may be of any size, those of
// keys that a row does not see or that weigh nothing among them.  So every column
// has a factor fe of its own that puts the largest p x vscale it has met (decayed
// with m, looked at where m moves) at 4: 2^-16 of that product before f16 loses bits,
// off by 2^-27 of it below.  Where a step's scales could take a product past 2^15
// (vscale above 2^5 times that largest one) the products themselves are looked at, and only if
// one does the factor changes.  O is rescaled by old over new product, never above 1,
// so that it cannot overflow.  Scales that vary: 32 columns 129 us with factors of e^0.5
// (one standard deviation), 134 with e^1, 139 with e^2 (182 and 189 us if every such step
// rescaled).
//
// Measured (one GPU, launches back to back; shares of the measured copy rate,
// 6,779 GB/s): 4 columns, FP8 32 x 16K-32K tokens 127 us (98%), 4 x 512K 314 us
// (104%), BF16 32 x 16K-32K 237 us (101%), NVFP4 32 x 16K-64K 173 us (65%: the
// dequantization's issue slots); 16 columns, FP8 16 x 32K 95 us (86%), NVFP4 8 x 64K 86
// us (52%); 32 columns (8 new tokens), BF16 8 x 64K 182 us (87%), FP8 129 us (63%),
// NVFP4 8 x 128K 224 us (40%; tensor pipe 43%, issue slots 40%, two warps a scheduler
// waiting for each other's results); 61 ragged BF16 sequences of 48 columns 82 us
// (51%; tensor pipe 50%); one sequence of 4K tokens 8.1 us.  Products rounded to E4M3: 4
// columns 229 us, 16 columns 107, 32 columns 273.
//
// Registers are what the wide instances lack: with 24 columns and more each of them spills
// (92 to 268 bytes of stores a thread, a stack of 56 to 176: mostly the producers', whose share is 40 or
// 24), with 16 all but BF16 (FP8 44, by blocks 28, INT8 80, over lists 124 and 132, NVFP4 84), with 8 NVFP4 (44, products
// rounded 60) and FP8 (8).
//
// Caches with one scale for each block and head (INT8, FP8).  A unit is a block, so its two
// scales are two numbers of the stage: K's goes into the columns' factors (where keys are masked into the
// logits), V's times fe is one factor of the weights; nothing is left of the FP8 format's work for
// each key.  INT8 becomes f16 exactly by 1024 + (x + 128) - 1152 (5 instructions for 4 elements, E4M3's
// 2 or 3).  The producer asks for the scales behind the block's copies and completes the stage's phase
// when they are there.  Measured: 4 columns, FP8 32 x 16K-32K 123 us (99% of the copy rate,
// 6,702 GB/s), INT8 4 x 512K 306 us (105%); 32 columns (8 x 128K, 8 new tokens) INT8 239 us
// (67%; tensor pipe 42%, issue slots 40%, two warps a scheduler), FP8 226; 24 columns 209 and 191, 16 columns
// 175 (92%); one sequence of 4K tokens 8.8 us: lengths and table 1.6, first tile 3.0, its unit 4.5, the
// warps' join 5.5, the last CTA's end seen by the join's launch 6.2, joined 8.2 (when it took 9.4).
//
// SEL: the sparse attend over selection lists (caches with block scales).  The new tokens are
// sequences of their own, a (token, KV head)'s units the entries of its list, its runs cut
// as above.  A list counts topk units, or as many as its sequence has blocks where those are fewer
// (32 tokens on 300 to 900 with 16 places 15.2 and 13.9 us, with 32 18.0 and 13.9; 64 of 32 places 21.2 and 15.1).  The
// producer holds a list in its lanes, leaves out what cannot be seen, is named twice or outside the pool, and
// says where each unit's keys begin.  Measured: 32 tokens x 4 heads x 16 blocks of INT8 19.8 us in a graph (10.1 at
// the copy rate; 4 blocks 12 us: what a call costs at least is launch, lists, first tiles and join), 64 of FP8
// (8 x 128K, 8 new tokens) 28.2 (18.1); the kernel for FP8 with token scales takes 30 and 44.  A prompt's
// chunk reads its blocks once for each token: 8,192 tokens on 64K 1.73 (FP8) and 2.13 ms (INT8), where the
// key-block-major attend of the FP8 format takes 0.58.
//
// A masked key's logit is replaced, not multiplied; in units that hold masked
// keys V is masked in registers too, so NaN or infinity in rows past the end of a
// sequence, or in a later token's row, reaches no output (0 x inf is NaN).
#pragma once

#include "msa_device.cuh"
#include "msa_internal.h"

namespace msa {

constexpr int kDenseWpg = 4;             // consumer warps of a team
// An MMA's sum is ready after 21 cycles, and a scheduler could start one every 8:
// a warp alternates this many sums (with two or eight the operator takes as long).
constexpr int kDenseChains = 4;
// What a segment's end takes over selection lists, in units (short segments, so that a unit's own share
// counts more than the end's: 64 tokens of 16 blocks 29.8 us with two, 29.2 with one).
constexpr int kSelEnd = 1;
constexpr float kDensePShift = 7.f;      // log2 of the scale of P (NVFP4)
constexpr float kDenseTop = 4.f;         // FP8: P x vscale of a column's largest product so far
constexpr float kDenseLeast = 6.1e-36f;  // ... which counts as 2^-117 at least: 2^8 x fe stays finite
constexpr float kDenseLazy = 8.f;        // a logit (log2) above the reference by this moves it
constexpr float kDenseNone = -3.0e38f;   // FP8: the reference before a row's first key

template <int FMT>
struct DenseTraits;
template <>
struct DenseTraits<FMT_FP8> {
  static constexpr int SK = 128, TILE = 128 * 128, SC = 512;  // keys, bytes of a K or V tile, of its scales
};
template <>
struct DenseTraits<FMT_I8B> {  // a unit is a block: its two scales come with the stage's facts
  static constexpr int SK = 128, TILE = 128 * 128, SC = 0;
};
template <>
struct DenseTraits<FMT_F8B> : DenseTraits<FMT_I8B> {};
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

// What the producer says of a stage over caches with block scales.
struct __align__(16) DenseStage {
  int32_t ok, key0;  // whether it holds keys, the position of the first
  float ks, vs;
};

// Formats of one byte an element, and those with a scale for each block.
template <int FMT>
constexpr bool kByBlock = fmt_by_block(FMT);
template <int FMT>
constexpr bool kBytes = FMT == FMT_FP8 || kByBlock<FMT>;

// NN: tiles of 8 query columns a warp takes; NCG: groups of such columns in a unit.
template <int FMT, int NN, int NCG>
struct DenseLayout {
  using T = DenseTraits<FMT>;
  // NVFP4's dequantization keeps three teams busy where two are enough for the
  // others (one token 173 us, 188 with two; 16 columns 86 and 93); with 24 columns
  // and more the accumulators leave no room for a third.
  static constexpr int TEAMS = (NN <= 2 && FMT == FMT_NVFP4) ? 3 : 2;
  // Where an equal share is too small, the consumers take registers over from the
  // producers; their warps come in fours then (the producers' four hold idle ones).
  // Three teams of one column tile do better with equal shares (173 us, 182 so).
  // (INT8's conversions want a few more: 64 columns 221 us, 224 with the others' shares; 24 209 and 218; but one group of
  // 32 243 and 238; FP8 by blocks, 24 columns 200 and 197.)
  static constexpr bool WIDE = NN >= 3, MOVE = WIDE || (TEAMS == 3 && NN == 2);
  static constexpr bool MORE = FMT == FMT_I8B && !(NN == 4 && NCG == 1);
  static constexpr int REGS_P = WIDE ? (MORE ? 24 : 40) : 56, REGS_C = WIDE ? (MORE ? 240 : 232) : 152;
  static constexpr int CONSUMERS = 32 * kDenseWpg * TEAMS;
  static constexpr int THREADS = CONSUMERS + (MOVE ? 128 : 32 * TEAMS);
  static_assert(!MOVE || 128 * REGS_P + CONSUMERS * REGS_C <= (65536 / THREADS / 8 * 8) * THREADS, "shares of the launch's registers");
  static constexpr int MT = (NN + 1) / 2;        // 16-row tiles of a warp's queries
  static constexpr int WROWS = 8 * NN;           // columns of a warp
  static constexpr int ROWS = WROWS * NCG;       // of a unit
  static constexpr int KGW = kDenseWpg / NCG;    // warps that share a group's columns, each its keys
  static constexpr size_t STAGE = 2 * (size_t)T::TILE;  // K tile, V tile
  static constexpr size_t SCALES = 2 * (size_t)T::SC;   // their scales, in a region of their own
  static constexpr int END = NN == 1 ? 2 : NN == 2 ? 3 : 4;  // what a segment's end takes, in units
  static constexpr int MT_OWN = 8 / KGW;         // output tiles a warp takes when the warps of a group join (NN > 1)
  static constexpr int MROW = kDim + 4;          // padded row of that join's area (NN = 1)
  static constexpr int QROW = 272;               // a query row, padded (conflict-free reads)
  // per team
  static constexpr size_t MERGE_BYTES = NN == 1 ? kDenseWpg * WROWS * MROW * 4 : kDenseWpg * (KGW - 1) * MT_OWN * 512;
  static constexpr size_t ML_BYTES = (size_t)kDenseWpg * WROWS * 16;  // m, l, a weight
  static constexpr size_t QSLOT = (size_t)ROWS * QROW;
  static constexpr size_t CF_BYTES = (ROWS * 4 + 15) / 16 * 16;
  static constexpr size_t FIXED = MERGE_BYTES + ML_BYTES + 2 * QSLOT + CF_BYTES + 2 * sizeof(DenseFacts) + 320;
  // Two stages a team: some 20 MB on their way over the GPU.  More make the memory
  // slower, not faster: 4 x 512K FP8 tokens 320 us with two, 335 with three, NVFP4
  // verify 226 with two and 236 with the four that fit.
  static constexpr int NST = 2;
  // the tiles of all teams first (1 KB alignment), then each team's block
  static constexpr size_t TILES = STAGE * NST * TEAMS;
  static constexpr size_t SC = 0;
  static constexpr size_t MERGE = SC + SCALES * NST;
  static constexpr size_t ML = MERGE + MERGE_BYTES;
  static constexpr size_t Q = ML + ML_BYTES;
  static constexpr size_t CF = Q + 2 * QSLOT;
  static constexpr size_t FACTS = CF + CF_BYTES;
  static constexpr size_t BARS = FACTS + 2 * sizeof(DenseFacts);
  static constexpr size_t STAGES = BARS + 8 * (2 * NST + 4);  // 4 bytes each, or a DenseStage
  static constexpr size_t STAGES_BYTES = NST * (kByBlock<FMT> ? sizeof(DenseStage) : 4);
  static constexpr size_t TEAM = (STAGES + STAGES_BYTES + 16 + 127) / 128 * 128;
  static constexpr size_t SMEM = TILES + TEAMS * TEAM + 1024;
  static_assert(SMEM <= 227 * 1024, "stages");
  static_assert(STAGE % 1024 == 0 && MERGE_BYTES % 16 == 0 && ML_BYTES % 16 == 0 && QSLOT % 16 == 0, "alignment");
  static_assert(STAGES % 16 == 0, "DenseStage");
};

// One team's shared memory.
struct DenseTeam {
  uint8_t* tiles;   // ring of stages
  uint8_t* mem;     // scales, merge area, queries, facts
  uint64_t *full, *empty, *ifull, *iempty;
  int* stage_ok;
  DenseStage* stage;  // block scales: in its place
  int* dead;
  DenseFacts* facts;
  int id;           // team of the grid: the run it takes
};

namespace dense {

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
// int8 as f16, exact: 1024 + u of u = x + 128, less 1152.  w: the codes with their top
// bits turned; sel: the bytes taken (4: the exponent's).
__device__ __forceinline__ uint32_t i8x2_to_f16x2(uint32_t w, uint32_t sel) {
  uint32_t d;
  const uint32_t h = __byte_perm(w, 0x64646464u, sel);
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h), "r"(0x64806480u));
  return d;
}
// The four bytes of w as f16: the low two in h0, the high two in h1.
template <int FMT>
__device__ __forceinline__ void bytes_to_f16(uint32_t w, uint32_t& h0, uint32_t& h1) {
  if constexpr (FMT == FMT_I8B) {
    w ^= 0x80808080u;
    h0 = i8x2_to_f16x2(w, 0x4140);
    h1 = i8x2_to_f16x2(w, 0x4342);
  } else {
    h0 = e4m3x2_to_f16x2(w);
    h1 = e4m3x2_hi_to_f16x2(w);
  }
}
// The same with the even bytes in h0, the odd ones in h1.
template <int FMT>
__device__ __forceinline__ void bytes_apart_to_f16(uint32_t w, uint32_t& h0, uint32_t& h1) {
  if constexpr (FMT == FMT_I8B) {
    w ^= 0x80808080u;
    h0 = i8x2_to_f16x2(w, 0x4240);
    h1 = i8x2_to_f16x2(w, 0x4341);
  } else {
    w = __byte_perm(w, 0u, 0x3120);
    h0 = e4m3x2_to_f16x2(w);
    h1 = e4m3x2_hi_to_f16x2(w);
  }
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
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(a, fmaxf(b, c)); }
__device__ __forceinline__ float2 lds_f2(const float* p) { return *reinterpret_cast<const float2*>(p); }

__device__ __forceinline__ bool is_dead(const int* flag) { return *reinterpret_cast<const volatile int*>(flag) != 0; }
__device__ __forceinline__ void set_dead(int* flag, DeviceStatus* st, int detail) {
  if (!is_dead(flag)) raise_flag(st, FLAG_TIMEOUT, detail);
  *reinterpret_cast<volatile int*>(flag) = 1;
}
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(done)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return done != 0;
}
// Bounded wait of a warp.  A plain test first: a try_wait may suspend, which takes
// some 200 cycles even where the phase is complete.
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, const int* dead) {
  if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  if (is_dead(dead)) return false;
  return mbar_wait_warp(bar, parity);
}

// Units of a sequence of length T (0: malformed or empty).
template <int SK>
__device__ __forceinline__ int units_of(int T, int max_nb) {
  return (T < 1 || T > max_nb * kBlock) ? 0 : (T + SK - 1) / SK;
}

// The same with END more for the segment's end.
template <int SK, int END>
__device__ __forceinline__ int slots_of(int T, int max_nb) {
  const int un = units_of<SK>(T, max_nb);
  return un > 0 ? un + END : 0;
}

// The query token of a column (SEL: tokens are sequences).  What a call fetches of code for the first time is
// latency in its start and ends, so it is kept small.
template <bool SEL>
__device__ __forceinline__ int token_of(int col, int r) {
  return SEL ? 0 : col / r;
}

// Places of a list (SEL): no more than the sequence has blocks, and one at least, whose segment writes the row.
__device__ __forceinline__ int places_of(int T, int q, int max_nb, int topk) {
  const int blocks = T >= q && T <= max_nb * kBlock ? (T - 1) / kBlock + 1 : 1;
  return blocks < topk ? blocks : topk;
}
// The lane of the k-th set bit of a mask that has more than k (else anything from 0 to 31).
__device__ __forceinline__ int nth_lane(uint32_t mask, int k) {
  int at = 0;
#pragma unroll
  for (int step = 16; step > 0; step >>= 1)
    if (__popc(mask & ((1u << (at + step)) - 1u)) <= k) at += step;
  return at;
}

__device__ __forceinline__ uint32_t warp_sum(uint32_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// The run [u0, u1) of team c, of `total` units cut evenly into as many as there are teams (no unit: the last ones).
// One division; where the runs with one unit more lie only has to be the same for all, so that fp32 will do.
__device__ __forceinline__ void run_of(uint32_t c, uint32_t teams, uint32_t total, uint32_t& u0, uint32_t& u1) {
  const uint32_t each = total / teams, more = total - each * teams;
  const float rate = each == 0 ? 1.f : __fdividef((float)(int)more, (float)(int)teams);
  auto start = [&](uint32_t i) {
    const uint32_t extra = (uint32_t)(int)((float)(int)i * rate);
    return i * each + (i == teams || extra > more ? more : extra);
  };
  u0 = start(c);
  u1 = start(c + 1);
}

// ---------------------------------------------------------------- the producer warp

template <int FMT, int NN, int NCG, bool SEL>
__device__ void producer(const CUtensorMap* tmk, const CUtensorMap* tmv, const DenseParams& p, const DenseTeam& tm,
                         int lane) {
  using TR = DenseTraits<FMT>;
  using LY = DenseLayout<FMT, NN, NCG>;
  constexpr int NST = LY::NST;
  constexpr bool BLK = kByBlock<FMT>;
  uint64_t *full = tm.full, *empty = tm.empty, *ifull = tm.ifull, *iempty = tm.iempty;
  int* dead = tm.dead;
  const int S = p.S, max_nb = p.max_nb;
  using U = uint32_t;  // (the host launches no more units at once)
  const U GC = (U)p.G * (U)p.CG;
  // Units in all, then the run of this team: [u0, u1).  Every segment has END units
  // more than its keys, which stand for its end (the join, the output, the next
  // one's start), so that runs with many short segments are not the last: without it
  // 61 ragged sequences of 48 columns take 14% longer.
  int mine0 = 0;  // the length of sequence `lane`: a batch of up to 32 is read once
  const U teams = (U)gridDim.x * LY::TEAMS, c = (U)tm.id;
  U u0 = 0, u1 = 0;
  int s = 0;  // the sequence that holds u0: sb units (x GC) come before it
  U sb = 0;
  U pick0_row = 0;  // SEL: the list that the run begins in, on its way
  int pick0 = -1;
  if constexpr (SEL) {
    // Where all sequences have topk blocks, every token has the same number of places and the first list is
    // asked for together with the lengths; else the places follow the lengths.
    const U R = (U)S / (U)p.q_real, list = GC * (U)(p.topk + kSelEnd);
    run_of(c, teams, (U)S * list, u0, u1);
    s = (int)(u0 / list);
    sb = (U)s * list;
    if (u1 > u0) {
      pick0_row = (U)s * p.G + (u0 - sb) / ((U)(p.topk + kSelEnd) * p.CG);
      if (lane < p.topk) pick0 = __ldcg(p.topk_idx + (size_t)pick0_row * p.topk + lane);
    }
    bool full = true;
#pragma unroll 1
    for (U at = lane; at < R; at += 32) {
      const int T = __ldcg(p.seq_lens + at);
      if (at < 32) mine0 = T;
      full = full && places_of(T, p.q_real, max_nb, p.topk) == p.topk;
    }
    if (__builtin_expect(!__all_sync(0xffffffffu, full), 0)) {
      const U per = GC * (U)p.q_real;
      U total = 0;
#pragma unroll 1
      for (U at = lane; at < R; at += 32)
        total += places_of(at < 32 ? mine0 : __ldcg(p.seq_lens + at), p.q_real, max_nb, p.topk) + kSelEnd;
      __syncwarp();
      run_of(c, teams, warp_sum(total) * per, u0, u1);
      s = 0;
      sb = 0;
#pragma unroll 1
      for (U s0 = 0; s0 < R && u1 > u0; s0 += 32) {
        const bool real = s0 + lane < R;
        const int T = s0 == 0 ? mine0 : real ? __ldcg(p.seq_lens + s0 + lane) : 0;
        const U mine = real ? per * (U)(places_of(T, p.q_real, max_nb, p.topk) + kSelEnd) : 0;
        const U incl = warp_scan(mine, lane);
        const uint32_t over = __ballot_sync(0xffffffffu, sb + incl > u0);
        if (over) {
          const int l = __ffs(over) - 1;
          sb += __shfl_sync(0xffffffffu, incl - mine, l);
          const U token = __shfl_sync(0xffffffffu, mine, l) / (U)p.q_real, i = (u0 - sb) / token;
          s = (int)((s0 + l) * (U)p.q_real + i);
          sb += i * token;
          break;
        }
        sb += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
  } else {
    U total = 0;
    mine0 = lane < S ? __ldcg(p.seq_lens + lane) : 0;
    total = slots_of<TR::SK, LY::END>(mine0, max_nb);
    // (1,000 short sequences 61 us, 64 with one load at a time; more of this code is more to fetch for all)
#pragma unroll 2
    for (int at = lane + 32; at < S; at += 32) total += slots_of<TR::SK, LY::END>(__ldcg(p.seq_lens + at), max_nb);
    __syncwarp();
    run_of(c, teams, warp_sum(total) * GC, u0, u1);
    if (u1 > u0) {
      for (int s0 = 0; s0 < S; s0 += 32) {
        const int T = s0 == 0 ? mine0 : s0 + lane < S ? __ldcg(p.seq_lens + s0 + lane) : 0;
        const U mine = GC * slots_of<TR::SK, LY::END>(T, max_nb);
        const U incl = warp_scan(mine, lane);
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
  }
  // what the combine reads: the segment the run begins in, and whether it began before
  U u = u0;
  int bi = 0, ii = 0;
  bool ok = true;
  bool first = true;
#pragma unroll 1
  while (u < u1 && ok) {
    int T, un, sr = s;
    if constexpr (SEL) {
      sr = (int)((uint32_t)s / (uint32_t)p.q_real);
      T = sr < 32 ? __shfl_sync(0xffffffffu, mine0, sr & 31) : __ldcg(p.seq_lens + sr);
      un = places_of(T, p.q_real, max_nb, p.topk);
    } else {
      T = s < 32 ? __shfl_sync(0xffffffffu, mine0, s & 31) : __ldcg(p.seq_lens + s);
      un = units_of<TR::SK>(T, max_nb);
    }
    if (un == 0) {  // an empty sequence holds no units
      ++s;
      continue;
    }
    const U in_s = u - sb;
    const int span = un + (SEL ? kSelEnd : LY::END), gc = (int)(in_s / (U)span), k0 = (int)(in_s - (U)gc * span);
    if (k0 >= un) {  // another run's segment end
      u += span - k0;
      if ((U)gc + 1 == GC) {
        sb += (U)span * GC;
        ++s;
      }
      continue;
    }
    const U left = u1 - u;
    const int n = left < (U)(un - k0) ? (int)left : un - k0;
    const int g = (int)((uint32_t)gc / (uint32_t)p.CG), cg = gc - g * p.CG;
    const bool cut_start = k0 > 0, cut_end = k0 + n < un;
    const int sg = (int)((U)s * GC + gc);
    if (first && lane == 0) p.info[c] = make_int2(sg, cut_start ? 1 : 0);
    first = false;
    // the first 32 block-table entries, on their way while the segment is published
    const int32_t* row = p.block_table + (size_t)sr * max_nb;
    constexpr int UPB = kBlock / TR::SK;  // units a block
    int b_have = SEL ? 0 : k0 / UPB;      // entries [b_have, b_have + 32), one a lane
    int entry = -1, pick = -1;
    float ks_mine = 0.f, vs_mine = 0.f;   // BLK: the scales of this lane's block
    if constexpr (SEL) {
      // the whole list, one entry a lane (topk <= 32)
      const U list = (U)s * p.G + g;
      if (list == pick0_row && u == u0) pick = pick0;
      else if (lane < p.topk) pick = __ldcg(p.topk_idx + (size_t)list * p.topk + lane);
      // keys that token s sees; 0: a malformed sequence, every entry of its lists is left out
      const bool good = T >= p.q_real && T <= max_nb * kBlock;
      if (!good && lane == 0) raise_flag(p.status, FLAG_BAD_SEQLEN, T);
      T = good ? T - p.q_real + (s - sr * p.q_real) + 1 : 0;
      const bool seen = pick >= 0 && pick <= (T - 1) >> 7;  // (an arithmetic shift: T = 0 sees none)
      const uint32_t same = __match_any_sync(0xffffffffu, seen ? pick : -1 - lane);
      const bool take = seen && (same & ((1u << lane) - 1u)) == 0;
      if (pick >= 0 && !take) raise_flag(p.status, FLAG_BAD_SELECT, pick);
      if (take) {
        entry = __ldcg(row + pick);
        if (entry < 0 || entry >= p.num_blocks) {
          raise_flag(p.status, FLAG_BAD_BLOCK, entry);
          entry = -1;
        }
      }
      // the entries that count to the list's first places: there are no more of them than places
      const uint32_t taken = __ballot_sync(0xffffffffu, take);
      if (__builtin_expect((taken & (taken + 1u)) != 0u, 0)) {
        const int at = nth_lane(taken, lane);
        const int e = __shfl_sync(0xffffffffu, entry, at), k = __shfl_sync(0xffffffffu, pick, at);
        entry = lane < __popc(taken) ? e : -1;
        pick = lane < __popc(taken) ? k : -1;
      }
    } else {
      entry = (b_have + lane) * UPB < k0 + n ? __ldcg(row + b_have + lane) : -1;
    }
    // publish the segment and its query rows
    const int slot = ii & 1, use = ii >> 1;
    if (use > 0 && !ring_wait(&iempty[slot], (uint32_t)((use - 1) & 1), dead)) {
      set_dead(dead, p.status, sg);
      ok = false;
      break;
    }
    const int qrow_bytes = p.q_fp8 ? 128 : 256;
    const int c0 = cg * p.cper;
    const int nrows = p.cols - c0 < p.cper ? p.cols - c0 : p.cper;
    if (lane == 0) {
      DenseFacts& f = tm.facts[slot];
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
    fence_proxy_async();
    for (int row = lane; row < nrows; row += 32) {
      const int col = c0 + row, i = token_of<SEL>(col, p.r), h = col - i * p.r;
      const size_t src = ((size_t)s * (SEL ? 1 : p.Q) + i) * ((size_t)p.G * p.r) + (size_t)g * p.r + h;
      bulk_g2s(tm.mem + LY::Q + (size_t)slot * LY::QSLOT + (size_t)row * LY::QROW,
               static_cast<const uint8_t*>(p.q) + src * qrow_bytes, (uint32_t)qrow_bytes, &ifull[slot]);
    }
    ++ii;
    // its tiles
#pragma unroll 1
    for (int k = k0; k < k0 + n; ++k) {
      const int b = k / UPB, half = k - b * UPB;
      if (!SEL && b >= b_have + 32) {
        b_have = b;
        entry = (b + lane) * UPB < k0 + n ? __ldcg(row + b + lane) : -1;
      }
      if (SEL ? k == k0 : b == b_have && (k == k0 || half == 0)) {  // new entries: the ones outside the pool
        if (!SEL && (b + lane) * UPB < k0 + n && (entry < 0 || entry >= p.num_blocks)) {
          raise_flag(p.status, FLAG_BAD_BLOCK, entry);
          entry = -1;
        }
      }
      const int ph = __shfl_sync(0xffffffffu, entry, b - b_have);
      const int st = bi % NST, ub = bi / NST;
      if (ub > 0 && !ring_wait(&empty[st], (uint32_t)((ub - 1) & 1), dead)) {
        set_dead(dead, p.status, sg);
        ok = false;
        break;
      }
      if constexpr (BLK) {
        // The copies first (their fence waits for loads on their way); then the scales of the new
        // entries, which the phase waits for (this lane's arrival).
        if (lane == 0 && ph >= 0) {
          uint8_t* stg = tm.tiles + (size_t)st * LY::STAGE;
          const int y = (int)(((size_t)ph * p.G + g) * kBlock);
          fence_proxy_async();
          mbar_expect_tx_only(&full[st], (uint32_t)LY::STAGE);
          const uint64_t pol = p.stream ? l2_policy_evict_first() : l2_policy_evict_normal();
          tma_load_2d_hint(stg, tmk, 0, y, &full[st], pol);
          tma_load_2d_hint(stg + TR::TILE, tmv, 0, y, &full[st], pol);
        }
        if (SEL ? k == k0 : b == b_have && (k == k0 || half == 0)) {
          if (entry >= 0) {
            const size_t at = (size_t)entry * p.G + g;
            ks_mine = __ldcg(reinterpret_cast<const float*>(p.k_sc) + at);
            vs_mine = __ldcg(reinterpret_cast<const float*>(p.v_sc) + at);
          }
        }
        DenseStage f;
        f.ok = ph >= 0;
        f.key0 = kBlock * (SEL ? __shfl_sync(0xffffffffu, pick, b) : k);
        f.ks = __shfl_sync(0xffffffffu, ks_mine, b - b_have);
        f.vs = __shfl_sync(0xffffffffu, vs_mine, b - b_have);
        if (lane == 0) {
          tm.stage[st] = f;
          mbar_arrive(&full[st]);
        }
      } else if (lane == 0) {
        tm.stage_ok[st] = ph >= 0 ? 1 : 0;
        if (ph >= 0) {
          uint8_t* stg = tm.tiles + (size_t)st * LY::STAGE;
          const size_t tile = (size_t)ph * p.G + g;
          const int y = (int)(tile * kBlock) + half * TR::SK;
          fence_proxy_async();
          mbar_expect_tx(&full[st], (uint32_t)(LY::STAGE + LY::SCALES));
          // (made here: two registers more over the loop spill, NVFP4 with one token 173 to 184 us)
          const uint64_t pol = p.stream ? l2_policy_evict_first() : l2_policy_evict_normal();
          if constexpr (FMT == FMT_BF16) {
            tma_load_2d_hint(stg, tmk, 0, y, &full[st], pol);
            tma_load_2d_hint(stg + TR::SK * 128, tmk, 64, y, &full[st], pol);
            tma_load_2d_hint(stg + TR::TILE, tmv, 0, y, &full[st], pol);
            tma_load_2d_hint(stg + TR::TILE + TR::SK * 128, tmv, 64, y, &full[st], pol);
          } else {
            tma_load_2d_hint(stg, tmk, 0, y, &full[st], pol);
            tma_load_2d_hint(stg + TR::TILE, tmv, 0, y, &full[st], pol);
            uint8_t* sc = tm.mem + LY::SC + (size_t)st * LY::SCALES;
            bulk_g2s_hint(sc, p.k_sc + tile * TR::SC, TR::SC, &full[st], pol);
            bulk_g2s_hint(sc + TR::SC, p.v_sc + tile * TR::SC, TR::SC, &full[st], pol);
          }
        } else {
          mbar_arrive(&full[st]);  // a rejected block: an empty phase keeps the ring in step
        }
      }
      ++bi;
    }
    u += n;  // from the last key's unit on, the next round passes the segment's end
  }
  if (first && lane == 0) p.info[c] = make_int2(-1, 0);  // a run without keys
  if (ok) {
    const int slot = ii & 1, use = ii >> 1;
    if (use > 0 && !ring_wait(&iempty[slot], (uint32_t)((use - 1) & 1), dead)) {
      set_dead(dead, p.status, -1);
    } else if (lane == 0) {
      tm.facts[slot].n = -1;
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

constexpr int kDenseKSteps = 8;  // 16-dim steps of the first product

__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Where dim d of a query row is kept, so that a k step's 16 columns are the dims
// K's fragments hold in the same slots.  The order of the dims is free as long as
// both agree; d even, pairs stay together.
template <int FMT>
__device__ __forceinline__ int q_place(int d) {
  if constexpr (kBytes<FMT>) {  // K's slots 2j, 2j + 1 and 2j + 8, 2j + 9 hold dims 4j .. 4j + 3
    const int ks = d >> 4, j = (d >> 2) & 3, hi = (d >> 1) & 1;
    return 16 * ks + 8 * hi + 2 * j;
  } else if constexpr (FMT == FMT_NVFP4) {  // a lane's 32 consecutive dims, four a step
    const int j = d >> 5, ks = (d >> 2) & 7, hi = (d >> 1) & 1;
    return 16 * ks + 8 * hi + 2 * j;
  } else {
    return d;
  }
}

// The segment's query rows, in place, into the form of their fragments (16-bit
// rows of 256 bytes), and each row's logit factor (log2 domain).  One warp a row.
template <int FMT, int QROW>
__device__ __forceinline__ void convert_q(uint8_t* qs, float* cf, int nrows, int rows, bool q_fp8, float q_scale, float cst,
                                          int warp, int lane) {
#pragma unroll 1
  for (int row = warp; row < rows; row += kDenseWpg) {
    uint8_t* r = qs + (size_t)row * QROW;
    if (row >= nrows) {  // no such column: zeros
      *reinterpret_cast<uint2*>(r + 8 * lane) = make_uint2(0u, 0u);
      if (lane == 0) cf[row] = 1.f;
      continue;
    }
    if (q_fp8) {
      // widened exactly
      const uint32_t w = *reinterpret_cast<const uint32_t*>(r + 4 * lane);
      __syncwarp();
      uint32_t h[2];
      if constexpr (FMT == FMT_BF16) {
        const float2 a = e4m3x2_to_float2((uint16_t)w), b = e4m3x2_to_float2((uint16_t)(w >> 16));
        h[0] = pack_bf16x2(a.x, a.y);
        h[1] = pack_bf16x2(b.x, b.y);
      } else {
        h[0] = e4m3x2_to_f16x2(w);
        h[1] = e4m3x2_hi_to_f16x2(w);
      }
      *reinterpret_cast<uint32_t*>(r + 2 * q_place<FMT>(4 * lane)) = h[0];
      *reinterpret_cast<uint32_t*>(r + 2 * q_place<FMT>(4 * lane + 2)) = h[1];
      if (lane == 0) cf[row] = fmaxf(q_scale * cst, 1.2e-38f);
      continue;
    }
    if constexpr (FMT == FMT_BF16) {
      if (lane == 0) cf[row] = fmaxf(cst, 1.2e-38f);
      continue;  // as they are
    }
    const uint2 w = *reinterpret_cast<const uint2*>(r + 8 * lane);
    __syncwarp();
    const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
    // The largest e with amax 2^e <= 2^14, from the exponent and mantissa (magnitudes' bits order as they do, infinity and
    // NaN above all): on the way of every segment's first logits (three short sequences of 40 columns 13.2 us; 15.0 by divisions and ldexpf).
    uint32_t m = max(max(__float_as_uint(a.x) & 0x7fffffffu, __float_as_uint(a.y) & 0x7fffffffu),
                     max(__float_as_uint(b.x) & 0x7fffffffu, __float_as_uint(b.y) & 0x7fffffffu));
    m = __reduce_max_sync(0xffffffffu, m);
    const bool bad = m >= 0x7f800000u;
    const int e = bad || m == 0u ? 0 : min(126, 141 - (int)(m >> 23) - ((m & 0x7fffffu) != 0u ? 1 : 0));
    // A query row that is not finite has no finite logits; the reduced formats
    // would hide that, so it is NaN (the logits of masked keys are replaced all the
    // same).  The factor is kept off zero: it multiplies -inf.
    const float ps = bad ? __int_as_float(0x7fc00000) : pow2i(e);
    *reinterpret_cast<uint32_t*>(r + 2 * q_place<FMT>(4 * lane)) = pack_f16x2(a.x * ps, a.y * ps);
    *reinterpret_cast<uint32_t*>(r + 2 * q_place<FMT>(4 * lane + 2)) = pack_f16x2(b.x * ps, b.y * ps);
    if (lane == 0) cf[row] = fmaxf(pow2i(-e) * cst, 1.2e-38f);
  }
}

// Lane addresses into a stage's tiles.  Rows are swizzled: the 16-byte chunk c of
// row r sits at chunk c ^ (r & 7) (128-byte rows) or c ^ ((r >> 1) & 3) (64-byte
// rows), so stepping through a row is an XOR on bits 4 to 6 of the address and
// stepping by 8 rows leaves the swizzle alone.
template <int FMT>
__device__ __forceinline__ uint32_t k_lane(uint32_t tile, int lane) {
  if constexpr (FMT == FMT_NVFP4) {
    const int g8 = lane >> 2, j = lane & 3;  // 16 bytes of key g8
    return tile + g8 * 64 + ((j ^ ((g8 >> 1) & 3)) << 4);
  } else {
    return tile + (lane & 7) * 128 + (((lane >> 3) ^ (lane & 7)) << 4);  // ldmatrix: 8 keys x 4 chunks
  }
}
template <int FMT>
__device__ __forceinline__ uint32_t v_lane(uint32_t tile, int lane) {  // ldmatrix.trans: 16 keys x 2 chunks
  const int row = (lane & 7) + (lane & 8);
  if constexpr (FMT == FMT_NVFP4) return tile + row * 64 + (((lane >> 4) ^ ((lane >> 1) & 3)) << 4);
  else return tile + row * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
}

// S of KC keys from key row kb of the tile.  kl: k_lane of the tile; ql[m]: this
// lane's ldmatrix address of the query rows of tile m.  REG: the fragments are in aq.
template <int FMT, bool NVR, int KC, int MT, bool REG>
__device__ __forceinline__ void logits(uint32_t kl, const uint8_t* ksc, const uint32_t (&ql)[MT], int kb, int lane,
                                       const uint32_t (&aq)[kDenseKSteps][4], float (&sacc)[KC / 8][MT][4]) {
  using TR = DenseTraits<FMT>;
  constexpr int NT = KC / 8;
  constexpr int TG = NT < kDenseChains / MT ? NT : kDenseChains / MT;  // key tiles whose MMAs alternate
  kl += kb * (FMT == FMT_NVFP4 ? 64 : 128);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) sacc[t][m][0] = sacc[t][m][1] = sacc[t][m][2] = sacc[t][m][3] = 0.f;
  if constexpr (FMT == FMT_NVFP4) {
    const uint8_t* sc = ksc + (kb + (lane >> 2)) * 8 + 2 * (lane & 3);
    uint32_t w[NT][4], s2[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[t][0]), "=r"(w[t][1]), "=r"(w[t][2]), "=r"(w[t][3])
                   : "r"(kl + t * 512));
      s2[t] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(sc + t * 64));
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // 8 dims: two k steps
      uint32_t a[2][MT][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if constexpr (REG) {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[i][m][e] = aq[2 * q + i][e];
          } else {
            ldmatrix_x4(a[i][m], ql[m] + (2 * q + i) * 32);
          }
        }
#pragma unroll
      for (int t0 = 0; t0 < NT; t0 += TG) {
        uint32_t h[TG][4];
#pragma unroll
        for (int u = 0; u < TG; ++u) {
          const uint32_t sx = s2[t0 + u], sd = q < 2 ? __byte_perm(sx, sx, 0x1010) : __byte_perm(sx, sx, 0x3232);
          e2m1x8_to_f16(w[t0 + u][q], h[u]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            h[u][i] = hmul2(h[u][i], sd);
            if constexpr (NVR) h[u][i] = e4m3_round_f16x2(h[u][i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int u = 0; u < TG; ++u)
#pragma unroll
            for (int m = 0; m < MT; ++m) mma_f16_k16(sacc[t0 + u][m], a[i][m], h[u][2 * i], h[u][2 * i + 1]);
      }
    }
  } else if constexpr (kBytes<FMT>) {  // a register's four dims of a key: both halves of a k step
#pragma unroll
    for (int kp = 0; kp < 2; ++kp) {
      uint32_t b[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) ldmatrix_x4(b[t], (kl ^ (kp << 6)) + t * 1024);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t a[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if constexpr (REG) {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[m][e] = aq[4 * kp + i][e];
          } else {
            ldmatrix_x4(a[m], ql[m] + (4 * kp + i) * 32);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          uint32_t b0, b1;
          bytes_to_f16<FMT>(b[t][i], b0, b1);
#pragma unroll
          for (int m = 0; m < MT; ++m) mma_f16_k16(sacc[t][m], a[m], b0, b1);
        }
      }
    }
  } else {
#pragma unroll
    for (int kp = 0; kp < 4; ++kp) {
      uint32_t a[2][MT][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if constexpr (REG) {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[i][m][e] = aq[2 * kp + i][e];
          } else {
            ldmatrix_x4(a[i][m], ql[m] + (2 * kp + i) * 32);
          }
        }
#pragma unroll
      for (int t0 = 0; t0 < NT; t0 += TG) {
        uint32_t b[TG][4];
#pragma unroll
        for (int u = 0; u < TG; ++u)
          ldmatrix_x4(b[u], (kl ^ ((kp & 1) << 6)) + (kp >> 1) * (TR::SK * 128) + (t0 + u) * 1024);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int u = 0; u < TG; ++u)
#pragma unroll
            for (int m = 0; m < MT; ++m) mma_bf16_k16(sacc[t0 + u][m], a[i][m], b[u][2 * i], b[u][2 * i + 1]);
      }
    }
  }
}

// One accumulator tile += A B.  SOME: only the columns 2j (keep 1) and 2j + 1
// (keep 2) that are named (0 x NaN is NaN in every column of a product).
template <int FMT, bool SOME>
__device__ __forceinline__ void mma_cols(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, int keep) {
  if constexpr (!SOME) {
    if constexpr (FMT == FMT_BF16) mma_bf16_k16(d, a, b0, b1);
    else mma_f16_k16(d, a, b0, b1);
  } else {
    float t[4] = {d[0], d[1], d[2], d[3]};
    if constexpr (FMT == FMT_BF16) mma_bf16_k16(t, a, b0, b1);
    else mma_f16_k16(t, a, b0, b1);
    d[0] = keep & 1 ? t[0] : d[0];
    d[1] = keep & 2 ? t[1] : d[1];
    d[2] = keep & 1 ? t[2] : d[2];
    d[3] = keep & 2 ? t[3] : d[3];
  }
}

// O^T += V^T P over 16 keys from key row kb.  vl: v_lane of the tile; pb[n][2]: P's
// B fragments of column tile n (pl: the lo terms of bf16).  MASK: V of the keys
// beyond row klim of the tile counts as 0, and keep[n] names the columns added to.
template <int FMT, int NN, bool NVR, bool MASK>
__device__ __forceinline__ void pv16(uint32_t vl, const uint8_t* vs, int kb, int klim, int lane,
                                     const uint32_t (&pb)[NN][2], const uint32_t (&pl)[NN][2], float (&o)[8][NN][4],
                                     const int (&keep)[NN]) {
  using TR = DenseTraits<FMT>;
  const int j = lane & 3;
  vl += kb * (FMT == FMT_NVFP4 ? 64 : 128);
  uint32_t m0 = 0xffffffffu, m1 = 0xffffffffu;  // keys 2j, 2j + 1 and 2j + 8, 2j + 9 of the step
  if constexpr (MASK) {
    const int k = kb + 2 * j;
    m0 = (k <= klim ? 0xffffu : 0u) | (k + 1 <= klim ? 0xffff0000u : 0u);
    m1 = (k + 8 <= klim ? 0xffffu : 0u) | (k + 9 <= klim ? 0xffff0000u : 0u);
  }
  if constexpr (kBytes<FMT>) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t r[4];
      ldmatrix_x4_trans(r, vl ^ (c << 5));
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        // a register holds two dims of two keys: rows g8 take the even dim, rows g8 + 8 the odd one
        uint32_t a[4];
        bytes_apart_to_f16<FMT>(r[2 * q], a[0], a[1]);
        bytes_apart_to_f16<FMT>(r[2 * q + 1], a[2], a[3]);
        if constexpr (MASK) {
          a[0] &= m0;
          a[1] &= m0;
          a[2] &= m1;
          a[3] &= m1;
        }
#pragma unroll
        for (int n = 0; n < NN; ++n) mma_cols<FMT, MASK>(o[2 * c + q][n], a, pb[n][0], pb[n][1], keep[n]);
      }
    }
  } else if constexpr (FMT == FMT_BF16) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint32_t r[4];
      ldmatrix_x4_trans(r, (vl ^ ((c & 3) << 5)) + (c >> 2) * (TR::SK * 128));
      uint32_t a[4] = {r[0], r[2], r[1], r[3]};
      if constexpr (MASK) {
        a[0] &= m0;
        a[1] &= m0;
        a[2] &= m1;
        a[3] &= m1;
      }
#pragma unroll
      for (int n = 0; n < NN; ++n) mma_cols<FMT, MASK>(o[c][n], a, pb[n][0], pb[n][1], keep[n]);
#pragma unroll
      for (int n = 0; n < NN; ++n) mma_cols<FMT, MASK>(o[c][n], a, pl[n][0], pl[n][1], keep[n]);
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
      ldmatrix_x4_trans(r, vl ^ (cp << 5));
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int c = 2 * cp + q;
        uint32_t bb[2][4];  // [key half][dim 4 g8 + i of chunk c]
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
        for (int u = 0; u < 2; ++u) {
          const uint32_t a[4] = {bb[0][2 * u], bb[0][2 * u + 1], bb[1][2 * u], bb[1][2 * u + 1]};
#pragma unroll
          for (int n = 0; n < NN; ++n) mma_cols<FMT, MASK>(o[2 * c + u][n], a, pb[n][0], pb[n][1], keep[n]);
        }
      }
    }
  }
}

// Whether V of any key in tile rows [r0, r1) is not finite (whole warp).
template <int FMT>
__device__ __forceinline__ bool v_not_finite(const uint8_t* stg, const uint8_t* vs, int r0, int r1, int lane) {
  using TR = DenseTraits<FMT>;
  if constexpr (FMT == FMT_I8B) return false;
  bool bad = false;
  for (int row = r0; row < r1; ++row) {
    if constexpr (kBytes<FMT>) {
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

// The output dim of accumulator tile mt's row g8 (half 0) or g8 + 8 (half 1).
template <int FMT>
__device__ __forceinline__ int out_dim(int mt, int half, int g8) {
  if constexpr (kBytes<FMT>) return 16 * mt + 2 * g8 + half;
  else if constexpr (FMT == FMT_BF16) return 16 * mt + 8 * half + g8;
  else return 32 * (mt >> 1) + 4 * g8 + 2 * (mt & 1) + half;
}

template <int FMT, int NN, int NCG, bool NVR, bool SEL>
__device__ void consumer(const DenseParams& p, const DenseTeam& tm, int bar, int warp, int lane) {
  using TR = DenseTraits<FMT>;
  using LY = DenseLayout<FMT, NN, NCG>;
  constexpr int NST = LY::NST, MT = LY::MT, KGW = LY::KGW;
  constexpr int KW = TR::SK / KGW;             // keys of a warp in a unit
  constexpr int KC = KW < 32 ? KW : 32;        // keys a softmax step takes
  constexpr bool F16P = FMT != FMT_BF16, BLK = kByBlock<FMT>;
  constexpr float SHIFT = FMT == FMT_NVFP4 ? kDensePShift : 0.f;
  constexpr bool REG = NN == 1;                // query fragments held in registers
  constexpr int TEAM_THREADS = 32 * kDenseWpg;
  const int ct = warp / KGW, kw = (warp % KGW) * KW;  // column group, first key
  const int tid = warp * 32 + lane;
  const int g8 = lane >> 2, j = lane & 3;
  const int H = p.G * p.r;
  auto Q = [&] { return SEL ? 1 : p.Q; };  // (read where it is used: a register over the loop spills)
  int* dead = tm.dead;
  float4* ml = reinterpret_cast<float4*>(tm.mem + LY::ML);  // [warps][WROWS]: m, l, the scale of O or its weight
  float* cf = reinterpret_cast<float*>(tm.mem + LY::CF);      // [ROWS]
  int st = 0;
  uint32_t par = 0;
#pragma unroll 1
  for (int ii = 0;; ++ii) {
    const int slot = ii & 1;
    const bool got = ring_wait(&tm.ifull[slot], (uint32_t)((ii >> 1) & 1), dead);
    if (!got) set_dead(dead, p.status, ii);
    if (named_bar_or(bar, TEAM_THREADS, !got)) break;  // the team's consumers leave together
    const DenseFacts f = tm.facts[slot];
    if (f.n < 0) break;
    const int c0 = f.cg * p.cper;
    const int nrows = p.cols - c0 < p.cper ? p.cols - c0 : p.cper;
    uint8_t* qs = tm.mem + LY::Q + (size_t)slot * LY::QSLOT;
    convert_q<FMT, LY::QROW>(qs, cf, nrows, LY::ROWS, p.q_fp8 != 0, p.q_scale, p.col_const, warp, lane);
    named_bar_sync(bar, TEAM_THREADS);
    // ldmatrix addresses of the query tiles: row (lane & 7) + (lane & 8), column half
    // lane >> 4.  Where a tile has 8 rows only, the other 8 repeat them and are not used.
    uint32_t ql[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const bool half = 2 * m + 1 == NN;
      ql[m] = smem_u32(qs) + (ct * LY::WROWS + 16 * m + (lane & 7) + (half ? 0 : (lane & 8))) * LY::QROW + (lane >> 4) * 16;
    }
    uint32_t aq[kDenseKSteps][4];
    if constexpr (REG) {
#pragma unroll
      for (int ks = 0; ks < kDenseKSteps; ++ks) {
        ldmatrix_x4(aq[ks], ql[0] + ks * 32);
        aq[ks][1] = aq[ks][3] = 0u;
      }
    }

    // row state: the reference m_run (log2 domain), what is subtracted, and the raw logit that
    // moves it.  (FP8 subtracts m_run itself: four registers fewer where they spill, 2% with
    // 32 columns.)
    constexpr bool SAME = kBytes<FMT>;
    float m_run[NN], msub[NN], ylim[NN], colf[NN];
    float2 l_run[NN];
#pragma unroll
    for (int n = 0; n < NN; ++n) {
      m_run[n] = SAME ? kDenseNone : -INFINITY;
      ylim[n] = -INFINITY;
      msub[n] = SAME ? m_run[n] : 0.f;
      l_run[n] = make_float2(0.f, 0.f);
      colf[n] = cf[ct * LY::WROWS + 8 * n + g8];
    }
    float o[8][NN][4];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int n = 0; n < NN; ++n) o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.f;
    // FP8: P enters as P x vscale x fe, O is kept times fe (0: no product yet); vlim: the
    // largest scale that keeps every column within f16's range
    float fe[NN], vlim = -1.f;
#pragma unroll
    for (int n = 0; n < NN; ++n) fe[n] = 0.f;
    const int lim0 = f.T - Q();  // every row sees the keys up to here

#pragma unroll 1
    for (int k = f.k0; k < f.k0 + f.n; ++k) {
      const bool have = ring_wait(&tm.full[st], par, dead);
      if (!have) set_dead(dead, p.status, f.s);
      const uint32_t stg = smem_u32(tm.tiles + (size_t)st * LY::STAGE);
      const uint8_t* ksc = tm.mem + LY::SC + (size_t)st * LY::SCALES;  // scales of K, then of V
      const uint8_t* vsb = ksc + TR::SC;
      DenseStage sf = {};
      if constexpr (BLK) sf = tm.stage[st];
      if (have && (BLK ? sf.ok : tm.stage_ok[st])) {
        const uint32_t kl = k_lane<FMT>(stg, lane), vl = v_lane<FMT>(stg + TR::TILE, lane);
#pragma unroll 1
        for (int kb = kw; kb < kw + KW; kb += KC) {
          const int key0 = (SEL ? sf.key0 : k * TR::SK) + kb;  // position of the step's first key
          if (key0 >= f.T) break;
          float sacc[KC / 8][MT][4];
          logits<FMT, NVR, KC, MT, REG>(kl, ksc, ql, kb, lane, aq, sacc);
          const bool masked = key0 + KC - 1 > lim0;
          // ---- raw logits y (x = y colf), masked; does any pass the reference?
          float2 y[KC / 8][NN];
#pragma unroll
          for (int t = 0; t < KC / 8; ++t) {
            float2 ks = make_float2(1.f, 1.f);
            if constexpr (FMT == FMT_FP8) ks = lds_f2(reinterpret_cast<const float*>(ksc) + kb + 8 * t + 2 * j);
#pragma unroll
            for (int n = 0; n < NN; ++n) {
              float2 v = make_float2(sacc[t][n >> 1][2 * (n & 1)], sacc[t][n >> 1][2 * (n & 1) + 1]);
              if constexpr (FMT == FMT_FP8) v = mul2(v, ks);
              y[t][n] = v;
            }
          }
          // a block's scale goes to the columns' factors, or, where keys are masked, to the logits
          // (-inf times a factor that is 0 or NaN would be NaN)
          const float kf = BLK && !masked ? sf.ks : 1.f;
          if (BLK && masked) {
#pragma unroll
            for (int t = 0; t < KC / 8; ++t)
#pragma unroll
              for (int n = 0; n < NN; ++n) y[t][n] = mul2(y[t][n], make_float2(sf.ks, sf.ks));
          }
          if (masked) {
#pragma unroll
            for (int n = 0; n < NN; ++n) {
              const int row = ct * LY::WROWS + 8 * n + g8;
              const int lim = row < nrows ? lim0 + token_of<SEL>(c0 + row, p.r) - key0 : -1;
#pragma unroll
              for (int t = 0; t < KC / 8; ++t) {
                if (8 * t + 2 * j > lim) y[t][n].x = -INFINITY;
                if (8 * t + 2 * j + 1 > lim) y[t][n].y = -INFINITY;
              }
            }
          }
          float mx[NN];
          bool over = false;
#pragma unroll
          for (int n = 0; n < NN; ++n) {
            mx[n] = fmaxf(y[0][n].x, y[0][n].y);
#pragma unroll
            for (int t = 1; t < KC / 8; ++t) mx[n] = max3(mx[n], y[t][n].x, y[t][n].y);
            if constexpr (BLK) mx[n] *= kf;
            over |= mx[n] > ylim[n];
          }
          const bool moved = __any_sync(0xffffffffu, over);
          if (moved) {
            // the row's new reference
#pragma unroll
            for (int n = 0; n < NN; ++n) {
              mx[n] = fmaxf(mx[n], __shfl_xor_sync(0xffffffffu, mx[n], 1));
              mx[n] = fmaxf(mx[n], __shfl_xor_sync(0xffffffffu, mx[n], 2));
              const float mnew = fmaxf(m_run[n], mx[n] * colf[n]);
              const float ref = !SAME && mnew == -INFINITY ? 0.f : mnew;
              const float alpha = ex2(m_run[n] - ref);  // the first time 0 x 0
              m_run[n] = mnew;
              msub[n] = ref - SHIFT;
              ylim[n] = (mnew + kDenseLazy) / colf[n];
              l_run[n].x *= alpha;
              l_run[n].y *= alpha;
              if constexpr (kBytes<FMT>) {
                fe[n] = fe[n] > 0.f ? fe[n] * __frcp_rn(alpha) : 0.f;  // O itself follows below
              } else {
                // the accumulators hold the columns 2j, 2j + 1
                const float w0 = __shfl_sync(0xffffffffu, alpha, 8 * j);
                const float w1 = __shfl_sync(0xffffffffu, alpha, 8 * j + 4);
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                  o[t][n][0] *= w0;
                  o[t][n][1] *= w1;
                  o[t][n][2] *= w0;
                  o[t][n][3] *= w1;
                }
              }
            }
          }
          // ---- FP8: V's scales; does P x vscale x fe keep to f16's range?
          float2 vs[BLK ? 1 : KC / 8];
          float fv[NN];  // block scales: fe x vscale
          if constexpr (kBytes<FMT>) {
            float vm = 0.f;
            if constexpr (BLK) {
              vs[0] = make_float2(sf.vs, sf.vs);
              vm = fabsf(sf.vs);
            }
#pragma unroll
            for (int t = 0; t < (BLK ? 0 : KC / 8); ++t) {
              vs[t] = lds_f2(reinterpret_cast<const float*>(vsb) + kb + 8 * t + 2 * j);
              if (masked) {  // the scale of a row that holds no key may be anything
                if (key0 + 8 * t + 2 * j >= f.T) vs[t].x = 0.f;
                if (key0 + 8 * t + 2 * j + 1 >= f.T) vs[t].y = 0.f;
              }
              vm = max3(vm, fabsf(vs[t].x), fabsf(vs[t].y));
            }
#pragma unroll
            for (int t = 0; t < KC / 8; ++t)
#pragma unroll
              for (int n = 0; n < NN; ++n) {
                const float cn = BLK ? colf[n] * kf : colf[n];
                const float2 x = fma2(y[t][n], make_float2(cn, cn), make_float2(-m_run[n], -m_run[n]));
                y[t][n] = make_float2(ex2(x.x), ex2(x.y));  // the weights
                if constexpr (BLK) l_run[n] = add2(l_run[n], y[t][n]);
              }
            const bool look = moved || __any_sync(0xffffffffu, vm > vlim);
            if (look) {
              // the products themselves (times 2^-10, so that they are finite): few of the large
              // scales meet a large weight
              float top[NN];
              bool grow = moved;
#pragma unroll
              for (int n = 0; n < NN; ++n) {
                top[n] = 0.f;
#pragma unroll
                for (int t = 0; t < KC / 8; ++t) {
                  const float2 a = mul2(y[t][n], mul2(vs[BLK ? 0 : t], make_float2(0x1p-10f, 0x1p-10f)));
                  top[n] = max3(top[n], fabsf(a.x) < INFINITY ? fabsf(a.x) : 0.f, fabsf(a.y) < INFINITY ? fabsf(a.y) : 0.f);
                }
                grow |= fe[n] > 0.f ? top[n] * fe[n] > 32.f : top[n] > 0.f;
              }
              if (__any_sync(0xffffffffu, grow)) {
                vlim = INFINITY;
#pragma unroll
                for (int n = 0; n < NN; ++n) {
                  top[n] = fmaxf(top[n], __shfl_xor_sync(0xffffffffu, top[n], 1));
                  top[n] = fmaxf(top[n], __shfl_xor_sync(0xffffffffu, top[n], 2));
                  const float kept = fe[n] > 0.f ? kDenseTop * __frcp_rn(fe[n]) : 0.f;  // the former one
                  const float most = fmaxf(kept, 1024.f * top[n]);
                  float w = 1.f;  // of O, never above 1
                  if (!(kept == most && kept >= kDenseLeast)) {
                    const float inv = __frcp_rn(fminf(fmaxf(most, kDenseLeast), 3.0e38f));
                    w = kept * inv;
                    fe[n] = most > 0.f ? kDenseTop * inv : 0.f;
                  }
                  vlim = fminf(vlim, fe[n] > 0.f ? 128.f * __frcp_rn(fe[n]) : -1.f);  // a weight is 2^8 at most
                  // the accumulators hold the columns 2j, 2j + 1
                  const float w0 = __shfl_sync(0xffffffffu, w, 8 * j);
                  const float w1 = __shfl_sync(0xffffffffu, w, 8 * j + 4);
#pragma unroll
                  for (int t = 0; t < 8; ++t) {
                    o[t][n][0] *= w0;
                    o[t][n][1] *= w1;
                    o[t][n][2] *= w0;
                    o[t][n][3] *= w1;
                  }
                }
              }
            }
            if constexpr (BLK) {
              // |vscale| <= vlim: fe x vscale is 128 at most.  Else a product with a small weight
              // keeps to the range, but fe x vscale may not: one after the other.
              const bool apart = look && __any_sync(0xffffffffu, vm > vlim);
#pragma unroll
              for (int n = 0; n < NN; ++n) {
                fv[n] = apart ? sf.vs : fe[n] * sf.vs;
                if (apart) {
#pragma unroll
                  for (int t = 0; t < KC / 8; ++t) y[t][n] = mul2(y[t][n], make_float2(fe[n], fe[n]));
                }
              }
            }
          }
          // ---- P, its row sums, and P's fragments: keys 2j, 2j + 1 of tile t
          uint32_t ph[KC / 8][NN], plo[KC / 8][NN];
#pragma unroll
          for (int t = 0; t < KC / 8; ++t) {
#pragma unroll
            for (int n = 0; n < NN; ++n) {
              float2 q = y[t][n];
              if constexpr (!kBytes<FMT>) {
                const float2 x = fma2(q, make_float2(colf[n], colf[n]), make_float2(-msub[n], -msub[n]));
                q = make_float2(ex2(x.x), ex2(x.y));
              }
              if constexpr (!BLK) l_run[n] = add2(l_run[n], q);
              if constexpr (kBytes<FMT>) {
                const float2 v = BLK ? mul2(q, make_float2(fv[n], fv[n])) : mul2(mul2(q, make_float2(fe[n], fe[n])), vs[BLK ? 0 : t]);
                if (masked) {  // a masked weight stays 0 beside a scale that is not finite
                  q.x = q.x == 0.f ? 0.f : v.x;
                  q.y = q.y == 0.f ? 0.f : v.y;
                } else {
                  q = v;
                }
              }
              if constexpr (F16P) {
                ph[t][n] = pack_f16x2(q.x, q.y);
                plo[t][n] = 0u;
              } else {
                const uint32_t h = pack_bf16x2(q.x, q.y);
                const float2 hv = bf16x2_to_float2(h);
                ph[t][n] = h;
                plo[t][n] = pack_bf16x2(q.x - hv.x, q.y - hv.y);
              }
            }
          }
          // ---- O^T += V^T P
#define MSA_DENSE_PV(MASK, KLIM, KEEP)                                                        \
  _Pragma("unroll") for (int h = 0; h < KC / 16; ++h) {                                       \
    uint32_t pb[NN][2], pl[NN][2];                                                            \
    _Pragma("unroll") for (int n = 0; n < NN; ++n) {                                          \
      pb[n][0] = ph[2 * h][n];                                                                \
      pb[n][1] = ph[2 * h + 1][n];                                                            \
      pl[n][0] = plo[2 * h][n];                                                               \
      pl[n][1] = plo[2 * h + 1][n];                                                           \
    }                                                                                         \
    pv16<FMT, NN, NVR, MASK>(vl, vsb, kb + 16 * h, KLIM, lane, pb, pl, o, KEEP);              \
  }
          int keep[NN];
#pragma unroll
          for (int n = 0; n < NN; ++n) keep[n] = 3;
          if (!masked) {
            MSA_DENSE_PV(false, 0, keep)
          } else {
            // tile rows up to the last key of the sequence; with several new tokens a
            // row between lim0 and there is seen by some of them only, and if its V is
            // not finite each token goes by itself, up to its own position
            const int klast = f.T - 1 - (key0 - kb);
            int r0 = lim0 + 1 - (key0 - kb), r1 = klast + 1;
            r0 = r0 < kb ? kb : r0;
            r1 = r1 > kb + KC ? kb + KC : r1;
            const bool apart =
                Q() > 1 && v_not_finite<FMT>(tm.tiles + (size_t)st * LY::STAGE, vsb, r0, r1, lane);
#pragma unroll 1
            for (int i = apart ? 0 : Q() - 1; i < Q(); ++i) {
              if (apart) {
#pragma unroll
                for (int n = 0; n < NN; ++n) {
                  const int col = c0 + ct * LY::WROWS + 8 * n + 2 * j;
                  keep[n] = (token_of<SEL>(col, p.r) == i ? 1 : 0) | (token_of<SEL>(col + 1, p.r) == i ? 2 : 0);
                }
              }
              MSA_DENSE_PV(true, klast - (Q() - 1 - i), keep)
            }
          }
#undef MSA_DENSE_PV
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&tm.empty[st]);
      if (++st == NST) {
        st = 0;
        par ^= 1u;
      }
    }
    fence_proxy_async();  // the query rows were rewritten in place; the next copy into them comes after that
    __syncwarp();
    if (lane == 0) mbar_arrive(&tm.iempty[slot]);

    // ---------------- the segment's result: the warps of a column group hold different keys
#pragma unroll
    for (int n = 0; n < NN; ++n) {
      const float osc = kBytes<FMT> ? (fe[n] > 0.f ? __frcp_rn(fe[n]) : 0.f) : (FMT == FMT_NVFP4 ? p.v_global : 1.f);
      float l = l_run[n].x + l_run[n].y;
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (j == 0) ml[warp * LY::WROWS + 8 * n + g8] = make_float4(m_run[n], l, osc, 0.f);
    }
    const bool whole = f.part < 0;
    if constexpr (NN == 1) {
      // Few columns: all of them through shared memory, then a thread a row and four
      // dims.  The code runs once a segment, so its size counts (instruction fetches):
      // only the stores out of the accumulators are unrolled.  256 sequences of 100 to
      // 1,000 tokens: 41.9 us, 43.1 in two halves, and 53 in the other way (below).
      float* mo = reinterpret_cast<float*>(tm.mem + LY::MERGE);  // [warps][WROWS][MROW]
#pragma unroll
      for (int c = 0; c < 2; ++c) {  // column 2j + c
        float* row = mo + (warp * LY::WROWS + 2 * j + c) * LY::MROW;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          const float(&v)[4] = o[mt][0];
          const int d = out_dim<FMT>(mt, 0, g8);
          if constexpr (FMT == FMT_NVFP4) {
            const float(&v1)[4] = o[mt | 1][0];
            if (!(mt & 1)) *reinterpret_cast<float4*>(row + d) = make_float4(v[c], v[c + 2], v1[c], v1[c + 2]);
          } else if constexpr (kBytes<FMT>) {
            *reinterpret_cast<float2*>(row + d) = make_float2(v[c], v[c + 2]);
          } else {
            row[d] = v[c];
            row[out_dim<FMT>(mt, 1, g8)] = v[c + 2];
          }
        }
      }
      named_bar_sync(bar, TEAM_THREADS);
#pragma unroll 1
      for (int x = tid; x < nrows * 32; x += TEAM_THREADS) {
        const int row = x >> 5, d = 4 * (x & 31);
        float4 v[KGW];
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < KGW; ++w) {
          v[w] = ml[w * LY::WROWS + row];
          M = fmaxf(M, v[w].x);
        }
        const float ms = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < KGW; ++w) {
          const float fw = ex2(v[w].x - ms);
          L += fw * v[w].y;
          const float4 ov = *reinterpret_cast<const float4*>(mo + (w * LY::WROWS + row) * LY::MROW + d);
          acc.x += fw * (ov.x * v[w].z);
          acc.y += fw * (ov.y * v[w].z);
          acc.z += fw * (ov.z * v[w].z);
          acc.w += fw * (ov.w * v[w].z);
        }
        if (whole) {
          const float inv = L == 0.f ? 0.f : 1.f / L;
          const int col = c0 + row, i = token_of<SEL>(col, p.r), h = col - i * p.r;
          const size_t orow = ((size_t)f.s * Q() + i) * H + (size_t)f.g * p.r + h;
          uint2 pk;
          pk.x = pack_bf16x2(acc.x * inv, acc.y * inv);
          pk.y = pack_bf16x2(acc.z * inv, acc.w * inv);
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + orow * kDim + d) = pk;
          if (d == 0 && p.lse) p.lse[orow] = L == 0.f ? -INFINITY : (M - SHIFT + log2f(L)) * 0.69314718055994531f;
        } else {
          *reinterpret_cast<float4*>(p.part_o + ((size_t)f.part * LY::ROWS + row) * kDim + d) = acc;
          if (d == 0) p.part_ml[(size_t)f.part * LY::ROWS + row] = make_float2(M, L);
        }
      }
      named_bar_sync(bar, TEAM_THREADS);  // the merge area is free again
    } else {
      // Many columns: each warp takes 1 / KGW of the output tiles from the others, as
      // they lie in the lanes (16 bytes a lane, no bank conflicts), and writes them.
      // 61 ragged sequences of 48 columns take 7% longer the other way.
      float4* mo = reinterpret_cast<float4*>(tm.mem + LY::MERGE);  // [warps][receivers][tiles][lanes]
      named_bar_sync(bar, TEAM_THREADS);
      if (tid < LY::ROWS) {  // a thread a column: the weights of its group's warps
        const int at = tid / LY::WROWS * KGW * LY::WROWS + tid % LY::WROWS;
        float4 v[KGW];
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < KGW; ++w) {
          v[w] = ml[at + w * LY::WROWS];
          M = fmaxf(M, v[w].x);
        }
        const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < KGW; ++w) {
          v[w].x = ex2(v[w].x - ms);
          L += v[w].x * v[w].y;
        }
        const float inv = whole ? (L == 0.f ? 0.f : 1.f / L) : 1.f;
#pragma unroll
        for (int w = 0; w < KGW; ++w) ml[at + w * LY::WROWS].w = v[w].x * inv;
        if (tid < nrows) {
          if (!whole) {
            p.part_ml[(size_t)f.part * LY::ROWS + tid] = make_float2(M, L);
          } else if (p.lse) {
            const int col = c0 + tid, i = token_of<SEL>(col, p.r), h = col - i * p.r;
            p.lse[((size_t)f.s * Q() + i) * H + (size_t)f.g * p.r + h] =
                L == 0.f ? -INFINITY : (M - SHIFT + log2f(L)) * 0.69314718055994531f;
          }
        }
      }
      named_bar_sync(bar, TEAM_THREADS);
      const int me = warp % KGW, grp = warp - me;
#pragma unroll
      for (int n = 0; n < NN; ++n) {
        const float4* own = ml + warp * LY::WROWS + 8 * n + 2 * j;
        const float2 oc = make_float2(own[0].z, own[1].z), wc = make_float2(own[0].w, own[1].w);  // columns 2j, 2j + 1
        // where this lane writes: BF16 lanes hold dims 8 apart and pair up with a neighbour's, one column each
        size_t at[2];
        bool live[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int row = ct * LY::WROWS + 8 * n + 2 * j + (FMT == FMT_BF16 ? (g8 & 1) : c);
          live[c] = row < nrows;
          const int col = c0 + row, i = token_of<SEL>(col, p.r), h = col - i * p.r;
          at[c] = whole ? (((size_t)f.s * Q() + i) * H + (size_t)f.g * p.r + h) * kDim
                        : ((size_t)f.part * LY::ROWS + row) * kDim;
        }
#pragma unroll
        for (int w = 0; w < KGW; ++w)
#pragma unroll
          for (int u = 0; u < LY::MT_OWN; ++u) {
            float(&v)[4] = o[w * LY::MT_OWN + u][n];
            v[0] = v[0] * oc.x * wc.x;
            v[1] = v[1] * oc.y * wc.y;
            v[2] = v[2] * oc.x * wc.x;
            v[3] = v[3] * oc.y * wc.y;
            if (w != me)
              mo[((warp * (KGW - 1) + (w < me ? w : w - 1)) * LY::MT_OWN + u) * 32 + lane] = make_float4(v[0], v[1], v[2], v[3]);
          }
        named_bar_sync(bar, TEAM_THREADS);
#pragma unroll
        for (int u = 0; u < LY::MT_OWN; ++u) {
          float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < KGW; ++w) {  // in the order of the keys
            const float(&mine)[4] = o[w * LY::MT_OWN + u][n];
            float4 x = make_float4(mine[0], mine[1], mine[2], mine[3]);
            if (w != me) x = mo[(((grp + w) * (KGW - 1) + (me < w ? me : me - 1)) * LY::MT_OWN + u) * 32 + lane];
            a[0] += x.x;
            a[1] += x.y;
            a[2] += x.z;
            a[3] += x.w;
          }
          const int mt = me * LY::MT_OWN + u;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float2 v;
            int dim;
            if constexpr (FMT == FMT_BF16) {
              const bool odd = g8 & 1;
              const float got = __shfl_xor_sync(0xffffffffu, odd ? a[2 * c] : a[2 * c + 1], 4);
              v = odd ? make_float2(got, a[2 * c + 1]) : make_float2(a[2 * c], got);
              dim = out_dim<FMT>(mt, c, g8 & ~1);
            } else {
              v = make_float2(a[c], a[c + 2]);
              dim = out_dim<FMT>(mt, 0, g8);
            }
            if (live[c]) {
              if (whole) *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + at[c] + dim) = pack_bf16x2(v.x, v.y);
              else *reinterpret_cast<float2*>(p.part_o + at[c] + dim) = v;
            }
          }
        }
        named_bar_sync(bar, TEAM_THREADS);  // the merge area is free again
      }
    }
  }
}

// One CTA an SM.  Two teams are ten warps with up to 168 registers a thread, or, WIDE,
// twelve launched with 168, of which the producers' four keep 40 and the consumers'
// eight take 232 (128 x 40 + 256 x 232 = 384 x 168 = 64,512 registers; MORE: 24 and 240); three teams
// are fifteen with up to 128, or sixteen launched with 128, the producers' four with 56
// then and the consumers' twelve with 152 (128 x 56 + 384 x 152 = 512 x 128).
template <int FMT, int NN, int NCG, bool NVR, bool SEL>
__global__ void __launch_bounds__(DenseLayout<FMT, NN, NCG>::THREADS, 1)
    dense_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const DenseParams p) {
  using LY = DenseLayout<FMT, NN, NCG>;
  constexpr int NST = LY::NST, TEAMS = LY::TEAMS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool consumes = warp < TEAMS * kDenseWpg;
  const int team = consumes ? warp / kDenseWpg : warp - TEAMS * kDenseWpg;
  DenseTeam tm;
  tm.tiles = base + (size_t)team * NST * LY::STAGE;
  tm.mem = base + LY::TILES + (size_t)team * LY::TEAM;
  tm.full = reinterpret_cast<uint64_t*>(tm.mem + LY::BARS);
  tm.empty = tm.full + NST;
  tm.ifull = tm.empty + NST;
  tm.iempty = tm.ifull + 2;
  tm.stage_ok = reinterpret_cast<int*>(tm.mem + LY::STAGES);
  tm.stage = reinterpret_cast<DenseStage*>(tm.mem + LY::STAGES);
  tm.dead = reinterpret_cast<int*>(tm.mem + LY::STAGES + LY::STAGES_BYTES);
  tm.facts = reinterpret_cast<DenseFacts*>(tm.mem + LY::FACTS);
  tm.id = blockIdx.x * TEAMS + team;
  if (!consumes && team < TEAMS && lane == 0) {
    for (int st = 0; st < NST; ++st) {
      mbar_init(&tm.full[st], 1);
      mbar_init(&tm.empty[st], kDenseWpg);
    }
    for (int sl = 0; sl < 2; ++sl) {
      mbar_init(&tm.ifull[sl], 1);
      mbar_init(&tm.iempty[sl], kDenseWpg);
    }
    *tm.dead = 0;
    fence_mbar_init();
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
  }
  __syncthreads();
  pdl_wait();               // (nothing of the memory has been touched)
  pdl_launch_dependents();  // the combine's CTAs may take their place as soon as this grid's leave room
  if (!consumes) {
    if constexpr (LY::MOVE) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(LY::REGS_P));
    if (team < TEAMS) producer<FMT, NN, NCG, SEL>(&tmk, &tmv, p, tm, lane);
  } else {
    if constexpr (LY::MOVE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(LY::REGS_C));
    // sequences without keys (and malformed ones) have no units: their rows here
    for (int s = SEL ? p.S : blockIdx.x + warp * gridDim.x; s < p.S; s += gridDim.x * TEAMS * kDenseWpg) {
      const int T = __ldcg(p.seq_lens + s);
      if (T >= 1 && T <= p.max_nb * kBlock) continue;
      if (T != 0 && lane == 0) raise_flag(p.status, FLAG_BAD_SEQLEN, T);
      const long rows = (long)p.Q * p.G * p.r;
      uint2* orow = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + (size_t)s * rows * kDim);
      for (long x = lane; x < rows * 32; x += 32) orow[x] = make_uint2(0u, 0u);
      if (p.lse)
        for (long x = lane; x < rows; x += 32) p.lse[(size_t)s * rows + x] = -INFINITY;
    }
    consumer<FMT, NN, NCG, NVR, SEL>(p, tm, 1 + team, warp % kDenseWpg, lane);
  }
}

template <int FMT, int NN, int NCG, bool NVR, bool SEL = false>
cudaError_t launch_one(const CUtensorMap* tk, const CUtensorMap* tv, const DenseParams& p, int num_sms, cudaStream_t st) {
  using LY = DenseLayout<FMT, NN, NCG>;
  static_assert(LY::ROWS == dense_rows(NN, NCG) && LY::TEAMS == dense_teams(FMT, NN), "the plan's sizes");
  auto kern = dense_kernel<FMT, NN, NCG, NVR, SEL>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), (int)LY::SMEM, allowed);
  if (e != cudaSuccess) return e;
  if constexpr (LY::MOVE) {
    // the consumers would wait for ever for registers that the launch did not bring
    static const int regs = [&] {
      cudaFuncAttributes fa;
      return cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : 0;
    }();
    if (regs / 8 * 8 * LY::THREADS < 128 * LY::REGS_P + LY::CONSUMERS * LY::REGS_C) return cudaErrorLaunchOutOfResources;
  }
  return launch_behind(kern, dim3((unsigned)num_sms), dim3(LY::THREADS), LY::SMEM, st, *tk, *tv, p);
}

// The instance for the columns of a group (dense_shape).
template <int FMT, bool SEL>
cudaError_t launch_shape(const CUtensorMap* tk, const CUtensorMap* tv, const DenseParams& p, int num_sms, cudaStream_t st) {
  const DenseShape sh = dense_shape(p.cper);
  if (sh.ncg == 2)
    return sh.nn == 3 ? launch_one<FMT, 3, 2, false, SEL>(tk, tv, p, num_sms, st) : launch_one<FMT, 4, 2, false, SEL>(tk, tv, p, num_sms, st);
  switch (sh.nn) {
    case 1: return launch_one<FMT, 1, 1, false, SEL>(tk, tv, p, num_sms, st);
    case 2: return launch_one<FMT, 2, 1, false, SEL>(tk, tv, p, num_sms, st);
    case 3: return launch_one<FMT, 3, 1, false, SEL>(tk, tv, p, num_sms, st);
    default: return launch_one<FMT, 4, 1, false, SEL>(tk, tv, p, num_sms, st);
  }
}

}  // namespace dense
}  // namespace msa
