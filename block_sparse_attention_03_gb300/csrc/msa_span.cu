// Spans of tokens into and out of the paged caches: the insert of new K and V rows
// into a cache with one scale for each block of 128 tokens and head, and the read of
// tokens back as bf16 rows out of a cache of any format.
//
// Insert, for a block, a head and K or V (Q = 127 for INT8, 448 for E4M3):
//   need = max(amax / Q, 2^-126), amax over the finite new elements;
//   scale = need where the block's first row is new, else old x 2^k, the least k >= 0
//   with old x 2^k >= need; held codes become round(code x 2^-k) where k > 0;
//   code = round(x / scale).
// Growing by powers of two moves E4M3 codes exactly (down to their subnormals) and
// keeps INT8's accumulated roundings below 1/2 + 1/4 + ... = one step of the present scale,
// however often a block grows; the price is up to one of INT8's seven bits.
// k compares exponents and mantissas, so it needs no division and cannot overflow.
// The quotients are divide2()'s, correctly rounded, so that the codes are those of a division.
//
// Split.  An item is a block, a head, and K or V: its scale needs all of its new rows, and the
// blocks are independent.  The lengths are on the device: a CTA sums up the blocks that 256
// spans touch and takes every n-th of them.  A CTA an item (prompts, chunks), its rows in registers
// between the maximum and the quotients, the next item's on their way into shared memory
// meanwhile; a warp an item where spans bring a step's few tokens.  No atomics on data: equal
// calls give equal bits.
//
// Insert bound: HBM in the limit, 256 bytes in and 128 out a row.  Measured (one GPU, back to
// back in a graph; of 6,702 GB/s copied): a prompt of 8,192 tokens x 4 heads 5.9 us (64%, of which some
// 3 are the launch and the chain lengths - sums - table - rows), 64 spans of 700 to 900 tokens x 8 heads 46 us
// (87%), 253 ragged ones of up to 200 29 us (68%: items of 55 rows on average, of whose 420 instructions
// a warp 170 are the item's own; issue slots 69% busy), 32 requests of one token 2.8 us, 8,000 of them 23 us.
// All of these without growth.  A block that grows has its held codes read and written once the maximum is known: where
// every block does, 32 requests of one token 11.5 us (a warp moves up to 16 KB), the 253 ragged ones 51, the prompt 5.8.
// Two rows' copies ahead (48 KB an SM on their way) do as well as three or a ring filled as far
// as it goes (32 and 38 us for the ragged ones: fewer CTAs, or more to do for each item); rows read twice
// instead, out of the L2, by teams of one to four warps 34 to 56 us (a block of 128 rows is too long for one).
//
// Read bound: HBM, mostly the writes.  A thread has eight rows' loads on their way before it
// stores the first; one item a CTA in hardware's order rather than a grid that stays (8 prefixes of
// 16K to 32K tokens 94 us, 96% of the copy rate; 109 so).  One prefix of 4K tokens 3.5 us, 61 ragged
// spans out of NVFP4 8.7 us (61%: two rounds of the chain above).
#include "msa_device.cuh"
#include "msa_internal.h"

namespace msa {

namespace {

constexpr int kSpanThreads = 256;
constexpr int kSpanWarps = kSpanThreads / 32;
constexpr int kRowsPerThread = kBlock / (2 * kSpanWarps);  // a half warp takes a row

// What a CTA knows of 256 sequences: the blocks their spans touch, summed up.
struct SpanChunk {
  int32_t first[kSpanThreads], end[kSpanThreads], off[kSpanThreads];
  int32_t before[kSpanThreads];  // blocks touched by the sequences in front
  int32_t warp_sum[kSpanWarps];
};

// One block of one span.  (The insert looks up 32 of a CTA's blocks at once, one a lane.)
struct SpanBlock {
  int n, at;  // its tokens, the first one's row in the block
  int row;    // and in the call's tensors
  int had;    // tokens that the block held in front of the span
  int phys;   // the block table's entry
};

// Which chunks of 256 sequences are a CTA's, and its place among the CTAs that share them: CTA
// (x, y) takes head and K or V x, and the chunks y mod their number, + gridDim.y, ... where there are more
// chunks than CTAs.
struct SpanWalk {
  int s0, step;
  uint32_t rank, size;
};
__device__ __forceinline__ SpanWalk span_walk(const SpanParams& p) {
  const uint32_t chunks = ((uint32_t)p.S + kSpanThreads - 1) / kSpanThreads, groups = min(chunks, gridDim.y);
  if (groups == 1) return {0, kSpanThreads, blockIdx.y, gridDim.y};
  const uint32_t group = blockIdx.y % groups;
  return {(int)group * kSpanThreads, (int)groups * kSpanThreads, blockIdx.y / groups, (gridDim.y - group + groups - 1) / groups};
}

// The spans s0 .. s0 + 255: returns how many blocks they touch.  Block i of those, in
// (sequence, position) order, goes to worker i mod their number.  (The host bounds
// num_tokens so that 256 spans touch fewer than 2^31 blocks.)
__device__ __forceinline__ int load_chunk(const SpanParams& p, SpanChunk& c, int s0, bool again) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = s0 + tid;
  int first = 0, end = 0, off = 0, count = 0;
  if (s < p.S) {
    first = p.first[s];
    end = p.end[s];
    off = p.offsets[s];
    if (end > first) {
      uint32_t bad = 0;
      if (first < 0 || end > p.max_nb * kBlock) bad = FLAG_BAD_SEQLEN;
      else if (off < 0 || off > p.num_tokens - (end - first)) bad = FLAG_NO_ROOM;
      if (bad == 0) count = (end - 1) / kBlock - first / kBlock + 1;
      else if (blockIdx.x == 0) raise_flag(p.status, bad, s);
    }
  }
  int incl = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (again) __syncthreads();  // the former chunk has been read
  if (lane == 31) c.warp_sum[warp] = incl;
  c.first[tid] = first;
  c.end[tid] = end;
  c.off[tid] = off;
  __syncthreads();
  int total = 0, front = 0;
#pragma unroll
  for (int w = 0; w < kSpanWarps; ++w) {
    const int v = c.warp_sum[w];
    if (w < warp) front += v;
    total += v;
  }
  c.before[tid] = front + incl - count;
  __syncthreads();
  return total;
}

// Block i of the chunk's.
__device__ __forceinline__ SpanBlock find_block(const SpanParams& p, const SpanChunk& c, int s0, int i) {
  int at = 0;  // the last sequence with no more than i blocks before it: it touches one itself
#pragma unroll
  for (int step = kSpanThreads / 2; step > 0; step >>= 1)
    if (c.before[at + step] <= i) at += step;
  const int first = c.first[at], blk = first / kBlock + (i - c.before[at]);
  const int p0 = max(first, blk * kBlock);
  SpanBlock b;
  b.n = min(c.end[at], (blk + 1) * kBlock) - p0;
  b.row = c.off[at] + (p0 - first);
  b.at = p0 % kBlock;
  b.had = max(0, first - blk * kBlock);
  b.phys = p.block_table[(size_t)(s0 + at) * p.max_nb + blk];
  return b;
}
__device__ __forceinline__ SpanBlock from_lane(const SpanBlock& b, int lane) {
  SpanBlock r;
  r.n = __shfl_sync(0xffffffffu, b.n, lane);
  r.at = __shfl_sync(0xffffffffu, b.at, lane);
  r.row = __shfl_sync(0xffffffffu, b.row, lane);
  r.had = __shfl_sync(0xffffffffu, b.had, lane);
  r.phys = __shfl_sync(0xffffffffu, b.phys, lane);
  return r;
}

__device__ __forceinline__ bool in_pool(const SpanParams& p, int phys) { return phys >= 0 && phys < p.num_blocks; }

// ---------------------------------------------------------------- insert

// Four elements as codes, rounded to nearest even.  SAFE: any fp32 values; else
// |z| < 2^21, for INT8 below 127.5.
template <int FMT, bool SAFE>
__device__ __forceinline__ uint32_t block_codes(float2 a, float2 b) {
  if constexpr (FMT == FMT_F8B) {
    return (uint32_t)pack_e4m3x2(a.x, a.y) | ((uint32_t)pack_e4m3x2(b.x, b.y) << 16);
  } else {
    float z[4] = {a.x, a.y, b.x, b.y};
    if constexpr (SAFE) {
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = z[i] == z[i] ? fminf(fmaxf(z[i], -127.f), 127.f) : 0.f;
    }
    // 1.5 x 2^23 + z has the rounded z, two's complement, in its lowest byte
    const float2 m = make_float2(12582912.f, 12582912.f);
    const float2 x = add2(make_float2(z[0], z[1]), m), y = add2(make_float2(z[2], z[3]), m);
    return __byte_perm(__byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x0040),
                       __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x0040), 0x5410);
  }
}

// Four held codes x 2^-k.
template <int FMT>
__device__ __forceinline__ uint32_t move_codes(uint32_t w, float f) {
  float2 a, b;
  if constexpr (FMT == FMT_F8B) {
    a = e4m3x2_to_float2((uint16_t)w);
    b = e4m3x2_to_float2((uint16_t)(w >> 16));
  } else {
    a = make_float2((float)(int8_t)w, (float)(int8_t)(w >> 8));
    b = make_float2((float)(int8_t)(w >> 16), (float)(int8_t)(w >> 24));
  }
  const float2 f2 = make_float2(f, f);
  return block_codes<FMT, false>(mul2(a, f2), mul2(b, f2));
}

__device__ __forceinline__ bool normal_positive(float v) {
  return __float_as_uint(v) - 0x00800000u < 0x7f000000u;
}

// The least k >= 0 with a x 2^k >= b, for normal positive a and b.
__device__ __forceinline__ int growth(float a, float b) {
  const uint32_t u = __float_as_uint(a), v = __float_as_uint(b);
  const int k = (int)(v >> 23) - (int)(u >> 23) + ((v & 0x7fffffu) > (u & 0x7fffffu) ? 1 : 0);
  return k > 0 ? k : 0;
}

// The larger magnitude of two pairs of bf16, half by half, under any sign; NaN if either is.
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t larger(uint32_t m, const uint4& x) {
  return larger2(m, larger2(larger2(x.x, x.y), larger2(x.z, x.w)));
}
// The bits of the larger half's magnitude: they order as the values do, NaN above all.
__device__ __forceinline__ uint32_t magnitude(uint32_t m) { return max(m & 0x7fffu, (m >> 16) & 0x7fffu); }
constexpr uint32_t kNotFinite = 0x7f80u;
// The same of the finite elements only.
__device__ __forceinline__ uint32_t larger_finite(uint32_t m, const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = w[j] & 0x7fffu, hi = (w[j] >> 16) & 0x7fffu;
    m = max(m, max(lo < kNotFinite ? lo : 0u, hi < kNotFinite ? hi : 0u));
  }
  return m;
}

// The block's scale for the largest magnitude m (bits) and, in `k`, by how many powers of two the
// held codes shrink.
template <int FMT>
__device__ __forceinline__ float block_scale(uint32_t m, bool held, float old, int& k) {
  constexpr float kLeast = 1.17549435e-38f;  // 2^-126
  const float need = fmaxf(__fdiv_rn(__uint_as_float(m << 16), FMT == FMT_I8B ? 127.f : 448.f), kLeast);
  k = 0;
  if (!held) return need;
  const float s = normal_positive(old) ? old : kLeast;
  k = growth(s, need);
  return __uint_as_float(__float_as_uint(s) + ((uint32_t)k << 23));  // below 2 need: no overflow
}

// `had` rows of held codes x 2^-k, by `threads` threads.
template <int FMT>
__device__ __forceinline__ void shrink(uint8_t* data, int had, int k, int tid, int threads) {
  const float f = pow2i(k < 126 ? -k : -126);  // (a smaller factor leaves nothing of a code either)
#pragma unroll 4
  for (int i = tid; i < had * 8; i += threads) {
    uint4 w = *reinterpret_cast<const uint4*>(data + 16 * i);
    w.x = move_codes<FMT>(w.x, f);
    w.y = move_codes<FMT>(w.y, f);
    w.z = move_codes<FMT>(w.z, f);
    w.w = move_codes<FMT>(w.w, f);
    *reinterpret_cast<uint4*>(data + 16 * i) = w;
  }
}

// Eight elements' codes: finite ones and a scale that divides() takes (r2: its reciprocal, n2: minus it) ...
template <int FMT>
__device__ __forceinline__ uint2 quantize(const uint4& x, float2 r2, float2 n2) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
  float2 z[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) z[j] = divide2(make_float2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u)), r2, n2);
  return make_uint2(block_codes<FMT, false>(z[0], z[1]), block_codes<FMT, false>(z[2], z[3]));
}
// ... and any.
template <int FMT>
__device__ __forceinline__ uint2 quantize_any(const uint4& x, float s) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
  float2 z[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    z[j] = make_float2(__fdiv_rn(__uint_as_float(u[j] << 16), s), __fdiv_rn(__uint_as_float(u[j] & 0xffff0000u), s));
  return make_uint2(block_codes<FMT, true>(z[0], z[1]), block_codes<FMT, true>(z[2], z[3]));
}

// A CTA an item.  Items on their way at once are each in a stage of 32 KB of shared memory; a
// thread copies and reads the same bytes, so the copies need no barrier.
constexpr int kInsertStages = 2;
constexpr int kInsertCtas = 3;  // CTAs an SM
constexpr int kStride = 2 * kSpanWarps;  // a half warp takes a row: rows between a thread's

template <int FMT>
__global__ void __launch_bounds__(kSpanThreads, kInsertCtas) block_insert_kernel(const SpanParams p) {
  extern __shared__ uint4 s_rows[];  // [stages][rows of a thread][threads]
  __shared__ SpanChunk chunk;
  __shared__ __align__(16) uint32_t s_max[2][kSpanWarps];
  static_assert(kSpanWarps == 8, "all_max");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l16 = lane & 15;
  const int row0 = 2 * warp + (lane >> 4);  // this thread's rows: row0 + kStride i
  const int h = blockIdx.x >> 1;
  const bool is_v = blockIdx.x & 1;
  const long step = is_v ? p.v_stride : p.k_stride;
  const __nv_bfloat16* const rows = (is_v ? p.v_in : p.k_in) + h * kDim + 8 * l16 + row0 * step;
  uint8_t* const codes = is_v ? p.vc : p.kc;
  float* const scales = is_v ? p.vs : p.ks;
  int turn = 0;  // the half of s_max: an item's reads end before the item after next writes

  auto fetch = [&](const SpanBlock& b, int stage) {
    const __nv_bfloat16* src = rows + (long)b.row * step;
    const uint32_t dst = smem_u32(s_rows + stage * (kRowsPerThread * kSpanThreads) + tid);
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      if (kStride * i >= b.n) break;
      if (row0 + kStride * i < b.n) cp_async16(dst + i * (kSpanThreads * 16), src);
      src += kStride * step;
    }
  };
  auto scale_of = [&](const SpanBlock& b) { return b.had > 0 && in_pool(p, b.phys) ? scales[(size_t)b.phys * p.H + h] : 0.f; };
  auto all_max = [&](uint32_t v) {  // of the CTA; one barrier
    v = __reduce_max_sync(0xffffffffu, v);
    if (lane == 0) s_max[turn][warp] = v;
    __syncthreads();
    const uint4 a = *reinterpret_cast<const uint4*>(s_max[turn]), c = *reinterpret_cast<const uint4*>(s_max[turn] + 4);
    turn ^= 1;
    return max(max(max(a.x, a.y), max(a.z, a.w)), max(max(c.x, c.y), max(c.z, c.w)));
  };
  auto insert = [&](const SpanBlock& b, float old, int stage) {
    const uint4* mine = s_rows + stage * (kRowsPerThread * kSpanThreads) + tid;
    uint4 x[kRowsPerThread];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      if (kStride * i >= b.n) break;
      if (row0 + kStride * i < b.n) {
        x[i] = mine[i * kSpanThreads];
        m = larger(m, x[i]);
      }
    }
    m = all_max(magnitude(m));
    const bool finite = m < kNotFinite;
    if (!finite) {  // again
      m = 0;
#pragma unroll 1
      for (int i = 0; row0 + kStride * i < b.n; ++i) m = larger_finite(m, mine[i * kSpanThreads]);
      m = all_max(m);
    }
    const size_t head = (size_t)b.phys * p.H + h;
    uint8_t* const data = codes + head * (kBlock * kDim);
    int k;
    const float s = block_scale<FMT>(m, b.had > 0, old, k);
    if (k > 0) shrink<FMT>(data, b.had, k, tid, kSpanThreads);
    if (tid == 0) scales[head] = s;
    uint8_t* const dst = data + (b.at + row0) * kDim + 8 * l16;
    if (finite && divides(s)) {
      const float inv = __frcp_rn(s);
#pragma unroll
      for (int i = 0; i < kRowsPerThread; ++i) {
        if (kStride * i >= b.n) break;
        if (row0 + kStride * i < b.n)
          *reinterpret_cast<uint2*>(dst + kStride * i * kDim) = quantize<FMT>(x[i], make_float2(inv, inv), make_float2(-s, -s));
      }
    } else {
#pragma unroll 1
      for (int i = 0; row0 + kStride * i < b.n; ++i)
        *reinterpret_cast<uint2*>(dst + kStride * i * kDim) = quantize_any<FMT>(mine[i * kSpanThreads], s);
    }
  };

  pdl_wait();
  const SpanWalk w = span_walk(p);
  uint32_t i = w.rank;  // this CTA's next block among those of the chunk
  for (int s0 = w.s0; s0 < p.S; s0 += w.step) {
    const uint32_t total = load_chunk(p, chunk, s0, s0 > w.s0);
    const int count = i < total ? (int)((total - 1 - i) / w.size) + 1 : 0;  // this CTA's blocks of the chunk
    SpanBlock b[kInsertStages], some;  // what is on its way, b[0] first; the next ones, one a lane
    auto start = [&](int k, int stage) {  // block k of the CTA's
      if (k < count) {
        if ((k & 31) == 0) some = find_block(p, chunk, s0, (int)min(i + (k + lane) * w.size, total - 1));
        fetch(b[kInsertStages - 1] = from_lane(some, k & 31), stage);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kInsertStages - 1; ++k) {
      start(k, k);
      b[k] = b[kInsertStages - 1];
    }
    float old = count > 0 ? scale_of(b[0]) : 0.f;
    int stage = 0;
#pragma unroll 1
    for (int k = 0; k < count; ++k) {
      start(k + kInsertStages - 1, stage == 0 ? kInsertStages - 1 : stage - 1);
      const float next = k + 1 < count ? scale_of(b[1]) : 0.f;
      cp_async_wait<kInsertStages - 1>();
      if (in_pool(p, b[0].phys)) insert(b[0], old, stage);
      else if (blockIdx.x == 0 && tid == 0) raise_flag(p.status, FLAG_BAD_BLOCK, b[0].phys);
#pragma unroll
      for (int j = 0; j + 1 < kInsertStages; ++j) b[j] = b[j + 1];
      old = next;
      stage = stage + 1 == kInsertStages ? 0 : stage + 1;
    }
    i = i + count * w.size - total;
  }
}

// A warp an item, for spans of a step's few tokens: eight rows at a time, what one round does not
// hold read again for the quotients.
constexpr int kFewCtas = 4;  // CTAs an SM
constexpr int kFewHeld = 4;  // rows a thread holds
// Tokens a span, on average over all of the call's, empty ones too (the lengths are on the device), up to which it
// is used, so that a prompt among many empty spans goes through it: 16,384 tokens in one of 512 spans 24 us, by itself 8.5 (4 heads);
// 2,048 in one of 64 16.3, by itself 3.6.  Spans alike: where the blocks' items are more than the CTAs of the
// other kernel (256 spans of 16 tokens, 8 items each 5.4 us, the other 7.4; of 32 8.3 and 9.1; of 64 19.5 and
// 14.6), and where they are not (32 spans of 8 tokens 3.3 us, the other 3.4; of 16 3.9 and 3.5).
constexpr long kFewTokensMany = 32, kFewTokens = 8;

template <int FMT>
__global__ void __launch_bounds__(kSpanThreads, kFewCtas) block_insert_few_kernel(const SpanParams p) {
  __shared__ SpanChunk chunk;
  constexpr int ROUND = 2 * kFewHeld;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l16 = lane & 15, row0 = lane >> 4;
  const int h = blockIdx.x >> 1;
  const bool is_v = blockIdx.x & 1;
  const long step = is_v ? p.v_stride : p.k_stride;
  const __nv_bfloat16* const rows = (is_v ? p.v_in : p.k_in) + h * kDim + 8 * l16 + row0 * step;
  uint8_t* const codes = is_v ? p.vc : p.kc;
  float* const scales = is_v ? p.vs : p.ks;

  auto load = [&](const __nv_bfloat16* src) { return *reinterpret_cast<const uint4*>(src); };
  auto insert = [&](const SpanBlock& b) {
    const size_t head = (size_t)b.phys * p.H + h;
    uint8_t* const data = codes + head * (kBlock * kDim);
    const __nv_bfloat16* const src = rows + (long)b.row * step;
    const float old = b.had > 0 ? scales[head] : 0.f;
    uint4 x[kFewHeld];
    uint32_t m = 0;
    auto round = [&](int r) {
#pragma unroll
      for (int i = 0; i < kFewHeld; ++i)
        x[i] = r + row0 + 2 * i < b.n ? load(src + (r + 2 * i) * step) : make_uint4(0u, 0u, 0u, 0u);
    };
#pragma unroll 1
    for (int r = 0; r < b.n; r += ROUND) {
      round(r);
#pragma unroll
      for (int i = 0; i < kFewHeld; ++i) m = larger(m, x[i]);
    }
    m = __reduce_max_sync(0xffffffffu, magnitude(m));
    const bool finite = m < kNotFinite;
    if (!finite) {  // again
      m = 0;
#pragma unroll 1
      for (int r = 0; row0 + r < b.n; r += 2) m = larger_finite(m, load(src + r * step));
      m = __reduce_max_sync(0xffffffffu, m);
    }
    int k;
    const float s = block_scale<FMT>(m, b.had > 0, old, k);
    if (k > 0) shrink<FMT>(data, b.had, k, lane, 32);
    __syncwarp();  // every lane has the old scale
    if (lane == 0) scales[head] = s;
    uint8_t* const dst = data + (b.at + row0) * kDim + 8 * l16;
    if (finite && divides(s)) {
      const float inv = __frcp_rn(s);
#pragma unroll 1
      for (int r = 0; r < b.n; r += ROUND) {
        if (b.n > ROUND) round(r);
#pragma unroll
        for (int i = 0; i < kFewHeld; ++i) {
          if (r + 2 * i >= b.n) break;
          const uint2 c = quantize<FMT>(x[i], make_float2(inv, inv), make_float2(-s, -s));
          if (r + row0 + 2 * i < b.n) *reinterpret_cast<uint2*>(dst + (r + 2 * i) * kDim) = c;
        }
      }
    } else {
#pragma unroll 1
      for (int r = 0; row0 + r < b.n; r += 2) *reinterpret_cast<uint2*>(dst + r * kDim) = quantize_any<FMT>(load(src + r * step), s);
    }
  };

  pdl_wait();
  const SpanWalk w = span_walk(p);
  const uint32_t workers = w.size * kSpanWarps;
  uint32_t i = w.rank * kSpanWarps + warp;  // this warp's next block among those of the chunk
  for (int s0 = w.s0; s0 < p.S; s0 += w.step) {
    const uint32_t total = load_chunk(p, chunk, s0, s0 > w.s0);
    const int count = i < total ? (int)((total - 1 - i) / workers) + 1 : 0;
    SpanBlock some;  // the next ones, one a lane
#pragma unroll 1
    for (int k = 0; k < count; ++k) {
      if ((k & 31) == 0) some = find_block(p, chunk, s0, (int)min(i + (uint32_t)(k + lane) * workers, total - 1));
      const SpanBlock b = from_lane(some, k & 31);
      if (in_pool(p, b.phys)) insert(b);
      else if (blockIdx.x == 0 && lane == 0) raise_flag(p.status, FLAG_BAD_BLOCK, b.phys);
    }
    i = i + count * workers - total;
  }
}

// ---------------------------------------------------------------- read

// A half warp takes a row of a cache, a lane its elements [8 l16, 8 l16 + 8): the bits as they
// are stored, then as bf16.
struct Raw {
  uint4 w;
  float s;
};
template <int FMT>
__device__ __forceinline__ Raw load_row(const uint8_t* data, const float* scale, const uint8_t* sf, size_t row, int l16) {
  Raw r;
  if constexpr (FMT == FMT_BF16) {
    r.w = reinterpret_cast<const uint4*>(data + row * 256)[l16];
  } else if constexpr (FMT == FMT_NVFP4) {
    r.w.x = reinterpret_cast<const uint32_t*>(data + row * 64)[l16];
    r.w.y = sf[row * 8 + (l16 >> 1)];
  } else {
    const uint2 w = reinterpret_cast<const uint2*>(data + row * 128)[l16];
    r.w.x = w.x;
    r.w.y = w.y;
    if constexpr (FMT == FMT_FP8) r.s = scale[row];
  }
  return r;
}
// s: the scale of the tensor or of the block
template <int FMT>
__device__ __forceinline__ uint4 row_bf16(const Raw& r, float s, bool nv_round) {
  if constexpr (FMT == FMT_BF16) return r.w;
  float v[8];
  if constexpr (FMT == FMT_NVFP4) {
    const float e = e4m3_to_float((uint8_t)r.w.y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = e2m1x2_to_f16x2((r.w.x >> (8 * i)) & 0xffu);
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[2 * i] = __fmul_rn(x.x, e);
      v[2 * i + 1] = __fmul_rn(x.y, e);
      if (nv_round) {
        const float2 y = e4m3x2_to_float2(pack_e4m3x2(v[2 * i], v[2 * i + 1]));
        v[2 * i] = y.x;
        v[2 * i + 1] = y.y;
      }
    }
  } else {
    if constexpr (FMT == FMT_FP8) s = r.s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = (i < 2 ? r.w.x : r.w.y) >> (16 * (i & 1));
      if constexpr (FMT == FMT_I8B) {
        v[2 * i] = (float)(int8_t)h;
        v[2 * i + 1] = (float)(int8_t)(h >> 8);
      } else {
        const float2 y = e4m3x2_to_float2((uint16_t)h);
        v[2 * i] = y.x;
        v[2 * i + 1] = y.y;
      }
    }
  }
  return make_uint4(pack_bf16x2(__fmul_rn(v[0], s), __fmul_rn(v[1], s)), pack_bf16x2(__fmul_rn(v[2], s), __fmul_rn(v[3], s)),
                    pack_bf16x2(__fmul_rn(v[4], s), __fmul_rn(v[5], s)), pack_bf16x2(__fmul_rn(v[6], s), __fmul_rn(v[7], s)));
}

constexpr int kReadCtas = 4;   // CTAs an SM
constexpr int kReadMost = 64;  // and in all: one after the other, as SMs come free

template <int FMT>
__global__ void __launch_bounds__(kSpanThreads, kReadCtas) cache_read_kernel(const SpanParams p) {
  __shared__ SpanChunk chunk;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l16 = lane & 15;
  const int h = blockIdx.x % p.H;
  const bool is_v = p.k_out == nullptr || (int)blockIdx.x >= p.H;
  const long step = is_v ? p.v_stride : p.k_stride;
  __nv_bfloat16* rows = (is_v ? p.v_out : p.k_out) + h * kDim + 8 * l16;
  const uint8_t* data = is_v ? p.vc : p.kc;
  const uint8_t* sf = is_v ? p.vsf : p.ksf;
  const float* scale = is_v ? p.vs : p.ks;
  const int row0 = 2 * warp + (lane >> 4);  // this thread's rows: row0 + 16 i
  pdl_wait();
  const SpanWalk w = span_walk(p);
  uint32_t i = w.rank;  // this CTA's next block among those of the chunk
  for (int s0 = w.s0; s0 < p.S; s0 += w.step) {
    const uint32_t total = load_chunk(p, chunk, s0, s0 > w.s0);
    for (; i < total; i += w.size) {
      const SpanBlock b = find_block(p, chunk, s0, i);
      if (!in_pool(p, b.phys)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) raise_flag(p.status, FLAG_BAD_BLOCK, b.phys);
        continue;
      }
      const size_t head = (size_t)b.phys * p.H + h, from = head * kBlock + b.at + row0;
      __nv_bfloat16* dst = rows + ((long)b.row + row0) * step;
      Raw x[kRowsPerThread];  // all of them on their way before the first is used
#pragma unroll
      for (int k = 0; k < kRowsPerThread; ++k)
        if (row0 + 16 * k < b.n) x[k] = load_row<FMT>(data, scale, sf, from + 16 * k, l16);
      const float s = FMT == FMT_NVFP4 ? (is_v ? p.vg : p.kg) : FMT == FMT_I8B || FMT == FMT_F8B ? scale[head] : 1.f;
#pragma unroll
      for (int k = 0; k < kRowsPerThread; ++k)
        if (row0 + 16 * k < b.n) __stcs(reinterpret_cast<uint4*>(dst + 16 * k * step), row_bf16<FMT>(x[k], s, p.nv_round));
    }
    i -= total;
  }
}

// Blocks that spans with `tokens` tokens in all touch at most: n tokens min(n, n / 128 + 2).
long most_blocks(const SpanParams& p) {
  const long tokens = p.num_tokens, spans = p.S < p.num_tokens ? p.S : p.num_tokens;
  const long blocks = tokens / kBlock + 2 * spans;
  return blocks < tokens ? blocks : tokens;
}

// CTAs: (heads x K and V, blocks over `each` a CTA), `ctas` in all at most.
dim3 span_grid(const SpanParams& p, int subs, int ctas, int each = 1) {
  const long blocks = (most_blocks(p) + each - 1) / each, cap = ctas > subs ? ctas / subs : 1;
  return dim3((unsigned)subs, (unsigned)(blocks > cap ? cap : blocks));
}

template <int FMT>
cudaError_t launch_insert_fmt(const SpanParams& p, int num_sms, cudaStream_t st) {
  const bool many = most_blocks(p) * 2 * p.H > (long)num_sms * kInsertCtas;
  if (p.num_tokens <= (many ? kFewTokensMany : kFewTokens) * p.S) {
    return launch_behind(block_insert_few_kernel<FMT>, span_grid(p, 2 * p.H, num_sms * kFewCtas, kSpanWarps), dim3(kSpanThreads), 0, st, p);
  }
  const int smem = kInsertStages * kRowsPerThread * kSpanThreads * (int)sizeof(uint4);
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(block_insert_kernel<FMT>), smem, allowed);
  if (e != cudaSuccess) return e;
  return launch_behind(block_insert_kernel<FMT>, span_grid(p, 2 * p.H, num_sms * kInsertCtas), dim3(kSpanThreads), smem, st, p);
}

}  // namespace

cudaError_t launch_block_insert(const SpanParams& p, int fmt, int num_sms, cudaStream_t st) {
  return fmt == FMT_I8B ? launch_insert_fmt<FMT_I8B>(p, num_sms, st) : launch_insert_fmt<FMT_F8B>(p, num_sms, st);
}

cudaError_t launch_cache_read(const SpanParams& p, int fmt, int num_sms, cudaStream_t st) {
  const dim3 grid = span_grid(p, ((p.k_out != nullptr) + (p.v_out != nullptr)) * p.H, num_sms * kReadMost);
  switch (fmt) {
    case FMT_BF16: return launch_behind(cache_read_kernel<FMT_BF16>, grid, dim3(kSpanThreads), 0, st, p);
    case FMT_FP8: return launch_behind(cache_read_kernel<FMT_FP8>, grid, dim3(kSpanThreads), 0, st, p);
    case FMT_NVFP4: return launch_behind(cache_read_kernel<FMT_NVFP4>, grid, dim3(kSpanThreads), 0, st, p);
    case FMT_I8B: return launch_behind(cache_read_kernel<FMT_I8B>, grid, dim3(kSpanThreads), 0, st, p);
    case FMT_F8B: return launch_behind(cache_read_kernel<FMT_F8B>, grid, dim3(kSpanThreads), 0, st, p);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace msa
