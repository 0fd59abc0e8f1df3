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

// One block of one span.
struct SpanBlock {
  int p0, n;     // its first token's position, tokens
  int row;       // the row of that token in the call's tensors
  int phys;      // the block in the pool
  int first;     // the span's first position
};

// Calls f(block, sub) for the items (block touched, sub < subs) that are this CTA's:
// item i of all, in (sequence, block, sub) order, goes to CTA i mod the grid.
template <class F>
__device__ __forceinline__ void walk_spans(const SpanParams& p, int subs, SpanChunk& c, const F& f) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long base = 0;  // items in front of this chunk's
  for (int s0 = 0; s0 < p.S; s0 += kSpanThreads) {
    const int s = s0 + tid;
    int first = 0, end = 0, off = 0, count = 0;
    if (s < p.S) {
      first = __ldg(p.first + s);
      end = __ldg(p.end + s);
      off = __ldg(p.offsets + s);
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
    __syncthreads();  // the former chunk has been read
    if (lane == 31) c.warp_sum[warp] = incl;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kSpanWarps; ++w) {
      const int v = c.warp_sum[w];
      if (w < warp) incl += v;
      total += v;
    }
    c.first[tid] = first;
    c.end[tid] = end;
    c.off[tid] = off;
    c.before[tid] = incl - count;
    __syncthreads();
    const long items = (long)total * subs;
    // the first of this chunk's items that is this CTA's
    long i = ((long)blockIdx.x - base % gridDim.x + gridDim.x) % gridDim.x;
    for (; i < items; i += gridDim.x) {
      const int pair = (int)(i / subs), sub = (int)(i - (long)pair * subs);
      int at = 0;  // the last sequence with no more than `pair` blocks before it: it touches one itself
#pragma unroll
      for (int step = kSpanThreads / 2; step > 0; step >>= 1)
        if (c.before[at + step] <= pair) at += step;
      const int blk = c.first[at] / kBlock + (pair - c.before[at]);
      SpanBlock b;
      b.first = c.first[at];
      b.p0 = max(b.first, blk * kBlock);
      b.n = min(c.end[at], (blk + 1) * kBlock) - b.p0;
      b.row = c.off[at] + (b.p0 - b.first);
      b.phys = __ldg(p.block_table + (size_t)(s0 + at) * p.max_nb + blk);
      if (b.phys < 0 || b.phys >= p.num_blocks) {
        if (sub == 0 && tid == 0) raise_flag(p.status, FLAG_BAD_BLOCK, b.phys);
        continue;
      }
      f(b, sub);
    }
    base += items;
  }
}

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

template <int FMT>
__global__ void __launch_bounds__(kSpanThreads) block_insert_kernel(const SpanParams p) {
  __shared__ SpanChunk chunk;
  __shared__ uint32_t s_max[2][kSpanWarps];
  constexpr float Q = FMT == FMT_I8B ? 127.f : 448.f;
  constexpr float kLeast = 1.17549435e-38f;  // 2^-126
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l16 = lane & 15;
  int turn = 0;  // the half of s_max: an item's reads end before the item after next writes
  walk_spans(p, 2 * p.H, chunk, [&](const SpanBlock& b, int sub) {
    const int h = sub >> 1;
    const bool is_v = sub & 1;
    const __nv_bfloat16* src = (is_v ? p.v_in : p.k_in) + (long)b.row * (is_v ? p.v_stride : p.k_stride) + h * kDim + 8 * l16;
    const long step = is_v ? p.v_stride : p.k_stride;
    const size_t head = (size_t)b.phys * p.H + h;
    uint8_t* data = (is_v ? p.vc : p.kc) + head * (kBlock * kDim);
    float* scale = (is_v ? p.vs : p.ks) + head;
    const int had = max(0, b.first - b.p0 / kBlock * kBlock);
    const float old = had > 0 ? *scale : 0.f;
    // this half warp's rows, and the largest magnitude (as bits: they order as the values do)
    uint4 x[kRowsPerThread];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      const int r = 2 * kSpanWarps * i + 2 * warp + (lane >> 4);
      x[i] = r < b.n ? *reinterpret_cast<const uint4*>(src + r * step) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      const uint32_t w[4] = {x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu, x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu};
      m = __vmaxu2(m, __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3])));
    }
    auto all_max = [&](uint32_t v) {  // of the CTA; one barrier
      v = max(v & 0xffffu, v >> 16);
      v = __reduce_max_sync(0xffffffffu, v);
      if (lane == 0) s_max[turn][warp] = v;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kSpanWarps; ++w) v = max(v, s_max[turn][w]);
      turn ^= 1;
      return v;
    };
    m = all_max(m);
    const bool finite = m < 0x7f80u;
    if (!finite) {  // again, over the finite elements
      uint32_t f = 0;
#pragma unroll
      for (int i = 0; i < kRowsPerThread; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = w[j] & 0x7fffu, hi = (w[j] >> 16) & 0x7fffu;
          f = max(f, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
      }
      m = all_max(f);
    }
    const float need = fmaxf(__fdiv_rn(__uint_as_float(m << 16), Q), kLeast);
    float s = need;
    int k = 0;
    if (had > 0) {
      s = normal_positive(old) ? old : kLeast;
      k = growth(s, need);
      if (k > 0) {
        // (s x 2^k is below 2 need: no overflow; a factor below 2^-126 leaves nothing of a code)
        s = __uint_as_float(__float_as_uint(s) + ((uint32_t)k << 23));
        const float f = pow2i(k < 126 ? -k : -126);
        for (int i = tid; i < had * 8; i += kSpanThreads) {
          uint4 w = *reinterpret_cast<const uint4*>(data + 16 * i);
          w.x = move_codes<FMT>(w.x, f);
          w.y = move_codes<FMT>(w.y, f);
          w.z = move_codes<FMT>(w.z, f);
          w.w = move_codes<FMT>(w.w, f);
          *reinterpret_cast<uint4*>(data + 16 * i) = w;
        }
      }
    }
    if (tid == 0) *scale = s;
    uint8_t* dst = data + (b.p0 % kBlock) * kDim + 8 * l16;
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      const int r = 2 * kSpanWarps * i + 2 * warp + (lane >> 4);
      if (2 * kSpanWarps * i >= b.n) break;
      const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      float2 y[4], z[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = make_float2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u));
      divide(y, s, finite, z);
      uint2 c;
      if (finite) c = make_uint2(block_codes<FMT, false>(z[0], z[1]), block_codes<FMT, false>(z[2], z[3]));
      else c = make_uint2(block_codes<FMT, true>(z[0], z[1]), block_codes<FMT, true>(z[2], z[3]));
      if (r < b.n) *reinterpret_cast<uint2*>(dst + r * kDim) = c;
    }
  });
}

// ---------------------------------------------------------------- read

// Eight elements [8 l16, 8 l16 + 8) of a cache row, as bf16.
template <int FMT>
__device__ __forceinline__ uint4 read_row(const uint8_t* __restrict__ data, const float* __restrict__ scale,
                                          const uint8_t* __restrict__ sf, float g, bool nv_round, size_t row, int l16) {
  if constexpr (FMT == FMT_BF16) return __ldg(reinterpret_cast<const uint4*>(data + row * 256) + l16);
  float v[8];
  float s;
  if constexpr (FMT == FMT_NVFP4) {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(data + row * 64) + l16);
    const float e = e4m3_to_float(__ldg(sf + row * 8 + (l16 >> 1)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = e2m1x2_to_f16x2((w >> (8 * i)) & 0xffu);
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[2 * i] = __fmul_rn(x.x, e);
      v[2 * i + 1] = __fmul_rn(x.y, e);
      if (nv_round) {
        const float2 y = e4m3x2_to_float2(pack_e4m3x2(v[2 * i], v[2 * i + 1]));
        v[2 * i] = y.x;
        v[2 * i + 1] = y.y;
      }
    }
    s = g;
  } else {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(data + row * 128) + l16);
    s = __ldg(scale + (FMT == FMT_FP8 ? row : row / kBlock));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = (i < 2 ? w.x : w.y) >> (16 * (i & 1));
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

template <int FMT>
__global__ void __launch_bounds__(kSpanThreads) cache_read_kernel(const SpanParams p) {
  __shared__ SpanChunk chunk;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l16 = lane & 15;
  const int sides = (p.k_out != nullptr) + (p.v_out != nullptr);
  walk_spans(p, sides * p.H, chunk, [&](const SpanBlock& b, int sub) {
    const int h = sub / sides;
    const bool is_v = p.k_out == nullptr || sub - h * sides == 1;
    const size_t row0 = ((size_t)b.phys * p.H + h) * kBlock + b.p0 % kBlock;
    const long step = is_v ? p.v_stride : p.k_stride;
    __nv_bfloat16* dst = (is_v ? p.v_out : p.k_out) + (long)b.row * step + h * kDim + 8 * l16;
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      const int r = 2 * kSpanWarps * i + 2 * warp + (lane >> 4);
      if (r < b.n)
        *reinterpret_cast<uint4*>(dst + r * step) = read_row<FMT>(is_v ? p.vc : p.kc, is_v ? p.vs : p.ks, is_v ? p.vsf : p.ksf,
                                                                  is_v ? p.vg : p.kg, p.nv_round, row0 + r, l16);
    }
  });
}

// CTAs for the items of spans with `tokens` tokens in all: a span of n tokens touches
// at most min(n, n / 128 + 2) blocks.
unsigned span_grid(const SpanParams& p, int subs, int num_sms, int per_sm) {
  const long tokens = p.num_tokens, spans = p.S < p.num_tokens ? p.S : p.num_tokens;
  long blocks = tokens / kBlock + 2 * spans;
  if (blocks > tokens) blocks = tokens;
  long grid = blocks * subs;
  const long cap = (long)num_sms * per_sm;
  if (grid > cap) grid = cap;
  return (unsigned)(grid < 1 ? 1 : grid);
}

}  // namespace

cudaError_t launch_block_insert(const SpanParams& p, int fmt, int num_sms, cudaStream_t st) {
  const unsigned grid = span_grid(p, 2 * p.H, num_sms, 4);
  if (fmt == FMT_I8B) block_insert_kernel<FMT_I8B><<<grid, kSpanThreads, 0, st>>>(p);
  else block_insert_kernel<FMT_F8B><<<grid, kSpanThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const SpanParams& p, int fmt, int num_sms, cudaStream_t st) {
  const unsigned grid = span_grid(p, ((p.k_out != nullptr) + (p.v_out != nullptr)) * p.H, num_sms, 8);
  switch (fmt) {
    case FMT_BF16: cache_read_kernel<FMT_BF16><<<grid, kSpanThreads, 0, st>>>(p); break;
    case FMT_FP8: cache_read_kernel<FMT_FP8><<<grid, kSpanThreads, 0, st>>>(p); break;
    case FMT_NVFP4: cache_read_kernel<FMT_NVFP4><<<grid, kSpanThreads, 0, st>>>(p); break;
    case FMT_I8B: cache_read_kernel<FMT_I8B><<<grid, kSpanThreads, 0, st>>>(p); break;
    case FMT_F8B: cache_read_kernel<FMT_F8B><<<grid, kSpanThreads, 0, st>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace msa
