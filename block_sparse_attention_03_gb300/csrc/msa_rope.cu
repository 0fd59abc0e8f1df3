// Rotary insert: the per-head RMS norm and rotary positions of q, k, the index
// queries and the index key, and the insert of k, v and the index key into the
// paged caches, in one pass over the projection's output (model page,
// MiniMaxM3SparseAttention: per-head norm and partial rotary positions before
// the caches are written; vLLM Day-0 blog, section "QKV GEMM + norm + RoPE + KV
// 插入融合").
//
//   y = x * rsqrt(mean x^2 + eps) * (offset + w)          (optional, per head)
//   pair i of a row, at the position p of its axis: angle = 2 pi p turns_i,
//   (a, b) -> (a cos - b sin, a sin + b cos)
// in fp32, rounded once where it is stored: a bf16 or e4m3 query, or the cache's
// format by msa_cache_insert's rules.
//
// The angle's fraction of a turn is the top half of p x turns_i mod 2^64
// (turns_i: turns a position x 2^64), exact for any 32-bit position to 2^-32 of
// a turn, with no table of cosines to read and no largest position.
//
// Bound: HBM (a token's rows are read once and written once).  Half a warp takes
// a row, 16 bytes a lane; a warp takes one token and, for many tokens, all of its
// rows, so that its 64 sines and cosines (two a lane, exchanged through shared
// memory) are used for every head; with few tokens its rows are spread over
// several warps, which compute them again.
#include "msa_device.cuh"
#include "msa_internal.h"

namespace msa {

namespace {

constexpr int kRopeWarps = 4;
constexpr int kBatch = 4;  // row pairs a warp has in flight

// e2m1 codes of (lo, hi), round to nearest even, saturating at +-6, +0 for zero magnitudes.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{ .reg .b8 t; cvt.rn.satfinite.e2m1x2.f32 t, %1, %2; cvt.u32.u8 %0, t; }" : "=r"(r) : "f"(hi), "f"(lo));
  if ((r & 0x7u) == 0u) r &= 0xF0u;
  if ((r & 0x70u) == 0u) r &= 0x0Fu;
  return r;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return (uint32_t)pack_e4m3x2(a, b) | ((uint32_t)pack_e4m3x2(c, d) << 16);
}

// What a row is.
enum Kind : int { KIND_Q = 0, KIND_IQ = 1, KIND_K = 2, KIND_IK = 3, KIND_V = 4, KIND_NONE = 5 };

struct Row {
  int kind, head;
};
// rows of a token in the order q, index q, k, v, index k
__device__ __forceinline__ Row row_of(const RopeParams& p, int r) {
  if (r < p.Hq) return {KIND_Q, r};
  r -= p.Hq;
  if (r < p.Giq) return {KIND_IQ, r};
  r -= p.Giq;
  if (r < p.H) return {KIND_K, r};
  r -= p.H;
  if (r < p.H) return {KIND_V, r};
  r -= p.H;
  if (r < p.Gik) return {KIND_IK, 0};
  return {KIND_NONE, 0};
}

__device__ __forceinline__ const __nv_bfloat16* row_src(const RopeParams& p, long t, Row w) {
  switch (w.kind) {
    case KIND_Q: return p.q + t * p.q_stride + w.head * kDim;
    case KIND_IQ: return p.iq + t * p.iq_stride + w.head * kDim;
    case KIND_K: return p.k + t * p.k_stride + w.head * kDim;
    case KIND_V: return p.v + t * p.v_stride + w.head * kDim;
    default: return p.ik + t * p.ik_stride;
  }
}

// One cache row of 16 lanes x 8 elements (every lane of the warp takes part in
// the shuffles; `put` says whether this half stores).
template <int FMT>
__device__ __forceinline__ void put_row(const float (&y)[8], bool put, uint8_t* __restrict__ data,
                                        float* __restrict__ scale, uint8_t* __restrict__ sf, float g, long row, int l16) {
  if constexpr (FMT == FMT_BF16) {
    if (!put) return;
    uint4 w;
    w.x = pack_bf16x2(y[0], y[1]);
    w.y = pack_bf16x2(y[2], y[3]);
    w.z = pack_bf16x2(y[4], y[5]);
    w.w = pack_bf16x2(y[6], y[7]);
    *reinterpret_cast<uint4*>(data + row * 256 + 16 * l16) = w;
    return;
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
  if constexpr (FMT == FMT_FP8) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (!put) return;
    const float s = m > 0.f ? __fdiv_rn(m, 448.f) : 1.f;
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = __fdiv_rn(y[i], s);
    uint2 w;
    w.x = e4m3x4(z[0], z[1], z[2], z[3]);
    w.y = e4m3x4(z[4], z[5], z[6], z[7]);
    *reinterpret_cast<uint2*>(data + row * 128 + 8 * l16) = w;
    if (l16 == 0) scale[row] = s;
  } else {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));  // 16 elements: two lanes
    if (!put) return;
    const uint32_t code = pack_e4m3x2(__fdiv_rn(m, __fmul_rn(6.f, g)), 0.f) & 0xffu;
    const float den = __fmul_rn(e4m3_to_float((uint8_t)code), g);
    uint32_t w = 0;
    if (den > 0.f) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w |= e2m1x2(__fdiv_rn(y[2 * i], den), __fdiv_rn(y[2 * i + 1], den)) << (8 * i);
    }
    *reinterpret_cast<uint32_t*>(data + row * 64 + 4 * l16) = w;
    if ((l16 & 1) == 0) sf[row * 8 + (l16 >> 1)] = (uint8_t)code;
  }
}

template <int KVF, int IF>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ uint64_t s_turns[64];
  __shared__ int s_axis[64];
  __shared__ float2 s_cs[kRopeWarps][64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l16 = lane & 15, half = lane >> 4;
  const int pairs = p.rope.rotary_dim >> 1;
  if (threadIdx.x < 64) {
    s_turns[threadIdx.x] = p.rope.turns[threadIdx.x];
    s_axis[threadIdx.x] = p.rope.axis[threadIdx.x];
  }
  __syncthreads();
  const int rows = p.Hq + p.Giq + 2 * p.H + p.Gik;
  const int row_pairs = (rows + 1) >> 1;
  const int per = (row_pairs + p.chunks - 1) / p.chunks;  // row pairs a warp takes
  const long items = (long)p.num_tokens * p.chunks;
  const bool adjacent = p.rope.layout == MSA_ROPE_ADJACENT;
  // this lane's 8 dims: the pairs they belong to, and whether they are the second of them
  const int d0 = 8 * l16;
  const bool rot = d0 < 2 * pairs;
  const int shift = pairs >> 3;  // lanes between the halves of a pair ("halves" layout)
  const bool second = d0 >= pairs;
  const int partner = (lane & 16) | ((second ? l16 - shift : l16 + shift) & 15);
#pragma unroll 1
  for (long it = (long)blockIdx.x * kRopeWarps + warp; it < items; it += (long)gridDim.x * kRopeWarps) {
    const long t = it / p.chunks;
    const int ch = (int)(it - t * p.chunks);
    const int pr0 = ch * per, pr1 = min(row_pairs, pr0 + per);
    const int slot = __ldg(p.slots + t);
    // cosines and sines of this token: pairs lane, lane + 32
    __syncwarp();
#pragma unroll
    for (int i = lane; i < 64; i += 32) {
      if (i < pairs) {
        const int pos = __ldg(p.positions + (size_t)s_axis[i] * p.num_tokens + t);
        const uint64_t f = (uint64_t)(int64_t)pos * s_turns[i];
        float sn, cs;
        sincospif((float)(int32_t)(f >> 32) * 4.656612873077393e-10f, &sn, &cs);  // x 2^-31: half turns
        s_cs[warp][i] = make_float2(cs, sn);
      }
    }
    __syncwarp();
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float2 v = make_float2(1.f, 0.f);
      if (rot) {
        const int dim = d0 + i;
        const int pair = adjacent ? dim >> 1 : (second ? dim - pairs : dim);
        v = s_cs[warp][pair];
        // out = own x cos + partner x sin, the first of a pair taking -sin
        if (adjacent ? (i & 1) == 0 : !second) v.y = -v.y;
      }
      c[i] = v.x;
      s[i] = v.y;
    }
    const bool live = slot >= 0;
    const int blk = slot >> 7, off = slot & 127;
    if (live && blk >= p.num_blocks && ch == 0 && lane == 0) raise_flag(p.status, FLAG_BAD_BLOCK, slot);
    const bool store = live && blk < p.num_blocks;
#pragma unroll 1
    for (int pr = pr0; pr < pr1; pr += kBatch) {
      uint4 raw[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int r = 2 * (pr + b) + half;
        raw[b] = make_uint4(0u, 0u, 0u, 0u);
        if (pr + b < pr1 && r < rows)
          raw[b] = *reinterpret_cast<const uint4*>(row_src(p, t, row_of(p, r)) + d0);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (pr + b >= pr1) break;
        const int r = 2 * (pr + b) + half;
        const Row w = r < rows ? row_of(p, r) : Row{KIND_NONE, 0};
        const uint32_t u[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[2 * i] = __uint_as_float(u[i] << 16);
          y[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
        const bool turns = w.kind <= KIND_IK;
        if (p.norm) {
          float q = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) q = fmaf(y[i], y[i], q);
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
          const __nv_bfloat16* wp = turns ? p.w[w.kind] : nullptr;
          if (wp) {
            const float inv = rsqrtf(fmaf(q, 1.f / kDim, p.eps));
            const uint4 ww = __ldg(reinterpret_cast<const uint4*>(wp + d0));
            const uint32_t g[4] = {ww.x, ww.y, ww.z, ww.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              y[2 * i] = y[2 * i] * inv * (__uint_as_float(g[i] << 16) + p.w_offset);
              y[2 * i + 1] = y[2 * i + 1] * inv * (__uint_as_float(g[i] & 0xffff0000u) + p.w_offset);
            }
          }
        }
        if (adjacent) {
          if (turns && rot) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const float a = y[i], d = y[i + 1];
              y[i] = fmaf(a, c[i], d * s[i]);
              y[i + 1] = fmaf(d, c[i + 1], a * s[i + 1]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float o = __shfl_sync(0xffffffffu, y[i], partner);
            if (turns && rot) y[i] = fmaf(y[i], c[i], o * s[i]);
          }
        }
        // ---- out
        const bool query = w.kind <= KIND_IQ;
        if (query) {
          const int heads = w.kind == KIND_Q ? p.Hq : p.Giq;
          uint8_t* out = w.kind == KIND_Q ? p.q_out : p.iq_out;
          const bool fp8 = (w.kind == KIND_Q ? p.q_fp8 : p.iq_fp8) != 0;
          const size_t e = ((size_t)t * heads + w.head) * kDim + d0;
          if (fp8) {
            const float iv = w.kind == KIND_Q ? p.q_inv : p.iq_inv;
            uint2 o;
            o.x = e4m3x4(y[0] * iv, y[1] * iv, y[2] * iv, y[3] * iv);
            o.y = e4m3x4(y[4] * iv, y[5] * iv, y[6] * iv, y[7] * iv);
            *reinterpret_cast<uint2*>(out + e) = o;
          } else {
            uint4 o;
            o.x = pack_bf16x2(y[0], y[1]);
            o.y = pack_bf16x2(y[2], y[3]);
            o.z = pack_bf16x2(y[4], y[5]);
            o.w = pack_bf16x2(y[6], y[7]);
            *reinterpret_cast<uint4*>(out + 2 * e) = o;
          }
        }
        const bool kv = w.kind == KIND_K || w.kind == KIND_V, ik = w.kind == KIND_IK;
        if (__any_sync(0xffffffffu, kv)) {
          const long row = ((long)blk * p.H + w.head) * kBlock + off;
          const bool isk = w.kind == KIND_K;
          put_row<KVF>(y, kv && store, isk ? p.kc : p.vc, isk ? p.ks : p.vs, isk ? p.ksf : p.vsf, isk ? p.kg : p.vg, row,
                       l16);
        }
        if (__any_sync(0xffffffffu, ik))
          put_row<IF>(y, ik && store, p.ic, p.is, p.isf, p.ig, (long)blk * kBlock + off, l16);
      }
    }
  }
}

template <int KVF>
cudaError_t launch_kv(const RopeParams& p, unsigned grid, cudaStream_t st) {
  switch (p.idx_fmt) {
    case FMT_BF16: rope_kernel<KVF, FMT_BF16><<<grid, 32 * kRopeWarps, 0, st>>>(p); break;
    case FMT_FP8: rope_kernel<KVF, FMT_FP8><<<grid, 32 * kRopeWarps, 0, st>>>(p); break;
    case FMT_NVFP4: rope_kernel<KVF, FMT_NVFP4><<<grid, 32 * kRopeWarps, 0, st>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(RopeParams p, int num_sms, cudaStream_t st) {
  // one warp a token where that fills the GPU (32 warps an SM); with fewer
  // tokens a token's rows go to as many warps as there are row pairs at most
  const int row_pairs = (p.Hq + p.Giq + 2 * p.H + p.Gik + 1) / 2;
  long chunks = ((long)num_sms * 32 + p.num_tokens - 1) / p.num_tokens;
  if (chunks > row_pairs) chunks = row_pairs;
  if (chunks < 1) chunks = 1;
  p.chunks = (int)chunks;
  const long items = (long)p.num_tokens * chunks;
  long grid = (items + kRopeWarps - 1) / kRopeWarps;
  const long cap = (long)num_sms * 64;
  if (grid > cap) grid = cap;
  switch (p.kv_fmt) {
    case FMT_BF16: return launch_kv<FMT_BF16>(p, (unsigned)grid, st);
    case FMT_FP8: return launch_kv<FMT_FP8>(p, (unsigned)grid, st);
    case FMT_NVFP4: return launch_kv<FMT_NVFP4>(p, (unsigned)grid, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace msa
