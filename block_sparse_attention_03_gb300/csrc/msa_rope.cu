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
// (turns_i: turns a position x 2^64), with no table of cosines to read and no largest
// position.  The product is exact for any 32-bit position; the fraction is then
// rounded to fp32 (2^-25 of half a turn), and turns_i, made from a double, is off by
// 2^-56 of a turn at most (2^-24 of half a turn at the farthest position).
//
// Bound: latency.  A token's rows are read once and written once, but neither the
// DRAM (33 to 38% of its peak cycles) nor the issue slots (59 to 66%: 257 instructions for
// the 16 elements a lane has of four rows) are full: the 24 warps an SM that 80
// registers allow have one quad each on its way, 24 KB an SM where the copy rate at some 800 ns
// needs 36, and wait for shuffles and shared memory in between.  (80 registers
// spill: up to 48 bytes a thread for halves, none for adjacent pairs.)  Measured (one GPU, launches back to back, of 6,779
// GB/s): 8,192 tokens into FP8 29.6 us (56%), 16,384 into BF16 51.6 us (70%), NVFP4
// 56.4 us (56%), adjacent pairs 55.9 and 58.5 us, 24,571 into NVFP4 with three axes
// and e4m3 queries 78 us (50%), 32 tokens 4.4 us.  A quarter of
// a warp takes a row, 16 elements a lane, chosen so that both elements of a pair
// are in one lane (eight at i and eight at i + rotary_dim / 2; no exchange between
// lanes); a warp takes four heads of one kind at a time, so that what a row is is
// a uniform branch and finding it, its loads, sums and stores are shared by
// many elements; fp32 operations go two at a time (f32x2).  What the loop needs to
// know of a row comes from a table that the CTA writes once (code of its own for
// each kind in place of the table: 32.7 us for the 8,192 tokens, the larger loop's
// instruction fetches).
//
// Split: the quads of rows of all tokens, in order, are cut into equal runs, one
// per warp of a grid that fills the GPU: a prompt leaves no uneven last wave, and
// a decode step's few tokens still spread over as many warps as they have quads.
// A warp computes a token's 64 sines and cosines (two a lane, exchanged through
// shared memory) once for all its quads of that token.
//
// The formats' rules divide by the row's (or group's) scale.  The quotient is
// formed by Markstein's method (Computation of elementary functions on the IBM
// RISC System/6000, 1990): with y = RN(1/s), q = RN(x y), r = RN(x - q s) exact,
// RN(q + r y) is the correctly rounded quotient, so the codes are those of an
// IEEE division at three operations an element; scales near the ends of fp32's
// range, where r could underflow or y overflow, and elements whose quotient is
// infinite take the division itself.
#include "msa_device.cuh"
#include "msa_internal.h"

namespace msa {

namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeCtas = 3;  // CTAs an SM (registers)

// e2m1 codes of (lo, hi), round to nearest even, saturating at +-6, +0 for zero magnitudes.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{ .reg .b8 t; cvt.rn.satfinite.e2m1x2.f32 t, %1, %2; cvt.u32.u8 %0, t; }" : "=r"(r) : "f"(hi), "f"(lo));
  if ((r & 0x7u) == 0u) r &= 0xF0u;
  if ((r & 0x70u) == 0u) r &= 0x0Fu;
  return r;
}

__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b) {
  return (uint32_t)pack_e4m3x2(a.x, a.y) | ((uint32_t)pack_e4m3x2(b.x, b.y) << 16);
}

// fma2 rounded down: a sum that is zero is -0.
__device__ __forceinline__ float2 fma2_down(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{ .reg .b64 x, y, z, w; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7}; fma.rm.f32x2 w, x, y, z; "
      "mov.b64 {%0, %1}, w; }"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// y[i] / s, correctly rounded (see above).  fits: no quotient is infinite (its
// remainder would be NaN).
// The sign of a zero is kept: the remainder is exact, and as -0 where it is zero it
// leaves q = -0 alone.
template <int N>
__device__ __forceinline__ void divide(const float2 (&y)[N], float s, bool fits, float2 (&z)[N]) {
  if (s >= 8.27e-25f && s <= 1.2e24f && fits) {  // 2^-80 to 2^80
    const float r = __frcp_rn(s);
    const float2 r2 = make_float2(r, r), n2 = make_float2(-s, -s);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 q = mul2(y[i], r2);
      z[i] = fma2(fma2_down(q, n2, y[i]), r2, q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = make_float2(__fdiv_rn(y[i].x, s), __fdiv_rn(y[i].y, s));
  }
}

// What a row is.
enum Kind : int { KIND_Q = 0, KIND_IQ = 1, KIND_K = 2, KIND_IK = 3, KIND_V = 4 };

// What the loop needs to know of a row (of one head of one kind).
struct __align__(16) RowDesc {
  const uint8_t* src;   // token 0
  long src_step;        // bytes between tokens
  uint8_t* out;         // queries: token 0 of the output; caches: the data (null: no such head)
  int out_step;         // queries: bytes between tokens; caches: the head's first row
  int kind;             // of all rows of a quad
};

__device__ __forceinline__ uint4 bf16x8(const float2* y) {
  return make_uint4(pack_bf16x2(y[0].x, y[0].y), pack_bf16x2(y[1].x, y[1].y), pack_bf16x2(y[2].x, y[2].y),
                    pack_bf16x2(y[3].x, y[3].y));
}
// the same of elements that are bf16 values: their bits (the rounding has one NaN only)
__device__ __forceinline__ uint4 bf16x8_bits(const float2* y) {
  auto top = [](float2 v) { return __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632); };
  return make_uint4(top(y[0]), top(y[1]), top(y[2]), top(y[3]));
}
__device__ __forceinline__ uint2 e4m3x8(const float2* y) { return make_uint2(e4m3x4(y[0], y[1]), e4m3x4(y[2], y[3])); }
__device__ __forceinline__ float amax8(const float2* y) {
  return fmaxf(fmaxf(fmaxf(fabsf(y[0].x), fabsf(y[0].y)), fmaxf(fabsf(y[1].x), fabsf(y[1].y))),
               fmaxf(fmaxf(fabsf(y[2].x), fabsf(y[2].y)), fmaxf(fabsf(y[3].x), fabsf(y[3].y))));
}

// One cache row of 8 lanes, elements [dA, dA + 8) (y[0..3]) and [dB, dB + 8) a lane
// (every lane of the warp takes part in the exchanges; `put`: this row is stored;
// `raw`: as it came).
template <int FMT>
__device__ __forceinline__ void put_row(const float2 (&y)[8], int dA, int dB, bool put, bool raw,
                                        uint8_t* __restrict__ data, float* __restrict__ scale, uint8_t* __restrict__ sf, float g, long row,
                                        float* chunk_max, int l8) {
  if constexpr (FMT == FMT_BF16) {
    if (put) {
      *reinterpret_cast<uint4*>(data + row * 256 + 2 * dA) = raw ? bf16x8_bits(y) : bf16x8(y);
      *reinterpret_cast<uint4*>(data + row * 256 + 2 * dB) = raw ? bf16x8_bits(y + 4) : bf16x8(y + 4);
    }
    return;
  }
  const float ma = amax8(y), mb = amax8(y + 4);
  if constexpr (FMT == FMT_FP8) {
    float m = fmaxf(ma, mb);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (!put) return;
    const float s = m > 0.f ? __fdiv_rn(m, 448.f) : 1.f;
    float2 z[8];
    divide(y, s, true, z);  // s follows the row's maximum: 448 at most, or s is infinite
    *reinterpret_cast<uint2*>(data + row * 128 + dA) = e4m3x8(z);
    *reinterpret_cast<uint2*>(data + row * 128 + dB) = e4m3x8(z + 4);
    if (l8 == 0) scale[row] = s;
  } else {
    // the largest of each 16-element group, from those of its two 8-element chunks
    // (in the row's order in shared memory; a group may lie in two halves)
    chunk_max[dA >> 3] = ma;
    chunk_max[dB >> 3] = mb;
    __syncwarp();
    const float2 a2 = *reinterpret_cast<const float2*>(chunk_max + (dA >> 4) * 2);
    const float2 b2 = *reinterpret_cast<const float2*>(chunk_max + (dB >> 4) * 2);
    __syncwarp();
    if (!put) return;
    const float g6 = __fmul_rn(6.f, g);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float m = k ? fmaxf(b2.x, b2.y) : fmaxf(a2.x, a2.y);
      const int d = k ? dB : dA;
      const uint32_t code = pack_e4m3x2(__fdiv_rn(m, g6), 0.f) & 0xffu;
      const float den = __fmul_rn(e4m3_to_float((uint8_t)code), g);
      uint32_t w = 0;
      if (den > 0.f) {
        const float2 v[4] = {y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]};
        float2 z[4];
        divide(v, den, m * __frcp_rn(den) <= 3.0e38f, z);  // the group's scale saturates
#pragma unroll
        for (int i = 0; i < 4; ++i) w |= e2m1x2(z[i].x, z[i].y) << (8 * i);
      }
      *reinterpret_cast<uint32_t*>(data + row * 64 + (d >> 1)) = w;
      if ((d & 8) == 0) sf[row * 8 + (d >> 4)] = (uint8_t)code;
    }
  }
}

template <int KVF, int IF, bool ADJ>
__global__ void __launch_bounds__(32 * kRopeWarps, kRopeCtas) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ RowDesc s_rows[];  // four a quad
  __shared__ uint64_t s_turns[64];
  __shared__ __align__(16) float s_w[4][kDim];           // offset + norm weight
  __shared__ __align__(16) float2 s_cs[kRopeWarps][64];  // cosines, sines
  __shared__ __align__(16) float s_max[kRopeWarps][4][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l8 = lane & 7, sub = lane >> 3;
  const int pairs = p.rope.rotary_dim >> 1;
  // quads of rows, kind after kind: where each ends
  const int e0 = (p.Hq + 3) >> 2, e1 = e0 + ((p.Giq + 3) >> 2), e2 = e1 + ((p.H + 3) >> 2), e3 = e2 + ((p.H + 3) >> 2),
            e4 = e3 + p.Gik;
  auto describe = [&](int r) {
    const int qd = r >> 2;
    RowDesc d;
    const int h = r - 4 * (qd < e0 ? 0 : qd < e1 ? e0 : qd < e2 ? e1 : qd < e3 ? e2 : e3);
    int heads = p.H;
    const __nv_bfloat16* src;
    long step;
    d.out = nullptr;
    if (qd < e1) {
      const bool q = qd < e0;
      d.kind = q ? KIND_Q : KIND_IQ;
      heads = q ? p.Hq : p.Giq;
      src = q ? p.q : p.iq;
      step = q ? p.q_stride : p.iq_stride;
      const int es = (q ? p.q_fp8 : p.iq_fp8) ? 1 : 2;
      if (h < heads) d.out = (q ? p.q_out : p.iq_out) + (size_t)h * kDim * es;
      d.out_step = heads * kDim * es;
    } else {
      d.kind = qd < e2 ? KIND_K : qd < e3 ? KIND_V : KIND_IK;
      if (qd >= e3) heads = 1;
      src = qd < e2 ? p.k : qd < e3 ? p.v : p.ik;
      step = qd < e2 ? p.k_stride : qd < e3 ? p.v_stride : p.ik_stride;
      if (h < heads) d.out = qd < e2 ? p.kc : qd < e3 ? p.vc : p.ic;
      d.out_step = h * kBlock;
    }
    // (a quarter without a head reads the last one's row again)
    d.src = reinterpret_cast<const uint8_t*>(src + (long)min(h, heads - 1) * kDim);
    d.src_step = 2 * step;
    return d;
  };
  // this lane's elements [dA, dA + 8) and [dB, dB + 8)
  int dA, dB;
  bool rot;
  if constexpr (ADJ) {
    dA = 16 * l8;
    dB = dA + 8;
    rot = dA < 2 * pairs;
  } else {
    const int rl = pairs >> 3;  // lanes that hold pairs; the others the rest of the row
    rot = l8 < rl;
    dA = rot ? 8 * l8 : 2 * pairs + 8 * (l8 - rl);
    dB = rot ? pairs + 8 * l8 : kDim / 2 + pairs + 8 * (l8 - rl);
  }

  // this warp's run of quads, [u, u1) of num_tokens x e4
  const long quads = (long)p.num_tokens * e4, warps = (long)gridDim.x * kRopeWarps;
  const long w = (long)blockIdx.x * kRopeWarps + warp;
  // (w quads / warps, in parts that keep the divisions to 32 bits where the total is)
  const bool small = (quads >> 32) == 0;
  const long each = small ? (long)((uint32_t)quads / (uint32_t)warps) : quads / warps;
  const uint32_t rest = (uint32_t)(quads - each * warps);  // warps are at most some thousands
  const long u0 = w * each + (uint32_t)w * rest / (uint32_t)warps;
  const long u1 = (w + 1) * each + (uint32_t)(w + 1) * rest / (uint32_t)warps;
  int t = small ? (int)((uint32_t)u0 / (uint32_t)e4) : (int)(u0 / e4);
  int qd = (int)(u0 - (long)t * e4);
  int left = (int)(u1 - u0);

  // The first reads, of memory, and then what the CTA keeps of the heads and weights.
  int axis[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) axis[k] = (p.axis_bits[0][k] >> lane & 1) | (p.axis_bits[1][k] >> lane & 1) << 1;
  // the slot and positions of a token, and the raw elements of a quad's rows, are
  // read one ahead
  int slot_n = -1, pos_n[2] = {0, 0};
  auto fetch = [&](int tt) {
    slot_n = __ldg(p.slots + tt);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (lane + 32 * k < pairs) pos_n[k] = __ldg(p.positions + (size_t)axis[k] * p.num_tokens + tt);
  };
  uint4 a1, b1;
  auto load = [&](int tt, const RowDesc& d) {
    const uint8_t* src = d.src + tt * d.src_step;
    a1 = *reinterpret_cast<const uint4*>(src + 2 * dA);
    b1 = *reinterpret_cast<const uint4*>(src + 2 * dB);
  };
  if (left > 0) fetch(t);
  if (threadIdx.x < 64) s_turns[threadIdx.x] = p.rope.turns[threadIdx.x];
  for (int i = threadIdx.x; i < 4 * kDim; i += 32 * kRopeWarps) {
    const __nv_bfloat16* w = p.w[i / kDim];
    s_w[i / kDim][i % kDim] = w ? __bfloat162float(w[i % kDim]) + p.w_offset : 1.f;
  }
  for (int r = threadIdx.x; r < 4 * e4; r += 32 * kRopeWarps) s_rows[r] = describe(r);
  __syncthreads();
  if (left > 0) load(t, s_rows[4 * qd + sub]);
#pragma unroll 1
  while (left > 0) {
    const int slot = slot_n;
    // cosines and sines of this token: pairs lane, lane + 32
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = lane + 32 * k;
      if (i < pairs) {
        const uint64_t f = (uint64_t)(int64_t)pos_n[k] * s_turns[i];
        float sn, cs;
        sincospif((float)(int32_t)(f >> 32) * 4.656612873077393e-10f, &sn, &cs);  // x 2^-31: half turns
        s_cs[warp][i] = make_float2(cs, sn);
      }
    }
    __syncwarp();
    if (left > e4 - qd) fetch(t + 1);
    // halves: pair dA + i for element i of both parts; adjacent: each pair's sine and cosine
    float2 c[4], s[4], cb[ADJ ? 4 : 1], sb[ADJ ? 4 : 1];
    if (rot) {
      const int first = ADJ ? dA >> 1 : dA;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(&s_cs[warp][first + 2 * i]);
        if constexpr (ADJ) {
          // pairs first + 2i and first + 2i + 1: out = own x cos + other x (-sin, sin)
          float2* cc = i < 2 ? c + 2 * i : cb + 2 * (i - 2);
          float2* ss = i < 2 ? s + 2 * i : sb + 2 * (i - 2);
          cc[0] = make_float2(v.x, v.x);
          ss[0] = make_float2(-v.y, v.y);
          cc[1] = make_float2(v.z, v.z);
          ss[1] = make_float2(-v.w, v.w);
        } else {
          c[i] = make_float2(v.x, v.z);
          s[i] = make_float2(v.y, v.w);
        }
      }
    }
    const bool live = slot >= 0;
    const int blk = slot >> 7, off = slot & 127;
    if (live && blk >= p.num_blocks && qd == 0 && lane == 0) raise_flag(p.status, FLAG_BAD_BLOCK, slot);
    const bool store = live && blk < p.num_blocks;
    const long row0 = (long)blk * p.H * kBlock + off;

    const int end = min(e4, qd + left);
    left -= end - qd;
#pragma unroll 1
    for (; qd < end; ++qd) {
      const uint32_t u[8] = {a1.x, a1.y, a1.z, a1.w, b1.x, b1.y, b1.z, b1.w};
      if (qd + 1 < end) load(t, s_rows[4 * (qd + 1) + sub]);
      else if (left > 0) load(t + 1, s_rows[sub]);
      const RowDesc& d = s_rows[4 * qd + sub];
      const int kind = d.kind;  // the same in all rows of the quad
      uint8_t* const out = d.out;
      float2 y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
      if (kind != KIND_V) {
        if (p.w[kind]) {
          float2 q2 = mul2(y[0], y[0]), q3 = mul2(y[4], y[4]);
#pragma unroll
          for (int i = 1; i < 4; ++i) {
            q2 = fma2(y[i], y[i], q2);
            q3 = fma2(y[4 + i], y[4 + i], q3);
          }
          q2 = add2(q2, q3);
          float q = q2.x + q2.y;
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
          const float inv = rsqrtf(fmaf(q, 1.f / kDim, p.eps));
          const float2 i2 = make_float2(inv, inv);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 g = *reinterpret_cast<const float4*>(&s_w[kind][(i < 2 ? dA : dB - 8) + 4 * i]);
            y[2 * i] = mul2(mul2(y[2 * i], i2), make_float2(g.x, g.y));
            y[2 * i + 1] = mul2(mul2(y[2 * i + 1], i2), make_float2(g.z, g.w));
          }
        }
        if (rot) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 a = y[i], b = y[4 + i];
            if constexpr (ADJ) {
              y[i] = fma2(a, c[i], mul2(make_float2(a.y, a.x), s[i]));
              y[4 + i] = fma2(b, cb[i], mul2(make_float2(b.y, b.x), sb[i]));
            } else {
              y[i] = fma2(a, c[i], mul2(b, make_float2(-s[i].x, -s[i].y)));
              y[4 + i] = fma2(b, c[i], mul2(a, s[i]));
            }
          }
        }
      }
      if (kind <= KIND_IQ) {
        uint8_t* const o = out + (long)t * d.out_step;
        if (kind == KIND_Q ? p.q_fp8 : p.iq_fp8) {
          const float iv = kind == KIND_Q ? p.q_inv : p.iq_inv;
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = mul2(y[i], make_float2(iv, iv));
          if (out) {
            *reinterpret_cast<uint2*>(o + dA) = e4m3x8(y);
            *reinterpret_cast<uint2*>(o + dB) = e4m3x8(y + 4);
          }
        } else if (out) {
          *reinterpret_cast<uint4*>(o + 2 * dA) = bf16x8(y);
          *reinterpret_cast<uint4*>(o + 2 * dB) = bf16x8(y + 4);
        }
      } else if (kind == KIND_IK) {
        put_row<IF>(y, dA, dB, store && out, false, out, p.is, p.isf, p.ig, (long)blk * kBlock + off, s_max[warp][sub], l8);
      } else {
        const bool isk = kind == KIND_K;
        put_row<KVF>(y, dA, dB, store && out, !isk, out, isk ? p.ks : p.vs, isk ? p.ksf : p.vsf, isk ? p.kg : p.vg, row0 + d.out_step,
                     s_max[warp][sub], l8);
      }
    }
    qd = 0;
    ++t;
  }
}

int rope_quads(const RopeParams& p) {
  return (p.Hq + 3) / 4 + (p.Giq + 3) / 4 + 2 * ((p.H + 3) / 4) + p.Gik;
}

template <int KVF, int IF>
cudaError_t launch_layout(const RopeParams& p, unsigned grid, cudaStream_t st) {
  const size_t smem = 4 * (size_t)rope_quads(p) * sizeof(RowDesc);
  auto kern = p.rope.layout == MSA_ROPE_ADJACENT ? rope_kernel<KVF, IF, true> : rope_kernel<KVF, IF, false>;
  if (smem > 32768) {  // with the static part more than the 48 KB a launch has unasked
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<grid, 32 * kRopeWarps, smem, st>>>(p);
  return cudaGetLastError();
}

template <int KVF>
cudaError_t launch_kv(const RopeParams& p, unsigned grid, cudaStream_t st) {
  switch (p.idx_fmt) {
    case FMT_BF16: return launch_layout<KVF, FMT_BF16>(p, grid, st);
    case FMT_FP8: return launch_layout<KVF, FMT_FP8>(p, grid, st);
    case FMT_NVFP4: return launch_layout<KVF, FMT_NVFP4>(p, grid, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int num_sms, cudaStream_t st) {
  const long quads = (long)p.num_tokens * rope_quads(p);
  long grid = (quads + kRopeWarps - 1) / kRopeWarps;
  const long cap = (long)num_sms * kRopeCtas;
  if (grid > cap) grid = cap;
  switch (p.kv_fmt) {
    case FMT_BF16: return launch_kv<FMT_BF16>(p, (unsigned)grid, st);
    case FMT_FP8: return launch_kv<FMT_FP8>(p, (unsigned)grid, st);
    case FMT_NVFP4: return launch_kv<FMT_NVFP4>(p, (unsigned)grid, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace msa
