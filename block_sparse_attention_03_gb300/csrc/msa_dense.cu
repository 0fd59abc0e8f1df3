// The join of the dense attend's cut segments (msa_dense.cuh): out =
// sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i over the partials of one (sequence,
// KV head, column group), in the order of the runs, so that the result does
// not depend on timing.
//
// CTA c takes the segment that crosses the border between the runs c - 1 and
// c, if it is the first border the segment crosses; the runs' own notes
// (DenseParams::info) say so, so nothing is counted or searched.  Partials stay
// in L2 (8 rows x 512 B a run); the launch overlaps the attend's tail (a
// programmatic dependent launch) and its latency is what it costs.
#include "msa_dense.cuh"

namespace msa {

namespace {

constexpr int kJoinWarps = 16;

// rows: of a partial; shift: log2 of P's scale, which l carries.
__global__ void __launch_bounds__(32 * kJoinWarps) dense_combine_kernel(const DenseParams p, int rows, float shift) {
  __shared__ float so[kJoinWarps][132];
  __shared__ float sm[kJoinWarps][2];
  __shared__ int s_parts;
  const int c = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) s_parts = gridDim.x;
  pdl_wait();
  const int2 me = __ldcg(p.info + c);
  if (me.x < 0 || me.y == 0) return;
  const int2 before = __ldcg(p.info + c - 1);  // a run that begins inside a segment is not the first
  if (before.x == me.x && before.y != 0) return;
  __syncthreads();
  // the runs c, c + 1, ... that begin inside the segment; part 0 is the end of run c - 1
  for (int i = c + tid; i < (int)gridDim.x; i += 32 * kJoinWarps) {
    const int2 x = __ldcg(p.info + i);
    if (x.x != me.x || x.y == 0) {
      atomicMin(&s_parts, i);
      break;
    }
  }
  __syncthreads();
  const int parts = s_parts - c + 1;
  const int gc = me.x % (p.G * p.CG), s = me.x / (p.G * p.CG);
  const int g = gc / p.CG, cg = gc - g * p.CG;
  const int c0 = cg * p.cper;
  const int nrows = p.cols - c0 < p.cper ? p.cols - c0 : p.cper;
  // few rows: several warps share a row's partials
  int ns = 1;
  while (ns < kJoinWarps && nrows * ns * 2 <= kJoinWarps) ns *= 2;
  const int per = kJoinWarps / ns;  // rows at a time
  for (int r0 = 0; r0 < nrows; r0 += per) {
    const int row = r0 + warp / ns, sl = warp % ns;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < nrows) {
      for (int t0 = sl; t0 < parts; t0 += 4 * ns) {
        float2 v[4];
        float4 o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + i * ns;
          v[i] = make_float2(-INFINITY, 0.f);
          o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (t < parts) {
            const size_t at = (size_t)(t == 0 ? 2 * (c - 1) + 1 : 2 * (c + t - 1)) * rows + row;
            v[i] = __ldcg(p.part_ml + at);
            o[i] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * kDim) + lane);
          }
        }
        float mn = M;
#pragma unroll
        for (int i = 0; i < 4; ++i) mn = fmaxf(mn, v[i].x);
        const float ms = mn == -INFINITY ? 0.f : mn;
        const float a = dense::ex2(M - ms);
        L *= a;
        acc.x *= a;
        acc.y *= a;
        acc.z *= a;
        acc.w *= a;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w = dense::ex2(v[i].x - ms);
          L += w * v[i].y;
          acc.x += w * o[i].x;
          acc.y += w * o[i].y;
          acc.z += w * o[i].z;
          acc.w += w * o[i].w;
        }
        M = mn;
      }
    }
    if (ns > 1) {
      __syncthreads();
      *reinterpret_cast<float4*>(&so[warp][4 * lane]) = acc;
      if (lane == 0) {
        sm[warp][0] = M;
        sm[warp][1] = L;
      }
      __syncthreads();
      if (sl == 0) {
        float mn = M;
        for (int i = 1; i < ns; ++i) mn = fmaxf(mn, sm[warp + i][0]);
        const float ms = mn == -INFINITY ? 0.f : mn;
        L = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < ns; ++i) {
          const float w = dense::ex2(sm[warp + i][0] - ms);
          const float4 o = *reinterpret_cast<const float4*>(&so[warp + i][4 * lane]);
          L += w * sm[warp + i][1];
          acc.x += w * o.x;
          acc.y += w * o.y;
          acc.z += w * o.z;
          acc.w += w * o.w;
        }
        M = mn;
      }
    }
    if (row < nrows && sl == 0) {
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const int col = c0 + row, i = col / p.r, h = col - i * p.r;
      const size_t orow = ((size_t)s * p.Q + i) * ((size_t)p.G * p.r) + (size_t)g * p.r + h;
      uint2 pk;
      pk.x = pack_bf16x2(acc.x * inv, acc.y * inv);
      pk.y = pack_bf16x2(acc.z * inv, acc.w * inv);
      *(reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + orow * kDim) + lane) = pk;
      if (lane == 0 && p.lse) p.lse[orow] = L == 0.f ? -INFINITY : (M - shift + log2f(L)) * 0.69314718055994531f;
    }
  }
}

}  // namespace

cudaError_t launch_dense_combine(const DenseParams& p, int fmt, int num_sms, cudaStream_t st) {
  const DenseShape sh = dense_shape(p.cper);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(num_sms * dense_teams(fmt, sh.nn)));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dense_combine_kernel, p, dense_rows(sh.nn, sh.ncg),
                            fmt != FMT_BF16 ? kDensePShift : 0.f);
}

}  // namespace msa
