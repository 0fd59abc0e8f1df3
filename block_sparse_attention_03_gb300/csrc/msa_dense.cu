// The join of the dense attend's cut segments (msa_dense.cuh): out =
// sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i over the partials of one (sequence,
// KV head, column group), in the order of the runs, so that the result does
// not depend on timing.
//
// The runs' own notes (DenseParams::info: the segment a run begins in, and
// whether it began before) say which partials belong together, so nothing is
// counted.  A CTA takes the segment that crosses the border in front of run c, if
// it is the first border the segment crosses; or, where there are fewer segments
// than runs, a segment, whose borders it finds among the notes.  Partials stay in
// L2 and the launch overlaps the attend's tail (a programmatic dependent
// launch): latency is what it costs, so a CTA has a few rows, its warps share a
// row's partials where rows are few, and each has eight partials in flight (four
// where segments are many and have few partials each).  Measured behind the attend:
// 3 to 5 us after its last CTA.  Rows a CTA: one up to 8 columns, then four (8 x
// 64K tokens of 32 columns: 1.4 us longer in all with eight, 4.3 with one).
#include "msa_dense.cuh"

namespace msa {

namespace {

constexpr int kJoinWarps = 8;
constexpr int kJoinThreads = 32 * kJoinWarps;

// runs: in the grid of the attend; rows: of a partial; cta_rows: a CTA's share of
// them (blockIdx.y); shift: log2 of P's scale, which l carries.
template <bool BY_SEGMENT>
__global__ void __launch_bounds__(kJoinThreads, BY_SEGMENT ? 3 : 4) dense_combine_kernel(const DenseParams p, int runs, int rows, int cta_rows,
                                                                     float shift) {
  constexpr int kJoinBatch = BY_SEGMENT ? 8 : 4;  // partials of a row a warp has in flight
  __shared__ __align__(16) float so[kJoinWarps][132];  // (read and written as float4)
  __shared__ float sm[kJoinWarps][2];
  __shared__ int s_first, s_end, s_more;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int c, sg;  // the segment, and the first run that begins inside it
  if (BY_SEGMENT && tid == 0) {
    s_first = runs;
    s_end = 0;
  }
  __syncthreads();
  pdl_wait();
  if constexpr (BY_SEGMENT) {
    sg = blockIdx.x;
#pragma unroll 1
    for (int i = tid; i < runs; i += 2 * kJoinThreads) {  // (two loads at once, for some 300 notes: 0.3 us)
      const int2 x = __ldcg(p.info + i), y = i + kJoinThreads < runs ? __ldcg(p.info + i + kJoinThreads) : make_int2(-1, 0);
      if (x.x == sg && x.y != 0) {
        atomicMin(&s_first, i);
        atomicMax(&s_end, i + 1);
      }
      if (y.x == sg && y.y != 0) {
        atomicMin(&s_first, i + kJoinThreads);
        atomicMax(&s_end, i + kJoinThreads + 1);
      }
    }
    __syncthreads();
    c = s_first;
    if (c == runs) return;  // whole: its team has written it
  } else {
    c = blockIdx.x + 1;  // nothing begins inside a segment before run 1
    if (warp == 0) {  // (all CTAs read the same few lines of notes: one warp each, 2% of a sparse call less than all of them)
      const int2 me = __ldcg(p.info + c), before = __ldcg(p.info + c - 1);
      const int2 x = c + 1 + lane < runs ? __ldcg(p.info + c + 1 + lane) : make_int2(-1, 0);
      const uint32_t ends = __ballot_sync(0xffffffffu, x.x != me.x || x.y == 0);
      if (lane == 0) {
        // (it begins with this run, or crossed an earlier border)
        s_first = me.x >= 0 && me.y != 0 && !(before.x == me.x && before.y != 0) ? me.x : -1;
        s_end = ends ? c + __ffs(ends) : runs;
        s_more = ends == 0;
      }
    }
    __syncthreads();
    sg = s_first;
    if (sg < 0) return;
    if (s_more) {  // a long one
      for (int i = c + 33 + tid; i < runs; i += kJoinThreads) {
        const int2 y = __ldcg(p.info + i);
        if (y.x != sg || y.y == 0) atomicMin(&s_end, i);
      }
      __syncthreads();
    }
  }
  // part 0 is the end of run c - 1, the others the starts of the runs c to s_end - 1
  const int parts = s_end - c + 1;
  const int gc = sg % (p.G * p.CG), s = sg / (p.G * p.CG);
  const int g = gc / p.CG, cg = gc - g * p.CG;
  const int c0 = cg * p.cper;
  const int nrows = p.cols - c0 < p.cper ? p.cols - c0 : p.cper;
  const int first = blockIdx.y * cta_rows, end = min(nrows, first + cta_rows);
  if (first >= end) return;
  // few rows: several warps share a row's partials
  int ns = 1;
  while (ns < kJoinWarps && (end - first) * ns * 2 <= kJoinWarps) ns *= 2;
  const int per = kJoinWarps / ns;  // rows at a time
  for (int r0 = first; r0 < end; r0 += per) {
    const int row = r0 + warp / ns, sl = warp % ns;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < end) {
      for (int t0 = sl; t0 < parts; t0 += kJoinBatch * ns) {
        float2 v[kJoinBatch];
        float4 o[kJoinBatch];
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
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
        for (int i = 0; i < kJoinBatch; ++i) mn = fmaxf(mn, v[i].x);
        const float ms = mn == -INFINITY ? 0.f : mn;
        const float a = dense::ex2(M - ms);
        L *= a;
        acc.x *= a;
        acc.y *= a;
        acc.z *= a;
        acc.w *= a;
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
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
    if (row < end && sl == 0) {
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
  const int runs = num_sms * dense_teams(fmt, sh.nn), rows = dense_rows(sh.nn, sh.ncg);
  const long segments = (long)p.S * p.G * p.CG;
  const float shift = fmt == FMT_NVFP4 ? kDensePShift : 0.f;
  // few segments: each has many partials, so its rows go to CTAs of their own
  const bool by_segment = segments <= runs / 4;
  const int cta_rows = by_segment ? (p.cper <= 8 ? 1 : 4) : (p.cper < kJoinWarps ? p.cper : kJoinWarps);
  const dim3 grid((unsigned)(by_segment ? segments : runs - 1), (unsigned)((p.cper + cta_rows - 1) / cta_rows));
  return launch_behind(by_segment ? dense_combine_kernel<true> : dense_combine_kernel<false>, grid, dim3(kJoinThreads), 0, st, p, runs,
                       rows, cta_rows, shift);
}

}  // namespace msa
