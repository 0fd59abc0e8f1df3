// Block tables, slot maps, positions and lengths of a step, from the requests'
// lengths and a stack of free blocks, in one launch and without the host.
//
// With c_s tokens cached and n_s new (n_s = -1: the request has ended):
//   wants_s = ceil((c_s + n_s) / 128) - ceil(c_s / 128)   blocks it takes
//   back_s  = ceil(c_s / 128) if it has ended             blocks it gives back
// and three exclusive sums over the requests (tokens, wants, back) say where each
// one's tokens, new blocks and returned blocks lie.  The returned blocks go on
// top of the stack in the requests' order, the new ones come off its top in the
// same order: the i-th block taken is the stack's entry total - 1 - i.
//
// Latency is all there is (some kilobytes): every CTA computes the sums by
// itself in shared memory, so there is no second launch and no wait between
// CTAs, and then takes its share of the tokens, new blocks and returned blocks,
// finding the request of each by bisection.  A new token's slot is computed from
// the stack, not read from the table entry another CTA writes.  Measured: 32
// requests of one token 3.8 us, 253 requests with up to 64K tokens and 36 that end
// 5.6 us, 0.4 of them for the look at the returned blocks (an empty kernel's launch
// takes about 2).
#include "msa_device.cuh"
#include "msa_internal.h"

namespace msa {

namespace {

constexpr int kTabThreads = 512;

// Sums saturate at kMost, past any count that can be granted, so that no set of
// lengths wraps around (a saturating sum of sizes is associative).
constexpr int kMost = 1 << 30;
__device__ __forceinline__ int sat_add(int a, int b) {  // 0 <= a, b <= kMost; two of kMost pass an int's range
  return (int)min((unsigned)a + (unsigned)b, (unsigned)kMost);
}

// Exclusive sums in place of three arrays of n sizes <= kMost (n <= kMaxTableSeqs);
// the totals land at [n].
__device__ void scan3(int* a, int* b, int* c, int n, int* warp_sums) {
  constexpr int W = kTabThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + kTabThreads - 1) / kTabThreads;
  const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
  int x[3] = {0, 0, 0};
  for (int i = i0; i < i1; ++i) {
    x[0] = sat_add(x[0], a[i]);
    x[1] = sat_add(x[1], b[i]);
    x[2] = sat_add(x[2], c[i]);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int t = __shfl_up_sync(0xffffffffu, x[k], o);
      if (lane >= o) x[k] = sat_add(x[k], t);
    }
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < 3; ++k) warp_sums[k * W + warp] = x[k];
  __syncthreads();
  int base[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    // every warp scans the warps' sums by itself
    int w = lane < W ? warp_sums[k * W + lane] : 0;
#pragma unroll
    for (int o = 1; o < W; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w = sat_add(w, t);
    }
    const int all = __shfl_sync(0xffffffffu, w, W - 1);
    const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    const int left = __shfl_up_sync(0xffffffffu, x[k], 1);
    base[k] = sat_add(warp > 0 ? before : 0, lane > 0 ? left : 0);
    if (tid == 0) (k == 0 ? a : k == 1 ? b : c)[n] = all;
  }
  for (int i = i0; i < i1; ++i) {
    const int ta = a[i], tb = b[i], tc = c[i];
    a[i] = base[0];
    b[i] = base[1];
    c[i] = base[2];
    base[0] = sat_add(base[0], ta);
    base[1] = sat_add(base[1], tb);
    base[2] = sat_add(base[2], tc);
  }
  __syncthreads();
}

// The last s with at[s] <= x (at: n + 1 exclusive sums, at[0] = 0 <= x < at[n]); among equal sums the one that holds x.
__device__ __forceinline__ int owner(const int* at, int n, int x) {
  int lo = 0, hi = n;  // at[lo] <= x < at[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int blocks_of(int t) { return (t + kBlock - 1) / kBlock; }

__global__ void __launch_bounds__(kTabThreads) tables_kernel(const TablesParams p) {
  extern __shared__ int sm[];
  __shared__ int warp_sums[3 * kTabThreads / 32];
  __shared__ int s_taken;
  const int S = p.num_seqs, tid = threadIdx.x;
  int* tok = sm;               // [S + 1] first token of each request
  int* want = tok + S + 1;     // [S + 1] first new block
  int* back = want + S + 1;    // [S + 1] first returned block
  int* cached = back + S + 1;  // [S] -1: malformed
  const long limit = (long)p.max_nb * kBlock;
  if (tid == 0) s_taken = 0;
  const int count_in = __ldg(p.free_count);
  for (int s = tid; s < S; s += kTabThreads) {
    const int c = __ldg(p.cached + s), n = __ldg(p.fresh + s);
    const bool good = c >= 0 && n >= -1 && (long)c + max(n, 0) <= limit;
    if (!good && blockIdx.x == 0) raise_flag(p.status, FLAG_BAD_SEQLEN, s);
    const int add = good ? max(n, 0) : 0;
    cached[s] = good ? c : -1;
    tok[s] = add;
    want[s] = add > 0 ? blocks_of(c + add) - blocks_of(c) : 0;
    back[s] = good && n < 0 ? blocks_of(c) : 0;
  }
  __syncthreads();
  scan3(tok, want, back, S, warp_sums);
  const int count = min(max(count_in, 0), p.free_cap);
  const int room = p.free_cap - count;
  auto ended = [&](int s) { return cached[s] >= 0 && __ldg(p.fresh + s) < 0; };
  auto in_pool = [&](int b) { return b >= 0 && b < p.num_blocks; };
  // Returned entries outside the pool are no blocks: they are left out, or they would
  // come around again.  Every CTA looks at all that the stack has room for (a round of
  // loads for each 512).
  bool odd = false;
  for (int r = tid; r < min(back[S], room); r += kTabThreads) {
    const int s = owner(back, S, r);
    odd |= !in_pool(p.block_table[(size_t)s * p.max_nb + (r - back[s])]);
  }
  for (int r = room + blockIdx.x * kTabThreads + tid; r < back[S]; r += gridDim.x * kTabThreads) {  // dropped: flagged only
    const int s = owner(back, S, r), e = p.block_table[(size_t)s * p.max_nb + (r - back[s])];
    if (!in_pool(e)) raise_flag(p.status, FLAG_BAD_BLOCK, e);
  }
  const bool gaps = __syncthreads_or(odd);
  if (gaps) {
    for (int s = tid >> 5; s < S; s += kTabThreads / 32) {  // a warp a request
      int good = 0;
      const int n = ended(s) ? blocks_of(cached[s]) : 0;
      for (int b0 = 0; b0 < n; b0 += 32) {
        const int b = b0 + (tid & 31);
        const int e = b < n ? p.block_table[(size_t)s * p.max_nb + b] : 0;
        if (b < n && !in_pool(e) && blockIdx.x == 0) raise_flag(p.status, FLAG_BAD_BLOCK, e);
        good += __popc(__ballot_sync(0xffffffffu, b < n && in_pool(e)));
      }
      if ((tid & 31) == 0) back[s] = good;
    }
    __syncthreads();
    if (tid == 0) {
      int sum = 0;
      for (int s = 0; s <= S; ++s) {
        const int n = s < S ? back[s] : 0;
        back[s] = sum;
        sum = sat_add(sum, n);
      }
    }
    __syncthreads();
  }
  // the r-th returned block
  auto returned = [&](int r) -> int {
    const int s = owner(back, S, r);
    const int32_t* row = p.block_table + (size_t)s * p.max_nb;
    int i = r - back[s];
    if (gaps)
      for (int b = 0, left = i + 1; left > 0; ++b)  // back[] counted `left` blocks or more in this row
        if (in_pool(row[b])) {
          i = b;
          --left;
        }
    return row[i];
  };
  if (blockIdx.x == 0 && tid == 0 && count != count_in) raise_flag(p.status, FLAG_BAD_BLOCK, count);
  const int given = min(back[S], room);  // returned blocks the stack has room for
  const int total = count + given;
  // the blocks taken: those of the requests that are granted, a prefix of all
  // (a request is granted if its blocks are there and its tokens have places)
  for (int s = tid; s < S; s += kTabThreads)
    if (want[s + 1] <= total && tok[s + 1] <= p.max_tokens) atomicMax(&s_taken, want[s + 1]);
  __syncthreads();
  const int taken = s_taken;
  const int gtid = blockIdx.x * kTabThreads + tid, gn = gridDim.x * kTabThreads;

  // the i-th block taken; -1 (and the flag) if the stack names a block outside the pool
  auto stack_at = [&](int i) -> int {
    const int at = total - 1 - i;
    int b;
    if (at < count) {
      b = __ldg(p.free_blocks_in + at);
    } else {
      b = returned(at - count);
    }
    if (b < 0 || b >= p.num_blocks) {
      raise_flag(p.status, FLAG_BAD_BLOCK, b);
      return -1;
    }
    return b;
  };
  auto granted = [&](int s) { return want[s + 1] <= total && tok[s + 1] <= p.max_tokens; };

  // lengths and token offsets
  for (int s = gtid; s < S; s += gn) {
    const int add = tok[s + 1] - tok[s];
    const int c = cached[s];
    int len = c < 0 || ended(s) ? 0 : c;
    if (add > 0) {
      if (granted(s)) len = c + add;
      else raise_flag(p.status, FLAG_NO_ROOM, s);
    }
    p.seq_lens[s] = len;
    p.offsets[s] = tok[s];
  }
  if (gtid == 0) {
    p.offsets[S] = tok[S];
    *p.free_count_out = total - taken;
    if (back[S] > room) raise_flag(p.status, FLAG_NO_ROOM, -1);
  }
  // slots and positions of the new tokens, padding behind them
  for (int t = gtid; t < p.max_tokens; t += gn) {
    int slot = -1, pos = 0;
    if (t < tok[S]) {
      const int s = owner(tok, S, t);
      const int c = cached[s];
      pos = c + (t - tok[s]);
      if (granted(s)) {
        const int b = pos / kBlock, had = blocks_of(c);
        int blk;
        if (b < had) {
          blk = p.block_table[(size_t)s * p.max_nb + b];
          if (blk < 0 || blk >= p.num_blocks) {
            raise_flag(p.status, FLAG_BAD_BLOCK, blk);
            blk = -1;
          }
        } else {
          blk = stack_at(want[s] + b - had);
        }
        if (blk >= 0) slot = blk * kBlock + pos % kBlock;
      }
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
  // the new blocks into the tables
  for (int i = gtid; i < taken; i += gn) {
    const int s = owner(want, S, i);
    p.block_table[(size_t)s * p.max_nb + blocks_of(cached[s]) + (i - want[s])] = stack_at(i);
  }
  // the returned blocks that stay on the stack (entries at and above `count`:
  // nothing reads those in this call)
  for (int r = gtid; r < min(given, total - taken - count); r += gn) p.free_blocks[count + r] = returned(r);
}

}  // namespace

cudaError_t launch_tables(const TablesParams& p, int num_sms, cudaStream_t st) {
  const size_t smem = ((size_t)p.num_seqs * 4 + 3) * sizeof(int);
  cudaError_t e = cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  // one token a thread, up to two CTAs an SM: a thread's chain of dependent
  // reads (bisection, table, stack) is the kernel's time, so each has one
  // (253 requests, 64K tokens: 9.2 us with four tokens a thread)
  const long work = p.max_tokens > p.num_seqs ? p.max_tokens : p.num_seqs;
  long grid = (work + kTabThreads - 1) / kTabThreads;
  if (grid > 2 * num_sms) grid = 2 * num_sms;
  if (grid < 1) grid = 1;
  tables_kernel<<<(unsigned)grid, kTabThreads, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace msa
