// C ABI of libmsa (declared in include/msa.h): argument checks, workspace
// carving, TMA descriptor encoding and the launch chains of each entry point.
#include <cmath>
#include <cstring>
#include <mutex>

#include "msa_cut.h"
#include "msa_device.cuh"
#include "msa_internal.h"

using namespace msa;

namespace {

// ---------------------------------------------------------------- device facts

int sm_count() {
  static int cache[64];
  static bool init[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (!init[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    cache[dev] = n;
    init[dev] = true;
  }
  return cache[dev];
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 2-D map over rows of 128 elements (FP8: 128 B, BF16: 256 B); one box is
// 128 rows x 128 bytes with the 128-byte swizzle.
bool encode_rows(CUtensorMap* m, const void* base, long rows, bool bf16) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {128, (cuuint64_t)rows};
  cuuint64_t strides[1] = {bf16 ? 256ull : 128ull};
  cuuint32_t box[2] = {bf16 ? 64u : 128u, 128u};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                  const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// The dense attend's maps: rows of 128 elements of an FP8 (128 B), BF16 (256 B, in
// boxes of 128 B) or NVFP4 (64 B) cache; a box holds the rows of one unit, each
// under the swizzle of its width (conflict-free ldmatrix).
bool encode_unit_rows(CUtensorMap* m, const void* base, long rows, int fmt) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const bool bf16 = fmt == FMT_BF16, fp4 = fmt == FMT_NVFP4;
  cuuint64_t dims[2] = {fp4 ? 64ull : 128ull, (cuuint64_t)rows};
  cuuint64_t strides[1] = {bf16 ? 256ull : (fp4 ? 64ull : 128ull)};
  cuuint32_t box[2] = {bf16 || fp4 ? 64u : 128u, (cuuint32_t)dense_unit_keys(fmt)};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                  const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  fp4 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// ---------------------------------------------------------------- checks

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// 32-bit arrays and the status word: a misaligned access would end the context
template <typename... P>
bool aligned4(P... p) {
  return ((... | reinterpret_cast<uintptr_t>(static_cast<const void*>(p))) & 3u) == 0;
}

int fmt_of(msa_dtype_t d) {
  switch (d) {
    case MSA_DTYPE_BF16: return FMT_BF16;
    case MSA_DTYPE_FP8_E4M3: return FMT_FP8;
    case MSA_DTYPE_NVFP4: return FMT_NVFP4;
    default: return -1;
  }
}

// formats of K and V
int kv_fmt_of(msa_dtype_t d) {
  switch (d) {
    case MSA_DTYPE_INT8_BLOCK: return FMT_I8B;
    case MSA_DTYPE_FP8_BLOCK: return FMT_F8B;
    default: return fmt_of(d);
  }
}

bool by_block(const msa_cache_t* c) { return fmt_by_block(kv_fmt_of(c->kv_dtype)); }

int next_pow2(int x) {
  int p = 1;
  while (p < x) p <<= 1;
  return p;
}

msa_status_t check_batch(const msa_batch_t* b) {
  if (!b || !b->seq_lens || !b->block_table) return MSA_ERR_INVALID_ARGUMENT;
  if (b->num_seqs < 1 || b->q_per_seq < 1 || b->max_blocks_per_seq < 1) return MSA_ERR_INVALID_ARGUMENT;
  if ((long)b->max_blocks_per_seq * kBlock > (1l << 30)) return MSA_ERR_UNSUPPORTED;
  if ((long)b->q_per_seq > (long)b->max_blocks_per_seq * kBlock) return MSA_ERR_INVALID_ARGUMENT;
  return MSA_OK;
}

msa_status_t check_cfg(const msa_config_t* c) {
  if (!c) return MSA_ERR_INVALID_ARGUMENT;
  if (c->topk != 4 && c->topk != 8 && c->topk != 16 && c->topk != 32) return MSA_ERR_UNSUPPORTED;
  if (c->init_blocks < 0 || c->local_blocks < 0 || c->init_blocks + c->local_blocks > c->topk - 1)
    return MSA_ERR_INVALID_ARGUMENT;
  if (!(c->index_scale > 0.f) || !std::isfinite(c->index_scale)) return MSA_ERR_INVALID_ARGUMENT;
  if (!(c->sm_scale > 0.f) || !std::isfinite(c->sm_scale)) return MSA_ERR_INVALID_ARGUMENT;
  if (c->score_type != MSA_SCORE_MAX) return MSA_ERR_UNSUPPORTED;
  if (c->prefill_select != MSA_PREFILL_SELECT_TOPK && c->prefill_select != MSA_PREFILL_SELECT_INDEXER)
    return MSA_ERR_INVALID_ARGUMENT;
  return MSA_OK;
}

msa_status_t check_cache(const msa_cache_t* c, bool need_index, bool need_kv) {
  if (c && c->nvfp4_mode != MSA_NVFP4_EXACT && c->nvfp4_mode != MSA_NVFP4_E4M3_PRODUCT) return MSA_ERR_INVALID_ARGUMENT;
  if (!c) return MSA_ERR_INVALID_ARGUMENT;
  if (c->block_size != kBlock || c->head_dim != kDim || c->index_dim != kDim) return MSA_ERR_UNSUPPORTED;
  if (c->num_kv_heads < 1 || c->num_kv_heads > 8) return MSA_ERR_UNSUPPORTED;
  if (c->num_blocks < 1 || (long)c->num_blocks * c->num_kv_heads * kBlock >= (1l << 31)) return MSA_ERR_UNSUPPORTED;
  if (need_index) {
    const int f = fmt_of(c->index_dtype);
    if (f < 0) return MSA_ERR_UNSUPPORTED;
    if (!c->idx || !aligned16(c->idx)) return MSA_ERR_INVALID_ARGUMENT;
    if (f == FMT_FP8 && (!c->idx_scale || !aligned16(c->idx_scale))) return MSA_ERR_INVALID_ARGUMENT;
    if (f == FMT_NVFP4 && (!c->idx_sf || !aligned16(c->idx_sf) || !(c->idx_global > 0.f))) return MSA_ERR_INVALID_ARGUMENT;
  }
  if (need_kv) {
    const int f = kv_fmt_of(c->kv_dtype);
    if (f < 0) return MSA_ERR_UNSUPPORTED;
    if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return MSA_ERR_INVALID_ARGUMENT;
    if ((f == FMT_FP8 || fmt_by_block(f)) && (!c->k_scale || !c->v_scale || !aligned16(c->k_scale) || !aligned16(c->v_scale)))
      return MSA_ERR_INVALID_ARGUMENT;
    if (f == FMT_NVFP4 && (!c->k_sf || !c->v_sf || !aligned16(c->k_sf) || !aligned16(c->v_sf) ||
                           !(c->k_global > 0.f) || !(c->v_global > 0.f)))
      return MSA_ERR_INVALID_ARGUMENT;
  }
  return MSA_OK;
}

msa_status_t check_query(const msa_query_t* q) {
  if (!q || !q->data || !aligned16(q->data)) return MSA_ERR_INVALID_ARGUMENT;
  if (q->dtype != MSA_DTYPE_BF16 && q->dtype != MSA_DTYPE_FP8_E4M3) return MSA_ERR_UNSUPPORTED;
  if (q->dtype == MSA_DTYPE_FP8_E4M3 && !(q->scale > 0.f && std::isfinite(q->scale))) return MSA_ERR_INVALID_ARGUMENT;
  return MSA_OK;
}

// ---------------------------------------------------------------- workspace plan

FragGeom geom_for(int key_fmt, bool q_fp8, int cols) {
  FragGeom g;
  g.cols = cols;
  g.sp = (key_fmt == FMT_FP8 && !q_fp8) ? 2 : 1;
  g.ks = (key_fmt == FMT_FP8) ? 4 : 8;
  g.nt = next_pow2((cols + 7) / 8);
  return g;
}

struct DensePlan {
  int cols = 0, CG = 0, cper = 0, rows = 0;
  size_t off_info = 0, off_ml = 0, off_o = 0, total = 0;
};

struct Plan {
  int S = 0, Q = 0, chunks = 1;  // indexer: sequences / query tokens as it sees them (long chunks split)
  int Sa = 0, Qa = 0, chunks_a = 1;  // the same for the attend
  FragGeom gi, ga;          // indexer / attend query geometry
  int bps = 0, splits = 0, cap = 0, r = 0;
  bool direct = false;      // one query token: the attend reads the selection rows directly
  size_t off_status = 0, off_pooled = 0, off_uids = 0, off_umask = 0, off_ucount = 0, off_ctr = 0, off_qfa = 0,
         off_cfa = 0, off_po = 0, off_pml = 0, total = 0;
  int nctr = 0;             // attend counters: splits finished per (sequence, group)
  // prefill chunks over an FP8 cache: the key-block-major attend (selection lists,
  // one partial per (token, head, slot), a combine pass)
  bool k2q = false;
  // ... whose selection the tcgen05 indexer makes in its epilogue (candidate
  // lists and a merge launch instead of the pooled scores and a top-k launch)
  bool pisel = false;
  size_t off_plists = 0;
  // block scales: the dense attend's kernel over selection lists, its parts behind the others
  bool blk = false;
  DensePlan dense;
  size_t off_kcnt = 0, off_koff = 0, off_kcur = 0, off_kitem = 0, off_kent = 0, off_klist = 0, off_kpo = 0,
         off_kpml = 0, off_kq = 0, off_kqf = 0;
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// A prefill chunk (more than 8 new tokens a sequence) over an FP8 index
// cache: the tcgen05 indexer, with the query tokens as the MMA's M side.
bool tc_indexer(const msa_cache_t* c, const msa_batch_t* b) {
  const int G = c->num_kv_heads;
  return fmt_of(c->index_dtype) == FMT_FP8 && b->q_per_seq > 8 && (G == 1 || G == 2 || G == 4 || G == 8);
}

// Units of a launch of the dense attend, which counts them in 32 bits (a 64-bit count takes a short call 0.2 to 0.5 us):
// larger batches go in several.  A sequence's, by the width of its table (64 keys each at least, 4 for an end), are
// below 2^31; so are those of a token's lists.
constexpr long kMaxUnits = (1l << 32) - 1;
long sequence_units(int G, const DensePlan& pl, int max_nb) { return (long)G * pl.CG * (2l * max_nb + 4); }
long list_units(int G, const DensePlan& pl, int topk) { return (long)G * pl.CG * (topk + 1); }

// The dense attend's kernel for `seqs` sequences of q new tokens; its workspace from byte o on.
msa_status_t dense_plan_at(const msa_cache_t* c, long seqs, int q, int hq, size_t o, DensePlan& pl) {
  const int G = c->num_kv_heads;
  if (hq < G || hq % G != 0) return MSA_ERR_INVALID_ARGUMENT;
  if (hq / G > 64 || q > 8) return MSA_ERR_UNSUPPORTED;
  pl.cols = q * (hq / G);
  pl.CG = (pl.cols + 63) / 64;
  pl.cper = (pl.cols + pl.CG - 1) / pl.CG;
  const DenseShape sh = dense_shape(pl.cper);
  pl.rows = dense_rows(sh.nn, sh.ncg);
  if (seqs * G * pl.CG >= (1l << 31)) return MSA_ERR_UNSUPPORTED;
  const size_t ctas = (size_t)sm_count() * dense_teams(kv_fmt_of(c->kv_dtype), sh.nn);  // runs
  pl.off_info = o; o = align256(o + ctas * sizeof(int2));
  pl.off_ml = o; o = align256(o + 2 * ctas * pl.rows * sizeof(float2));
  pl.off_o = o; o = align256(o + 2 * ctas * pl.rows * kDim * sizeof(float));
  pl.total = o;
  return MSA_OK;
}

msa_status_t make_dense_plan(const msa_cache_t* c, const msa_batch_t* b, int hq, DensePlan& pl) {
  return dense_plan_at(c, b->num_seqs, b->q_per_seq, hq, 256, pl);  // behind the status word
}

// Plan for the given problem.  iq_fp8 / q_fp8: query dtypes (E4M3 or bf16).
msa_status_t make_plan(const msa_cache_t* c, const msa_batch_t* b, const msa_config_t* cfg, int hq, bool iq_fp8,
                       bool q_fp8, Plan& pl, bool allow_pisel = true) {
  // more than 8 new tokens per sequence (a prefill chunk): split into virtual
  // sequences of the largest of 8, 4, 2, 1 tokens dividing the count
  int QV = b->q_per_seq;
  if (QV > 8) {
    QV = 8;
    while (b->q_per_seq % QV) QV >>= 1;
  }
  pl.chunks = b->q_per_seq / QV;
  pl.S = b->num_seqs * pl.chunks;
  pl.Q = QV;
  // The attend runs every new token as its own one-token sequence (speculative
  // verify and prefill chunks alike): the tokens' selections overlap little, so
  // a union over 8 tokens streams each block for 32 query columns of which
  // about 4 chose it, four times the work per block for the few blocks saved.
  pl.Qa = 1;
  pl.chunks_a = b->q_per_seq / pl.Qa;
  pl.Sa = b->num_seqs * pl.chunks_a;
  const int Q = pl.Q, G = c->num_kv_heads;
  const int S = pl.Sa, Qa = pl.Qa;  // the attend's units size the buffers below
  if (hq < G || hq % G != 0) return MSA_ERR_INVALID_ARGUMENT;
  pl.r = hq / G;
  const int fi = fmt_of(c->index_dtype), fa = kv_fmt_of(c->kv_dtype);
  pl.gi = geom_for(fi < 0 ? FMT_FP8 : fi, iq_fp8, Q * G);
  pl.ga = geom_for(fa < 0 ? FMT_FP8 : fa, q_fp8, Qa * pl.r);
  if (!tc_indexer(c, b) && (pl.gi.nt > kMaxIndexerNT || pl.gi.nt * pl.gi.sp > 8)) return MSA_ERR_UNSUPPORTED;
  pl.blk = fmt_by_block(fa);
  if (pl.blk) {
    pl.off_pooled = 256;
    const size_t pooled = (size_t)b->num_seqs * b->q_per_seq * G * b->max_blocks_per_seq * 4;
    const msa_status_t s = dense_plan_at(c, (long)b->num_seqs * b->q_per_seq, 1, hq, align256(256 + pooled), pl.dense);
    pl.total = pl.dense.total;
    if (s == MSA_OK && b->q_per_seq * list_units(G, pl.dense, cfg->topk) > kMaxUnits) return MSA_ERR_UNSUPPORTED;
    return s;
  }
  if (pl.ga.cols > kMaxAttendCols || pl.ga.nt * pl.ga.sp > 8) return MSA_ERR_UNSUPPORTED;
  pl.cap = Qa * cfg->topk;
  pl.direct = (Qa == 1);
  // a union never holds more blocks than a sequence has
  const int cap_eff = pl.cap < b->max_blocks_per_seq ? pl.cap : b->max_blocks_per_seq;
  pl.bps = attend_blocks_per_split(cap_eff, (long)S * G, 2 * sm_count());
  pl.splits = (cap_eff + pl.bps - 1) / pl.bps;
  pl.nctr = S * G;  // splits finished per (sequence, group)
  size_t o = 0;
  pl.off_status = o; o = align256(o + 256);
  pl.k2q = fa == FMT_FP8 && b->q_per_seq > 8 && (pl.r == 1 || pl.r == 2 || pl.r == 4 || pl.r == 8);
  // (16 list entries a thread, 16-bit block ids)
  pl.pisel = allow_pisel && cfg->prefill_select == MSA_PREFILL_SELECT_INDEXER && pl.k2q && tc_indexer(c, b) &&
             cfg->topk <= 16 && b->max_blocks_per_seq <= 65536;
  pl.off_pooled = o;
  if (!pl.pisel) o = align256(o + (size_t)b->num_seqs * b->q_per_seq * G * b->max_blocks_per_seq * 4);
  pl.off_uids = o; o = align256(o + (size_t)S * G * pl.cap * 4);
  pl.off_umask = o; o = align256(o + (size_t)S * G * pl.cap * 4);
  pl.off_ucount = o; o = align256(o + (size_t)S * G * 4);
  pl.off_ctr = o; o = align256(o + (size_t)pl.nctr * 4);
  pl.off_qfa = o; o = align256(o + (size_t)S * G * pl.ga.words_per_unit() * 4);
  pl.off_cfa = o; o = align256(o + (size_t)S * G * pl.ga.nt * 8 * 4);
  pl.off_po = o; o = align256(o + (size_t)S * G * pl.splits * pl.ga.cols * 128 * 4);
  pl.off_pml = o; o = align256(o + (size_t)S * G * pl.splits * pl.ga.cols * 2 * 4);
  if (pl.pisel) {
    // a list slot per (CTA, query tile it touches): at most tiles + min(CTAs,
    // units) slots of 128 rows x 4 lists x 16 keys
    const size_t tiles = (size_t)b->num_seqs * ((b->q_per_seq + 128 / G - 1) / (128 / G));
    const size_t units = tiles * (size_t)((b->max_blocks_per_seq + 1) / 2);
    const size_t ctas = (size_t)prefill_indexer_grid(sm_count());
    pl.off_plists = o; o = align256(o + (tiles + (units < ctas ? units : ctas)) * 128 * 64 * 8);
  }
  if (pl.k2q) {
    const size_t L = (size_t)b->num_seqs * G * b->max_blocks_per_seq;
    const size_t E = (size_t)b->num_seqs * b->q_per_seq * G * cfg->topk;
    const size_t P = E * pl.r;
    if (P >= ((size_t)1 << 31)) return MSA_ERR_UNSUPPORTED;  // the list kernels count entries and partials in 32 bits
    pl.off_kcnt = o; o = align256(o + L * 4);
    pl.off_koff = o; o = align256(o + L * 4);
    pl.off_kcur = o; o = align256(o + L * 4);
    pl.off_kitem = o; o = align256(o + (L + 1) * 4);
    pl.off_kent = o; o = align256(o + E * 4 + 16);  // the attend copies entries from 16-byte boundaries
    pl.off_klist = o; o = align256(o + E * 4);
    pl.off_kpo = o; o = align256(o + P * 128 * 2);
    pl.off_kpml = o; o = align256(o + P * 4 * 4);
    const size_t R = (size_t)b->num_seqs * b->q_per_seq * hq;  // query rows (token, head)
    pl.off_kq = o; o = align256(o + (q_fp8 ? 0 : R * 256));
    pl.off_kqf = o; o = align256(o + (q_fp8 ? 0 : R * 4));
  }
  pl.total = o;
  return MSA_OK;
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

BatchDev batch_dev(const msa_batch_t* b, const Plan& pl) {
  BatchDev d;
  d.seq_lens = b->seq_lens;
  d.block_table = b->block_table;
  d.S = pl.S;
  d.Q = pl.Q;
  d.max_nb = b->max_blocks_per_seq;
  d.chunks = pl.chunks;
  d.q_real = b->q_per_seq;
  return d;
}

// the attend's view of the batch (its own virtual sequences)
BatchDev batch_dev_att(const msa_batch_t* b, const Plan& pl) {
  BatchDev d = batch_dev(b, pl);
  d.S = pl.Sa;
  d.Q = pl.Qa;
  d.chunks = pl.chunks_a;
  return d;
}

msa_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA; }

// ---------------------------------------------------------------- stages of the path

msa_status_t run_indexer(const msa_cache_t* c, const msa_batch_t* b, const msa_config_t* cfg, const msa_query_t* iq,
                         const Plan& pl, void* ws, float* pooled, cudaStream_t st, bool select = false) {
  const int G = c->num_kv_heads;
  const int fi = fmt_of(c->index_dtype);
  CUtensorMap tm;
  const CUtensorMap* tmp = nullptr;
  if (fi != FMT_NVFP4) {
    if (!encode_rows(&tm, c->idx, (long)c->num_blocks * kBlock, fi == FMT_BF16)) return MSA_ERR_CUDA;
    tmp = &tm;
  }
  if (tc_indexer(c, b)) {
    // a prefill chunk: the queries fill the tensor cores' M side (tcgen05)
    PrefillIndexerParams pp;
    Plan real;
    real.S = b->num_seqs;
    real.Q = b->q_per_seq;
    real.chunks = 1;
    pp.batch = batch_dev(b, real);
    pp.G = G;
    pp.num_blocks = c->num_blocks;
    pp.idx_scale = c->idx_scale;
    pp.index_q = iq->data;
    pp.iq_fp8 = iq->dtype == MSA_DTYPE_FP8_E4M3;
    pp.iq_scale = pp.iq_fp8 ? iq->scale : 1.f;
    pp.col_const = cfg->index_scale;
    pp.pooled = pooled;
    pp.lists = select ? at<uint64_t>(ws, pl.off_plists) : nullptr;
    pp.topk = cfg->topk;
    pp.init_blocks = cfg->init_blocks;
    pp.local_blocks = cfg->local_blocks;
    pp.status = at<DeviceStatus>(ws, pl.off_status);
    return cuda_status(launch_prefill_indexer(tmp, pp, sm_count(), st));
  }
  IndexerParams ip;
  ip.batch = batch_dev(b, pl);
  ip.G = G;
  ip.num_blocks = c->num_blocks;
  ip.idx = static_cast<const uint8_t*>(c->idx);
  ip.idx_sf = static_cast<const uint8_t*>(c->idx_sf);
  ip.idx_scale = c->idx_scale;
  ip.index_q = iq->data;
  ip.iq_fp8 = iq->dtype == MSA_DTYPE_FP8_E4M3;
  ip.iq_scale = ip.iq_fp8 ? iq->scale : 1.f;
  ip.col_const = cfg->index_scale * (fi == FMT_NVFP4 ? c->idx_global : 1.f);
  ip.nv_round = c->nvfp4_mode == MSA_NVFP4_E4M3_PRODUCT ? 1 : 0;
  ip.geom = pl.gi;
  ip.pooled = pooled;
  ip.status = at<DeviceStatus>(ws, pl.off_status);
  // first kernel of the call: plain stream order, so every earlier write to the
  // caches and queries is complete and visible before it reads them
  return cuda_status(launch_indexer(fi, tmp, ip, sm_count(), st, false));
}

// fill the attend query-fragment job of a top-k / union launch
template <typename P>
void set_frag_job(P& kp, const msa_cache_t* c, const msa_config_t* cfg, const msa_query_t* q, int hq, const Plan& pl,
                  void* ws) {
  const int fa = fmt_of(c->kv_dtype);
  kp.q = q->data;
  kp.q_fp8 = q->dtype == MSA_DTYPE_FP8_E4M3;
  kp.q_scale = kp.q_fp8 ? q->scale : 1.f;
  kp.col_const = cfg->sm_scale * 1.4426950408889634f * (fa == FMT_NVFP4 ? c->k_global : 1.f);
  kp.key_fmt = fa;
  kp.r = pl.r;
  kp.hq = hq;
  kp.geom = pl.ga;
  kp.frag = at<uint32_t>(ws, pl.off_qfa);
  kp.colf = at<float>(ws, pl.off_cfa);
}

struct FragJob {
  const msa_cache_t* c;
  const msa_query_t* q;
  int hq;
};

msa_status_t run_topk(const msa_batch_t* b, const msa_config_t* cfg, int G, const float* pooled, int32_t* topk_idx,
                      float* topk_score, void* ws, const Plan* pl, cudaStream_t st, bool pdl, bool clear_ctr,
                      const FragJob* frag_job = nullptr, bool warp_rows = false) {
  TopkParams tp;
  // positions T - Q + i are the same with or without virtual sequences: the real batch
  Plan real;
  real.S = b->num_seqs;
  real.Q = b->q_per_seq;
  real.chunks = 1;
  tp.batch = batch_dev(b, real);
  tp.G = G;
  tp.topk = cfg->topk;
  tp.init_blocks = cfg->init_blocks;
  tp.local_blocks = cfg->local_blocks;
  tp.pooled = pooled;
  tp.topk_idx = topk_idx;
  tp.topk_score = topk_score;
  tp.status = pl ? at<DeviceStatus>(ws, pl->off_status) : static_cast<DeviceStatus*>(ws);
  tp.zero = (clear_ctr && pl) ? at<int32_t>(ws, pl->off_ctr) : nullptr;  // for the attend that follows
  tp.nzero = (clear_ctr && pl) ? pl->nctr : 0;
  tp.frag = nullptr;
  tp.colf = nullptr;
  if (frag_job && pl) set_frag_job(tp, frag_job->c, cfg, frag_job->q, frag_job->hq, *pl, ws);
  // one warp per row: for many short rows with nothing else to do (no scores,
  // fragments or counters)
  if (warp_rows && !topk_score && !tp.frag && !tp.zero) return cuda_status(launch_topk_warp(tp, st, pdl));
  return cuda_status(launch_topk(tp, st, pdl));
}

// The prefill selection from the candidate lists the tcgen05 indexer left (Plan::pisel).
msa_status_t run_pisel(const msa_batch_t* b, const msa_config_t* cfg, int G, int32_t* topk_idx, const Plan& pl,
                       void* ws, cudaStream_t st) {
  Plan real;
  real.S = b->num_seqs;
  real.Q = b->q_per_seq;
  real.chunks = 1;
  PiSelectParams sp;
  sp.batch = batch_dev(b, real);
  sp.G = G;
  sp.topk = cfg->topk;
  sp.init_blocks = cfg->init_blocks;
  sp.local_blocks = cfg->local_blocks;
  sp.grid = prefill_indexer_grid(sm_count());
  sp.lists = at<uint64_t>(ws, pl.off_plists);
  sp.topk_idx = topk_idx;
  sp.status = at<DeviceStatus>(ws, pl.off_status);
  return cuda_status(launch_prefill_select(sp, st));
}

msa_status_t run_attend(const msa_cache_t* c, const msa_batch_t* b, const msa_config_t* cfg, const msa_query_t* q,
                        int hq, const int32_t* topk_idx, void* out, float* lse, const Plan& pl, void* ws,
                        cudaStream_t st, bool prepared) {
  // prepared: the preceding top-k launch (one query token) already cleared the
  // counters and wrote the query fragments; otherwise the union kernel does both
  const int G = c->num_kv_heads;
  const int fa = fmt_of(c->kv_dtype);
  DeviceStatus* status = at<DeviceStatus>(ws, pl.off_status);
  const bool direct = prepared && pl.direct;
  UnionParams up;
  up.batch = batch_dev_att(b, pl);
  up.G = G;
  up.topk = cfg->topk;
  up.topk_idx = topk_idx;
  up.cap = pl.cap;
  up.u_ids = at<int32_t>(ws, pl.off_uids);
  up.u_mask = at<uint32_t>(ws, pl.off_umask);
  up.u_count = at<int32_t>(ws, pl.off_ucount);
  up.zero = at<int32_t>(ws, pl.off_ctr);  // for the attend that follows
  up.nzero = pl.nctr;
  set_frag_job(up, c, cfg, q, hq, pl, ws);
  up.status = status;
  if (!direct) {
    if (launch_union(up, st, true) != cudaSuccess) return MSA_ERR_CUDA;
  }

  CUtensorMap tk, tv;
  const CUtensorMap *tkp = nullptr, *tvp = nullptr;
  if (fa != FMT_NVFP4) {
    const long rows = (long)c->num_blocks * G * kBlock;
    if (!encode_rows(&tk, c->k, rows, fa == FMT_BF16) || !encode_rows(&tv, c->v, rows, fa == FMT_BF16))
      return MSA_ERR_CUDA;
    tkp = &tk;
    tvp = &tv;
  }
  AttendParams ap;
  ap.batch = batch_dev_att(b, pl);
  ap.G = G;
  ap.r = pl.r;
  ap.num_blocks = c->num_blocks;
  ap.k = static_cast<const uint8_t*>(c->k);
  ap.v = static_cast<const uint8_t*>(c->v);
  ap.k_sf = static_cast<const uint8_t*>(c->k_sf);
  ap.v_sf = static_cast<const uint8_t*>(c->v_sf);
  ap.k_scale = c->k_scale;
  ap.v_scale = c->v_scale;
  ap.v_global = c->v_global;
  ap.nv_round = c->nvfp4_mode == MSA_NVFP4_E4M3_PRODUCT ? 1 : 0;
  ap.q = q->data;
  ap.q_fp8 = q->dtype == MSA_DTYPE_FP8_E4M3;
  ap.q_scale = ap.q_fp8 ? q->scale : 1.f;
  ap.col_const = cfg->sm_scale * 1.4426950408889634f * (fa == FMT_NVFP4 ? c->k_global : 1.f);
  ap.geom = pl.ga;
  ap.direct = direct ? 1 : 0;
  ap.frag = up.frag;
  ap.colf = up.colf;
  ap.topk_idx = topk_idx;
  ap.topk = cfg->topk;
  ap.u_ids = up.u_ids;
  ap.u_mask = up.u_mask;
  ap.u_count = up.u_count;
  ap.cap = pl.cap;
  ap.bps = pl.bps;
  ap.splits = pl.splits;
  ap.work_ctr = nullptr;
  ap.sg_ctr = at<int32_t>(ws, pl.off_ctr);
  ap.part_o = at<float>(ws, pl.off_po);
  ap.part_ml = at<float>(ws, pl.off_pml);
  ap.out = out;
  ap.lse = lse;
  ap.status = status;
  if (launch_attend(fa, tkp, tvp, ap, sm_count(), st, true) != cudaSuccess) return MSA_ERR_CUDA;
  return MSA_OK;
}

// The key-block-major attend of a prefill chunk from the selection topk_idx.
msa_status_t run_k2q(const msa_cache_t* c, const msa_batch_t* b, const msa_config_t* cfg, const msa_query_t* q,
                     int hq, const int32_t* topk_idx, void* out, float* lse, const Plan& pl, void* ws,
                     cudaStream_t st) {
  const int G = c->num_kv_heads;
  if (!aligned16(ws)) return MSA_ERR_INVALID_ARGUMENT;  // the attend's bulk copies read from it
  CUtensorMap tk, tv;
  const long rows = (long)c->num_blocks * G * kBlock;
  if (!encode_rows(&tk, c->k, rows, false) || !encode_rows(&tv, c->v, rows, false)) return MSA_ERR_CUDA;
  Plan real;
  real.S = b->num_seqs;
  real.Q = b->q_per_seq;
  real.chunks = 1;
  K2qParams kp;
  kp.batch = batch_dev(b, real);
  kp.G = G;
  kp.r = hq / G;
  kp.topk = cfg->topk;
  kp.num_blocks = c->num_blocks;
  kp.topk_idx = topk_idx;
  kp.cnt = at<int32_t>(ws, pl.off_kcnt);
  kp.off = at<int32_t>(ws, pl.off_koff);
  kp.cur = at<int32_t>(ws, pl.off_kcur);
  kp.item_off = at<int32_t>(ws, pl.off_kitem);
  kp.entries = at<int32_t>(ws, pl.off_kent);
  kp.item_list = at<int32_t>(ws, pl.off_klist);
  kp.item_tokens = kBlock / kp.r;
  kp.k_scale = c->k_scale;
  kp.v_scale = c->v_scale;
  kp.q = q->data;
  kp.q_fp8 = q->dtype == MSA_DTYPE_FP8_E4M3;
  kp.q_scale = kp.q_fp8 ? q->scale : 1.f;
  kp.col_const = cfg->sm_scale * 1.4426950408889634f;
  kp.qsplit = at<uint8_t>(ws, pl.off_kq);
  kp.qrowf = at<float>(ws, pl.off_kqf);
  kp.part_o = at<uint16_t>(ws, pl.off_kpo);
  kp.part_ml = at<float>(ws, pl.off_kpml);
  kp.out = out;
  kp.lse = lse;
  kp.status = at<DeviceStatus>(ws, pl.off_status);
  if (launch_k2q_build(kp, sm_count(), st) != cudaSuccess) return MSA_ERR_CUDA;
  if (launch_k2q_attend(&tk, &tv, kp, sm_count(), st) != cudaSuccess) return MSA_ERR_CUDA;
  if (launch_k2q_combine(kp, sm_count(), st) != cudaSuccess) return MSA_ERR_CUDA;
  return MSA_OK;
}

// ---------------------------------------------------------------- the dense attend


// topk_idx: the sparse attend over these selections (caches with block scales), else null.
msa_status_t run_dense(const msa_cache_t* c, const msa_batch_t* b, const msa_config_t* cfg, const msa_query_t* q, int hq,
                       const int32_t* topk_idx, void* out, float* lse, const DensePlan& pl, void* ws, cudaStream_t st) {
  const int G = c->num_kv_heads, fmt = kv_fmt_of(c->kv_dtype), sms = sm_count();
  const long rows = (long)c->num_blocks * G * kBlock;
  CUtensorMap tk, tv;
  if (!encode_unit_rows(&tk, c->k, rows, fmt) || !encode_unit_rows(&tv, c->v, rows, fmt)) return MSA_ERR_CUDA;
  DenseParams p;
  p.S = topk_idx ? b->num_seqs * b->q_per_seq : b->num_seqs;
  p.Q = topk_idx ? 1 : b->q_per_seq;
  p.topk_idx = topk_idx;
  p.topk = cfg->topk;
  p.q_real = b->q_per_seq;
  p.G = G;
  p.r = hq / G;
  p.cols = pl.cols;
  p.CG = pl.CG;
  p.cper = pl.cper;
  p.max_nb = b->max_blocks_per_seq;
  p.num_blocks = c->num_blocks;
  p.q_fp8 = q->dtype == MSA_DTYPE_FP8_E4M3;
  p.q_scale = p.q_fp8 ? q->scale : 1.f;
  p.col_const = cfg->sm_scale * 1.4426950408889634f * (fmt == FMT_NVFP4 ? c->k_global : 1.f);
  p.k_sc = static_cast<const uint8_t*>(fmt == FMT_NVFP4 ? c->k_sf : static_cast<const void*>(c->k_scale));
  p.v_sc = static_cast<const uint8_t*>(fmt == FMT_NVFP4 ? c->v_sf : static_cast<const void*>(c->v_scale));
  p.v_global = c->v_global;
  // A small cache stays in the 129 MB L2 by itself; a larger one is a stream that would push the
  // partials and the next kernels' code out, so its lines are the first to go.  Four BF16
  // sequences, default and so: 16 MB 12.6 and 14.5 us, 32 MB 16.6 and 16.5, 64 MB 22.7 and 21.7, 128 MB
  // 32.9 and 31.4 (with a cold L2 41.5 and 37.0).  The host knows no lengths: the table's width bounds
  // them, so a small cache under a wide table counts as a large one.
  const double row = fmt == FMT_BF16 ? 512. : fmt == FMT_FP8 ? 264. : fmt == FMT_NVFP4 ? 144. : 256.;
  // Over selection lists the same, but for a prompt's chunk, whose tokens share blocks: they stay (1,024 tokens on
  // 256K 281 and 262 us, 8,192 on 64K 1,940 and 1,858; a verify step's whole path, 8 x 128K x 8 tokens, 99 with its
  // blocks the first to go and 108 without).
  p.stream = (!topk_idx || b->q_per_seq <= 8) && (double)p.S * (topk_idx ? cfg->topk : p.max_nb) * kBlock * G * row > 32e6;
  p.info = at<int2>(ws, pl.off_info);
  p.part_ml = at<float2>(ws, pl.off_ml);
  p.part_o = at<float>(ws, pl.off_o);
  p.lse = nullptr;
  p.status = at<DeviceStatus>(ws, 0);
  const long tokens = b->q_per_seq, units = topk_idx ? tokens * list_units(G, pl, cfg->topk) : sequence_units(G, pl, p.max_nb);
  for (long s0 = 0; s0 < b->num_seqs;) {
    const DenseCut cut = dense_cut(s0, b->num_seqs, units, kMaxUnits, tokens, hq, p.max_nb, G, cfg->topk);
    s0 += cut.n;
    p.S = (int)(topk_idx ? cut.n * tokens : cut.n);
    p.seq_lens = b->seq_lens + cut.s0;
    p.block_table = b->block_table + cut.table;
    if (topk_idx) p.topk_idx = topk_idx + cut.lists;
    p.q = static_cast<const uint8_t*>(q->data) + (size_t)cut.row * kDim * (p.q_fp8 ? 1 : 2);
    p.out = static_cast<uint8_t*>(out) + (size_t)cut.row * kDim * 2;
    if (lse) p.lse = lse + cut.row;
    cudaError_t e;
    if (fmt == FMT_BF16) e = launch_dense_bf16(&tk, &tv, p, sms, st);
    else if (fmt == FMT_FP8) e = launch_dense_fp8(&tk, &tv, p, sms, st);
    else if (fmt == FMT_I8B) e = topk_idx ? launch_dense_int8_sel(&tk, &tv, p, sms, st) : launch_dense_int8(&tk, &tv, p, sms, st);
    else if (fmt == FMT_F8B) e = topk_idx ? launch_dense_fp8b_sel(&tk, &tv, p, sms, st) : launch_dense_fp8b(&tk, &tv, p, sms, st);
    else if (c->nvfp4_mode == MSA_NVFP4_E4M3_PRODUCT) e = launch_dense_nvfp4_rounded(&tk, &tv, p, sms, st);
    else e = launch_dense_nvfp4(&tk, &tv, p, sms, st);
    if (e == cudaSuccess) e = launch_dense_combine(p, fmt, sms, st);
    if (e != cudaSuccess) return MSA_ERR_CUDA;
  }
  return MSA_OK;
}

// The path's second half over a cache with block scales: the top-k of the pooled scores and the
// attend over its lists.  (A warp a row for a prompt chunk's many rows, as elsewhere.)
msa_status_t run_select_dense(const msa_cache_t* c, const msa_batch_t* b, const msa_config_t* cfg, const msa_query_t* q, int hq,
                              const float* pooled, int32_t* topk_idx, void* out, float* lse, const Plan& pl, void* ws,
                              cudaStream_t st) {
  const msa_status_t s = run_topk(b, cfg, c->num_kv_heads, pooled, topk_idx, nullptr, ws, &pl, st, true, false, nullptr,
                                  b->q_per_seq > 8);
  if (s != MSA_OK) return s;
  return run_dense(c, b, cfg, q, hq, topk_idx, out, lse, pl.dense, ws, st);
}

msa_status_t check_rope(const msa_rope_t* r) {
  if (!r) return MSA_ERR_INVALID_ARGUMENT;
  if (r->rotary_dim < 16 || r->rotary_dim > kDim || r->rotary_dim % 16 != 0) return MSA_ERR_UNSUPPORTED;
  if (r->axes < 1 || r->axes > MSA_ROPE_MAX_AXES) return MSA_ERR_UNSUPPORTED;
  if (r->layout != MSA_ROPE_HALVES && r->layout != MSA_ROPE_ADJACENT) return MSA_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < r->rotary_dim / 2; ++i)
    if (r->axis[i] >= r->axes) return MSA_ERR_INVALID_ARGUMENT;
  return MSA_OK;
}

// rows of one projection: tokens `stride` elements apart, heads side by side
bool rows_ok(const msa_rows_t* r) { return r && r->data && aligned16(r->data) && r->stride >= 0 && r->stride % 8 == 0; }

// Bytes from a on; whether two such pieces of memory meet.
struct Piece {
  const void* p;
  size_t n;
};
bool meet(const Piece& a, const Piece& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.n > 0 && b.n > 0 && x < y + b.n && y < x + a.n;
}
Piece rows_piece(const msa_rows_t* r, int tokens, int heads) {
  return {r ? r->data : nullptr, ((size_t)(tokens - 1) * r->stride + (size_t)heads * kDim) * 2};
}
// The K and V side of a cache: data, then scales.
void cache_pieces(const msa_cache_t* c, Piece (&out)[4]) {
  const size_t blocks = (size_t)c->num_blocks * c->num_kv_heads, rows = blocks * kBlock;
  const int f = kv_fmt_of(c->kv_dtype);
  const size_t data = rows * (f == FMT_BF16 ? 256 : f == FMT_NVFP4 ? 64 : 128);
  const size_t scales = f == FMT_BF16 ? 0 : f == FMT_NVFP4 ? rows * 8 : f == FMT_FP8 ? rows * 4 : blocks * 4;
  out[0] = {c->k, data};
  out[1] = {c->v, data};
  out[2] = {f == FMT_NVFP4 ? c->k_sf : c->k_scale, scales};
  out[3] = {f == FMT_NVFP4 ? c->v_sf : c->v_scale, scales};
}
// Whether what a span call writes meets what it reads: the cache (insert) or the rows (read) against the
// others, the lengths, the table and the status word.
bool span_overlap(const msa_cache_t* c, const msa_spans_t* sp, int tokens, const msa_rows_t* k, const msa_rows_t* v,
                  const void* ws, bool insert) {
  Piece cache[4], other[8];
  cache_pieces(c, cache);
  int n = 0;
  if (k) other[n++] = rows_piece(k, tokens, c->num_kv_heads);
  if (v) other[n++] = rows_piece(v, tokens, c->num_kv_heads);
  const int rows = n;
  const size_t words = 4 * (size_t)sp->num_seqs;
  other[n++] = {sp->first, words};
  other[n++] = {sp->end, words};
  other[n++] = {sp->token_offsets, words};
  other[n++] = {sp->block_table, words * sp->max_blocks_per_seq};
  other[n++] = {ws, sizeof(DeviceStatus)};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < (insert ? n : rows); ++j)
      if (meet(cache[i], other[j])) return true;
    for (int j = 0; insert && j < i; ++j)
      if (meet(cache[i], cache[j])) return true;
  }
  if (insert) return false;
  for (int i = 0; i < rows; ++i)
    for (int j = rows; j < n; ++j)
      if (meet(other[i], other[j])) return true;
  if (rows == 2 && meet(other[0], other[1])) {
    // slices of the same rows side by side are fine: the same stride, and no token's K on another's V
    if (k->stride != v->stride) return true;
    const int64_t d = (int64_t)(reinterpret_cast<intptr_t>(v->data) - reinterpret_cast<intptr_t>(k->data)) / 2;
    const int64_t row = (int64_t)c->num_kv_heads * kDim, step = tokens > 1 ? k->stride : 0;
    const int64_t m = step > 0 ? d / step : 0;  // the tokens whose rows are nearest
    for (int64_t t = m - 1; t <= m + 1; ++t)
      if (t > -tokens && t < tokens && d - t * step < row && t * step - d < row) return true;
  }
  return false;
}

// What the insert and the read of spans share.
msa_status_t span_params(const msa_cache_t* c, const msa_spans_t* sp, int num_tokens, const msa_rows_t* k, const msa_rows_t* v,
                         void* ws, size_t ws_bytes, SpanParams& p) {
  const msa_status_t s = check_cache(c, false, true);
  if (s != MSA_OK) return s;
  if (!sp || sp->num_seqs < 1 || sp->max_blocks_per_seq < 1 || num_tokens < 0 || !sp->first || !sp->end || !sp->token_offsets ||
      !sp->block_table || !ws || !aligned4(sp->first, sp->end, sp->token_offsets, sp->block_table, ws))
    return MSA_ERR_INVALID_ARGUMENT;
  if ((long)sp->max_blocks_per_seq * kBlock > (1l << 30) || num_tokens > (1 << 27)) return MSA_ERR_UNSUPPORTED;
  if (ws_bytes < 256) return MSA_ERR_WORKSPACE_TOO_SMALL;
  std::memset(&p, 0, sizeof(p));
  p.S = sp->num_seqs;
  p.max_nb = sp->max_blocks_per_seq;
  p.num_tokens = num_tokens;
  p.H = c->num_kv_heads;
  p.num_blocks = c->num_blocks;
  p.first = sp->first;
  p.end = sp->end;
  p.offsets = sp->token_offsets;
  p.block_table = sp->block_table;
  if (k) p.k_stride = k->stride;
  if (v) p.v_stride = v->stride;
  p.kc = static_cast<uint8_t*>(const_cast<void*>(c->k));
  p.vc = static_cast<uint8_t*>(const_cast<void*>(c->v));
  p.ks = const_cast<float*>(c->k_scale);
  p.vs = const_cast<float*>(c->v_scale);
  p.ksf = static_cast<const uint8_t*>(c->k_sf);
  p.vsf = static_cast<const uint8_t*>(c->v_sf);
  p.kg = c->k_global;
  p.vg = c->v_global;
  p.nv_round = c->nvfp4_mode == MSA_NVFP4_E4M3_PRODUCT;
  p.status = static_cast<DeviceStatus*>(ws);
  return MSA_OK;
}

}  // namespace

// ====================================================================== C ABI

extern "C" {

const char* msa_status_string(msa_status_t s) {
  switch (s) {
    case MSA_OK: return "MSA_OK";
    case MSA_ERR_INVALID_ARGUMENT: return "MSA_ERR_INVALID_ARGUMENT";
    case MSA_ERR_UNSUPPORTED: return "MSA_ERR_UNSUPPORTED";
    case MSA_ERR_WORKSPACE_TOO_SMALL: return "MSA_ERR_WORKSPACE_TOO_SMALL";
    case MSA_ERR_CUDA: return "MSA_ERR_CUDA";
    case MSA_ERR_DEVICE_FAULT: return "MSA_ERR_DEVICE_FAULT";
    case MSA_ERR_TIMEOUT: return "MSA_ERR_TIMEOUT";
    default: return "MSA_ERR_UNKNOWN";
  }
}

size_t msa_workspace_size(const msa_cache_t* cache, const msa_batch_t* batch, const msa_config_t* cfg,
                          int32_t num_q_heads) {
  if (check_batch(batch) != MSA_OK || check_cfg(cfg) != MSA_OK || check_cache(cache, false, false) != MSA_OK)
    return 0;
  // the largest plan over query dtypes (a bf16 query against FP8 keys needs two terms)
  Plan pl;
  if (make_plan(cache, batch, cfg, num_q_heads, false, false, pl) != MSA_OK) {
    if (make_plan(cache, batch, cfg, num_q_heads, true, true, pl) != MSA_OK) return 0;
  }
  return pl.total;
}

msa_status_t msa_workspace_init(void* workspace, size_t workspace_bytes, msa_stream_t stream) {
  if (!workspace || workspace_bytes < 256) return MSA_ERR_INVALID_ARGUMENT;
  return cuda_status(cudaMemsetAsync(workspace, 0, 256, (cudaStream_t)stream));
}

msa_status_t msa_indexer_score(const msa_cache_t* cache, const msa_batch_t* batch, const msa_config_t* cfg,
                               const msa_query_t* index_q, float* pooled, void* workspace, size_t workspace_bytes,
                               msa_stream_t stream) {
  msa_status_t s;
  if ((s = check_batch(batch)) != MSA_OK || (s = check_cfg(cfg)) != MSA_OK || (s = check_cache(cache, true, false)) != MSA_OK ||
      (s = check_query(index_q)) != MSA_OK)
    return s;
  if (!pooled || !workspace) return MSA_ERR_INVALID_ARGUMENT;
  Plan pl;
  if ((s = make_plan(cache, batch, cfg, cache->num_kv_heads, index_q->dtype == MSA_DTYPE_FP8_E4M3, false, pl)) != MSA_OK)
    return s;
  if (workspace_bytes < pl.off_pooled) return MSA_ERR_WORKSPACE_TOO_SMALL;
  return run_indexer(cache, batch, cfg, index_q, pl, workspace, pooled, (cudaStream_t)stream);
}

msa_status_t msa_topk_blocks(const msa_batch_t* batch, const msa_config_t* cfg, int32_t num_groups,
                             const float* pooled, int32_t* topk_idx, float* topk_score, void* workspace,
                             size_t workspace_bytes, msa_stream_t stream) {
  msa_status_t s;
  if ((s = check_batch(batch)) != MSA_OK || (s = check_cfg(cfg)) != MSA_OK) return s;
  if (num_groups < 1 || num_groups > 8 || !pooled || !topk_idx || !workspace) return MSA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < 256) return MSA_ERR_WORKSPACE_TOO_SMALL;
  return run_topk(batch, cfg, num_groups, pooled, topk_idx, topk_score, workspace, nullptr, (cudaStream_t)stream, false,
                  false);
}

msa_status_t msa_sparse_attend(const msa_cache_t* cache, const msa_batch_t* batch, const msa_config_t* cfg,
                               const msa_query_t* q, int32_t num_q_heads, const int32_t* topk_idx, void* out,
                               float* lse, void* workspace, size_t workspace_bytes, msa_stream_t stream) {
  msa_status_t s;
  if ((s = check_batch(batch)) != MSA_OK || (s = check_cfg(cfg)) != MSA_OK || (s = check_cache(cache, false, true)) != MSA_OK ||
      (s = check_query(q)) != MSA_OK)
    return s;
  if (!topk_idx || !out || !workspace || !aligned16(out)) return MSA_ERR_INVALID_ARGUMENT;
  Plan pl;
  if ((s = make_plan(cache, batch, cfg, num_q_heads, true, q->dtype == MSA_DTYPE_FP8_E4M3, pl)) != MSA_OK) return s;
  if (workspace_bytes < pl.total) return MSA_ERR_WORKSPACE_TOO_SMALL;
  if (pl.blk) {
    if (!aligned16(workspace) || !aligned4(batch->seq_lens, batch->block_table, topk_idx, lse)) return MSA_ERR_INVALID_ARGUMENT;
    return run_dense(cache, batch, cfg, q, num_q_heads, topk_idx, out, lse, pl.dense, workspace, (cudaStream_t)stream);
  }
  if (pl.k2q) return run_k2q(cache, batch, cfg, q, num_q_heads, topk_idx, out, lse, pl, workspace, (cudaStream_t)stream);
  return run_attend(cache, batch, cfg, q, num_q_heads, topk_idx, out, lse, pl, workspace, (cudaStream_t)stream, false);
}

msa_status_t msa_decode(const msa_cache_t* cache, const msa_batch_t* batch, const msa_config_t* cfg,
                        const msa_query_t* index_q, const msa_query_t* q, int32_t num_q_heads, int32_t* topk_idx,
                        void* out, float* lse, void* workspace, size_t workspace_bytes, msa_stream_t stream) {
  msa_status_t s;
  if ((s = check_batch(batch)) != MSA_OK || (s = check_cfg(cfg)) != MSA_OK || (s = check_cache(cache, true, true)) != MSA_OK ||
      (s = check_query(index_q)) != MSA_OK || (s = check_query(q)) != MSA_OK)
    return s;
  if (!topk_idx || !out || !workspace || !aligned16(out)) return MSA_ERR_INVALID_ARGUMENT;
  Plan pl;
  if ((s = make_plan(cache, batch, cfg, num_q_heads, index_q->dtype == MSA_DTYPE_FP8_E4M3,
                     q->dtype == MSA_DTYPE_FP8_E4M3, pl)) != MSA_OK)
    return s;
  if (workspace_bytes < pl.total) return MSA_ERR_WORKSPACE_TOO_SMALL;
  if (pl.blk && (!aligned16(workspace) || !aligned4(batch->seq_lens, batch->block_table, topk_idx, lse)))
    return MSA_ERR_INVALID_ARGUMENT;
  cudaStream_t st = (cudaStream_t)stream;
  float* pooled = at<float>(workspace, pl.off_pooled);
  if ((s = run_indexer(cache, batch, cfg, index_q, pl, workspace, pooled, st, pl.pisel)) != MSA_OK) return s;
  if (pl.blk) return run_select_dense(cache, batch, cfg, q, num_q_heads, pooled, topk_idx, out, lse, pl, workspace, st);
  if (pl.k2q) {
    if ((s = pl.pisel ? run_pisel(batch, cfg, cache->num_kv_heads, topk_idx, pl, workspace, st)
                      : run_topk(batch, cfg, cache->num_kv_heads, pooled, topk_idx, nullptr, workspace, &pl, st, true,
                                 false, nullptr, true)) != MSA_OK)
      return s;
    return run_k2q(cache, batch, cfg, q, num_q_heads, topk_idx, out, lse, pl, workspace, st);
  }
  const FragJob fj = {cache, q, num_q_heads};
  if ((s = run_topk(batch, cfg, cache->num_kv_heads, pooled, topk_idx, nullptr, workspace, &pl, st, true, true,
                    pl.direct ? &fj : nullptr)) != MSA_OK)
    return s;
  return run_attend(cache, batch, cfg, q, num_q_heads, topk_idx, out, lse, pl, workspace, st, true);
}

msa_status_t msa_cache_insert(const msa_cache_t* cache, int32_t num_tokens, const int32_t* slot_mapping,
                              const void* k, const void* v, const void* index_k, void* workspace,
                              size_t workspace_bytes, msa_stream_t stream) {
  msa_status_t s;
  if ((s = check_cache(cache, index_k != nullptr, true)) != MSA_OK) return s;
  if (num_tokens < 0 || !workspace || !aligned4(workspace, slot_mapping)) return MSA_ERR_INVALID_ARGUMENT;
  if (cache->num_kv_heads > 8) return MSA_ERR_UNSUPPORTED;
  const bool blk = by_block(cache);  // K and V have an insert of their own
  if (blk && (k || v)) return MSA_ERR_UNSUPPORTED;
  if (workspace_bytes < 256) return MSA_ERR_WORKSPACE_TOO_SMALL;
  if (num_tokens == 0) return MSA_OK;
  if (!slot_mapping || (!blk && (!k || !v)) || !aligned16(k) || !aligned16(v) || (index_k && !aligned16(index_k)))
    return MSA_ERR_INVALID_ARGUMENT;
  InsertParams p;
  std::memset(&p, 0, sizeof(p));
  p.num_tokens = num_tokens;
  p.H = blk ? 0 : cache->num_kv_heads;
  p.num_blocks = cache->num_blocks;
  p.kv_fmt = blk ? FMT_BF16 : fmt_of(cache->kv_dtype);
  p.idx_fmt = index_k ? fmt_of(cache->index_dtype) : FMT_BF16;
  p.slots = slot_mapping;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.ik = static_cast<const __nv_bfloat16*>(index_k);
  // the insert writes through the cache's pointers
  p.kc = static_cast<uint8_t*>(const_cast<void*>(cache->k));
  p.vc = static_cast<uint8_t*>(const_cast<void*>(cache->v));
  p.ic = static_cast<uint8_t*>(const_cast<void*>(cache->idx));
  p.ks = const_cast<float*>(cache->k_scale);
  p.vs = const_cast<float*>(cache->v_scale);
  p.is = const_cast<float*>(cache->idx_scale);
  p.ksf = static_cast<uint8_t*>(const_cast<void*>(cache->k_sf));
  p.vsf = static_cast<uint8_t*>(const_cast<void*>(cache->v_sf));
  p.isf = static_cast<uint8_t*>(const_cast<void*>(cache->idx_sf));
  p.kg = cache->k_global;
  p.vg = cache->v_global;
  p.ig = cache->idx_global;
  p.status = static_cast<DeviceStatus*>(workspace);
  return cuda_status(launch_insert(p, sm_count(), (cudaStream_t)stream));
}

msa_status_t msa_block_insert(const msa_cache_t* cache, const msa_spans_t* spans, int32_t num_tokens,
                              const msa_rows_t* k, const msa_rows_t* v, void* workspace, size_t workspace_bytes,
                              msa_stream_t stream) {
  SpanParams p;
  const msa_status_t s = span_params(cache, spans, num_tokens, k, v, workspace, workspace_bytes, p);
  if (s != MSA_OK) return s;
  if (!by_block(cache)) return MSA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return MSA_OK;
  if (!rows_ok(k) || !rows_ok(v) || span_overlap(cache, spans, num_tokens, k, v, workspace, true))
    return MSA_ERR_INVALID_ARGUMENT;
  p.k_in = static_cast<const __nv_bfloat16*>(k->data);
  p.v_in = static_cast<const __nv_bfloat16*>(v->data);
  return cuda_status(launch_block_insert(p, kv_fmt_of(cache->kv_dtype), sm_count(), (cudaStream_t)stream));
}

msa_status_t msa_cache_read(const msa_cache_t* cache, const msa_spans_t* spans, int32_t num_tokens, const msa_rows_t* k,
                            const msa_rows_t* v, void* workspace, size_t workspace_bytes, msa_stream_t stream) {
  SpanParams p;
  const msa_status_t s = span_params(cache, spans, num_tokens, k, v, workspace, workspace_bytes, p);
  if (s != MSA_OK) return s;
  if (num_tokens == 0 || (!k && !v)) return MSA_OK;
  // the rows are written: heads side by side, no two tokens on top of each other
  const int64_t row = (int64_t)cache->num_kv_heads * kDim;
  if ((k && (!rows_ok(k) || (num_tokens > 1 && k->stride < row))) || (v && (!rows_ok(v) || (num_tokens > 1 && v->stride < row))) ||
      span_overlap(cache, spans, num_tokens, k, v, workspace, false))
    return MSA_ERR_INVALID_ARGUMENT;
  p.k_out = k ? static_cast<__nv_bfloat16*>(const_cast<void*>(k->data)) : nullptr;
  p.v_out = v ? static_cast<__nv_bfloat16*>(const_cast<void*>(v->data)) : nullptr;
  return cuda_status(launch_cache_read(p, kv_fmt_of(cache->kv_dtype), sm_count(), (cudaStream_t)stream));
}

size_t msa_dense_workspace_size(const msa_cache_t* cache, const msa_batch_t* batch, int32_t num_q_heads) {
  DensePlan pl;
  if (check_batch(batch) != MSA_OK || check_cache(cache, false, false) != MSA_OK ||
      make_dense_plan(cache, batch, num_q_heads, pl) != MSA_OK)
    return 0;
  return pl.total;
}

msa_status_t msa_dense_attend(const msa_cache_t* cache, const msa_batch_t* batch, const msa_config_t* cfg,
                              const msa_query_t* q, int32_t num_q_heads, void* out, float* lse, void* workspace,
                              size_t workspace_bytes, msa_stream_t stream) {
  msa_status_t s;
  if ((s = check_batch(batch)) != MSA_OK || (s = check_cfg(cfg)) != MSA_OK || (s = check_cache(cache, false, true)) != MSA_OK ||
      (s = check_query(q)) != MSA_OK)
    return s;
  if (!out || !workspace || !aligned16(out) || !aligned16(workspace) || !aligned4(batch->seq_lens, batch->block_table, lse))
    return MSA_ERR_INVALID_ARGUMENT;
  DensePlan pl;
  if ((s = make_dense_plan(cache, batch, num_q_heads, pl)) != MSA_OK) return s;
  if (workspace_bytes < pl.total) return MSA_ERR_WORKSPACE_TOO_SMALL;
  return run_dense(cache, batch, cfg, q, num_q_heads, nullptr, out, lse, pl, workspace, (cudaStream_t)stream);
}

msa_status_t msa_rope_init(msa_rope_t* rope, int32_t rotary_dim, double theta, int32_t axes, const int32_t* sections,
                           int32_t layout) {
  if (!rope || !sections || !(theta > 0.0) || !std::isfinite(theta)) return MSA_ERR_INVALID_ARGUMENT;
  if (axes < 1 || axes > MSA_ROPE_MAX_AXES || rotary_dim < 16 || rotary_dim > kDim || rotary_dim % 16 != 0)
    return MSA_ERR_UNSUPPORTED;
  std::memset(rope, 0, sizeof(*rope));
  rope->rotary_dim = rotary_dim;
  rope->axes = axes;
  rope->layout = layout;
  const int pairs = rotary_dim / 2;
  int i = 0;
  for (int a = 0; a < axes; ++a) {
    if (sections[a] < 0 || sections[a] > pairs - i) return MSA_ERR_INVALID_ARGUMENT;
    for (int k = 0; k < sections[a]; ++k) rope->axis[i++] = (uint8_t)a;
  }
  if (i != pairs) return MSA_ERR_INVALID_ARGUMENT;
  for (i = 0; i < pairs; ++i) {
    double turns = std::pow(theta, -2.0 * i / rotary_dim) / 6.283185307179586476925;
    turns -= std::floor(turns);  // whole turns change nothing (theta < 1)
    rope->turns[i] = (uint64_t)std::ldexp(turns, 64);
  }
  return check_rope(rope);
}

msa_status_t msa_rope_insert(const msa_cache_t* cache, const msa_rope_t* rope, int32_t num_tokens,
                             const int32_t* positions, const int32_t* slot_mapping, int32_t num_q_heads,
                             const msa_rows_t* q, const msa_query_t* q_out, const msa_rows_t* index_q,
                             const msa_query_t* index_q_out, const msa_rows_t* k, const msa_rows_t* v,
                             const msa_rows_t* index_k, const msa_qk_norm_t* norm, void* workspace,
                             size_t workspace_bytes, msa_stream_t stream) {
  msa_status_t s;
  if ((s = check_cache(cache, index_k != nullptr, true)) != MSA_OK || (s = check_rope(rope)) != MSA_OK) return s;
  if (num_tokens < 0 || !workspace || !aligned4(workspace, positions, slot_mapping)) return MSA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < 256) return MSA_ERR_WORKSPACE_TOO_SMALL;
  if (num_q_heads < 1 || num_q_heads > 1024) return MSA_ERR_UNSUPPORTED;
  const bool blk = by_block(cache);  // K and V have an insert of their own
  if (blk && (k || v)) return MSA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return MSA_OK;
  if (!positions || !slot_mapping || !rows_ok(q) || (!blk && (!rows_ok(k) || !rows_ok(v))) || (index_q && !rows_ok(index_q)) ||
      (index_k && !rows_ok(index_k)) || (index_q != nullptr) != (index_q_out != nullptr))
    return MSA_ERR_INVALID_ARGUMENT;
  if ((s = check_query(q_out)) != MSA_OK || (index_q && (s = check_query(index_q_out)) != MSA_OK)) return s;
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  p.rope = *rope;
  static_assert(MSA_ROPE_MAX_AXES <= 4, "two bits an axis");
  for (int i = 0; i < rope->rotary_dim / 2; ++i)
    for (int b = 0; b < 2; ++b) p.axis_bits[b][i >> 5] |= (uint32_t)(rope->axis[i] >> b & 1) << (i & 31);
  p.num_tokens = num_tokens;
  p.Hq = num_q_heads;
  p.H = blk ? 0 : cache->num_kv_heads;
  p.Giq = index_q ? cache->num_kv_heads : 0;
  p.Gik = index_k ? 1 : 0;
  p.num_blocks = cache->num_blocks;
  p.kv_fmt = blk ? FMT_BF16 : fmt_of(cache->kv_dtype);
  p.idx_fmt = index_k ? fmt_of(cache->index_dtype) : FMT_BF16;
  p.positions = positions;
  p.slots = slot_mapping;
  p.q = static_cast<const __nv_bfloat16*>(q->data);
  p.q_stride = q->stride;
  if (!blk) {
    p.k = static_cast<const __nv_bfloat16*>(k->data);
    p.k_stride = k->stride;
    p.v = static_cast<const __nv_bfloat16*>(v->data);
    p.v_stride = v->stride;
  }
  if (index_q) {
    p.iq = static_cast<const __nv_bfloat16*>(index_q->data);
    p.iq_stride = index_q->stride;
    p.iq_out = static_cast<uint8_t*>(const_cast<void*>(index_q_out->data));
    p.iq_fp8 = index_q_out->dtype == MSA_DTYPE_FP8_E4M3;
    p.iq_inv = p.iq_fp8 ? 1.f / index_q_out->scale : 1.f;
  }
  if (index_k) {
    p.ik = static_cast<const __nv_bfloat16*>(index_k->data);
    p.ik_stride = index_k->stride;
  }
  p.q_out = static_cast<uint8_t*>(const_cast<void*>(q_out->data));
  p.q_fp8 = q_out->dtype == MSA_DTYPE_FP8_E4M3;
  p.q_inv = p.q_fp8 ? 1.f / q_out->scale : 1.f;
  if (!std::isfinite(p.q_inv) || !std::isfinite(p.iq_inv)) return MSA_ERR_INVALID_ARGUMENT;
  if (norm) {
    const void* w[4] = {norm->q, norm->index_q, norm->k, norm->index_k};
    if (!(norm->eps >= 0.f) || !std::isfinite(norm->eps) || !std::isfinite(norm->offset)) return MSA_ERR_INVALID_ARGUMENT;
    for (int i = 0; i < 4; ++i) {
      if (w[i] && !aligned16(w[i])) return MSA_ERR_INVALID_ARGUMENT;
      p.w[i] = static_cast<const __nv_bfloat16*>(w[i]);
    }
    p.eps = norm->eps;
    p.w_offset = norm->offset;
  }
  // the insert writes through the cache's pointers
  p.kc = static_cast<uint8_t*>(const_cast<void*>(cache->k));
  p.vc = static_cast<uint8_t*>(const_cast<void*>(cache->v));
  p.ic = static_cast<uint8_t*>(const_cast<void*>(cache->idx));
  p.ks = const_cast<float*>(cache->k_scale);
  p.vs = const_cast<float*>(cache->v_scale);
  p.is = const_cast<float*>(cache->idx_scale);
  p.ksf = static_cast<uint8_t*>(const_cast<void*>(cache->k_sf));
  p.vsf = static_cast<uint8_t*>(const_cast<void*>(cache->v_sf));
  p.isf = static_cast<uint8_t*>(const_cast<void*>(cache->idx_sf));
  p.kg = cache->k_global;
  p.vg = cache->v_global;
  p.ig = cache->idx_global;
  p.status = static_cast<DeviceStatus*>(workspace);
  return cuda_status(launch_rope(p, sm_count(), (cudaStream_t)stream));
}

msa_status_t msa_build_tables(int32_t num_seqs, int32_t num_blocks, const int32_t* cached_lens, const int32_t* new_lens,
                              int32_t max_blocks_per_seq, int32_t* block_table, int32_t free_capacity,
                              int32_t* free_blocks, const int32_t* free_count, int32_t* free_count_out,
                              int32_t* seq_lens, int32_t* token_offsets, int32_t max_tokens, int32_t* slot_mapping,
                              int32_t* positions, void* workspace, size_t workspace_bytes, msa_stream_t stream) {
  if (num_seqs < 1 || num_blocks < 1 || max_blocks_per_seq < 1 || free_capacity < 0 || max_tokens < 0)
    return MSA_ERR_INVALID_ARGUMENT;
  if (num_seqs > kMaxTableSeqs || (long)num_blocks * kBlock >= (1l << 31) || (long)max_blocks_per_seq * kBlock > (1l << 30) ||
      free_capacity >= (1 << 30) || max_tokens >= (1 << 30))
    return MSA_ERR_UNSUPPORTED;
  if (!cached_lens || !new_lens || !block_table || !free_count || !free_count_out || !seq_lens || !token_offsets ||
      !workspace || (free_capacity > 0 && !free_blocks) || (max_tokens > 0 && (!slot_mapping || !positions)))
    return MSA_ERR_INVALID_ARGUMENT;
  if (!aligned4(cached_lens, new_lens, block_table, free_blocks, free_count, free_count_out, seq_lens, token_offsets, slot_mapping,
                positions, workspace))
    return MSA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < 256) return MSA_ERR_WORKSPACE_TOO_SMALL;
  // the CTAs read the inputs while others write: what is written overlaps nothing else
  const struct {
    const int32_t* p;
    size_t n;
  } words[] = {{free_count_out, 1}, {seq_lens, (size_t)num_seqs}, {token_offsets, (size_t)num_seqs + 1},
               {slot_mapping, (size_t)max_tokens}, {positions, (size_t)max_tokens},
               {block_table, (size_t)num_seqs * max_blocks_per_seq}, {free_blocks, (size_t)free_capacity},
               {static_cast<const int32_t*>(workspace), sizeof(DeviceStatus) / 4},
               {free_count, 1}, {cached_lens, (size_t)num_seqs}, {new_lens, (size_t)num_seqs}};
  for (int i = 0; i < 8; ++i)  // written: the first eight
    for (int j = i + 1; j < 11; ++j)
      if (words[i].n > 0 && words[j].n > 0 && words[i].p < words[j].p + words[j].n && words[j].p < words[i].p + words[i].n)
        return MSA_ERR_INVALID_ARGUMENT;
  TablesParams p;
  p.num_seqs = num_seqs;
  p.num_blocks = num_blocks;
  p.max_nb = max_blocks_per_seq;
  p.free_cap = free_capacity;
  p.max_tokens = max_tokens;
  p.cached = cached_lens;
  p.fresh = new_lens;
  p.block_table = block_table;
  p.free_blocks_in = free_blocks;
  p.free_blocks = free_blocks;
  p.free_count = free_count;
  p.free_count_out = free_count_out;
  p.seq_lens = seq_lens;
  p.offsets = token_offsets;
  p.slots = slot_mapping;
  p.positions = positions;
  p.status = static_cast<DeviceStatus*>(workspace);
  return cuda_status(launch_tables(p, sm_count(), (cudaStream_t)stream));
}

msa_status_t msa_read_device_status(void* workspace, msa_stream_t stream, int32_t* detail) {
  if (!workspace) return MSA_ERR_INVALID_ARGUMENT;
  DeviceStatus h = {0, 0};
  cudaStream_t st = (cudaStream_t)stream;
  if (cudaMemcpyAsync(&h, workspace, sizeof(h), cudaMemcpyDeviceToHost, st) != cudaSuccess) return MSA_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return MSA_ERR_CUDA;
  if (cudaMemsetAsync(workspace, 0, sizeof(h), st) != cudaSuccess) return MSA_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return MSA_ERR_CUDA;
  if (detail) *detail = (int32_t)h.flags;
  if (h.flags & FLAG_TIMEOUT) return MSA_ERR_TIMEOUT;
  if (h.flags) return MSA_ERR_DEVICE_FAULT;
  return MSA_OK;
}

msa_status_t msa_dequant_debug(const msa_cache_t* cache, int32_t which, const int32_t* phys_blocks, int32_t n,
                               float* out, msa_stream_t stream) {
  if (which < 0 || which > 2 || n < 0 || (n > 0 && (!phys_blocks || !out))) return MSA_ERR_INVALID_ARGUMENT;
  msa_status_t s = check_cache(cache, which == 2, which != 2);
  if (s != MSA_OK) return s;
  const int f = which == 2 ? fmt_of(cache->index_dtype) : kv_fmt_of(cache->kv_dtype);
  return cuda_status(launch_dequant(f, which, *cache, phys_blocks, n, out, (cudaStream_t)stream));
}

}  // extern "C"

// ====================================================================== allocation-free decode
//
// Some callers cannot allocate device memory for a workspace: code that runs
// inside another framework's memory pool or allocator hooks, a plugin that
// must not call cudaMalloc (or torch's allocator) on its hot path, or a
// process whose device memory is fully reserved up front.  msa_decode_noalloc
// serves them with a fixed scratch area that lives in the library itself: the
// array below is part of the library's device image, so every GPU that loads
// libmsa holds these bytes until the process exits.

// MSA_NOALLOC_SCRATCH_BYTES (include/msa.h): the largest workspace it accepts.
static __device__ __align__(256) unsigned char msa_noalloc_scratch[MSA_NOALLOC_SCRATCH_BYTES];

namespace {

// Device address of msa_noalloc_scratch on the current device, looked up once
// per device (the host-side symbol is only a stand-in, never a device address).
// The cached address assumes the device's context lives as long as the
// process: a device reset (cudaDeviceReset) is not supported afterwards.
msa_status_t noalloc_scratch(void** out) {
  static std::mutex mu;
  static void* addr[64];
  static bool have[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MSA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  if (!have[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, msa_noalloc_scratch) != cudaSuccess || p == nullptr) return MSA_ERR_CUDA;
    addr[dev] = p;
    have[dev] = true;
  }
  *out = addr[dev];
  return MSA_OK;
}

}  // namespace

extern "C" msa_status_t msa_decode_noalloc(const msa_cache_t* cache, const msa_batch_t* batch,
                                           const msa_config_t* cfg, const msa_query_t* index_q,
                                           const msa_query_t* q, int32_t num_q_heads, int32_t* topk_idx,
                                           void* out, float* lse, int32_t* status_out, msa_stream_t stream) {
  msa_status_t s;
  if ((s = check_batch(batch)) != MSA_OK || (s = check_cfg(cfg)) != MSA_OK || (s = check_cache(cache, true, true)) != MSA_OK ||
      (s = check_query(index_q)) != MSA_OK || (s = check_query(q)) != MSA_OK)
    return s;
  if (!topk_idx || !out || !aligned16(out)) return MSA_ERR_INVALID_ARGUMENT;
  Plan pl;
  if ((s = make_plan(cache, batch, cfg, num_q_heads, index_q->dtype == MSA_DTYPE_FP8_E4M3,
                     q->dtype == MSA_DTYPE_FP8_E4M3, pl)) != MSA_OK)
    return s;
  if (pl.total > MSA_NOALLOC_SCRATCH_BYTES && pl.pisel &&
      (s = make_plan(cache, batch, cfg, num_q_heads, index_q->dtype == MSA_DTYPE_FP8_E4M3,
                     q->dtype == MSA_DTYPE_FP8_E4M3, pl, false)) != MSA_OK)  // pooled scores may still fit
    return s;
  if (pl.total > MSA_NOALLOC_SCRATCH_BYTES) return MSA_ERR_WORKSPACE_TOO_SMALL;
  if (pl.blk && !aligned4(batch->seq_lens, batch->block_table, topk_idx, lse)) return MSA_ERR_INVALID_ARGUMENT;
  void* ws = nullptr;
  if ((s = noalloc_scratch(&ws)) != MSA_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  // the status word must start at zero; every other region is written before it is read
  if (cudaMemsetAsync(ws, 0, 256, st) != cudaSuccess) return MSA_ERR_CUDA;
  float* pooled = at<float>(ws, pl.off_pooled);
  if ((s = run_indexer(cache, batch, cfg, index_q, pl, ws, pooled, st, pl.pisel)) != MSA_OK) return s;
  if (pl.blk) {
    if ((s = run_select_dense(cache, batch, cfg, q, num_q_heads, pooled, topk_idx, out, lse, pl, ws, st)) != MSA_OK) return s;
  } else if (pl.k2q) {
    // a prefill chunk over an FP8 cache: the same chain as msa_decode's
    if ((s = pl.pisel ? run_pisel(batch, cfg, cache->num_kv_heads, topk_idx, pl, ws, st)
                      : run_topk(batch, cfg, cache->num_kv_heads, pooled, topk_idx, nullptr, ws, &pl, st, true, false,
                                 nullptr, true)) != MSA_OK)
      return s;
    if ((s = run_k2q(cache, batch, cfg, q, num_q_heads, topk_idx, out, lse, pl, ws, st)) != MSA_OK) return s;
  } else {
    const FragJob fj = {cache, q, num_q_heads};
    if ((s = run_topk(batch, cfg, cache->num_kv_heads, pooled, topk_idx, nullptr, ws, &pl, st, true, true,
                      pl.direct ? &fj : nullptr)) != MSA_OK)
      return s;
    if ((s = run_attend(cache, batch, cfg, q, num_q_heads, topk_idx, out, lse, pl, ws, st, true)) != MSA_OK)
      return s;
  }
  if (status_out &&
      cudaMemcpyAsync(status_out, ws, 2 * sizeof(int32_t), cudaMemcpyDeviceToDevice, st) != cudaSuccess)
    return MSA_ERR_CUDA;
  return MSA_OK;
}
