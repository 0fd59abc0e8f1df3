// Dense attend over FP8 caches (msa_dense.cuh).
#include "msa_dense.cuh"

namespace msa {

namespace {

// E4M3 queries as they are; bf16 ones as two e4m3 terms (in the spare rows of
// the tile, or by a second MMA), and against K widened to f16 where the second
// MMA would make the tensor pipe the bound (more than 16 columns).
template <int NN, int NCG>
cudaError_t launch(const CUtensorMap* tk, const CUtensorMap* tv, const DenseParams& p, int num_sms, cudaStream_t st) {
  if constexpr (NN == 1) return dense::launch_one<FMT_FP8, NN, NCG, QM_ROWS, false>(tk, tv, p, num_sms, st);
  else if (p.q_fp8) return dense::launch_one<FMT_FP8, NN, NCG, QM_E4, false>(tk, tv, p, num_sms, st);
  else return dense::launch_one<FMT_FP8, NN, NCG, NN == 2 ? QM_E4X2 : QM_F16K, false>(tk, tv, p, num_sms, st);
}

}  // namespace

cudaError_t launch_dense_fp8(const CUtensorMap* tk, const CUtensorMap* tv, const DenseParams& p, int num_sms,
                             cudaStream_t st) {
  const DenseShape sh = dense_shape(p.cper);
  if (sh.ncg == 2) return sh.nn == 3 ? launch<3, 2>(tk, tv, p, num_sms, st) : launch<4, 2>(tk, tv, p, num_sms, st);
  switch (sh.nn) {
    case 1: return launch<1, 1>(tk, tv, p, num_sms, st);
    case 2: return launch<2, 1>(tk, tv, p, num_sms, st);
    case 3: return launch<3, 1>(tk, tv, p, num_sms, st);
    default: return launch<4, 1>(tk, tv, p, num_sms, st);
  }
}

}  // namespace msa
