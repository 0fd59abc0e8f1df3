// Dense attend over FP8 caches (msa_dense.cuh).
#include "msa_dense.cuh"

namespace msa {

namespace {

template <int NN, int NCG>
cudaError_t launch(const CUtensorMap* tk, const CUtensorMap* tv, const DenseParams& p, int num_sms, cudaStream_t st) {
  return dense::launch_one<FMT_FP8, NN, NCG, false>(tk, tv, p, num_sms, st);
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
