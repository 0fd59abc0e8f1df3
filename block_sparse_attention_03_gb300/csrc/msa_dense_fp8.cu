// Dense attend over FP8 caches (msa_dense.cuh).
#include "msa_dense.cuh"

namespace msa {

cudaError_t launch_dense_fp8(const CUtensorMap* tk, const CUtensorMap* tv, const DenseParams& p, int num_sms,
                             cudaStream_t st) {
  // a bf16 query of more than 8 columns needs a second MMA for its lo terms
  const bool two = !p.q_fp8;
  switch (dense_nt(p.cols)) {
    case 0: return dense::launch_one<FMT_FP8, 1, true, 1, false>(tk, tv, p, num_sms, st);
    case 1:
      return two ? dense::launch_one<FMT_FP8, 1, false, 2, false>(tk, tv, p, num_sms, st)
                 : dense::launch_one<FMT_FP8, 1, false, 1, false>(tk, tv, p, num_sms, st);
    case 2:
      return two ? dense::launch_one<FMT_FP8, 2, false, 2, false>(tk, tv, p, num_sms, st)
                 : dense::launch_one<FMT_FP8, 2, false, 1, false>(tk, tv, p, num_sms, st);
    default:
      return two ? dense::launch_one<FMT_FP8, 4, false, 2, false>(tk, tv, p, num_sms, st)
                 : dense::launch_one<FMT_FP8, 4, false, 1, false>(tk, tv, p, num_sms, st);
  }
}

}  // namespace msa
