// Dense attend over NVFP4 caches (products rounded to E4M3, MSA_NVFP4_E4M3_PRODUCT; msa_dense.cuh).
#include "msa_dense.cuh"

namespace msa {

cudaError_t launch_dense_nvfp4_rounded(const CUtensorMap* tk, const CUtensorMap* tv, const DenseParams& p, int num_sms,
                               cudaStream_t st) {
  const DenseShape sh = dense_shape(p.cper);
  if (sh.ncg == 2) return sh.nn == 3 ? dense::launch_one<FMT_NVFP4, 3, 2, true>(tk, tv, p, num_sms, st)
                                      : dense::launch_one<FMT_NVFP4, 4, 2, true>(tk, tv, p, num_sms, st);
  switch (sh.nn) {
    case 1: return dense::launch_one<FMT_NVFP4, 1, 1, true>(tk, tv, p, num_sms, st);
    case 2: return dense::launch_one<FMT_NVFP4, 2, 1, true>(tk, tv, p, num_sms, st);
    case 3: return dense::launch_one<FMT_NVFP4, 3, 1, true>(tk, tv, p, num_sms, st);
    default: return dense::launch_one<FMT_NVFP4, 4, 1, true>(tk, tv, p, num_sms, st);
  }
}

}  // namespace msa
