// Dense attend over BF16 caches (msa_dense.cuh).
#include "msa_dense.cuh"

namespace msa {

cudaError_t launch_dense_bf16(const CUtensorMap* tk, const CUtensorMap* tv, const DenseParams& p, int num_sms,
                              cudaStream_t st) {
  const DenseShape sh = dense_shape(p.cper);
  if (sh.ncg == 2) return sh.nn == 3 ? dense::launch_one<FMT_BF16, 3, 2, false>(tk, tv, p, num_sms, st)
                                      : dense::launch_one<FMT_BF16, 4, 2, false>(tk, tv, p, num_sms, st);
  switch (sh.nn) {
    case 1: return dense::launch_one<FMT_BF16, 1, 1, false>(tk, tv, p, num_sms, st);
    case 2: return dense::launch_one<FMT_BF16, 2, 1, false>(tk, tv, p, num_sms, st);
    case 3: return dense::launch_one<FMT_BF16, 3, 1, false>(tk, tv, p, num_sms, st);
    default: return dense::launch_one<FMT_BF16, 4, 1, false>(tk, tv, p, num_sms, st);
  }
}

}  // namespace msa
