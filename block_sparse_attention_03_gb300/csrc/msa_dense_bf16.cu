// Dense attend over BF16 caches (msa_dense.cuh).
#include "msa_dense.cuh"

namespace msa {

cudaError_t launch_dense_bf16(const CUtensorMap* tk, const CUtensorMap* tv, const DenseParams& p, int num_sms,
                              cudaStream_t st) {
  switch (dense_nt(p.cols)) {
    case 0: return dense::launch_one<FMT_BF16, 1, true, 1, false>(tk, tv, p, num_sms, st);
    case 1: return dense::launch_one<FMT_BF16, 1, false, 1, false>(tk, tv, p, num_sms, st);
    case 2: return dense::launch_one<FMT_BF16, 2, false, 1, false>(tk, tv, p, num_sms, st);
    default: return dense::launch_one<FMT_BF16, 4, false, 1, false>(tk, tv, p, num_sms, st);
  }
}

}  // namespace msa
