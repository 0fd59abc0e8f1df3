// Dense attend over INT8 caches with block scales (msa_dense.cuh).
#include "msa_dense.cuh"

namespace msa {

cudaError_t launch_dense_int8(const CUtensorMap* tk, const CUtensorMap* tv, const DenseParams& p, int num_sms, cudaStream_t st) {
  return dense::launch_shape<FMT_I8B, false>(tk, tv, p, num_sms, st);
}

}  // namespace msa
