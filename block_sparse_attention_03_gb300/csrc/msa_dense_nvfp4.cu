// Dense attend over NVFP4 caches (msa_dense.cuh).
#include "msa_dense.cuh"

namespace msa {

namespace {

template <bool NVR>
cudaError_t launch(const CUtensorMap* tk, const CUtensorMap* tv, const DenseParams& p, int num_sms, cudaStream_t st) {
  switch (dense_nt(p.cols)) {
    case 0: return dense::launch_one<FMT_NVFP4, 1, true, 1, NVR>(tk, tv, p, num_sms, st);
    case 1: return dense::launch_one<FMT_NVFP4, 1, false, 1, NVR>(tk, tv, p, num_sms, st);
    case 2: return dense::launch_one<FMT_NVFP4, 2, false, 1, NVR>(tk, tv, p, num_sms, st);
    default: return dense::launch_one<FMT_NVFP4, 4, false, 1, NVR>(tk, tv, p, num_sms, st);
  }
}

}  // namespace

cudaError_t launch_dense_nvfp4(const CUtensorMap* tk, const CUtensorMap* tv, const DenseParams& p, int num_sms,
                               bool round_e4m3, cudaStream_t st) {
  return round_e4m3 ? launch<true>(tk, tv, p, num_sms, st) : launch<false>(tk, tv, p, num_sms, st);
}

}  // namespace msa
