// decode_scores.cu -- the partial kernel of the CUDA-core decode that also
// leaves the score of every row and query head, for a weighing decode
// (evict.cu turns them into weights once the row's LSE is known).  A file of
// its own: it compiles beside decode.cu.
#include "decode_partial.cuh"

namespace pkv {

template <typename T, int D>
static cudaError_t dispatch_group_scores(int group, const CUtensorMap& tmk, const CUtensorMap& tmv,
                                         const DecodeArgs& a, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_partial<T, D, 1, true>(tmk, tmv, a, stream);
    case 2: return launch_partial<T, D, 2, true>(tmk, tmv, a, stream);
    case 4: return launch_partial<T, D, 4, true>(tmk, tmv, a, stream);
    case 8:
      if constexpr (!kIsMx<T>) return launch_partial<T, D, 8, true>(tmk, tmv, a, stream);
      return cudaErrorInvalidValue;
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_decode_partial_scores(int dtype, int head_dim, int group, const CUtensorMap& tmk,
                                         const CUtensorMap& tmv, const DecodeArgs& a,
                                         cudaStream_t stream) {
  if (dtype == PKV_MXFP8)
    return head_dim == 128 ? dispatch_group_scores<__nv_fp8_e4m3, 128>(group, tmk, tmv, a, stream)
                           : dispatch_group_scores<__nv_fp8_e4m3, 64>(group, tmk, tmv, a, stream);
  if (dtype == PKV_BF16)
    return head_dim == 128 ? dispatch_group_scores<__nv_bfloat16, 128>(group, tmk, tmv, a, stream)
                           : dispatch_group_scores<__nv_bfloat16, 64>(group, tmk, tmv, a, stream);
  return head_dim == 128 ? dispatch_group_scores<float, 128>(group, tmk, tmv, a, stream)
                         : dispatch_group_scores<float, 64>(group, tmk, tmv, a, stream);
}

}  // namespace pkv
