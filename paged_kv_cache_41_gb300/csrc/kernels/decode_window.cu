// decode_window.cu -- the partial kernel of the CUDA-core decode under a sliding
// window with sinks: of T rows the first S and the last W are seen.  The work
// split and the walk count only stages that hold a row that is seen (plan.cuh);
// boxes without one are not loaded, so their blocks may have been given back.
// A file of its own: it compiles beside decode.cu.
#include "decode_partial.cuh"

namespace pkv {

template <typename T, int D>
static cudaError_t dispatch_group_window(int group, const CUtensorMap& tmk, const CUtensorMap& tmv,
                                         const WindowArgs& a, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_partial<T, D, 1, false, true>(tmk, tmv, a, stream);
    case 2: return launch_partial<T, D, 2, false, true>(tmk, tmv, a, stream);
    case 4: return launch_partial<T, D, 4, false, true>(tmk, tmv, a, stream);
    case 8:
      if constexpr (!kIsMx<T>) return launch_partial<T, D, 8, false, true>(tmk, tmv, a, stream);
      return cudaErrorInvalidValue;
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_decode_partial_window(int dtype, int head_dim, int group, const CUtensorMap& tmk,
                                         const CUtensorMap& tmv, const DecodeArgs& args,
                                         cudaStream_t stream) {
  const WindowArgs a(args, kStageRows);
  if (dtype == PKV_MXFP8)
    return head_dim == 128 ? dispatch_group_window<__nv_fp8_e4m3, 128>(group, tmk, tmv, a, stream)
                           : dispatch_group_window<__nv_fp8_e4m3, 64>(group, tmk, tmv, a, stream);
  if (dtype == PKV_BF16)
    return head_dim == 128 ? dispatch_group_window<__nv_bfloat16, 128>(group, tmk, tmv, a, stream)
                           : dispatch_group_window<__nv_bfloat16, 64>(group, tmk, tmv, a, stream);
  return head_dim == 128 ? dispatch_group_window<float, 128>(group, tmk, tmv, a, stream)
                         : dispatch_group_window<float, 64>(group, tmk, tmv, a, stream);
}

}  // namespace pkv
