// decode_window.cu -- the decode of fp32 pools under a sliding window with sinks, on
// the CUDA cores: of T rows the first S and the last W are seen.  (bf16 and MXFP8
// pools: window_mma.cu.)
//
// The work split and the walk count only boxes that hold a row that is seen
// (plan.cuh); boxes without one are not loaded, so their blocks may have been given
// back.  Two splits of the partial kernel (decode_partial.cuh):
//   * balanced, as the plain decode's, for long windows: persistent CTAs, a scan
//     of the lengths, pieces cut anywhere and the plain decode's reduction;
//   * direct, for short ones, where no sequence shows many rows: a CTA takes
//     an equal part of one segment's stages and asks nothing but its length.  There is no
//     scan, and where segments alone fill the GPU no merge either: a CTA writes its segment.
// The merge of the direct split's parts serves window_mma.cu too.  A file of its
// own: it compiles beside decode.cu.
#include "decode_partial.cuh"

namespace pkv {

namespace {

// Merge the parts of each (sequence, query head)'s segment, or what its clusters
// made of them, by log-sum-exp, a warp each; segments that one CTA or cluster had
// whole, and empty ones, are written already.
template <typename T, int D>
__global__ void __launch_bounds__(128) window_merge_kernel(const WindowArgs a) {
  constexpr int EPL = D / 32;
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t rh = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (rh >= (int64_t)a.num_seqs * a.num_q_heads) return;
  const int r = (int)(rh / a.num_q_heads), qh = (int)(rh - (int64_t)r * a.num_q_heads);
  const int G = a.num_q_heads / a.num_kv_heads;
  const int nt = (plan_len(a, r, a.block_size, false) + kStageRows - 1) / kStageRows;
  // a record of each part (as direct_stages), or of each cluster of them
  const int w = (nt + a.parts - 1) / a.parts, each = max(a.cluster, 1);
  const int n = nt ? (nt + w * each - 1) / (w * each) : 0;
  if (n < 2) return;
  const int64_t rec0 = ((int64_t)r * a.num_kv_heads + qh / G) * (a.parts / each);
  auto rec = [&](int i) { return 2 * (rec0 + i) * G + qh % G; };
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) {
    const float l = a.rec_lse[rec(i)];
    M = fmaxf(M, l != l ? INFINITY : l);  // NaN is not passed over
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float acc[EPL] = {}, sum = 0.f;
  if (M != -INFINITY) {
    for (int i0 = 0; i0 < n; i0 += kMergeBatch) {
      float l[kMergeBatch], x[kMergeBatch][EPL];
#pragma unroll
      for (int u = 0; u < kMergeBatch; ++u) {
        l[u] = i0 + u < n ? a.rec_lse[rec(i0 + u)] : -INFINITY;
#pragma unroll
        for (int e = 0; e < EPL; ++e) x[u][e] = 0.f;
        if (i0 + u < n) VecLoad<float, EPL>::run(a.rec_o + rec(i0 + u) * D + lane * EPL, x[u]);
      }
#pragma unroll
      for (int u = 0; u < kMergeBatch; ++u) {
        if (l[u] == -INFINITY) continue;
        const float wt = exp2f(l[u] - M);
        sum += wt;
#pragma unroll
        for (int e = 0; e < EPL; ++e) acc[e] = fmaf(wt, x[u][e], acc[e]);
      }
    }
  }
  const bool nonempty = sum != 0.f;  // NaN stays
  T* out = static_cast<T*>(a.out) + rh * D + lane * EPL;
#pragma unroll
  for (int e = 0; e < EPL; ++e) store_out(out + e, nonempty ? acc[e] / sum : 0.f);
  if (lane == 0 && a.lse_out) a.lse_out[rh] = nonempty ? (M + log2f(sum)) * kLn2 : -INFINITY;
}

template <int D, int G>
cudaError_t launch_group(const CUtensorMap& tmk, const CUtensorMap& tmv, const WindowArgs& a,
                         cudaStream_t stream) {
  return a.parts ? launch_partial<float, D, G, false, true, true>(tmk, tmv, a, stream)
                 : launch_partial<float, D, G, false, true, false>(tmk, tmv, a, stream);
}

template <int D>
cudaError_t launch_dim(int group, const CUtensorMap& tmk, const CUtensorMap& tmv, const WindowArgs& a,
                       cudaStream_t stream) {
  cudaError_t e;
  switch (group) {
    case 1: e = launch_group<D, 1>(tmk, tmv, a, stream); break;
    case 2: e = launch_group<D, 2>(tmk, tmv, a, stream); break;
    case 4: e = launch_group<D, 4>(tmk, tmv, a, stream); break;
    case 8: e = launch_group<D, 8>(tmk, tmv, a, stream); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess || a.parts == 1) return e;
  return a.parts ? launch_window_merge(PKV_F32, D, a, stream) : launch_decode_reduce(PKV_F32, D, a, stream);
}

template <typename T>
cudaError_t merge(int head_dim, const WindowArgs& a, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.num_seqs * a.num_q_heads;
  return launch_pdl(head_dim == 128 ? window_merge_kernel<T, 128> : window_merge_kernel<T, 64>,
                    dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, stream, a);
}

}  // namespace

cudaError_t launch_window_merge(int dtype, int head_dim, const WindowArgs& a, cudaStream_t stream) {
  return dtype == PKV_F32 ? merge<float>(head_dim, a, stream) : merge<__nv_bfloat16>(head_dim, a, stream);
}

cudaError_t launch_decode_window(int head_dim, int group, const CUtensorMap& tmk, const CUtensorMap& tmv,
                                 const DecodeArgs& args, cudaStream_t stream) {
  const WindowArgs a(args, box_rows_for(args.block_size));
  return head_dim == 128 ? launch_dim<128>(group, tmk, tmv, a, stream)
                         : launch_dim<64>(group, tmk, tmv, a, stream);
}

}  // namespace pkv
