// decode.cu -- split-K paged attention decode on CUDA cores (GQA groups <= 8).
//
// What it computes ("M5.3 - KV Memory Layout and Exact Reuse", 0x0A and
// 0x0BA): for sequence r and query head h, attention of q[r, h] over the
// request-visible rows t < T_r of kv head h / G, where row t lives in physical
// block block_tables[r, t / P] at offset t % P.  The rows of one (sequence,
// kv head) are cut into pieces; each piece keeps an online softmax state
// (m, l, u) and emits (O_p = u / l, LSE_p = m + log l); pieces are merged by
// log-sum-exp, never by averaging normalised outputs, with empty pieces as
// the identity.
//
// Design (GB300):
//   * persistent, balanced CTAs: the work is the list of 32-row stages of
//     every (sequence, kv head) segment, sequence-major; every CTA scans the
//     lengths itself (a block-wide prefix sum, no planning launch), and CTA c
//     of C (one wave: four per SM) takes the c-th equal share of the work
//     units (plan.cuh: a stage costs two, a piece's fixed cost three).  Every
//     CTA does the same work whatever the length mix, there is no tail wave,
//     and a CTA crosses segment boundaries without draining its pipeline;
//   * a segment a CTA covers whole is finished there (output written
//     directly); a segment cut by CTA boundaries leaves one (O, LSE) record
//     per piece -- at most two per CTA, for its first and last segments --
//     and a reduction kernel merges them;
//   * the G query heads of a kv head share every K/V byte the CTA reads;
//   * warp 0 also issues the loads: it walks the CTA's stages, holds the
//     current sequence's block ids 32 at a time (one coalesced load per 32
//     blocks, the next group in flight), and fills each 32-row stage with 4-D
//     TMA boxes (one block, or a 32-row slice of a larger block, of one kv
//     head) for K and V, tracked by mbarriers, plus a small descriptor of the
//     stage (sequence, head, valid rows, piece start / end) for the
//     consumers; a stage is refilled as soon as all four warps released it;
//   * warps consume 16-row chunks: each half-warp owns two token rows, each
//     lane 1/16 of head_dim; the 2G (row, head) partial dot products are
//     summed across the 16 lanes through a small per-warp shared scratch;
//     the row lands in lane bit 3; a vote on each lane's own score decides
//     whether the chunk needs the max over the warp's four rows (two
//     shuffles) and a rescale, and each lane sums its own rows' weights until
//     the piece end adds them; q . k and P . V use packed fp32x2 FMAs;
//   * full stages take a straight-line path with no row masking;
//   * at a piece's end the four warps merge through the stage's own tile
//     (released only afterwards), so the ring keeps streaming the next piece;
//   * the exponent base is only moved when the running max grows by more than
//     2^8 (exact: output and denominator keep the same base), so the
//     accumulator rescale is rare;
//   * scores are in base 2 (q is pre-multiplied by scale * log2 e);
//   * rows past the request's tail are never multiplied in, so stale or NaN
//     bytes in a recycled block cannot leak (M5.3 0x03G).
#include "decode_partial.cuh"

namespace pkv {

int decode_num_stages(int head_dim, int elem_bytes) {
  const int stage_bytes = 2 * kStageRows * head_dim * elem_bytes;
  int ns = (49 * 1024) / stage_bytes;  // 3 stages of 16 KiB: 4 CTAs per SM
  if (ns < 2) ns = 2;
  if (ns > 8) ns = 8;
  return ns;
}

// One warp per (sequence, query head): merge the pieces of its segment (and,
// in states mode, the extra states before them) by log-sum-exp.  A segment
// one CTA covered whole was written by that CTA (plain mode: nothing to do).
template <typename T, int D>
__global__ void __launch_bounds__(128) decode_reduce_kernel(const DecodeArgs a) {
  constexpr int EPL = D / 32;
  pdl_wait();  // the partial kernel's records and plan are complete
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t rh = (int64_t)blockIdx.x * 4 + warp;
  if (rh >= (int64_t)a.num_seqs * a.num_q_heads) return;
  const int r = (int)(rh / a.num_q_heads), qh = (int)(rh % a.num_q_heads);
  const int G = a.num_q_heads / a.num_kv_heads, h = qh / G, g = qh % G;
  const int Hkv = a.num_kv_heads, C = a.num_ctas;
  // the work split of plan.cuh, in units: segment (r, h) starts at unit
  // seg0, its stage i at seg0 + pu + su i, owned by CTA (start) / w
  const long long su = a.stage_units, pu = a.piece_units;
  const long long S = a.plan_pre[a.num_seqs] * Hkv;
  const long long pre = a.plan_pre[r], u = a.plan_pre[r + 1] - pre;
  const long long nt = u > 0 ? (u - pu) / su : 0;
  const int n_ext = a.st_o ? a.st_slot : 0;
  // Sources: extra states [0, n_ext), then either the whole-segment state
  // (states mode) or pieces c_first..c_last.
  const long long w = units_per_cta(S, C, su);
  int c_first = 0, n_pc = 0;  // pieces: CTAs c_first .. c_first + n_pc - 1
  bool whole_state = false;
  bool first_is_slot1 = false;
  if (nt > 0) {
    const long long seg0 = pre * Hkv + (long long)h * u;
    c_first = (int)((seg0 + pu) / w);
    const int c_last = (int)((seg0 + pu + su * (nt - 1)) / w);
    if (c_first == c_last) {
      // written whole by its CTA: to out, or to its state slot, which is
      // already the result when only states are wanted and none merge in
      if (!a.st_o || (!a.out && n_ext == 0)) return;
      whole_state = true;
    } else {
      n_pc = c_last - c_first + 1;
      // a cut segment's first piece is in slot 1 of its CTA when that CTA
      // owns an earlier stage: the stage just before, which starts at
      // seg0 - su, the last of the previous non-empty segment
      first_is_slot1 = seg0 > 0 && seg0 - su >= (long long)c_first * w;
    }
  }
  const float* ext_lse = a.st_o ? a.st_lse + rh * a.st_stride : nullptr;
  const float* ext_o = a.st_o ? a.st_o + rh * a.st_stride * D : nullptr;
  const int n_st = n_ext + (whole_state ? 1 : 0);
  auto piece_rec = [&](int i) -> int64_t {  // record of piece i (CTA c_first + i)
    const int64_t cc = c_first + i;
    return (2 * cc + (i == 0 && first_is_slot1 ? 1 : 0)) * G + g;
  };
  // Sources 0 .. n-1: lane i holds source i's LSE (sources past 32, rare,
  // are read again in pass 2); pass 2 loads the outputs kMergeBatch at a
  // time so their latencies overlap.
  const int n = n_st + n_pc;
  auto src_lse = [&](int i) -> float {
    return i < n_st ? ext_lse[i] : a.rec_lse[piece_rec(i - n_st)];
  };
  auto src_o = [&](int i) -> const float* {
    return i < n_st ? ext_o + (int64_t)i * D : a.rec_o + piece_rec(i - n_st) * D;
  };
  const float my0 = lane < n ? src_lse(lane) : -INFINITY;
  auto top = [](float l) { return l != l ? INFINITY : l; };  // NaN (a window's) is not passed over
  float M = top(my0);
  for (int i = lane + 32; i < n; i += 32) M = fmaxf(M, top(src_lse(i)));
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float acc[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
  float Lsum = 0.f;
  if (M != -INFINITY) {
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int m = min(32, n - i0);
      const float my = i0 == 0 ? my0 : (lane < m ? src_lse(i0 + lane) : -INFINITY);
      for (int u0 = 0; u0 < m; u0 += kMergeBatch) {
        float l[kMergeBatch], x[kMergeBatch][EPL];
#pragma unroll
        for (int u = 0; u < kMergeBatch; ++u) {
          l[u] = __shfl_sync(0xffffffffu, my, (u0 + u) & 31);
          if (u0 + u >= m) l[u] = -INFINITY;  // an empty state: the merge's identity
#pragma unroll
          for (int e = 0; e < EPL; ++e) x[u][e] = 0.f;
          if (l[u] != -INFINITY) VecLoad<float, EPL>::run(src_o(i0 + u0 + u) + lane * EPL, x[u]);
        }
#pragma unroll
        for (int u = 0; u < kMergeBatch; ++u) {
          if (l[u] == -INFINITY) continue;
          const float w = exp2f(l[u] - M);
          Lsum += w;
#pragma unroll
          for (int e = 0; e < EPL; ++e) acc[e] = fmaf(w, x[u][e], acc[e]);
        }
      }
    }
  }
  const bool nonempty = a.window ? Lsum != 0.f : Lsum > 0.f;  // a window's NaN stays
  if (!a.out) {  // states only: the merged pieces become the segment's state
    const int64_t slot = rh * a.st_stride + a.st_slot;
    float* so = a.st_o + slot * D + lane * EPL;
#pragma unroll
    for (int e = 0; e < EPL; ++e) so[e] = nonempty ? acc[e] / Lsum : 0.f;
    if (lane == 0) a.st_lse[slot] = nonempty ? M + log2f(Lsum) : -INFINITY;
    return;
  }
  T* out = static_cast<T*>(a.out) + rh * D + lane * EPL;
#pragma unroll
  for (int e = 0; e < EPL; ++e) store_out(out + e, nonempty ? acc[e] / Lsum : 0.f);
  if (lane == 0 && a.lse_out) a.lse_out[rh] = nonempty ? (M + log2f(Lsum)) * kLn2 : -INFINITY;
}

template <typename T, int D, int G>
static size_t partial_smem_bytes() {
  return decode_smem_layout(D, (int)sizeof(T), G, decode_num_stages(D, (int)sizeof(T))).total;
}

// Resident CTAs per SM of one partial-kernel instance, looked up once per
// device.
template <typename T, int D, int G>
static int resident_ctas() {
  static std::mutex mu;
  static int cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (!cached[dev]) {
    const size_t smem = partial_smem_bytes<T, D, G>();
    auto kern = decode_partial_kernel<T, D, G>;
    int per_sm = 0, sms = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kDecodeThreads, smem) !=
            cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return 0;
    cached[dev] = per_sm * sms;
  }
  return cached[dev];
}

template <typename T, int D>
static int resident_for_group(int group) {
  switch (group) {
    case 1: return resident_ctas<T, D, 1>();
    case 2: return resident_ctas<T, D, 2>();
    case 4: return resident_ctas<T, D, 4>();
    case 8:
      if constexpr (!kIsMx<T>) return resident_ctas<T, D, 8>();
      return 0;
    default: return 0;
  }
}

int decode_resident_ctas(int dtype, int head_dim, int group) {
  if (dtype == PKV_MXFP8) {
    if (group > 4) return 0;
    return head_dim == 128 ? resident_for_group<__nv_fp8_e4m3, 128>(group)
                           : resident_for_group<__nv_fp8_e4m3, 64>(group);
  }
  if (dtype == PKV_BF16)
    return head_dim == 128 ? resident_for_group<__nv_bfloat16, 128>(group)
                           : resident_for_group<__nv_bfloat16, 64>(group);
  return head_dim == 128 ? resident_for_group<float, 128>(group)
                         : resident_for_group<float, 64>(group);
}

template <typename T, int D>
static cudaError_t dispatch_group(int group, const CUtensorMap& tmk, const CUtensorMap& tmv,
                                  const DecodeArgs& a, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_partial<T, D, 1>(tmk, tmv, a, stream);
    case 2: return launch_partial<T, D, 2>(tmk, tmv, a, stream);
    case 4: return launch_partial<T, D, 4>(tmk, tmv, a, stream);
    case 8:
      if constexpr (!kIsMx<T>) return launch_partial<T, D, 8>(tmk, tmv, a, stream);
      return cudaErrorInvalidValue;
    default: return cudaErrorInvalidValue;
  }
}

template <typename T, int D>
static cudaError_t launch_reduce_t(const DecodeArgs& a, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.num_seqs * a.num_q_heads;
  return launch_pdl(decode_reduce_kernel<T, D>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0,
                    stream, a);
}

cudaError_t launch_decode_reduce(int dtype, int head_dim, const DecodeArgs& a,
                                 cudaStream_t stream) {
  if (dtype == PKV_BF16 || dtype == PKV_MXFP8)  // out is bf16 beside an MXFP8 pool
    return head_dim == 128 ? launch_reduce_t<__nv_bfloat16, 128>(a, stream)
                           : launch_reduce_t<__nv_bfloat16, 64>(a, stream);
  return head_dim == 128 ? launch_reduce_t<float, 128>(a, stream)
                         : launch_reduce_t<float, 64>(a, stream);
}

cudaError_t launch_paged_decode(int dtype, int head_dim, int group, const CUtensorMap& tmk,
                                const CUtensorMap& tmv, const DecodeArgs& a,
                                cudaStream_t stream) {
  cudaError_t e;
  if (a.window) return launch_decode_window(head_dim, group, tmk, tmv, a, stream);  // fp32
  if (a.scores)
    e = launch_decode_partial_scores(dtype, head_dim, group, tmk, tmv, a, stream);
  else if (dtype == PKV_MXFP8)
    e = head_dim == 128 ? dispatch_group<__nv_fp8_e4m3, 128>(group, tmk, tmv, a, stream)
                        : dispatch_group<__nv_fp8_e4m3, 64>(group, tmk, tmv, a, stream);
  else if (dtype == PKV_BF16)
    e = head_dim == 128 ? dispatch_group<__nv_bfloat16, 128>(group, tmk, tmv, a, stream)
                        : dispatch_group<__nv_bfloat16, 64>(group, tmk, tmv, a, stream);
  else
    e = head_dim == 128 ? dispatch_group<float, 128>(group, tmk, tmv, a, stream)
                        : dispatch_group<float, 64>(group, tmk, tmv, a, stream);
  if (e != cudaSuccess) return e;
  return launch_decode_reduce(dtype, head_dim, a, stream);
}

}  // namespace pkv
