// draft.cu -- attention of drafted tokens over a paged fp32 cache, on the CUDA
// cores.  (bf16 and MXFP8 pools: draft_tc.cu, on the tensor cores.)
//
// What it computes: sequence r holds ctx committed token rows and n drafted
// ones behind them (positions ctx .. ctx + n - 1, already in the cache).
// Drafted row i, query head h:
//   A_i = {t < ctx} + {ctx + j : bit j of mask_i},
//   lse = log sum_{t in A_i} exp(s_t),  s_t = scale q . k_t,
//   out = sum_{t in A_i} exp(s_t - lse) v_t,
// in one pass over the rows with a running maximum and sum (base 2, fp32).
//
// Design:
//   * a CTA takes kRT * 8 (token, query head) rows of one kv head -- all the
//     G heads of a token share its K/V -- and one contiguous split of the
//     sequence's rows, 32 at a time, in shared memory;
//   * thread (rg, kg) of 8 x 16 holds the scores of rows rg kRT .. and keys
//     kg, kg + 16, and the outputs of those rows at D / 16 columns;
//   * splits leave (O, LSE) states that a second kernel merges by
//     log-sum-exp; one split writes the result directly;
//   * a hidden row's weight is stored as -1 and skipped, not multiplied, so
//     an infinity or NaN in it cannot leak; rows past the last drafted one
//     are never read.
// The fp32 FMAs bound it, 256 per (row, key) at head_dim 128: fp32 operands
// would lose 16 bits on the tensor cores.  SIMT_US
#include <math.h>

#include "draft.cuh"

namespace pkv {

namespace {

constexpr int kDsThreads = 128;
constexpr int kDsKeys = 32;  // keys per tile
constexpr float kDsLn2 = 0.6931471805599453f;

template <int D, int kRT>
constexpr int draft_simt_smem() {
  return (8 * kRT * (D + 4) + kDsKeys * (D + 4) + kDsKeys * D + 8 * kRT * (kDsKeys + 1)) * 4 +
         8 * kRT * 8;
}

}  // namespace

template <int D, int kRT>
__global__ void __launch_bounds__(kDsThreads) draft_simt_kernel(const DraftArgs a) {
  constexpr int R = 8 * kRT;       // query rows per CTA
  constexpr int LD = D + 4;        // padded shared rows of Q and K
  constexpr int CPT = D / 16;      // output columns per thread
  constexpr int kVec = D / 8;      // 8-element vectors per row
  extern __shared__ __align__(16) float sm[];
  float* qs = sm;                           // [R][LD], scaled
  float* ks = qs + R * LD;                  // [keys][LD]
  float* vs = ks + kDsKeys * LD;            // [keys][D]
  float* ps = vs + kDsKeys * D;             // [R][keys + 1]
  uint64_t* mk = reinterpret_cast<uint64_t*>(ps + ((R * (kDsKeys + 1) + 1) & ~1));
  pdl_wait();
  pdl_launch_dependents();
  const int r = blockIdx.z, split = blockIdx.x;
  const int Hkv = a.num_kv_heads, G = a.num_q_heads / Hkv, P = a.block_size;
  const int tiles = gridDim.y / Hkv;
  const int h = blockIdx.y / tiles, tile = blockIdx.y % tiles;
  const DraftSeq s = draft_seq(a, r, split == 0 && blockIdx.y == 0 && threadIdx.x == 0);
  const int row_lo = tile * R, rows = min(R, s.n * G - row_lo);  // (token, head) rows
  if (rows <= 0) return;
  const int T_all = s.ctx + s.n;
  // the split's keys: equal shares, whole tiles
  const int per = (((T_all + a.num_splits - 1) / a.num_splits + kDsKeys - 1) / kDsKeys) * kDsKeys;
  const long long lo64 = (long long)split * per;
  const int t_lo = lo64 < T_all ? (int)lo64 : T_all, t_hi = min(T_all - t_lo, per) + t_lo;

  const int tid = threadIdx.x, rg = tid >> 4, kg = tid & 15;
  for (int i = tid; i < R * kVec; i += kDsThreads) {
    const int row = i / kVec, c = (i % kVec) * 8;
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (row < rows) {
      const int tok = (row_lo + row) / G, g = (row_lo + row) % G;
      VecLoad<float, 8>::run(static_cast<const float*>(a.q) + ((int64_t)(s.row0 + tok) * a.num_q_heads + h * G + g) * D + c,
                            f);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) qs[row * LD + c + e] = f[e] * a.qscale;
  }
  for (int i = tid; i < R; i += kDsThreads) mk[i] = i < rows ? draft_mask(a, s, (row_lo + i) / G) : 0;

  float m[kRT], l[kRT], o[kRT][CPT];
#pragma unroll
  for (int i = 0; i < kRT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < CPT; ++c) o[i][c] = 0.f;
  }
  for (int t0 = t_lo; t0 < t_hi; t0 += kDsKeys) {
    __syncthreads();  // the previous tile has been used
    for (int i = tid; i < kDsKeys * kVec; i += kDsThreads) {
      const int key = i / kVec, c = (i % kVec) * 8, t = t0 + key;
      float kf[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, vf[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (t < t_hi) {
        const int blk = __ldg(a.block_tables + (int64_t)r * a.max_blocks + t / P);
        if (blk >= 0 && (int64_t)blk < a.num_blocks) {
          const int64_t at = (((int64_t)blk * P + t % P) * Hkv + h) * D + c;
          VecLoad<float, 8>::run(static_cast<const float*>(a.k) + at, kf);
          VecLoad<float, 8>::run(static_cast<const float*>(a.v) + at, vf);
        } else if (c == 0) {
          atomicOr(a.err, PKV_DEVERR_BLOCK);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ks[key * LD + c + e] = kf[e];
        vs[key * D + c + e] = vf[e];
      }
    }
    __syncthreads();
    // ---- scores of rows rg kRT + i, keys kg and kg + 16
    float x[kRT][2];
#pragma unroll
    for (int i = 0; i < kRT; ++i) x[i][0] = x[i][1] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      const float4 k0 = *reinterpret_cast<const float4*>(ks + kg * LD + c);
      const float4 k1 = *reinterpret_cast<const float4*>(ks + (kg + 16) * LD + c);
#pragma unroll
      for (int i = 0; i < kRT; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(qs + (rg * kRT + i) * LD + c);
        x[i][0] = fmaf(q.x, k0.x, fmaf(q.y, k0.y, fmaf(q.z, k0.z, fmaf(q.w, k0.w, x[i][0]))));
        x[i][1] = fmaf(q.x, k1.x, fmaf(q.y, k1.y, fmaf(q.z, k1.z, fmaf(q.w, k1.w, x[i][1]))));
      }
    }
#pragma unroll
    for (int i = 0; i < kRT; ++i) {
      const int row = rg * kRT + i;
      bool seen[2];
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = t0 + kg + 16 * j, d = t - s.ctx;
        seen[j] = t < t_hi && (d < 0 || ((mk[row] >> d) & 1));  // d < n <= 64 where t < t_hi
        if (seen[j]) mx = fmaxf(mx, x[i][j]);
      }
#pragma unroll
      for (int w = 8; w >= 1; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float m_new = fmaxf(m[i], mx);
      const float base = m_new == -INFINITY ? 0.f : m_new;  // nothing seen yet
      const float alpha = exp2f(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float p = exp2f(x[i][j] - base);
        if (seen[j]) sum += p;
        ps[row * (kDsKeys + 1) + kg + 16 * j] = seen[j] ? p : -1.f;
      }
#pragma unroll
      for (int w = 8; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l[i] = l[i] * alpha + sum;
      m[i] = m_new;
#pragma unroll
      for (int c = 0; c < CPT; ++c) o[i][c] *= alpha;
    }
    __syncwarp();  // a row's weights are written and read by one half-warp
    const int nk = min(kDsKeys, t_hi - t0);
    for (int key = 0; key < nk; ++key) {
      float v[CPT];
#pragma unroll
      for (int c = 0; c < CPT; ++c) v[c] = vs[key * D + c * 16 + kg];
#pragma unroll
      for (int i = 0; i < kRT; ++i) {
        const float p = ps[(rg * kRT + i) * (kDsKeys + 1) + key];
        if (!(p < 0.f)) {  // a NaN weight counts
#pragma unroll
          for (int c = 0; c < CPT; ++c) o[i][c] = fmaf(p, v[c], o[i][c]);
        }
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < kRT; ++i) {
    const int row = rg * kRT + i;
    if (row >= rows) continue;
    const int tok = (row_lo + row) / G, g = (row_lo + row) % G;
    const int64_t qh = (int64_t)(s.row0 + tok) * a.num_q_heads + h * G + g;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
    const float lse2 = l[i] == 0.f ? -INFINITY : m[i] + log2f(l[i]);
    if (a.num_splits == 1) {
#pragma unroll
      for (int c = 0; c < CPT; ++c)
        static_cast<float*>(a.out)[qh * D + c * 16 + kg] = o[i][c] * inv;
      if (kg == 0 && a.lse_out) a.lse_out[qh] = lse2 * kDsLn2;
    } else {
      // states by (sequence, drafted row, head), whatever query row that is
      const int64_t st = (((int64_t)r * a.max_draft + tok) * a.num_q_heads + h * G + g) * a.num_splits + split;
#pragma unroll
      for (int c = 0; c < CPT; ++c) a.rec_o[st * D + c * 16 + kg] = o[i][c] * inv;
      if (kg == 0) a.rec_lse[st] = lse2;
    }
  }
}

// One warp per (sequence, drafted row, head): merge the row's split states.
template <int D>
__global__ void __launch_bounds__(128) draft_simt_merge_kernel(const DraftArgs a) {
  constexpr int EPL = D / 32;
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 4 + warp;
  const int r = blockIdx.y;
  const DraftSeq s = draft_seq(a, r, false);
  if (w >= (int64_t)s.n * a.num_q_heads) return;
  const int64_t qh = (int64_t)s.row0 * a.num_q_heads + w;
  const int S = a.num_splits;
  const int64_t st0 = ((int64_t)r * a.max_draft * a.num_q_heads + w) * S;
  const float* lse = a.rec_lse + st0;
  float M = -INFINITY;
  for (int i = 0; i < S; ++i) M = fmaxf(M, lse[i]);
  float acc[EPL], L = 0.f;
#pragma unroll
  for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
  for (int i = 0; i < S; ++i) {
    const float x = lse[i];
    if (x == -INFINITY) continue;  // an empty state
    const float wt = exp2f(x - M);  // NaN stays NaN
    L += wt;
    float f[EPL];
    VecLoad<float, EPL>::run(a.rec_o + (st0 + i) * D + lane * EPL, f);
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] = fmaf(wt, f[e], acc[e]);
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int e = 0; e < EPL; ++e)
    static_cast<float*>(a.out)[qh * D + lane * EPL + e] = acc[e] * inv;
  if (lane == 0 && a.lse_out) a.lse_out[qh] = L == 0.f ? -INFINITY : (M + log2f(L)) * kDsLn2;
}

template <int D, int kRT>
static cudaError_t launch_draft_simt_t(const DraftArgs& a, cudaStream_t stream) {
  constexpr int smem = draft_simt_smem<D, kRT>() + 16;
  auto kern = draft_simt_kernel<D, kRT>;
  static SmemAttrCache attr_cache;
  cudaError_t e = ensure_smem_limit(kern, smem, attr_cache);
  if (e != cudaSuccess) return e;
  const int G = a.num_q_heads / a.num_kv_heads;
  const int tiles = (a.max_draft * G + 8 * kRT - 1) / (8 * kRT);
  e = launch_pdl(kern, dim3((unsigned)a.num_splits, (unsigned)(a.num_kv_heads * tiles), (unsigned)a.num_seqs),
                 dim3(kDsThreads), smem, stream, a);
  if (e != cudaSuccess || a.num_splits == 1) return e;
  return launch_pdl(draft_simt_merge_kernel<D>,
                    dim3((unsigned)((a.max_draft * a.num_q_heads + 3) / 4), (unsigned)a.num_seqs), dim3(128), 0,
                    stream, a);
}

int draft_simt_rows(int rows) { return rows <= 8 ? 8 : 32; }

cudaError_t launch_draft_simt(int head_dim, const DraftArgs& a, cudaStream_t stream) {
  const int rows = a.max_draft * (a.num_q_heads / a.num_kv_heads);
  if (head_dim == 128) return rows <= 8 ? launch_draft_simt_t<128, 1>(a, stream) : launch_draft_simt_t<128, 4>(a, stream);
  return rows <= 8 ? launch_draft_simt_t<64, 1>(a, stream) : launch_draft_simt_t<64, 4>(a, stream);
}

}  // namespace pkv
