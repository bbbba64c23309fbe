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
//   * a CTA takes 16 kRT (token, query head) rows of one kv head -- all the
//     G heads of a token share its K/V -- and one contiguous split of the
//     sequence's rows, 32 at a time, through two buffers that cp.async fills;
//   * thread (rg, kg) of 16 x 16 holds the scores of rows rg kRT .. and keys
//     kg, kg + 16, and the outputs of those rows at columns 4 kg .. + 3 of
//     every 64: three shared-memory wavefronts for every eight FMAs;
//   * splits leave (O, LSE) states that a second kernel merges by
//     log-sum-exp; one split writes the result directly;
//   * a hidden row's weight is stored as -1 and skipped, not multiplied, so
//     an infinity or NaN in it cannot leak; rows past the last drafted one
//     are never read.  Tiles without hidden rows look at no weight's sign.
// The fp32 FMAs bound it, 256 per (row, key) at head_dim 128.  (One TF32 term on
// the tensor cores would lose 13 bits of an operand; sums of several terms, and
// packed FMAs here, are untried.)  16 requests with trees of 5 to 27, 32 query
// and 8 kv heads: 748 us, 24 TFLOP/s, of the 74 that the FMAs can do.
#include <math.h>

#include <type_traits>

#include "draft.cuh"

namespace pkv {

namespace {

constexpr int kDsThreads = 256;
constexpr int kDsKeys = 32;  // keys per tile
constexpr int kDsPs = kDsKeys + 4;  // padded shared rows of weights
constexpr float kDsLn2 = 0.6931471805599453f;

template <int D, int kRT>
constexpr int draft_simt_smem() {
  return (16 * kRT * (D + 4) + 2 * kDsKeys * (D + 4) + 2 * kDsKeys * D + 16 * kRT * kDsPs) * 4 + 16 * kRT * 8;
}

// 16 bytes, or zeros.
__device__ __forceinline__ void cp_async16_or_zero(void* smem, const void* g, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(smem)), "l"(g), "r"(valid ? 16 : 0)
               : "memory");
}

}  // namespace

template <int D, int kRT>
__global__ void __launch_bounds__(kDsThreads, 2) draft_simt_kernel(const DraftArgs a) {
  constexpr int R = 16 * kRT;      // query rows per CTA
  constexpr int LD = D + 4;        // padded shared rows of Q and K
  constexpr int NQ = D / 64;       // quads of output columns per thread
  constexpr int kVec = D / 4;      // 16-byte vectors per row
  extern __shared__ __align__(16) float sm[];
  float* qs = sm;                           // [R][LD], scaled
  float* ks = qs + R * LD;                  // [2][keys][LD]
  float* vs = ks + 2 * kDsKeys * LD;        // [2][keys][D]
  float* ps = vs + 2 * kDsKeys * D;         // [R][kDsPs]
  uint64_t* mk = reinterpret_cast<uint64_t*>(ps + R * kDsPs);
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
  const int per = (((T_all - 1) / a.num_splits + kDsKeys) / kDsKeys) * kDsKeys;
  const long long lo64 = (long long)split * per;
  const int t_lo = lo64 < T_all ? (int)lo64 : T_all, t_hi = min(T_all - t_lo, per) + t_lo;

  const int tid = threadIdx.x, rg = tid >> 4, kg = tid & 15;
  auto load = [&](int t0, int buf) {  // the tile's K and V; zeros past the split and for bad blocks
#pragma unroll
    for (int n = 0; n < kDsKeys * kVec / kDsThreads; ++n) {
      const int i = tid + n * kDsThreads, key = i / kVec, c = (i % kVec) * 4, t = t0 + key;
      bool valid = t < t_hi;
      int64_t at = 0;
      if (valid) {
        const int blk = __ldg(a.block_tables + (int64_t)r * a.max_blocks + t / P);
        valid = blk >= 0 && (int64_t)blk < a.num_blocks;
        if (valid) at = (((int64_t)blk * P + t % P) * Hkv + h) * D + c;
        else if (c == 0) atomicOr(a.err, PKV_DEVERR_BLOCK);
      }
      cp_async16_or_zero(ks + (buf * kDsKeys + key) * LD + c, static_cast<const float*>(a.k) + at, valid);
      cp_async16_or_zero(vs + (buf * kDsKeys + key) * D + c, static_cast<const float*>(a.v) + at, valid);
    }
  };
  if (t_lo < t_hi) load(t_lo, 0);
  asm volatile("cp.async.commit_group;" ::: "memory");
  for (int i = tid; i < R * kVec; i += kDsThreads) {
    const int row = i / kVec, c = (i % kVec) * 4;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < rows) {
      const int tok = (row_lo + row) / G, g = (row_lo + row) % G;
      f = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) +
                                                ((int64_t)(s.row0 + tok) * a.num_q_heads + h * G + g) * D + c));
    }
    *reinterpret_cast<float4*>(qs + row * LD + c) =
        make_float4(f.x * a.qscale, f.y * a.qscale, f.z * a.qscale, f.w * a.qscale);
  }
  for (int i = tid; i < R; i += kDsThreads) mk[i] = i < rows ? draft_mask(a, s, (row_lo + i) / G) : 0;

  float m[kRT], l[kRT], o[kRT][4 * NQ];
#pragma unroll
  for (int i = 0; i < kRT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < 4 * NQ; ++c) o[i][c] = 0.f;
  }
  int buf = 0;
  for (int t0 = t_lo; t0 < t_hi; t0 += kDsKeys, buf ^= 1) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // this tile is here, and the previous one has been used
    if (t0 + kDsKeys < t_hi) load(t0 + kDsKeys, buf ^ 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    if ((tid >> 5) * 2 * kRT >= rows) continue;  // a warp without rows only loads
    const float* kt = ks + buf * kDsKeys * LD;
    const float* vt = vs + buf * kDsKeys * D + kg * 4;
    // ---- scores of rows rg kRT + i, keys kg and kg + 16
    float x[kRT][2];
#pragma unroll
    for (int i = 0; i < kRT; ++i) x[i][0] = x[i][1] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      const float4 k0 = *reinterpret_cast<const float4*>(kt + kg * LD + c);
      const float4 k1 = *reinterpret_cast<const float4*>(kt + (kg + 16) * LD + c);
#pragma unroll
      for (int i = 0; i < kRT; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(qs + (rg * kRT + i) * LD + c);
        x[i][0] = fmaf(q.x, k0.x, fmaf(q.y, k0.y, fmaf(q.z, k0.z, fmaf(q.w, k0.w, x[i][0]))));
        x[i][1] = fmaf(q.x, k1.x, fmaf(q.y, k1.y, fmaf(q.z, k1.z, fmaf(q.w, k1.w, x[i][1]))));
      }
    }
    const bool clean = t0 + kDsKeys <= min(s.ctx, t_hi);  // every row sees every key
#pragma unroll
    for (int i = 0; i < kRT; ++i) {
      const int row = rg * kRT + i;
      bool seen[2];
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = t0 + kg + 16 * j, d = t - s.ctx;
        seen[j] = clean || (t < t_hi && (d < 0 || ((mk[row] >> d) & 1)));  // d < n <= 64 where t < t_hi
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
        ps[row * kDsPs + kg + 16 * j] = seen[j] ? p : -1.f;
      }
#pragma unroll
      for (int w = 8; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l[i] = l[i] * alpha + sum;
      m[i] = m_new;
#pragma unroll
      for (int c = 0; c < 4 * NQ; ++c) o[i][c] *= alpha;
    }
    __syncwarp();  // a row's weights are written and read by one half-warp
    auto add = [&](auto hidden) {
#pragma unroll 2
      for (int key = 0; key < kDsKeys; key += 4) {
        float4 p4[kRT];
#pragma unroll
        for (int i = 0; i < kRT; ++i) p4[i] = *reinterpret_cast<const float4*>(ps + (rg * kRT + i) * kDsPs + key);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float4 v[NQ];
#pragma unroll
          for (int c = 0; c < NQ; ++c) v[c] = *reinterpret_cast<const float4*>(vt + (key + k) * D + c * 64);
#pragma unroll
          for (int i = 0; i < kRT; ++i) {
            const float p = k == 0 ? p4[i].x : k == 1 ? p4[i].y : k == 2 ? p4[i].z : p4[i].w;
            if (decltype(hidden)::value && p < 0.f) continue;  // a NaN weight counts
#pragma unroll
            for (int c = 0; c < NQ; ++c) {
              o[i][4 * c] = fmaf(p, v[c].x, o[i][4 * c]);
              o[i][4 * c + 1] = fmaf(p, v[c].y, o[i][4 * c + 1]);
              o[i][4 * c + 2] = fmaf(p, v[c].z, o[i][4 * c + 2]);
              o[i][4 * c + 3] = fmaf(p, v[c].w, o[i][4 * c + 3]);
            }
          }
        }
      }
    };
    if (clean) add(std::false_type{});
    else add(std::true_type{});
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
    // states by (sequence, drafted row, head), whatever query row that is
    const int64_t st = (((int64_t)r * a.max_draft + tok) * a.num_q_heads + h * G + g) * a.num_splits + split;
    float* dst = (a.num_splits == 1 ? static_cast<float*>(a.out) + qh * D : a.rec_o + st * D) + kg * 4;
#pragma unroll
    for (int c = 0; c < NQ; ++c)
      *reinterpret_cast<float4*>(dst + c * 64) =
          make_float4(o[i][4 * c] * inv, o[i][4 * c + 1] * inv, o[i][4 * c + 2] * inv, o[i][4 * c + 3] * inv);
    if (kg == 0) {
      if (a.num_splits > 1) a.rec_lse[st] = lse2;
      else if (a.lse_out) a.lse_out[qh] = lse2 * kDsLn2;
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
  for (int i = lane; i < S; i += 32) M = fmaxf(M, lse[i]);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float acc[EPL], L = 0.f;
#pragma unroll
  for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
  constexpr int kBatch = 8;  // states loaded at once
  for (int i0 = 0; i0 < S; i0 += kBatch) {
    float x[kBatch], f[kBatch][EPL];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      x[i] = -INFINITY;
      if (i0 + i >= S) continue;
      x[i] = lse[i0 + i];
      VecLoad<float, EPL>::run(a.rec_o + (st0 + i0 + i) * D + lane * EPL, f[i]);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (x[i] == -INFINITY) continue;  // an empty state
      const float wt = exp2f(x[i] - M);  // NaN stays NaN
      L += wt;
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] = fmaf(wt, f[i][e], acc[e]);
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int e = 0; e < EPL; ++e)
    static_cast<float*>(a.out)[qh * D + lane * EPL + e] = acc[e] * inv;
  if (lane == 0 && a.lse_out) a.lse_out[qh] = L == 0.f ? -INFINITY : (M + log2f(L)) * kDsLn2;
}

template <int D, int kRT>
static cudaError_t launch_draft_simt_t(const DraftArgs& a, cudaStream_t stream) {
  constexpr int smem = draft_simt_smem<D, kRT>();
  auto kern = draft_simt_kernel<D, kRT>;
  static SmemAttrCache attr_cache;
  cudaError_t e = ensure_smem_limit(kern, smem, attr_cache);
  if (e != cudaSuccess) return e;
  const int G = a.num_q_heads / a.num_kv_heads;
  const int tiles = (a.max_draft * G + 16 * kRT - 1) / (16 * kRT);
  e = launch_pdl(kern, dim3((unsigned)a.num_splits, (unsigned)(a.num_kv_heads * tiles), (unsigned)a.num_seqs),
                 dim3(kDsThreads), smem, stream, a);
  if (e != cudaSuccess || a.num_splits == 1) return e;
  return launch_pdl(draft_simt_merge_kernel<D>,
                    dim3((unsigned)((a.max_draft * a.num_q_heads + 3) / 4), (unsigned)a.num_seqs), dim3(128), 0,
                    stream, a);
}

int draft_simt_rows(int rows) { return rows <= 16 ? 16 : 64; }

cudaError_t launch_draft_simt(int head_dim, const DraftArgs& a, cudaStream_t stream) {
  const bool few = draft_simt_rows(a.max_draft * (a.num_q_heads / a.num_kv_heads)) == 16;
  if (head_dim == 128) return few ? launch_draft_simt_t<128, 1>(a, stream) : launch_draft_simt_t<128, 4>(a, stream);
  return few ? launch_draft_simt_t<64, 1>(a, stream) : launch_draft_simt_t<64, 4>(a, stream);
}

}  // namespace pkv
