// window_mma.cu -- the decode of bf16 pools under a sliding window with sinks,
// on warp-level matrix instructions.
//
// What it computes: what decode_window.cu computes -- for sequence r and query
// head h, attention of q[r, h] over the rows t < S and t >= T - W of kv head h /
// G -- with the direct split: a CTA takes an equal part of one segment's 32-row
// stages and asks nothing but its length.
//
// Design (GB300): a window's segments are short and many, so what counts is how
// soon a CTA has its first rows, how many CTAs stream at once and how few
// instructions a row costs.  tcgen05's 128-row tiles want one CTA an SM and a
// prologue for each segment's piece (64 requests of 64/8 heads, window 128: 38.5 us on
// decode_tc.cu's kernel, 7.6 here; window 1024 76 / 44); the CUDA cores' decode is bound by its
// instructions (32/8 heads, window 1024: 58 / 43).  mma.sync needs no set-up and leaves
// DRAM the bound, and its 16 x 8 tiles fit up to eight query heads:
//   S [16 x 16 rows]  = Q [16 heads x D] K^T,     heads 8 .. 15 zero
//   O [16 x D]       += P [16 x 16 rows] V,       heads 0 .. 7 the upper bf16 term
// of the weights, 8 .. 15 what it leaves of them, so that the unused half of the tile
// carries the second term (a weight within 2^-16 of itself).  A 16-row chunk is 32
// matrix instructions and, loads and waits among them, 340 in all, where the CUDA-core
// kernel takes 920 for four heads.  Measured: 64 requests, 1024 + 4 rows,
// 32/8 heads 43.0 us, 6170 GB/s, 91% of a copy's rate; 2000 + 4 rows 97%.
//   * warp 2 fetches block ids sixteen stages at a time and fills a ring of 32-row
//     stages by TMA (the row-group tiles of launch.h, 128-byte swizzle, which
//     ldmatrix reads without bank conflicts);
//   * warps 0 and 1 take 16 rows of each stage: ldmatrix of K as the B operand,
//     of V transposed; the weights' layout as accumulators of S is that of the
//     A operand of P V, so they never leave registers;
//   * the exponent base moves only when a score passes it by 2^8; rows that are
//     not seen have weight 0, and their V is cleared in the fragments (0 x NaN);
//   * the two warps merge through the ring at the end.
#include <math.h>

#include "common.cuh"
#include "launch.h"
#include "plan.cuh"

namespace pkv {

namespace {

constexpr int kWmRows = 32;             // rows of a stage
constexpr int kWmThreads = 3 * 32;      // two warps of matrix work, one of loads
constexpr float kWmLn2 = 0.6931471805599453f;
// Stages of the ring: 48 KiB, four CTAs an SM.
constexpr int wm_stages(int d) { return d == 128 ? 3 : 6; }
constexpr int wm_tile(int d) { return kWmRows * d * 2; }  // bytes of a K (or V) tile
constexpr int wm_smem(int d) { return wm_stages(d) * 2 * wm_tile(d) + 1024; }  // +1024: alignment

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

}  // namespace

template <int D, int G>
__global__ void __launch_bounds__(kWmThreads, 4)
    window_mma_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                      const WindowArgs a) {
  constexpr int NS = wm_stages(D), kTile = wm_tile(D);
  constexpr int kAtom = D / 64 * 1024;  // bytes of an 8-row group, both halves
  __shared__ uint64_t full[NS], empty[NS];
  __shared__ float sm_m[2][8], sm_l[2][8];

  if (!a.plan_before_wait) pdl_wait();
  pdl_launch_dependents();
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  int4 d0;
  const int n = direct_stages<kWmRows>(a, &d0);
  const int r = d0.x, h = d0.y, i0 = d0.z;
  __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(a.out) + ((int64_t)r * a.num_q_heads + (int64_t)h * G) * D;
  float* const lse_out = a.lse_out ? a.lse_out + (int64_t)r * a.num_q_heads + (int64_t)h * G : nullptr;
  if (n < 0) {  // an empty sequence
    if (a.plan_before_wait) pdl_wait();
    for (int i = t; i < G * D; i += kWmThreads) store_out(out + i, 0.f);
    if (lse_out && t < G) lse_out[t] = -INFINITY;
  }
  if (n <= 0) return;  // the whole CTA leaves before any barrier
  const SegRows seg = seg_rows(a, r);
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);

  if (t == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);
    }
    fence_barrier_init();
  }
  __syncthreads();

  bool ok = true;
  int issued = 0;  // stages whose copies warp 2 started
  if (warp == 2) {
    // ============================================================== loads
    // A stage is one box of TB rows or two, K by lanes 0 and 1, V by 2 and 3.
    const int P = a.block_size, TB = a.box_rows;
    if (lane == 0) {
      prefetch_tensormap(&tmk);
      prefetch_tensormap(&tmv);
    }
    // lane 2 x + j: block and first row of box j of stage x of sixteen
    int blk = 0, brow = 0, x0 = 0;
    auto fetch = [&](int k0) {
      x0 = k0;
      const int k = k0 + (lane >> 1), j = lane & 1;
      if (k >= n) return;
      const StageRows sr = stage_rows<kWmRows>(a, seg, i0 + k);
      if (j * TB >= sr.nvalid) return;
      const int row = sr.row(j * TB), b = row / P;
      blk = __ldg(a.block_tables + (int64_t)r * a.max_blocks + b);
      brow = row - b * P;
      if (blk < 0 || (int64_t)blk >= a.num_blocks) {
        atomicOr(a.err, PKV_DEVERR_BLOCK);
        blk = (int)a.num_blocks;  // a zero-filled box out of range
        brow = 0;
      }
    };
    fetch(0);
    if (a.plan_before_wait) pdl_wait();  // the rows are read from here on
    for (int k = 0; k < n; ++k) {
      const int s = k % NS;
      if (k >= NS && !__all_sync(0xffffffffu, mbar_wait(&empty[s], ((k / NS) - 1) & 1))) {
        if (lane == 0) atomicOr(a.err, PKV_DEVERR_TIMEOUT);
        ok = false;
        break;
      }
      const int nbox = (stage_rows<kWmRows>(a, seg, i0 + k).nvalid + TB - 1) / TB;
      const int from = 2 * (k - x0) + (lane & 1);
      const int my_blk = __shfl_sync(0xffffffffu, blk, from), my_row = __shfl_sync(0xffffffffu, brow, from);
      if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(2 * nbox * TB * D * 2));
      __syncwarp();
      if (lane < 4 && (lane & 1) < nbox)
        tma_load_5d(ring + (size_t)s * 2 * kTile + (lane >> 1) * kTile + (lane & 1) * TB * D * 2,
                    lane < 2 ? &tmk : &tmv, 0, 0, 0, h,
                    (int)((int64_t)my_blk * (P / kRowGroup) + my_row / kRowGroup), &full[s]);
      issued = k + 1;
      if (k + 1 == x0 + 16 && k + 1 < n) fetch(k + 1);
    }
    // the last copies land before the CTA's shared memory is released, also
    // where a warp has given up waiting for them
    for (int k = issued > NS ? issued - NS : 0; k < issued; ++k) mbar_wait(&full[k % NS], (k / NS) & 1);
  } else {
    // ======================================================= matrix work
    const int hd = lane >> 2, quad = lane & 3;  // head, and pair of columns, of a fragment
    if (a.plan_before_wait) pdl_wait();
    uint32_t q[D / 16][2];
    {
      const uint32_t* qp = reinterpret_cast<const uint32_t*>(
          static_cast<const __nv_bfloat16*>(a.q) + ((int64_t)r * a.num_q_heads + (int64_t)h * G + hd) * D);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        q[kk][0] = hd < G ? __ldg(qp + kk * 8 + quad) : 0u;
        q[kk][1] = hd < G ? __ldg(qp + kk * 8 + 4 + quad) : 0u;
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    float m = -INFINITY, l = 0.f;  // of head hd; l: this lane's share
    // ldmatrix addresses: lane i names row i % 8 of matrix i / 8.  K: matrices
    // (rows 0-7, columns 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15); V: (rows
    // 0-7, columns 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15).
    const int mat = lane >> 3, r8 = lane & 7;
    const uint32_t base = smem_u32(ring) + (uint32_t)(warp * 2 * kAtom);  // this warp's two row groups
    const uint32_t krow = base + (uint32_t)((mat >> 1) * kAtom + r8 * 128);
    const uint32_t vrow = base + (uint32_t)(kTile + (mat & 1) * kAtom + r8 * 128);
    for (int k = 0; k < n; ++k) {
      const int s = k % NS;
      if (!__all_sync(0xffffffffu, mbar_wait(&full[s], (k / NS) & 1))) {
        if (lane == 0) atomicOr(a.err, PKV_DEVERR_TIMEOUT);
        ok = false;
        break;
      }
      const StageRows sr = stage_rows<kWmRows>(a, seg, i0 + k);
      const bool whole = sr.nvalid == kWmRows && sr.hide_hi == 0;
      if (warp * 16 < sr.nvalid) {
        const uint32_t off = (uint32_t)(s * 2 * kTile);
        // ---- scores of 16 rows: two tiles of eight
        float sc[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[x][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int c = 2 * kk + (mat & 1);  // 8-column chunk
          uint32_t b[4];
          ldsm4(krow + off + (c >> 3) * 1024 + (((c & 7) ^ r8) << 4), b);
          mma16816(sc[0], q[kk][0], 0u, q[kk][1], 0u, b[0], b[1]);
          mma16816(sc[1], q[kk][0], 0u, q[kk][1], 0u, b[2], b[3]);
        }
        // ---- weights
        float p[4];
        bool on[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = warp * 16 + (e >> 1) * 8 + quad * 2 + (e & 1);
          on[e] = whole || row_seen(row, sr.nvalid, sr.hide_lo, sr.hide_hi);
          p[e] = on[e] ? sc[e >> 1][e & 1] * a.qscale : -INFINITY;
        }
        float top = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3]));
        if (__any_sync(0xffffffffu, top > m + 8.0f)) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          if (top > m + 8.0f) {
            const float alpha = exp2f(m - top);
            m = top;
            l *= alpha;
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[j][e] *= alpha;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = p[e] == -INFINITY ? 0.f : exp2f(p[e] - m);
          l += p[e];
        }
        // two bf16 terms: a weight's upper half, cut off (so that neither term is
        // negative and an infinity of V stays one), and what that leaves
        const uint32_t hi0 = __byte_perm(__float_as_uint(p[0]), __float_as_uint(p[1]), 0x7632);
        const uint32_t hi1 = __byte_perm(__float_as_uint(p[2]), __float_as_uint(p[3]), 0x7632);
        const uint32_t lo0 = pack_bf16(p[0] - bf16lo(hi0), p[1] - bf16hi(hi0));
        const uint32_t lo1 = pack_bf16(p[2] - bf16lo(hi1), p[3] - bf16hi(hi1));
        // ---- P V; V of rows that are not seen is cleared
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (!whole) {
          keep0 = (on[0] ? 0xffffu : 0u) | (on[1] ? 0xffff0000u : 0u);
          keep1 = (on[2] ? 0xffffu : 0u) | (on[3] ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int j = 0; j < D / 8; j += 2) {
          const int c = j + (mat >> 1);
          uint32_t b[4];
          ldsm4_t(vrow + off + (c >> 3) * 1024 + (((c & 7) ^ r8) << 4), b);
          mma16816(o[j], hi0, lo0, hi1, lo1, b[0] & keep0, b[1] & keep1);
          mma16816(o[j + 1], hi0, lo0, hi1, lo1, b[2] & keep0, b[3] & keep1);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }
    // ---- merge the two warps through the ring (its last copies have landed)
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (quad == 0) {
      sm_m[warp][hd] = m;
      sm_l[warp][hd] = l;
    }
    named_barrier_sync(1, 64);  // both are done with the ring
    float* om = reinterpret_cast<float*>(ring);  // [2][8][D]
    if (hd < G) {
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
        *reinterpret_cast<float2*>(om + (warp * 8 + hd) * D + j * 8 + quad * 2) =
            make_float2(o[j][0] + o[j][2], o[j][1] + o[j][3]);
    }
    named_barrier_sync(1, 64);
    if (ok) {
      const int nt = (seg.len + kWmRows - 1) / kWmRows;
      const bool all = i0 == 0 && n == nt;
      const int64_t rec = 2 * (int64_t)blockIdx.x * G;
      for (int i = t * 4; i < G * D; i += 64 * 4) {
        const int g = i / D, e0 = i % D;
        const float m0 = sm_m[0][g], m1 = sm_m[1][g], M = fmaxf(m0, m1);
        const float w0 = M == -INFINITY ? 0.f : exp2f(m0 - M), w1 = M == -INFINITY ? 0.f : exp2f(m1 - M);
        const float sum = fmaf(w0, sm_l[0][g], w1 * sm_l[1][g]);
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        const float4 x = *reinterpret_cast<const float4*>(om + g * D + e0);
        const float4 y = *reinterpret_cast<const float4*>(om + (8 + g) * D + e0);
        const float v[4] = {fmaf(w0, x.x, w1 * y.x) * inv, fmaf(w0, x.y, w1 * y.y) * inv,
                            fmaf(w0, x.z, w1 * y.z) * inv, fmaf(w0, x.w, w1 * y.w) * inv};
        const float lse2 = sum > 0.f ? M + log2f(sum) : -INFINITY;
        if (all) {
          *reinterpret_cast<uint2*>(out + i) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
          if (e0 == 0 && lse_out) lse_out[g] = lse2 * kWmLn2;
        } else {
          *reinterpret_cast<float4*>(a.rec_o + rec * D + i) = make_float4(v[0], v[1], v[2], v[3]);
          if (e0 == 0) a.rec_lse[rec + g] = lse2;
        }
      }
    }
  }
}

template <int D, int G>
static int wm_resident() {
  static std::mutex mu;
  static int cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (!cached[dev]) {
    auto kern = window_mma_kernel<D, G>;
    int per_sm = 0, sms = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, wm_smem(D)) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kWmThreads, wm_smem(D)) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return 0;
    cached[dev] = per_sm * sms;
  }
  return cached[dev];
}

template <int D>
static int wm_resident_group(int group) {
  return group == 1 ? wm_resident<D, 1>() : group == 2 ? wm_resident<D, 2>() : group == 4 ? wm_resident<D, 4>()
                                                                              : wm_resident<D, 8>();
}

int window_mma_resident_ctas(int head_dim, int group) {
  return head_dim == 128 ? wm_resident_group<128>(group) : wm_resident_group<64>(group);
}

template <int D, int G>
static cudaError_t launch_wm(const CUtensorMap& tmk, const CUtensorMap& tmv, const WindowArgs& a,
                             cudaStream_t stream) {
  auto kern = window_mma_kernel<D, G>;
  static SmemAttrCache attr_cache;
  cudaError_t e = ensure_smem_limit(kern, wm_smem(D), attr_cache);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)a.num_ctas), dim3(kWmThreads), wm_smem(D), stream, tmk, tmv, a);
}

template <int D>
static cudaError_t launch_wm_group(int group, const CUtensorMap& tmk, const CUtensorMap& tmv,
                                   const WindowArgs& a, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_wm<D, 1>(tmk, tmv, a, stream);
    case 2: return launch_wm<D, 2>(tmk, tmv, a, stream);
    case 4: return launch_wm<D, 4>(tmk, tmv, a, stream);
    case 8: return launch_wm<D, 8>(tmk, tmv, a, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_window_mma(int head_dim, int group, const CUtensorMap& tmk, const CUtensorMap& tmv,
                              const DecodeArgs& args, cudaStream_t stream) {
  const WindowArgs a(args, box_rows_for(args.block_size));
  cudaError_t e = head_dim == 128 ? launch_wm_group<128>(group, tmk, tmv, a, stream)
                                  : launch_wm_group<64>(group, tmk, tmv, a, stream);
  if (e != cudaSuccess || a.parts == 1) return e;
  return launch_window_merge(PKV_BF16, head_dim, a, stream);
}

}  // namespace pkv
