// window_mma.cu -- the decode of bf16 and MXFP8 pools under a sliding window with
// sinks, on warp-level matrix instructions.
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
// carries the second term (a weight within 2^-16 + 2^-23 of itself).  A 16-row chunk is 32
// matrix instructions and, loads and waits among them, 340 in all, where the CUDA-core
// kernel takes 920 for four heads.  Measured: 64 requests, 1024 + 4 rows,
// 32/8 heads 43.8 us, 6050 GB/s, 89% of a copy's rate; 2000 + 4 rows 78.5 us, 98%.
//   * warp 2 fetches block ids sixteen stages at a time and fills a ring of 32-row
//     stages by TMA (the row-group tiles of launch.h, 128-byte swizzle, which
//     ldmatrix reads without bank conflicts);
//   * warps 0 and 1 take 16 rows of each stage: ldmatrix of K as the B operand,
//     of V transposed; the weights' layout as accumulators of S is that of the
//     A operand of P V, so they never leave registers;
//   * the exponent base moves only when a score passes it by 2^8; rows that are
//     not seen have weight 0, and their V is cleared in the fragments (0 x NaN);
//   * the two warps merge through the ring at the end, and the CTAs that share a
//     segment through distributed shared memory: up to eight parts are a cluster, each CTA
//     of it merges a share of the outputs, and one launch does the whole decode (one chat
//     of 516 rows 4.8 us, 8.9 with records and a merging launch; 8 x 16,448 rows, 64/8 heads 81 / 90).
//     CTAs without a stage leave; the cluster's barriers wait for those that are there.
// MXFP8 pools: tiles hold codes, and a warp widens them in its fragments, exactly (an
// E4M3 value times a power of two is a bf16 value, those from 2^-126 up).  ldmatrix moves pairs of codes, so
// a lane gets four codes of consecutive columns where the fragment wants two and two: K
// is contracted in that order of columns (q is loaded so), and V's tiles are the even
// and the odd columns of sixteen.  K's scales multiply the scores of their 32 columns,
// V's the codes as they are widened.  NaN codes, scales of 2^-127 (K) and above 2^7 (V)
// cost more instructions; a chunk without one, by a vote, skips them (in every call they
// made 64 requests, window 1024, 32/8 heads 79 us instead of 51).  A chunk's 900
// instructions bound it: two warps of matrix work a scheduler, half of its cycles issuing,
// the ALU pipe 46% busy, 168 registers (at 128, for five CTAs, 77 us).  Against the CUDA cores
// (one to four heads) and tcgen05's widened tiles (eight), 64 requests, window 128 / 1024:
//   32/8 heads  9.4 / 51.0 us against 12.3 / 69.7;  64/8   9.9 / 51.8 against 42.5 / 115.7;
//   8/8         9.1 / 50.5 against 8.8 / 47.4 (head_dim 64: 7.7 / 39.4 against 8.5 / 46.0).
#include <cooperative_groups.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "plan.cuh"

namespace pkv {

namespace cg = cooperative_groups;

namespace {

constexpr int kWmRows = 32;             // rows of a stage
constexpr int kWmThreads = 3 * 32;      // two warps of matrix work, one of loads
constexpr int kWmCluster = 8;           // CTAs of a cluster at most
constexpr float kWmLn2 = 0.6931471805599453f;
// Bytes of a K (or V) tile, of its scales, and stages of the ring: 48 KiB (32 for
// head_dim 64 over MXFP8), four CTAs an SM.
constexpr int wm_tile(bool mx, int d) { return kWmRows * d * (mx ? 1 : 2); }
constexpr int wm_scales(bool mx, int d) { return mx ? kWmRows * d / 32 : 0; }
constexpr int wm_stages(bool mx, int d) { return mx ? (d == 128 ? 6 : 8) : (d == 128 ? 3 : 6); }
constexpr int wm_smem(bool mx, int d) {
  return wm_stages(mx, d) * 2 * (wm_tile(mx, d) + wm_scales(mx, d)) + 1024;  // +1024: alignment
}

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
// The same onto zeros.
__device__ __forceinline__ void mma16816_new(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

}  // namespace

// Two of a word's four codes as the bits of two bf16, times 2^-120: s.eeee.mmm with s
// at 15, eeeemmm at 10 .. 4.  kHigh: bytes 1 and 3, else 0 and 2.
template <bool kHigh>
__device__ __forceinline__ uint32_t place_codes(uint32_t w) {
  return ((kHigh ? w >> 4 : w << 4) & 0x07f007f0u) | ((kHigh ? w : w << 8) & 0x80008000u);
}
// They times f1, as bf16; with kRare also times f2, and with the NaN codes (s.1111.111).
template <bool kHigh, bool kRare>
__device__ __forceinline__ uint32_t widen2(uint32_t w, uint32_t f1, uint32_t f2) {
  const uint32_t x = place_codes<kHigh>(w);
  __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&f1));
  if constexpr (kRare) v = __hmul2(v, *reinterpret_cast<const __nv_bfloat162*>(&f2));
  uint32_t y = *reinterpret_cast<const uint32_t*>(&v);
  if constexpr (kRare) {
    if ((x & 0x07f0u) == 0x07f0u) y |= 0x7fffu;
    if ((x & 0x07f00000u) == 0x07f00000u) y |= 0x7fff0000u;
  }
  return y;
}
// Bit 7 of a byte is set ...
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {  // ... in NaN codes
  return (w & 0x7f7f7f7fu) + 0x01010101u;
}
__device__ __forceinline__ uint32_t zero_scales(uint32_t s) {  // ... if one is 0 (in some byte)
  return (s - 0x01010101u) & ~s;
}
__device__ __forceinline__ uint32_t large_scales(uint32_t s) {  // ... in scales above 134
  return ((s & 0x7f7f7f7fu) + 0x79797979u) & s;
}

template <bool kMx, int D, int G>
__global__ void __launch_bounds__(kWmThreads, 4)
    window_mma_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                      const WindowArgs a) {
  constexpr int NS = wm_stages(kMx, D), kTile = wm_tile(kMx, D), kScales = wm_scales(kMx, D);
  constexpr int kAtom = kMx ? 8 * D : D / 64 * 1024;  // bytes of an 8-row group, all columns
  __shared__ uint64_t full[NS], empty[NS];
  __shared__ float sm_m[2][8], sm_l[2][8];
  __shared__ float sm_lse[8];  // of this part

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

  const int nt = (seg.len + kWmRows - 1) / kWmRows;
  const bool all = i0 == 0 && n == nt;
  float* const om = reinterpret_cast<float*>(ring);  // [2][8][D], later also the part's [G][D]
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
      if (lane == 0)
        mbar_arrive_expect_tx(&full[s], (uint32_t)(2 * nbox * TB * (kMx ? D + D / 32 : 2 * D)));
      __syncwarp();
      if constexpr (kMx) {
        if (lane < 4 && (lane & 1) < nbox) {
          tma_load_4d(ring + (size_t)s * 2 * kTile + (lane >> 1) * kTile + (lane & 1) * TB * D,
                      lane < 2 ? &tmk : &tmv, 0, h, my_row, my_blk, &full[s]);
        } else if (lane < 8 && lane >= 4 && (lane & 1) < nbox) {
          // the box's scale rows; of a bad block, block 0's (its codes are zeros)
          const int64_t sb = my_blk < a.num_blocks ? my_blk : 0;
          const uint8_t* src = (lane < 6 ? a.k_scales : a.v_scales) +
                               ((sb * a.num_kv_heads + h) * P + my_row) * (D / 32);
          bulk_load(ring + NS * 2 * kTile + (s * 2 + (lane < 6 ? 0 : 1)) * kScales + (lane & 1) * TB * (D / 32),
                    src, (uint32_t)(TB * (D / 32)), &full[s]);
        }
      } else if (lane < 4 && (lane & 1) < nbox)
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
        if constexpr (kMx) {  // columns 4 quad, + 2 against + 1, + 3
          const uint32_t w0 = hd < G ? __ldg(qp + kk * 8 + 2 * quad) : 0u;
          const uint32_t w1 = hd < G ? __ldg(qp + kk * 8 + 2 * quad + 1) : 0u;
          q[kk][0] = __byte_perm(w0, w1, 0x5410);
          q[kk][1] = __byte_perm(w0, w1, 0x7632);
        } else {
          q[kk][0] = hd < G ? __ldg(qp + kk * 8 + quad) : 0u;
          q[kk][1] = hd < G ? __ldg(qp + kk * 8 + 4 + quad) : 0u;
        }
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    float m = -INFINITY, l = 0.f;  // of head hd; l: this lane's share
    // ldmatrix addresses: lane i names row i % 8 of matrix i / 8.  bf16 K: matrices
    // (rows 0-7, columns 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15); V: (rows
    // 0-7, columns 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15).
    const int mat = lane >> 3, r8 = lane & 7;
    const uint32_t base = smem_u32(ring) + (uint32_t)(warp * 2 * kAtom);  // this warp's two row groups
    // Codes, K and V: (rows 0-7, 16 columns), (8-15, they), (0-7, the next 16), (8-15, those).
    const uint32_t krow = base + (uint32_t)(kMx ? (mat & 1) * kAtom + r8 * D : (mat >> 1) * kAtom + r8 * 128);
    const uint32_t vrow = kMx ? krow + kTile : base + (uint32_t)(kTile + (mat & 1) * kAtom + r8 * 128);
    // where 16-byte chunk c of a row of codes lies
    auto code_chunk = [&](int c) -> uint32_t {
      return (uint32_t)((D == 128 ? c ^ r8 : c ^ (r8 >> 1)) << 4);
    };
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
        // MXFP8: the scales of this lane's four rows
        uint32_t ksc[4] = {}, vsc[4] = {};
        if constexpr (kMx) {
          const unsigned char* at = ring + NS * 2 * kTile + s * 2 * kScales;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = warp * 16 + (e >> 1) * 8 + quad * 2 + (e & 1);
            if constexpr (D == 128) {
              ksc[e] = reinterpret_cast<const uint32_t*>(at)[row];
              vsc[e] = reinterpret_cast<const uint32_t*>(at + kScales)[row];
            } else {
              ksc[e] = reinterpret_cast<const uint16_t*>(at)[row] | 0x01010000u;
              vsc[e] = reinterpret_cast<const uint16_t*>(at + kScales)[row];
            }
          }
          uint32_t w[D / 32][4], odd = 0;
#pragma unroll
          for (int g = 0; g < D / 32; ++g) {
            ldsm4(krow + off + code_chunk(2 * g + (mat >> 1)), w[g]);
#pragma unroll
            for (int i = 0; i < 4; ++i) odd |= nan_codes(w[g][i]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) odd |= zero_scales(ksc[e]);
          auto scores = [&](auto rare) {
            constexpr uint32_t kUp = 0x7b807b80u;  // 2^120: codes as they are placed, to their values
#pragma unroll
            for (int g = 0; g < D / 32; ++g) {
              float part[2][4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {  // row group i & 1, chunk 2 g + (i >> 1)
                const int kk = 2 * g + (i >> 1);
                const uint32_t b0 = widen2<false, rare.value>(w[g][i], kUp, 0x3f803f80u);
                const uint32_t b1 = widen2<true, rare.value>(w[g][i], kUp, 0x3f803f80u);
                if (i < 2)
                  mma16816_new(part[i], q[kk][0], 0u, q[kk][1], 0u, b0, b1);
                else
                  mma16816(part[i & 1], q[kk][0], 0u, q[kk][1], 0u, b0, b1);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                // 0 is 2^-127, which fp32 here takes for 0: 2^-126 and a half of it
                const bool least = rare.value && ((ksc[e] >> (8 * g)) & 0xffu) == 0;
                const float f = least ? 0x1p-126f
                                      : __uint_as_float((g == 3 ? ksc[e] >> 1 : ksc[e] << (23 - 8 * g)) & 0x7f800000u);
                const float x = part[e >> 1][e & 1];
                sc[e >> 1][e & 1] = fmaf(least ? 0.5f * x : x, f, sc[e >> 1][e & 1]);
              }
            }
          };
          if (__any_sync(0xffffffffu, (odd & 0x80808080u) != 0))
            scores(std::true_type{});
          else
            scores(std::false_type{});
        }
#pragma unroll
        for (int kk = 0; kk < (kMx ? 0 : D / 16); ++kk) {
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
        // two bf16 terms: a weight's upper half, cut off, and what that leaves of p (1 +
        // 2^-23).  Neither is negative, nor 0 (above 2^-103) unless the weight is, so
        // that an infinity of V stays one in both products.
        constexpr float kMore = 1.f + 0x1p-23f;
        const uint32_t hi0 = __byte_perm(__float_as_uint(p[0]), __float_as_uint(p[1]), 0x7632);
        const uint32_t hi1 = __byte_perm(__float_as_uint(p[2]), __float_as_uint(p[3]), 0x7632);
        const uint32_t lo0 = pack_bf16(fmaf(p[0], kMore, -bf16lo(hi0)), fmaf(p[1], kMore, -bf16hi(hi0)));
        const uint32_t lo1 = pack_bf16(fmaf(p[2], kMore, -bf16lo(hi1)), fmaf(p[3], kMore, -bf16hi(hi1)));
        // ---- P V; V of rows that are not seen is cleared
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (!whole) {
          keep0 = (on[0] ? 0xffffu : 0u) | (on[1] ? 0xffff0000u : 0u);
          keep1 = (on[2] ? 0xffffu : 0u) | (on[3] ? 0xffff0000u : 0u);
        }
        if constexpr (kMx) {
          uint32_t w[D / 32][4], odd = 0;
#pragma unroll
          for (int g = 0; g < D / 32; ++g) {
            ldsm4_t(vrow + off + code_chunk(2 * g + (mat >> 1)), w[g]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              w[g][i] &= i & 1 ? keep1 : keep0;  // a word's halves are two rows
              odd |= nan_codes(w[g][i]);
            }
          }
          // scales past 2^7 take the second factor
#pragma unroll
          for (int e = 0; e < 4; ++e) odd |= large_scales(vsc[e]);
          auto values = [&](auto rare) {
#pragma unroll
            for (int g = 0; g < D / 32; ++g) {
              uint32_t f1[2], f2[2];  // of rows 2 quad, + 1, and those 8 further on
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t s2 = __byte_perm(vsc[2 * x], vsc[2 * x + 1], 0x0400u + 0x0101u * g) & 0x00ff00ffu;
                f1[x] = f2[x] = 0;
                if constexpr (rare.value) {
                  const uint32_t m2 = min(s2 & 0xffu, 134u) | min(s2 >> 16, 134u) << 16;
                  f1[x] = m2 * 0x80u + 0x3C003C00u;          // 2^(m - 7)
                  f2[x] = (s2 - m2) * 0x80u + 0x3F803F80u;   // 2^(s - m)
                } else {
                  f1[x] = s2 * 0x80u + 0x3C003C00u;          // 2^(s - 7)
                }
              }
#pragma unroll
              for (int y = 0; y < 2; ++y) {  // chunk 2 g + y: tiles of its even and odd columns
                const int j = 2 * (2 * g + y);
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const uint32_t b0 = z ? widen2<true, rare.value>(w[g][2 * y], f1[0], f2[0])
                                        : widen2<false, rare.value>(w[g][2 * y], f1[0], f2[0]);
                  const uint32_t b1 = z ? widen2<true, rare.value>(w[g][2 * y + 1], f1[1], f2[1])
                                        : widen2<false, rare.value>(w[g][2 * y + 1], f1[1], f2[1]);
                  mma16816(o[j + z], hi0, lo0, hi1, lo1, b0, b1);
                }
              }
            }
          };
          if (__any_sync(0xffffffffu, (odd & 0x80808080u) != 0))
            values(std::true_type{});
          else
            values(std::false_type{});
        }
#pragma unroll
        for (int j = 0; j < (kMx ? 0 : D / 8); j += 2) {
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
    if (hd < G) {
      float* to = om + (warp * 8 + hd) * D;
      if constexpr (kMx) {
#pragma unroll
        for (int j = 0; j < D / 8; j += 2)  // even and odd columns of sixteen
          *reinterpret_cast<float4*>(to + j * 8 + quad * 4) =
              make_float4(o[j][0] + o[j][2], o[j + 1][0] + o[j + 1][2], o[j][1] + o[j][3], o[j + 1][1] + o[j + 1][3]);
      } else {
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
          *reinterpret_cast<float2*>(to + j * 8 + quad * 2) = make_float2(o[j][0] + o[j][2], o[j][1] + o[j][3]);
      }
    }
    named_barrier_sync(1, 64);
    if (ok) {
      for (int i = t * 4; i < G * D; i += 64 * 4) {
        const int g = i / D, e0 = i % D;
        const float m0 = sm_m[0][g], m1 = sm_m[1][g], M = fmaxf(m0, m1);
        const float w0 = M == -INFINITY ? 0.f : exp2f(m0 - M), w1 = M == -INFINITY ? 0.f : exp2f(m1 - M);
        const float sum = fmaf(w0, sm_l[0][g], w1 * sm_l[1][g]);
        const float inv = sum != 0.f ? 1.f / sum : 0.f;  // NaN stays
        const float4 x = *reinterpret_cast<const float4*>(om + g * D + e0);
        const float4 y = *reinterpret_cast<const float4*>(om + (8 + g) * D + e0);
        const float v[4] = {fmaf(w0, x.x, w1 * y.x) * inv, fmaf(w0, x.y, w1 * y.y) * inv,
                            fmaf(w0, x.z, w1 * y.z) * inv, fmaf(w0, x.w, w1 * y.w) * inv};
        const float lse2 = sum != 0.f ? M + log2f(sum) : -INFINITY;
        if (all) {
          *reinterpret_cast<uint2*>(out + i) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
          if (e0 == 0 && lse_out) lse_out[g] = lse2 * kWmLn2;
        } else {
          *reinterpret_cast<float4*>(om + 16 * D + i) = make_float4(v[0], v[1], v[2], v[3]);
          if (e0 == 0) sm_lse[g] = lse2;
        }
      }
    }
  }
  if (all) return;
  // ---- merge the cluster's parts, each CTA a share of the outputs; CTAs without a
  // stage have left
  const int w = (nt + a.parts - 1) / a.parts, parts = (nt + w - 1) / w;  // as direct_stages
  const int part = blockIdx.x % a.parts, rank = part % a.cluster, np = min(parts - (part - rank), a.cluster);
  const int64_t rec = 2 * (int64_t)(blockIdx.x / a.cluster) * G;
  cg::cluster_group cluster = cg::this_cluster();
  __syncwarp();
  cluster.sync();
  for (int u = rank * kWmThreads + t; u < G * D / 4; u += np * kWmThreads) {
    const int g = u * 4 / D;
    float l[kWmCluster], M = -INFINITY;
    float4 x[kWmCluster];
#pragma unroll
    for (int i = 0; i < kWmCluster; ++i) {
      l[i] = -INFINITY;
      if (i < np) {
        l[i] = cluster.map_shared_rank(sm_lse, i)[g];
        x[i] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(om, i) + 16 * D + u * 4);
      }
      M = fmaxf(M, l[i] != l[i] ? INFINITY : l[i]);  // NaN is not passed over
    }
    float sum = 0.f, y[4] = {};
#pragma unroll
    for (int i = 0; i < kWmCluster; ++i) {
      if (i >= np || l[i] == -INFINITY) continue;
      const float wt = exp2f(l[i] - M);
      sum += wt;
      y[0] = fmaf(wt, x[i].x, y[0]);
      y[1] = fmaf(wt, x[i].y, y[1]);
      y[2] = fmaf(wt, x[i].z, y[2]);
      y[3] = fmaf(wt, x[i].w, y[3]);
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    const float lse2 = sum != 0.f ? M + log2f(sum) : -INFINITY;
    if (parts <= a.cluster) {
      *reinterpret_cast<uint2*>(out + u * 4) =
          make_uint2(pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv));
      if (u * 4 % D == 0 && lse_out) lse_out[g] = lse2 * kWmLn2;
    } else {
      *reinterpret_cast<float4*>(a.rec_o + rec * D + u * 4) =
          make_float4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
      if (u * 4 % D == 0) a.rec_lse[rec + g] = lse2;
    }
  }
  __syncwarp();
  cluster.sync();  // its shared memory has been read
}

template <bool kMx, int D, int G>
static int wm_resident() {
  static std::mutex mu;
  static int cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (!cached[dev]) {
    auto kern = window_mma_kernel<kMx, D, G>;
    constexpr int smem = wm_smem(kMx, D);
    int per_sm = 0, sms = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kWmThreads, smem) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return 0;
    cached[dev] = per_sm * sms;
  }
  return cached[dev];
}

// Clusters of `size` CTAs that can be resident at once.
template <bool kMx, int D, int G>
static int wm_clusters(int size) {
  static std::mutex mu;
  static int cached[64][kWmCluster + 1] = {};  // + 1
  int dev = 0;
  if (wm_resident<kMx, D, G>() <= 0 || cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  int& c = cached[dev][size];
  if (!c) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)size);
    cfg.blockDim = dim3(kWmThreads);
    cfg.dynamicSmemBytes = wm_smem(kMx, D);
    cudaLaunchAttribute attr = cluster_attr(size);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, window_mma_kernel<kMx, D, G>, &cfg) != cudaSuccess) return 0;
    c = n + 1;
  }
  return c - 1;
}

template <bool kMx, int D, int G>
static cudaError_t launch_wm(const CUtensorMap& tmk, const CUtensorMap& tmv, const WindowArgs& a,
                             cudaStream_t stream) {
  auto kern = window_mma_kernel<kMx, D, G>;
  constexpr int smem = wm_smem(kMx, D);
  static SmemAttrCache attr_cache;
  cudaError_t e = ensure_smem_limit(kern, smem, attr_cache);
  if (e != cudaSuccess) return e;
  if (a.cluster > 1)
    return launch_pdl_clusters(kern, dim3((unsigned)a.num_ctas), dim3(kWmThreads), smem, stream, a.cluster, tmk,
                               tmv, a);
  return launch_pdl(kern, dim3((unsigned)a.num_ctas), dim3(kWmThreads), smem, stream, tmk, tmv, a);
}

// Call f.operator()<kMx, D, G>() for the sizes of a call.  (MXFP8 with eight query
// heads a kv head and head_dim 64 is refused, as by the plain decode.)
template <bool kMx, int D, class F>
static auto wm_group(int group, F&& f) {
  if constexpr (!kMx || D == 128)
    if (group == 8) return f.template operator()<kMx, D, 8>();
  return group == 1   ? f.template operator()<kMx, D, 1>()
         : group == 2 ? f.template operator()<kMx, D, 2>()
                      : f.template operator()<kMx, D, 4>();
}
template <class F>
static auto wm_sizes(int dtype, int head_dim, int group, F&& f) {
  if (dtype == PKV_MXFP8)
    return head_dim == 128 ? wm_group<true, 128>(group, f) : wm_group<true, 64>(group, f);
  return head_dim == 128 ? wm_group<false, 128>(group, f) : wm_group<false, 64>(group, f);
}

namespace {
struct ResidentCall {
  template <bool kMx, int D, int G>
  int operator()() const {
    return wm_resident<kMx, D, G>();
  }
};
struct ClustersCall {
  int size;
  template <bool kMx, int D, int G>
  int operator()() const {
    return wm_clusters<kMx, D, G>(size);
  }
};
struct LaunchCall {
  const CUtensorMap &tmk, &tmv;
  const WindowArgs& a;
  cudaStream_t stream;
  template <bool kMx, int D, int G>
  cudaError_t operator()() const {
    return launch_wm<kMx, D, G>(tmk, tmv, a, stream);
  }
};
}  // namespace

int window_mma_resident_ctas(int dtype, int head_dim, int group) {
  return wm_sizes(dtype, head_dim, group, ResidentCall{});
}

int window_mma_resident_clusters(int dtype, int head_dim, int group, int size) {
  return wm_sizes(dtype, head_dim, group, ClustersCall{size});
}

cudaError_t launch_window_mma(int dtype, int head_dim, int group, const CUtensorMap& tmk,
                              const CUtensorMap& tmv, const DecodeArgs& args, cudaStream_t stream) {
  const WindowArgs a(args, box_rows_for(args.block_size));
  cudaError_t e = wm_sizes(dtype, head_dim, group, LaunchCall{tmk, tmv, a, stream});
  if (e != cudaSuccess || a.parts == a.cluster) return e;
  return launch_window_merge(dtype, head_dim, a, stream);
}

}  // namespace pkv
