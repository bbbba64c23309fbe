// rope_append.cu -- norms of queries and keys, their rotation by position, and
// the append of K and V, in one pass over a step's projections.
//
// What it computes (pkv_qk_norm_rope_append): for every head row x of q and k
//   x^ = x * rsqrt(mean x^2 + eps) * w               (where a weight is given)
//   (x^_a, x^_b) -> (x^_a c - x^_b s, x^_b c + x^_a s) for each pair j of the
// first `rot` elements, c and s the cosine and sine of pair j at the token's
// position on axis axis_of[j]; q goes to `out`, k and the untouched v to their
// slots of the pools (an MXFP8 pool: quantised straight from the 32-bit values).
//
// Design (GB300): the bytes are those of q, k and v once in and once out, so
// the whole is one kernel bound by memory.  A head row is held by head_dim / 8
// lanes, eight elements (a 16-byte load of bf16) each: the mean is three or
// four shuffles, and a pair's other half is eight shuffles away (or in the same
// lane, where pairs are interleaved).  Angles come from a table, so that far
// positions lose nothing: a lane reads its eight cosines and sines once for
// the kRows head rows of its token that it takes.
#include "common.cuh"
#include "launch.h"

namespace pkv {

namespace {

constexpr int kRopeThreads = 256;

template <int N>
__device__ __forceinline__ void store_row(float* p, const float (&y)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
}
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&y)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Four values as E4M3 codes of the scale 2^e.
__device__ __forceinline__ uint32_t mx_codes4(float a, float b, float c, float d, int e) {
  const float inv = mx_inverse_scale(e);
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c * inv, d * inv), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

}  // namespace

// Group of D / 8 lanes g takes head rows g % parts + parts * i (i < kRows) of
// token g / parts; rows 0 .. Hq - 1 are q's, then k's, then v's.
template <typename T, bool kMx, int D, bool kInter, int kRows>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeArgs a) {
  constexpr int LPR = D / 8;  // lanes of a head row
  pdl_launch_dependents();    // a decode after this append may be scheduled now
  const int Hq = a.num_q_heads, Hkv = a.num_kv_heads, H = Hq + 2 * Hkv;
  const int parts = (H + kRows - 1) / kRows;
  const int64_t g = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) / LPR;
  const int l = threadIdx.x % LPR;  // elements 8 l .. 8 l + 7
  const int64_t tok = g / parts;
  const int part = (int)(g - tok * parts);
  bool on = tok < a.num_tokens;

  // ---- the rows, and where they go
  float x[kRows][8];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int h = part + i * parts;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
    if (on && h < H) {
      const T* src = h < Hq ? static_cast<const T*>(a.q) + tok * a.q_stride + (int64_t)h * D
                     : h < Hq + Hkv
                         ? static_cast<const T*>(a.k) + tok * a.k_stride + (int64_t)(h - Hq) * D
                         : static_cast<const T*>(a.v) + tok * a.v_stride + (int64_t)(h - Hq - Hkv) * D;
      VecLoad<T, 8>::run(src + l * 8, x[i]);
    }
  }
  int64_t slot = on ? a.slots[tok] : -1;
  // positions: a negative one marks a row of no token
  int pos[kMaxAxes];
#pragma unroll
  for (int ax = 0; ax < kMaxAxes; ++ax) {
    pos[ax] = on && ax < a.axes ? a.positions[ax * a.pos_stride + tok] : 0;
  }
  bool skip = false, far = false;
#pragma unroll
  for (int ax = 0; ax < kMaxAxes; ++ax) {
    skip |= pos[ax] < 0;
    far |= pos[ax] >= a.max_positions;
  }
  if (on && far && !skip && part == 0 && l == 0) atomicOr(a.err, PKV_DEVERR_POSITION);
  on = on && !skip && !far;
  if (slot >= a.num_slots) {
    if (on && part == 0 && l == 0) atomicOr(a.err, PKV_DEVERR_SLOT);
    slot = -1;
  }

  // ---- this lane's cosines and sines
  constexpr int NP = kInter ? 4 : 8;  // pairs that its elements belong to
  const int half = a.rot / 2;
  const bool turned = 8 * l < a.rot;            // rot is a multiple of 16
  const bool second = !kInter && 8 * l >= half;  // its elements are the pairs' second ones
  const int j0 = kInter ? 4 * l : second ? 8 * l - half : 8 * l;
  float cs[NP], sn[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    cs[j] = 1.f;
    sn[j] = 0.f;
  }
  if (on && turned) {
    const int ax0 = a.axis_of[j0];
    if (a.uniform >> (j0 / NP) & 1) {  // one axis for all of them
      const int p = ax0 == 0 ? pos[0] : ax0 == 1 ? pos[1] : pos[2];
      const float* row = a.cos_sin + (int64_t)p * a.rot + j0;
      VecLoad<float, NP>::run(row, cs);
      VecLoad<float, NP>::run(row + half, sn);
    } else {
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int ax = a.axis_of[j0 + j];
        const int p = ax == 0 ? pos[0] : ax == 1 ? pos[1] : pos[2];
        const float* row = a.cos_sin + (int64_t)p * a.rot + j0 + j;
        cs[j] = row[0];
        sn[j] = row[half];
      }
    }
  }

#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int h = part + i * parts;
    const bool is_q = h < Hq, is_v = h >= Hq + Hkv;
    // ---- norm
    const float* w = is_q ? a.q_weight : a.k_weight;
    const bool normed = !is_v && w != nullptr;
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[i][e], x[i][e], ss);
#pragma unroll
    for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (normed) {
      const float inv = rsqrtf(ss * (1.f / D) + a.eps);
      float wf[8];
      VecLoad<float, 8>::run(w + l * 8, wf);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] *= inv * wf[e];
    }
    // ---- rotation
    float y[8];
    if constexpr (kInter) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[2 * j] = x[i][2 * j] * cs[j] - x[i][2 * j + 1] * sn[j];
        y[2 * j + 1] = x[i][2 * j + 1] * cs[j] + x[i][2 * j] * sn[j];
      }
    } else {
      const int other = second ? l - half / 8 : l + half / 8;
      float z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = __shfl_sync(0xffffffffu, x[i][e], other & (LPR - 1), LPR);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = x[i][e] * cs[e] + (second ? z[e] * sn[e] : -z[e] * sn[e]);
    }
    if (is_v || !turned) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = x[i][e];
    }
    // ---- to where it belongs
    const int hk = is_v ? h - Hq - Hkv : h - Hq;  // kv head
    if constexpr (kMx) {
      // the scale of a group of 32: four lanes
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[e]));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      if (!is_q && on && h < H && slot >= 0) {
        const int ex = mx_scale_exponent(amax);
        uint8_t* pool = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache);
        const int64_t blk = slot / a.block_size, off = slot - blk * a.block_size;
        *reinterpret_cast<uint2*>(pool + (slot * Hkv + hk) * D + l * 8) =
            make_uint2(mx_codes4(y[0], y[1], y[2], y[3], ex), mx_codes4(y[4], y[5], y[6], y[7], ex));
        if (l % 4 == 0)
          pool[a.plane_bytes + ((blk * Hkv + hk) * a.block_size + off) * (D / 32) + l / 4] =
              (uint8_t)(ex + 127);
      }
    } else if (!is_q && on && h < H && slot >= 0) {
      store_row(static_cast<T*>(is_v ? a.v_cache : a.k_cache) + (slot * Hkv + hk) * D + l * 8, y);
    }
    if (is_q && on) store_row(static_cast<T*>(a.out) + (tok * Hq + h) * D + l * 8, y);
  }
}

template <typename T, bool kMx, int D, bool kInter>
static cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t stream) {
  const int64_t H = a.num_q_heads + 2 * (int64_t)a.num_kv_heads;
  const int per_cta = kRopeThreads / (D / 8);
  // Few rows: one a group, so that every SM has some.  Many: four, so that a
  // token's angles are read once for four.
  const bool few = a.num_tokens * H <= 20000;
  const int64_t groups = a.num_tokens * (few ? H : (H + 3) / 4);
  const unsigned grid = (unsigned)((groups + per_cta - 1) / per_cta);
  if (few)
    rope_append_kernel<T, kMx, D, kInter, 1><<<grid, kRopeThreads, 0, stream>>>(a);
  else
    rope_append_kernel<T, kMx, D, kInter, 4><<<grid, kRopeThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, bool kMx>
static cudaError_t launch_rope_dim(const RopeArgs& a, int head_dim, bool inter, cudaStream_t stream) {
  if (head_dim == 128)
    return inter ? launch_rope_t<T, kMx, 128, true>(a, stream) : launch_rope_t<T, kMx, 128, false>(a, stream);
  return inter ? launch_rope_t<T, kMx, 64, true>(a, stream) : launch_rope_t<T, kMx, 64, false>(a, stream);
}

cudaError_t launch_rope_append(int dtype, int head_dim, bool interleaved, const RopeArgs& a,
                               cudaStream_t stream) {
  if (dtype == PKV_MXFP8) return launch_rope_dim<__nv_bfloat16, true>(a, head_dim, interleaved, stream);
  if (dtype == PKV_BF16) return launch_rope_dim<__nv_bfloat16, false>(a, head_dim, interleaved, stream);
  return launch_rope_dim<float, false>(a, head_dim, interleaved, stream);
}

}  // namespace pkv
