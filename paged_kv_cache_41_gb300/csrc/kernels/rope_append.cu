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
// lanes, two stretches of four elements each, laid out so that both halves of a
// pair lie in one lane (split pairs: elements 4 l and rot / 2 + 4 l on; those
// that are not rotated follow, eight a lane): the only shuffles are the three or four of
// the mean.  A group of lanes takes kRows head rows of one token and one kind
// (q, k or v), so that weight and angle are multiplied into four coefficients a
// pair once for all of them.  Angles come from a table, so that far positions lose
// nothing.  K rows of an MXFP8 pool are brought into order by shuffles before their
// groups of 32 are quantised; they are few beside the queries.  Each token's first
// group asks a later token's rows into L2.  32768 tokens of 32/8 heads, bf16: 123
// us, 6690 GB/s read and written, 98% of a copy's rate.
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace pkv {

namespace {

constexpr int kRopeThreads = 128;
// Bytes of q, k and v between a token and the one that its first group asks into
// L2: about what the resident groups have in hand.  There are not warps enough to cover DRAM's
// latency twice (positions, then angles): 32768 tokens (12 KiB each) take 138 us
// without, 124.2 / 123.0 / 123.4 / 125.4 with 300 / 600 / 1000 / 1500 of them
// between, 166 with 3000.
constexpr int64_t kRopeAheadBytes = 8 << 20;
// Elements of q, k and v up to which a group of lanes takes one head row, so that
// every SM has some; above, four, so that a token's weights and angles are multiplied
// once for four.  One against four, us, 32/8 heads, by millions of elements:
//   bf16, head_dim 128: 0.75 2.6 / 2.9, 1 2.90 / 2.91, 1.25 3.4 / 3.2, 2.5 4.9 / 3.7;
//   64/8 heads, head_dim 64: 1 2.9 / 3.1, 1.25 3.2 / 3.2, 2.5 4.7 / 3.6;
//   fp32, head_dim 128: 0.75 3.07 / 3.10, 1 3.3 / 3.2, 2.5 5.2 / 4.0; 64: 1 3.1 / 3.1, 1.25 3.4 / 3.3;
//   MXFP8, head_dim 128: 1 3.4 / 4.4, 2 4.8 / 4.9, 2.5 5.4 / 5.1, 5 8.6 / 7.6;
//   64: 1 3.0 / 5.3, 4 7.1 / 7.9, 8 13.0 / 13.3, 16 25.6 / 23.7; 64/8 heads 4 7.0 / 7.1, 8 13.2 / 12.1.
constexpr int64_t rope_few(bool mx, int d) { return mx ? (d == 128 ? 2200000 : 6000000) : 1100000; }

// Four consecutive elements as they lie in memory.
template <typename T>
struct Raw4;
template <>
struct Raw4<float> {
  float4 w;
  __device__ __forceinline__ void load(const float* p) { w = __ldg(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = w; }
  __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w; }
  __device__ __forceinline__ void set(const float (&x)[4]) { w = make_float4(x[0], x[1], x[2], x[3]); }
};
template <>
struct Raw4<__nv_bfloat16> {
  uint2 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    w = __ldg(reinterpret_cast<const uint2*>(p));
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = w; }
  __device__ __forceinline__ void get(float (&x)[4]) const {
    x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
  }
  __device__ __forceinline__ void set(const float (&x)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};

// Four values as E4M3 codes of the scale 2^e.
__device__ __forceinline__ uint32_t mx_codes4(float a, float b, float c, float d, int e) {
  const float inv = mx_inverse_scale(e);
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c * inv, d * inv), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

}  // namespace

// Quantise eight consecutive values a lane (lane l: elements 8 l ..), groups of
// 32 being four lanes, into row `hk` of slot `slot`.
template <int D>
__device__ __forceinline__ void store_mx(const RopeArgs& a, void* cache, const float (&y)[8], int64_t slot,
                                         int hk, int l, unsigned lanes) {
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[e]));
  amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, 2));
  if (slot < 0) return;
  const int ex = mx_scale_exponent(amax), Hkv = a.num_kv_heads;
  uint8_t* pool = static_cast<uint8_t*>(cache);
  const int64_t blk = slot / a.block_size, off = slot - blk * a.block_size;
  *reinterpret_cast<uint2*>(pool + (slot * Hkv + hk) * D + l * 8) =
      make_uint2(mx_codes4(y[0], y[1], y[2], y[3], ex), mx_codes4(y[4], y[5], y[6], y[7], ex));
  if (l % 4 == 0)
    pool[a.plane_bytes + ((blk * Hkv + hk) * a.block_size + off) * (D / 32) + l / 4] = (uint8_t)(ex + 127);
}

// Group g of D / 8 lanes takes up to kRows head rows of token g / parts: of
// its parts, the first ceil(Hq / kRows) are q's, then come k's and v's.
// kWhole: the whole head is rotated (rot = D), so that no lane asks whether its
// elements are: 32768 tokens 123.8 us, 125.2 where they ask.
// Four rows of 16-bit elements: 56 registers, nine CTAs an SM (32768 tokens 122 us; with
// eight CTAs 127, ten 125); quantising takes eight (8192 tokens 44.3 us; with seven
// 45.3).
template <typename T, bool kMx, int D, bool kInter, int kRows, bool kWhole>
__global__ void
__launch_bounds__(kRopeThreads, kRows == 4 && sizeof(T) == 2 ? (kMx ? 8 : 9) : 1)
    rope_append_kernel(const RopeArgs a) {
  constexpr int LPR = D / 8;  // lanes of a head row
  pdl_launch_dependents();    // a decode after this append may be scheduled now
  const int Hq = a.num_q_heads, Hkv = a.num_kv_heads;
  const int qparts = (Hq + kRows - 1) / kRows, kparts = (Hkv + kRows - 1) / kRows;
  const int parts = qparts + 2 * kparts;
  const unsigned g = blockIdx.x * (unsigned)(kRopeThreads / LPR) + threadIdx.x / LPR;  // at most 2^29
  const int l = threadIdx.x % LPR;
  const unsigned lanes = (LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1)) << ((threadIdx.x & 31) / LPR * LPR);
  const unsigned tok32 = g / (unsigned)parts;
  const int64_t tok = tok32;
  if (tok >= a.num_tokens) return;  // a group leaves together
  int part = (int)(g - tok32 * parts);
  const bool token_first = part == 0;
  const int kind = part < qparts ? 0 : part < qparts + kparts ? 1 : 2;  // q, k, v
  part -= kind == 0 ? 0 : kind == 1 ? qparts : qparts + kparts;
  const int heads = kind == 0 ? Hq : Hkv;
  const int h0 = part * kRows, nrows = min(kRows, heads - h0);
  const T* src = kind == 0   ? static_cast<const T*>(a.q) + tok * a.q_stride
                 : kind == 1 ? static_cast<const T*>(a.k) + tok * a.k_stride
                             : static_cast<const T*>(a.v) + tok * a.v_stride;
  src += (int64_t)h0 * D;
  // this lane's elements: o0 .. o0 + 3 and o1 .. o1 + 3
  const int half = a.rot / 2;
  const bool turned = 8 * l < a.rot && kind != 2;
  const bool split = !kInter && turned;
  const int o0 = split ? 4 * l : 8 * l, o1 = split ? half + 4 * l : 8 * l + 4;

  // ---- the rows, and where they go
  if (kRows > 1 && token_first && a.ahead > 0 && tok + a.ahead < a.num_tokens) {
    // a later token's rows and angles, into L2 (kRopeAheadBytes)
    const int64_t far_tok = tok + a.ahead;
    if (l == 0) prefetch_l2_bulk(static_cast<const T*>(a.q) + far_tok * a.q_stride, (uint32_t)(Hq * D * sizeof(T)));
    if (l == 1) prefetch_l2_bulk(static_cast<const T*>(a.k) + far_tok * a.k_stride, (uint32_t)(Hkv * D * sizeof(T)));
    if (l == 2) prefetch_l2_bulk(static_cast<const T*>(a.v) + far_tok * a.v_stride, (uint32_t)(Hkv * D * sizeof(T)));
    if (l >= 4 && l < 4 + a.axes && a.rot > 0) {
      const int p = a.positions[(l - 4) * a.pos_stride + far_tok];
      if (p >= 0 && p < a.max_positions) prefetch_l2_bulk(a.cos_sin + (int64_t)p * a.rot, (uint32_t)(a.rot * 4));
    }
  }
  Raw4<T> x[kRows][2];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int h = min(i, nrows - 1);  // past the last: it again, not stored
    x[i][0].load(src + h * D + o0);
    x[i][1].load(src + h * D + o1);
  }
  int64_t slot = a.slots[tok];
  // positions: a negative one marks a row of no token
  int pos[kMaxAxes] = {};
  bool skip = false, far = false;
#pragma unroll
  for (int ax = 0; ax < kMaxAxes; ++ax)
    if (ax < a.axes) {
      pos[ax] = a.positions[ax * a.pos_stride + tok];
      skip |= pos[ax] < 0;
      far |= pos[ax] >= a.max_positions;
    }
  if (skip || far) {
    if (!skip && token_first && l == 0) atomicOr(a.err, PKV_DEVERR_POSITION);
    return;
  }
  if (slot >= a.num_slots) {
    if (token_first && l == 0) atomicOr(a.err, PKV_DEVERR_SLOT);
    slot = -1;
  }
  void* cache = kind == 1 ? a.k_cache : a.v_cache;
  if (kind != 0 && slot < 0) return;
  if (kind == 2) {  // values go as they are
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (i >= nrows) break;
      if constexpr (kMx) {
        float y[8], z[4];
        x[i][0].get(z);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = z[e];
        x[i][1].get(z);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[4 + e] = z[e];
        store_mx<D>(a, cache, y, slot, h0 + i, l, lanes);
      } else {
        T* dst = static_cast<T*>(cache) + (slot * Hkv + h0 + i) * D;
        x[i][0].store(dst + o0);
        x[i][1].store(dst + o1);
      }
    }
    return;
  }

  // ---- coefficients: with w the weights of a pair (a, b), c and s its angle,
  //   y_a = x_a (w_a c) - x_b (w_b s),   y_b = x_b (w_b c) + x_a (w_a s)
  float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
  if (turned) {
    const int j0 = 4 * l;
    if (a.uniform >> l & 1) {  // one axis for all four
      const int ax = a.axis_of[j0];
      const float* row = a.cos_sin + (int64_t)(ax == 0 ? pos[0] : ax == 1 ? pos[1] : pos[2]) * a.rot + j0;
      VecLoad<float, 4>::run(row, cs);
      VecLoad<float, 4>::run(row + half, sn);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int ax = a.axis_of[j0 + j];
        const float* row = a.cos_sin + (int64_t)(ax == 0 ? pos[0] : ax == 1 ? pos[1] : pos[2]) * a.rot + j0 + j;
        cs[j] = row[0];
        sn[j] = row[half];
      }
    }
  }
  // element pairs of the lane: (first, second) of pair j
  auto first = [](int j) { return kInter ? 2 * j : j; };
  auto second = [](int j) { return kInter ? 2 * j + 1 : 4 + j; };
  // two pairs to a packed operation
  float2 aa[2], ab[2], bb[2], ba[2];
  const float* w = kind == 0 ? a.q_weight : a.k_weight;
  {
    float wt[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (w) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(w + o0)), v = __ldg(reinterpret_cast<const float4*>(w + o1));
      wt[0] = u.x, wt[1] = u.y, wt[2] = u.z, wt[3] = u.w;
      wt[4] = v.x, wt[5] = v.y, wt[6] = v.z, wt[7] = v.w;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 wa = make_float2(wt[first(2 * j)], wt[first(2 * j + 1)]);
      const float2 wb = make_float2(wt[second(2 * j)], wt[second(2 * j + 1)]);
      const float2 c2 = make_float2(cs[2 * j], cs[2 * j + 1]), s2 = make_float2(sn[2 * j], sn[2 * j + 1]);
      aa[j] = __fmul2_rn(wa, c2);
      ab[j] = __fmul2_rn(wb, make_float2(-s2.x, -s2.y));
      bb[j] = __fmul2_rn(wb, c2);
      ba[j] = __fmul2_rn(wa, s2);
    }
  }

#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (i >= nrows) break;
    float v[8];
    {
      float z[4];
      x[i][0].get(z);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = z[e];
      x[i][1].get(z);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 + e] = z[e];
    }
    float2 va[2], vb[2];  // the pairs' halves
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      va[j] = make_float2(v[first(2 * j)], v[first(2 * j + 1)]);
      vb[j] = make_float2(v[second(2 * j)], v[second(2 * j + 1)]);
    }
    if (w) {
      float2 s2 = __fmul2_rn(va[0], va[0]);
      s2 = __ffma2_rn(va[1], va[1], s2);
      s2 = __ffma2_rn(vb[0], vb[0], s2);
      s2 = __ffma2_rn(vb[1], vb[1], s2);
      float ss = s2.x + s2.y;
#pragma unroll
      for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(lanes, ss, o);
      const float inv = rsqrtf(ss * (1.f / D) + a.eps);
      const float2 i2 = make_float2(inv, inv);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        va[j] = __fmul2_rn(va[j], i2);
        vb[j] = __fmul2_rn(vb[j], i2);
      }
    }
    float y[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float2 ya = __ffma2_rn(va[j], aa[j], __fmul2_rn(vb[j], ab[j]));
      float2 yb = __ffma2_rn(vb[j], bb[j], __fmul2_rn(va[j], ba[j]));
      if (!kWhole && !turned) {  // by themselves: an infinity times a sine of 0 is NaN
        ya = __fmul2_rn(va[j], aa[j]);
        yb = __fmul2_rn(vb[j], bb[j]);
      }
      y[first(2 * j)] = ya.x;
      y[first(2 * j + 1)] = ya.y;
      y[second(2 * j)] = yb.x;
      y[second(2 * j + 1)] = yb.y;
    }
    if (kMx && kind == 1) {
      // into order: lane l wants elements 8 l .., the stretches 2 l and 2 l + 1
      float z[8];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int u = 2 * l + c;
        int from = l, which = c;  // interleaved, or not rotated: in order already
        if (!kInter && 4 * u < a.rot) {
          which = 4 * u >= half;
          from = which ? u - half / 4 : u;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float s0 = __shfl_sync(lanes, y[e], from, LPR), s1 = __shfl_sync(lanes, y[4 + e], from, LPR);
          z[4 * c + e] = which ? s1 : s0;
        }
      }
      store_mx<D>(a, cache, z, slot, h0 + i, l, lanes);
    } else {
      T* dst = kind == 0 ? static_cast<T*>(a.out) + (tok * Hq + h0 + i) * D
                         : static_cast<T*>(cache) + (slot * Hkv + h0 + i) * D;
      Raw4<T> o;
      const float lo[4] = {y[0], y[1], y[2], y[3]}, hi[4] = {y[4], y[5], y[6], y[7]};
      o.set(lo);
      o.store(dst + o0);
      o.set(hi);
      o.store(dst + o1);
    }
  }
}

template <typename T, bool kMx, int D, bool kInter>
static cudaError_t launch_rope_t(const RopeArgs& args, cudaStream_t stream) {
  RopeArgs a = args;
  const int64_t H = a.num_q_heads + 2 * (int64_t)a.num_kv_heads;
  const int per_cta = kRopeThreads / (D / 8);
  const bool few = a.num_tokens * H * D <= rope_few(kMx, D);
  const int64_t groups =
      a.num_tokens * (few ? H : (a.num_q_heads + 3) / 4 + 2 * ((a.num_kv_heads + 3) / 4));
  const unsigned grid = (unsigned)((groups + per_cta - 1) / per_cta);
  a.ahead = (int)std::max<int64_t>(kRopeAheadBytes / (H * D * (int64_t)sizeof(T)), 1);
  auto kern = few ? (a.rot == D ? rope_append_kernel<T, kMx, D, kInter, 1, true>
                                : rope_append_kernel<T, kMx, D, kInter, 1, false>)
                  : (a.rot == D ? rope_append_kernel<T, kMx, D, kInter, 4, true>
                                : rope_append_kernel<T, kMx, D, kInter, 4, false>);
  kern<<<grid, kRopeThreads, 0, stream>>>(a);
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
