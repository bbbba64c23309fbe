// verify.cu -- drafted tokens against the target's probabilities.
//
// What it computes (pkv_draft_verify): a walk down a request's tree of drafted
// tokens.  At node i with target row p and draft row q the children are tried
// in ascending order, with weights
//   r(v) = max(p(v) - c q(v), 0),   R = sum_v r(v),   c = 0 before the first
// child and R = 1 there: child x with number u is accepted where u q(x) R <
// r(x), else c grows by R and the next child is tried.  (Turning x down leaves
// the distribution max(p' - q, 0) / sum of it, p' = r / R; r's closed form
// follows because q >= 0: max(max(p - a q, 0) - b q, 0) = max(p - (a + b) q, 0).)
// Tokens that the draft chose outright (no q) are tried at their mass among
// what is left, u R < p(x), and their mass is taken out of p.  Where the walk
// ends the next token is the first v whose running sum of r passes u R.
//
// Design (GB300): the bytes are one row of p (and of q) a request, the rest is
// a chain of dependent steps.  A cluster of CTAs takes a request: each walks
// the tree by itself (64 nodes in shared memory), and where a sum over the
// vocabulary is wanted each warp of the cluster sums one segment and the sums are
// read through distributed shared memory.  The CTA whose segment holds the
// wanted place sums that segment again in eighths, one a warp, until what is left
// is two steps of a warp (64 requests: 21.3 us, 26.0 with one warp walking its
// segment alone, a step behind the other).
//   * Sums are whole numbers: a probability is held as a multiple of 2^-60
//     (exact from 2^-37 up, rounded below), so they are exact, do not depend on
//     how the row was cut, and a segment's second reading meets the place that
//     its sum promised.  Sums in fp32 would move the borders between tokens by
//     more than the smallest of them.
//   * The tests of single tokens are in 64 bits, u q < p exactly.
#include <cooperative_groups.h>

#include "common.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace pkv {

namespace {

constexpr int kVfThreads = 256;
constexpr int kVfWarps = kVfThreads / 32;
constexpr int kVfMaxCluster = 8;
constexpr int kVfWave = 560;  // CTAs that run at once; clusters of eight do not fill all 608 places
constexpr int kVfNodes = 64;  // PKV_MAX_DRAFT
static_assert(kVfWarps * kVfMaxCluster <= 64, "a warp holds two segments' sums a lane");
typedef unsigned long long u64;

// x held to [0, 1]; NaN counts as 0.
__device__ __forceinline__ float as_prob(float x) { return __saturatef(x); }

// A number of [0, 1] as a 2^-20 + b 2^-40 + c 2^-60, rounded to the nearest
// multiple of 2^-60.  Adding 8 leaves x as a multiple of 2^-20 in the low bits
// of the sum; what that left out is exact in fp32 and goes on in the same way.
// Seven additions and three integer ones a number, none of them in 64 bits: 64
// requests took 26.0 us so and 39.9 with mantissas shifted to their place (and
// twice the threads).
struct Limbs {
  int a, b, c;
};
constexpr float kLimb1 = 8.0f, kLimb2 = 12.0f * 0x1p-20f, kLimb3 = 12.0f * 0x1p-40f;
__device__ __forceinline__ Limbs limbs(float x) {
  const float t1 = __fadd_rn(x, kLimb1);
  const float r1 = __fsub_rn(x, __fsub_rn(t1, kLimb1));
  const float t2 = __fadd_rn(r1, kLimb2);
  const float r2 = __fsub_rn(r1, __fsub_rn(t2, kLimb2));
  const float t3 = __fadd_rn(r2, kLimb3);
  return {__float_as_int(t1) - __float_as_int(kLimb1), __float_as_int(t2) - __float_as_int(kLimb2),
          __float_as_int(t3) - __float_as_int(kLimb3)};
}
__device__ __forceinline__ u64 whole(const Limbs& x) {
  return (u64)(x.a * (1ll << 40) + x.b * (1ll << 20) + x.c);
}
__device__ __forceinline__ u64 fixed60(float x) { return whole(limbs(x)); }

// u of [0, 1) as a multiple of 2^-64.
__device__ __forceinline__ u64 fixed64(float u) {
  const uint32_t b = __float_as_uint(u);
  const int e = (int)(b >> 23);
  if (e == 0) return 0;
  const u64 m = (u64)((b & 0x7fffffu) | 0x800000u);
  const int s = e - 86;
  return s >= 0 ? m << s : (s > -24 ? m >> -s : 0);
}

// max(P - c Q, 0) of fixed numbers, c a multiple of 2^-56.
template <bool kOne>
__device__ __forceinline__ u64 rest(u64 p, u64 q, u64 c) {
  u64 cq = q;
  if constexpr (!kOne) {
    const u64 top = __umul64hi(q, c);
    cq = top >> 56 ? ~0ull : (top << 8) | ((q * c) >> 56);
  }
  return p > cq ? p - cq : 0;
}

// One row's weights of a request: p, and q where there is one.
struct VfRow {
  const float* p;
  const float* q;  // null: none is taken off
  u64 c;           // 2^56: once
};

// Elements v .. v + 3 of the row, held to [0, 1] (0 past the end).
template <bool kVec, bool kQ>
__device__ __forceinline__ void load4(const VfRow& row, int v, int end, float (&p)[4], float (&q)[4]) {
  if (kVec && v + 4 <= end) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(row.p + v));
    p[0] = x.x, p[1] = x.y, p[2] = x.z, p[3] = x.w;
    if constexpr (kQ) {
      const float4 y = __ldg(reinterpret_cast<const float4*>(row.q + v));
      q[0] = y.x, q[1] = y.y, q[2] = y.z, q[3] = y.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = v + i < end ? __ldg(row.p + v + i) : 0.f;
      if constexpr (kQ) q[i] = v + i < end ? __ldg(row.q + v + i) : 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[i] = as_prob(p[i]);
    if constexpr (kQ) q[i] = as_prob(q[i]);
  }
}

// ... and as weights.
template <bool kVec, bool kQ, bool kOne>
__device__ __forceinline__ void weights4(const VfRow& row, int v, int end, u64 (&w)[4]) {
  float p[4], q[4];
  load4<kVec, kQ>(row, v, end, p, q);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = fixed60(p[i]);
    if constexpr (kQ) w[i] = rest<kOne>(w[i], fixed60(q[i]), row.c);
  }
}

// The sum of the weights of [lo, hi), this lane's share.
template <bool kVec, bool kQ, bool kOne>
__device__ __forceinline__ u64 segment_sum(const VfRow& row, int lo, int hi, int lane) {
  u64 sum = 0;
  if constexpr (kQ && !kOne) {
#pragma unroll 2
    for (int v = lo + lane * 4; v < hi; v += 128) {
      u64 w[4];
      weights4<kVec, true, false>(row, v, hi, w);
      sum += (w[0] + w[1]) + (w[2] + w[3]);
    }
  } else {
    // limbs apart, in 32 bits: kRun numbers of 2^20 at most
    constexpr int kRun = 1024;
    for (int v0 = lo + lane * 4; v0 < hi; v0 += kRun / 4 * 128) {
      Limbs s = {0, 0, 0};
      const int stop = min(hi, v0 + kRun / 4 * 128);
#pragma unroll 2
      for (int v = v0; v < stop; v += 128) {
        float p[4], q[4];
        load4<kVec, kQ>(row, v, hi, p, q);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (kQ) {  // max(p - q, 0), the two apart
            const bool over = p[i] > q[i];
            const Limbs x = limbs(over ? p[i] : 0.f), y = limbs(over ? q[i] : 0.f);
            s.a += x.a - y.a;
            s.b += x.b - y.b;
            s.c += x.c - y.c;
          } else {
            const Limbs x = limbs(p[i]);
            s.a += x.a;
            s.b += x.b;
            s.c += x.c;
          }
        }
      }
      sum += whole(s);
    }
  }
  return sum;
}

// First element of [lo, hi) whose running sum passes `want`, the tokens of
// `out` (n of them) counting nothing; hi - 1 if none does.  A warp.
template <bool kVec>
__device__ __forceinline__ int segment_find(const VfRow& row, int lo, int hi, int lane, u64 want,
                                            const int* out, int n) {
  u64 before = 0;
  for (int v0 = lo; v0 < hi; v0 += 128) {
    const int v = v0 + lane * 4;
    u64 w[4];
    if (row.q)  // c = 1 like any other: one copy of the code
      weights4<kVec, true, false>(row, v, hi, w);
    else
      weights4<kVec, false, true>(row, v, hi, w);
    for (int k = 0; k < n; ++k) {
      const int d = out[k] - v;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (d == i) w[i] = 0;
    }
    const u64 mine = (w[0] + w[1]) + (w[2] + w[3]);
    u64 upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + upto > want);
    if (hit) {
      const int l = __ffs(hit) - 1;
      u64 run = before + upto - mine;
      int at = v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        run += w[i];
        if (run <= want) at = v + i + 1;
      }
      return __shfl_sync(0xffffffffu, at, l);
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return hi - 1;
}

}  // namespace

template <bool kVec>
__global__ void __launch_bounds__(kVfThreads, 4) draft_verify_kernel(const VerifyArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ int s_tok[kVfNodes], s_out[kVfNodes];  // tokens; those turned down here
  __shared__ u64 s_outw[kVfNodes];                   // ... and their mass, once each
  __shared__ float s_u[kVfNodes], s_p[kVfNodes], s_q[kVfNodes];
  __shared__ u64 s_kids[kVfNodes];
  __shared__ u64 s_ok;                    // children that pass their first trial
  __shared__ u64 seg[2][kVfWarps];        // this CTA's segments, by sum
  __shared__ u64 all[kVfWarps * kVfMaxCluster];
  __shared__ u64 part_sum[2][kVfWarps];
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int r = blockIdx.x / C;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int S = C * kVfWarps;             // segments of the row
  const int V = a.vocab;

  // ---- the request's nodes
  const int p0 = a.draft_ptr[r], p1 = a.draft_ptr[r + 1];
  const bool bad = p0 < 0 || p1 < p0 || p1 - p0 > a.max_draft || p1 > a.num_rows;
  const int n = bad ? 0 : p1 - p0;
  if (bad && rank == 0 && t == 0) atomicOr(a.err, PKV_DEVERR_LENGTH);
  if (n == 0) {  // the whole cluster leaves
    if (rank == 0) {
      for (int i = t; i < a.max_draft; i += kVfThreads) a.keep[(int64_t)r * a.max_draft + i] = -1;
      if (t == 0) {
        a.keep_lens[r] = 0;
        a.next_tokens[r] = -1;
      }
    }
    return;
  }
  if (t < kVfNodes) s_kids[t] = 0;
  if (t == 0) s_ok = 0;
  __syncthreads();
  if (t < n) {
    const int64_t row = (int64_t)p0 + t;
    const u64 mask = a.masks ? a.masks[row] : 0;
    // the parent: the last ancestor in the node's mask, or the node before
    const u64 older = a.masks ? mask & ((1ull << t) - 1) : t > 0 ? 1ull << (t - 1) : 0;
    const int up = older ? 63 - __clzll((long long)older) : -1;
    const int tok = a.tokens[row];
    float u = a.uniforms[row];
    u = u >= 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f;
    const bool known = tok >= 0 && tok < V;
    if (t > 0 && !known && rank == 0) atomicOr(a.err, PKV_DEVERR_TOKEN);
    float p = 0.f, q = 1.f;
    if (known && up >= 0) {
      p = as_prob(__ldg(a.target + (p0 + up) * a.target_stride + tok));
      if (a.draft) q = as_prob(__ldg(a.draft + (p0 + up) * a.draft_stride + tok));
    }
    s_tok[t] = tok;
    s_u[t] = u;
    s_p[t] = p;
    s_q[t] = q;
    if (known && up >= 0) {  // any other is never reached
      atomicOr(&s_kids[up], 1ull << t);
      if ((double)u * (double)q < (double)p) atomicOr(&s_ok, 1ull << t);
    }
  }
  __syncthreads();

  // ---- sums over the vocabulary, the whole cluster: every thread gets R
  const int per = (((V + S - 1) / S) + 127) & ~127;
  const int lo = (int)min((int64_t)(rank * kVfWarps + warp) * per, (int64_t)V), hi = min(lo + per, V);
  const u64 one = 1ull << 56;
  int sums = 0;
  auto range_sum = [&](const VfRow& row, int from, int to) -> u64 {  // a warp
    u64 sum = !row.q          ? segment_sum<kVec, false, true>(row, from, to, lane)
              : row.c == one ? segment_sum<kVec, true, true>(row, from, to, lane)
                             : segment_sum<kVec, true, false>(row, from, to, lane);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
  };
  auto total_of = [&](const VfRow& row) -> u64 {
    const u64 sum = range_sum(row, lo, hi);
    // two buffers in turn: one is written again only after every CTA has
    // passed the next sum's barrier, so has read this one's
    u64* mine = seg[sums & 1];
    if (lane == 0) mine[warp] = sum;
    ++sums;
    cluster.sync();
    if (t < S) all[t] = cluster.map_shared_rank(mine, t / kVfWarps)[t % kVfWarps];
    __syncthreads();
    u64 total = 0;
    for (int s = lane; s < S; s += 32) total += all[s];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    return total;
  };
  auto row_at = [&](int node, u64 c) {
    VfRow row;
    row.p = a.target + (p0 + node) * a.target_stride;
    row.q = a.draft && c ? a.draft + (p0 + node) * a.draft_stride : nullptr;
    row.c = c;
    return row;
  };

  // ---- the walk, the same in every thread of the cluster
  u64 kept = 1;       // accepted nodes
  int at = 0, n_out = 0;
  double c = 0.0, mass = 1.0;
  u64 kids = s_kids[0];
  auto fixed_c = [&](double x) { return (u64)(x * 0x1p56); };
  while (kids) {
    const int x = __ffsll((long long)kids) - 1;
    kids &= kids - 1;
    bool yes;
    double part = 0.0;
    if (n_out == 0) {
      yes = s_ok >> x & 1;
      part = s_p[x];
    } else if (a.draft) {
      part = fmax((double)s_p[x] - c * (double)s_q[x], 0.0);
      yes = (double)s_u[x] * (double)s_q[x] * mass < part;
    } else {
      bool twice = false;
      for (int k = 0; k < n_out; ++k) twice |= s_out[k] == s_tok[x];
      part = twice ? 0.0 : (double)s_p[x];
      yes = (double)s_u[x] * mass < part;
    }
    if (yes) {
      kept |= 1ull << x;
      at = x;
      n_out = 0;
      c = 0.0;
      mass = 1.0;
      kids = s_kids[x];
      continue;
    }
    __syncthreads();  // s_out is read above
    if (t == 0) {
      bool twice = false;
      for (int k = 0; k < n_out; ++k) twice |= s_out[k] == s_tok[x];
      s_out[n_out] = s_tok[x];
      s_outw[n_out] = twice ? 0 : fixed60(s_p[x]);
    }
    __syncthreads();
    ++n_out;
    if (a.draft) {
      c += mass;
      if (kids) mass = (double)total_of(row_at(at, fixed_c(c))) * 0x1p-60;
    } else {
      mass -= part;
    }
  }

  // ---- the next token
  VfRow row = row_at(at, a.draft ? fixed_c(c) : 0);
  int taken_out = a.draft ? 0 : n_out;  // tokens whose mass counts nothing
  u64 total = total_of(row);
  // the mass in [from, to) of the tokens that count nothing
  auto out_of = [&](int from, int to) -> u64 {
    u64 sum = 0;
    for (int k = 0; k < taken_out; ++k)
      if (s_out[k] >= from && s_out[k] < to) sum += s_outw[k];
    return sum;
  };
  if (taken_out) {
    __syncthreads();  // every warp has added all[] up
    if (t < S) {
      const int from = (int)min((int64_t)t * per, (int64_t)V);
      all[t] -= out_of(from, min(from + per, V));
    }
    __syncthreads();
    total = 0;
    for (int s = lane; s < S; s += 32) total += all[s];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (total == 0 && n_out > 0) {  // nothing is left: the target's own distribution
    row = row_at(at, 0);
    taken_out = 0;
    total = total_of(row);
  }
  const u64 want = __umul64hi(fixed64(s_u[0]), total);  // below total
  // The part that holds `want`, of n <= 64 parts one behind the other; what
  // stands before it is taken off.  The same in every lane.
  auto part_of = [&](const u64* sums_, int n_, u64& want_) -> int {
    const u64 x0 = 2 * lane < n_ ? sums_[2 * lane] : 0, x1 = 2 * lane + 1 < n_ ? sums_[2 * lane + 1] : 0;
    u64 upto = x0 + x1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const unsigned above = __ballot_sync(0xffffffffu, upto > want_);
    const int l = above ? __ffs(above) - 1 : 31;  // none: the rows have changed in between
    const u64 before = __shfl_sync(0xffffffffu, upto - x0 - x1, l), first = __shfl_sync(0xffffffffu, x0, l);
    const bool in_first = want_ - before < first;
    want_ -= in_first ? before : before + first;
    return min(2 * l + (in_first ? 0 : 1), n_ - 1);
  };
  if (total > 0) {
    u64 left = want;
    const int s = part_of(all, S, left);
    if (s / kVfWarps == rank) {
      int from = (int)min((int64_t)s * per, (int64_t)V), to = min(from + per, V);
      for (int b = 0; to - from > 256; b ^= 1) {
        const int sub = ((to - from + kVfWarps - 1) / kVfWarps + 127) & ~127;
        const int a0 = min(from + warp * sub, to), a1 = min(a0 + sub, to);
        const u64 sum = range_sum(row, a0, a1) - out_of(a0, a1);
        if (lane == 0) part_sum[b][warp] = sum;
        __syncthreads();
        const int w = part_of(part_sum[b], kVfWarps, left);
        from = min(from + w * sub, to);
        to = min(from + sub, to);
      }
      if (warp == 0) {
        const int v = segment_find<kVec>(row, from, to, lane, left, s_out, taken_out);
        if (lane == 0) a.next_tokens[r] = max(v, 0);
      }
    }
  }
  if (rank == 0) {
    if (t == 0 && total == 0) a.next_tokens[r] = -1;
    for (int i = t; i < a.max_draft; i += kVfThreads)
      if (i >= __popcll(kept)) a.keep[(int64_t)r * a.max_draft + i] = -1;
    if (t < kVfNodes && (kept >> t & 1))
      a.keep[(int64_t)r * a.max_draft + __popcll(kept & ((1ull << t) - 1))] = t;
    if (t == 0) a.keep_lens[r] = __popcll(kept);
  }
  cluster.sync();  // every CTA's sums have been read
}

cudaError_t launch_draft_verify(const VerifyArgs& a, cudaStream_t stream) {
  // CTAs of a request: no more than run at once (four an SM, in clusters), and no warp's
  // segment below 64 elements of the vocabulary (each is whole steps of 128, so some may
  // be empty).  With 1 / 2 / 4 / 8 CTAs, us, chains of 3:
  //   131072 words: 64 requests 58 / 33 / 22 / 17.0, 70 58 / 33 / 22 / 17.5, 76 59 / 34 / 23 /
  //   24, 140 64 / 39 / 28 / 32, 152 65 / 40 / 41 / 39; 32000 words: 256 22 / 17.2 / 22 / 32,
  //   304 23.1 / 18.6 / 28 / 40, 330 24.6 / 27.2 / 30 / 42;
  //   16 requests: 600 words 5.5 / 5.6 / 5.5 / 5.8, 1200 6.4 / 5.8 / 6.0 / 5.9, 2400 6.6 / 6.4 / 5.9 /
  //   5.9, 5000 7.4 / 7.0 / 6.4 / 5.9; 64 requests: 600 5.6 / 5.8 / 6.2 / 7.1, 2400 6.8 / 6.8 / 6.2 / 7.2.
  int C = 1;
  while (C < kVfMaxCluster && (int64_t)a.num_seqs * C * 2 <= kVfWave && C * 4 * kVfThreads < a.vocab)
    C *= 2;
  const bool vec = a.target_stride % 4 == 0 && (reinterpret_cast<uintptr_t>(a.target) & 15u) == 0 &&
                   (!a.draft || (a.draft_stride % 4 == 0 && (reinterpret_cast<uintptr_t>(a.draft) & 15u) == 0));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.num_seqs * C));
  cfg.blockDim = dim3(kVfThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return vec ? cudaLaunchKernelEx(&cfg, draft_verify_kernel<true>, a)
             : cudaLaunchKernelEx(&cfg, draft_verify_kernel<false>, a);
}

}  // namespace pkv
