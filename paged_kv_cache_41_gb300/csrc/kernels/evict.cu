// evict.cu -- keeping a paged cache inside a budget: the running attention
// weight of every cached row, the choice of the rows to keep by it, and the
// move of the kept rows together.
#include <cooperative_groups.h>
#include <math.h>

#include "common.cuh"
#include "launch.h"

namespace pkv {

// ------------------------------------------------------------------ weighing
// weights[r, c, t] = decay * weights[r, c, t] + sum over the G query heads h
// of kv head c of 2^(s_ht - lse_h), from the base-2 scores s that the decode
// left and the LSEs of its merge.  A thread per row, four rows in flight.
// Bound by its bytes: 4 G + 8 a row, beside the 4 D of K and V that the decode
// read for it (bf16), and partly still in L2.  64 requests, 279k rows, 32 query
// and 8 kv heads: 23 us beside the decode's 198, half of it this kernel and
// half the decode's writing of the scores; reading K again instead: 640 us.
namespace {

constexpr int kWeighThreads = 256;
constexpr int kWeighRows = 4;  // rows of a thread

}  // namespace

template <int G>
__global__ void __launch_bounds__(kWeighThreads) weigh_kernel(const WeighArgs a) {
  pdl_wait();
  const int r = blockIdx.z, c = blockIdx.y, Hkv = a.num_kv_heads;
  const int len = effective_len(__ldg(a.seq_lens + r), a.max_blocks, a.block_size, a.err, false);
  if (len > a.weights_rows && blockIdx.x == 0 && c == 0 && threadIdx.x == 0)
    atomicOr(a.err, PKV_DEVERR_LENGTH);
  const int64_t n = len < a.weights_rows ? len : a.weights_rows;
  const int64_t t0 = (int64_t)blockIdx.x * (kWeighThreads * kWeighRows) + threadIdx.x;
  if (t0 - threadIdx.x >= n) return;
  const int64_t rc = (int64_t)r * Hkv + c;
  float lse2[G];
#pragma unroll
  for (int g = 0; g < G; ++g) lse2[g] = __ldg(a.lse + rc * G + g) * 1.4426950408889634f;
  const float* s = a.scores + rc * a.scores_rows * G;
  float* w = a.weights + rc * a.weights_stride;
  float x[kWeighRows][G], old[kWeighRows];
#pragma unroll
  for (int i = 0; i < kWeighRows; ++i) {
    const int64_t t = t0 + i * kWeighThreads;
    if (t >= n) continue;
    if constexpr (G == 1)
      x[i][0] = s[t];
    else
      VecLoad<float, G>::run(s + t * G, x[i]);
    old[i] = w[t];
  }
#pragma unroll
  for (int i = 0; i < kWeighRows; ++i) {
    const int64_t t = t0 + i * kWeighThreads;
    if (t >= n) continue;
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      // a row that was not attended (a bad block) has score -inf and weight 0;
      // a head without an LSE (NaN scores) has no weights
      if (x[i][g] != -INFINITY) sum += lse2[g] == -INFINITY ? nanf("") : exp2f(x[i][g] - lse2[g]);
    }
    w[t] = fmaf(a.decay, old[i], sum);
  }
}

template <int G>
static cudaError_t launch_weigh_t(const WeighArgs& a, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.max_blocks * a.block_size, per = kWeighThreads * kWeighRows;
  return launch_pdl(weigh_kernel<G>,
                    dim3((unsigned)((rows + per - 1) / per), (unsigned)a.num_kv_heads, (unsigned)a.num_seqs),
                    dim3(kWeighThreads), 0, stream, a);
}

cudaError_t launch_weigh(const WeighArgs& a, cudaStream_t stream) {
  switch (a.num_q_heads / a.num_kv_heads) {
    case 1: return launch_weigh_t<1>(a, stream);
    case 2: return launch_weigh_t<2>(a, stream);
    case 4: return launch_weigh_t<4>(a, stream);
    case 8: return launch_weigh_t<8>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

// ------------------------------------------------------------------ selection
// Of the rows t < T of one (sequence, kv head): all where T <= budget, else
// the first num_sinks, the last num_recent and the k = budget - sinks -
// recent heaviest of those between, ties to the lowest index.
//
// The k-th largest weight is found by radix selection on an order-preserving
// integer key; then the kept indices are written in ascending order, from
// running counts.  The data is small (4 bytes a row), so the work on it and its
// barriers bound it, not its bytes: one CTA takes a row of weights (a cluster of
// up to eight where it does not fit) and reads it once, into shared memory.  A
// histogram of the keys' upper 11 bits leaves the rows of one bin (3% of a
// lognormal row); where they are few they are ranked against each other, else
// histograms of the next 11 and the last 10 bits follow.  64 requests, 8 kv
// heads, 512 to 8192 rows: 17.1 us (four passes of 8 bits over global memory:
// 44); 8 requests of 32768 to 65536 rows: 20.5 us (117).
namespace {

constexpr int kSelThreads = 1024;

// Larger weight, larger key: -0 counts as +0 and NaN below everything.  Takes
// the weight's bits, and they are loaded as integers: float operations would
// take subnormal weights for zero here.
__device__ __forceinline__ uint32_t weight_key(uint32_t u) {
  const uint32_t mag = u & 0x7fffffffu;
  if (mag > 0x7f800000u) return 0u;
  return (u & 0x80000000u) && mag ? ~u : (mag | 0x80000000u);
}

}  // namespace

namespace {

namespace cg = cooperative_groups;

constexpr int kScBins = 2048;
constexpr int kScList = 256;         // rows ranked against each other at most
constexpr int kScSlice = 48 * 1024;  // keys of a CTA at most (192 KiB)
constexpr uint32_t kScForced = 0xffffffffu;  // the key of a row kept for certain: no weight has it

}  // namespace

// Warp w of the cluster's CTA `rank` holds a contiguous run of its slice, 128
// consecutive rows at a time, four a lane.
template <int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 5 : 2) evict_select_cluster_kernel(const SelectArgs a) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint32_t keys[];  // this CTA's slice, padded with key 0
  __shared__ __align__(16) uint32_t hist[kScBins];  // of its keys, largest digit first
  // in CTA 0: key << 32 | ~row of the rows in the threshold's bin, so that a
  // larger word comes first
  __shared__ unsigned long long list[kScList];
  __shared__ uint32_t listed;
  __shared__ uint32_t warp_sum[kWarps], warp_above[kWarps], warp_at[kWarps];
  __shared__ uint32_t found[3];    // digit, rows wanted of its bin, rows in it
  __shared__ unsigned long long last;  // in CTA 0: the last kept candidate's word
  __shared__ uint32_t counts[2];   // this CTA's rows above the threshold, and at it
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int c = blockIdx.x / cs, r = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int T = __ldg(a.seq_lens + r);
  if (T < 0 || T > a.weights_rows) {
    if (c == 0 && rank == 0 && tid == 0) atomicOr(a.err, PKV_DEVERR_LENGTH);
    T = T < 0 ? 0 : (int)a.weights_rows;
  }
  int32_t* keep = a.keep + ((int64_t)r * a.num_kv_heads + c) * a.budget;
  const int kept = min(T, a.budget);
  if (c == 0 && rank == 0 && tid == 0) a.new_lens[r] = kept;
  const int me = rank * kThreads + tid, all = cs * kThreads;
  for (int j = kept + me; j < a.budget; j += all) keep[j] = -1;
  if (T <= a.budget) {  // the same for the whole cluster
    for (int j = me; j < T; j += all) keep[j] = j;
    return;
  }
  // every CTA of the cluster meets; one alone only needs its own threads
  auto meet = [&]() {
    if (cs > 1) cluster.sync();
    else __syncthreads();
  };
  const int slice = ((T + cs - 1) / cs + 3) & ~3;          // <= kScSlice
  const int n = (slice + 4 * kThreads - 1) / (4 * kThreads);  // fours of a thread
  const int first = rank * slice, len = min(T - first, slice);  // this CTA's rows (len may be <= 0)
  const int at0 = warp * 128 * n + lane * 4;               // this thread's: at0 + 128 i ..+3 of them
  const int lo = a.num_sinks, hi = T - a.num_recent;       // candidates: [lo, hi)
  const uint32_t* w = reinterpret_cast<const uint32_t*>(a.weights) +
                      ((int64_t)r * a.num_kv_heads + c) * a.weights_stride + first;
  const bool wide = (reinterpret_cast<uintptr_t>(w) & 15u) == 0;
  auto clear = [&]() {
    for (int i = tid; i < kScBins / 4; i += kThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0u, 0u, 0u, 0u);
  };
  clear();
  if (tid == 0) listed = 0;
  __syncthreads();
  uint32_t need = (uint32_t)(a.budget - a.num_sinks - a.num_recent);  // < hi - lo
  uint32_t prefix = kScForced - 1;  // the key's digits found so far; need 0: only forced rows are above
  uint32_t last_row = 0xffffffffu;  // of the rows at the key, keep those up to here ...
  bool ranked = false;              // ... where the candidates were ranked; else the first `need`
  // A thread reads only the keys it wrote.
#pragma unroll 2
  for (int i = 0; i < n; ++i) {
    const int at = at0 + 128 * i;
    if (at >= len) break;
    const int run = first + at - 4 * lane;  // the warp's 128 rows: all of them candidates, as a rule
    if (wide && run >= lo && run + 128 <= hi && run + 128 <= first + len) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(w + at));
      const uint32_t v[4] = {weight_key(x.x), weight_key(x.y), weight_key(x.z), weight_key(x.w)};
#pragma unroll
      for (int q = 0; q < 4; ++q) atomicAdd(&hist[kScBins - 1 - (v[q] >> 21)], 1u);
      *reinterpret_cast<uint4*>(keys + at) = make_uint4(v[0], v[1], v[2], v[3]);
      continue;
    }
    uint4 x;
    if (wide && at + 3 < len) {
      x = __ldg(reinterpret_cast<const uint4*>(w + at));
    } else {
      x.x = __ldg(w + at);
      x.y = at + 1 < len ? __ldg(w + at + 1) : 0u;
      x.z = at + 2 < len ? __ldg(w + at + 2) : 0u;
      x.w = at + 3 < len ? __ldg(w + at + 3) : 0u;
    }
    uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int t = first + at + q;
      v[q] = at + q >= len ? 0u : t < lo || t >= hi ? kScForced : weight_key(v[q]);
      if (at + q < len && v[q] != kScForced) atomicAdd(&hist[kScBins - 1 - (v[q] >> 21)], 1u);
    }
    *reinterpret_cast<uint4*>(keys + at) = make_uint4(v[0], v[1], v[2], v[3]);
  }
  // f(key, index in the slice) for this thread's keys whose upper bits are
  // `prefix`; a padding key passes as well, its index being >= len
  auto matching = [&](int shift, auto f) {
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int at = at0 + 128 * i;
      if (at >= len) break;
      const uint4 x = *reinterpret_cast<const uint4*>(keys + at);
      const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if ((v[q] >> shift) == prefix && at + q < len) f(v[q], at + q);
    }
  };
  int bits_left = 21;
  for (int pass = 0; need > 0 && pass < 3; ++pass) {
    const int bits = pass == 2 ? 10 : 11;
    if (pass > 0) {
      bits_left -= bits;
      meet();  // the others have read this CTA's histogram
      clear();
      __syncthreads();
      matching(bits_left + bits, [&](uint32_t key, int) {
        atomicAdd(&hist[kScBins - 1 - ((key >> bits_left) & ((1u << bits) - 1u))], 1u);
      });
    }
    meet();
    // the bin that holds the need-th largest digit, over the whole cluster:
    // thread t adds up bins kPer t ..
    constexpr int kPer = kScBins / kThreads;
    uint32_t v[kPer];
#pragma unroll
    for (int q = 0; q < kPer; ++q) v[q] = 0;
    for (int q = 0; q < cs; ++q) {
      const uint32_t* h = (cs > 1 ? cluster.map_shared_rank(hist, q) : hist) + tid * kPer;
#pragma unroll
      for (int p = 0; p < kPer / 2; ++p) {
        const uint2 x = reinterpret_cast<const uint2*>(h)[p];
        v[2 * p] += x.x;
        v[2 * p + 1] += x.y;
      }
    }
    uint32_t mine = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) mine += v[q];
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    uint32_t before = inc - mine + __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0u);
    if (before < need && need <= before + mine) {
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        if (before < need && need <= before + v[q]) {
          found[0] = (uint32_t)(kScBins - 1 - (kPer * tid + q));
          found[1] = need - before;
          found[2] = v[q];
        }
        before += v[q];
      }
    }
    __syncthreads();
    prefix = pass == 0 ? found[0] : (prefix << bits) | found[0];
    need = found[1];
    const uint32_t in_bin = found[2];
    if (in_bin <= (uint32_t)kScList) {
      // rank the bin's rows by (key, lowest row first), in CTA 0
      ranked = true;
      unsigned long long* to = cs > 1 ? cluster.map_shared_rank(list, 0) : list;
      uint32_t* nl = cs > 1 ? cluster.map_shared_rank(&listed, 0) : &listed;
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const int at = at0 + 128 * i;
        if (at >= len) break;
        const uint4 x = *reinterpret_cast<const uint4*>(keys + at);
        const uint32_t v[4] = {x.x, x.y, x.z, x.w};
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if ((v[q] >> bits_left) == prefix) m |= 1u << q;
        if (at + 3 >= len) m &= (1u << (len - at)) - 1u;  // not the padding
        if (m) {
          uint32_t place = atomicAdd(nl, (uint32_t)__popc(m));
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if ((m >> q) & 1u) to[place++] = ((unsigned long long)v[q] << 32) | (uint32_t)~(first + at + q);
        }
      }
      meet();
      if (rank == 0 && tid < in_bin) {
        const unsigned long long x = list[tid];
        uint32_t above = 0;
#pragma unroll 4
        for (uint32_t q = 0; q < in_bin; ++q) above += list[q] > x ? 1u : 0u;
        if (above == need - 1) last = x;
      }
      meet();
      const unsigned long long x = cs > 1 ? *cluster.map_shared_rank(&last, 0) : last;
      prefix = (uint32_t)(x >> 32);
      last_row = ~(uint32_t)x;
      break;
    }
  }
  // ---- keep every key above `prefix`, and of those at it the rows up to
  // last_row (ranked) or the first `need`: counts by warp, by CTA, by row.
  // Ranked: one bit a row says it all (padding lies past last_row), and a
  // thread's 4 n <= 48 of them wait in a register for the counts.
  uint64_t kept_bits = 0;
  // above and at of four rows: bits 0-3 and 4-7
  auto kinds = [&](int at) -> uint32_t {
    uint32_t m = 0;
    if (at < len) {
      const uint4 x = *reinterpret_cast<const uint4*>(keys + at);
      const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (ranked) {
          if (v[q] > prefix || (v[q] == prefix && (uint32_t)(first + at + q) <= last_row)) m |= 1u << q;
        } else {
          if (v[q] > prefix) m |= 1u << q;
          if (v[q] == prefix && at + q < len) m |= 16u << q;
        }
      }
    }
    return m;
  };
  uint32_t n_above = 0, n_at = 0;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const uint32_t m = kinds(at0 + 128 * i);
    kept_bits |= (uint64_t)(m & 15u) << (4 * i);
    n_above += __popc(m & 15u);
    n_at += __popc(m >> 4);
  }
  n_above = __reduce_add_sync(0xffffffffu, n_above);
  n_at = __reduce_add_sync(0xffffffffu, n_at);
  if (lane == 0) {
    warp_above[warp] = n_above;
    warp_at[warp] = n_at;
  }
  __syncthreads();
  uint32_t my_above = __reduce_add_sync(0xffffffffu, lane < warp ? warp_above[lane] : 0u);
  uint32_t my_at = __reduce_add_sync(0xffffffffu, lane < warp ? warp_at[lane] : 0u);
  if (cs > 1) {
    if (tid == kThreads - 1) {
      counts[0] = my_above + n_above;
      counts[1] = my_at + n_at;
    }
    cluster.sync();
    for (int q = 0; q < rank; ++q) {
      const uint32_t* x = cluster.map_shared_rank(counts, q);
      my_above += x[0];
      my_at += x[1];
    }
  }
  if (ranked) {
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int row = first + at0 + 128 * i;
      const uint32_t m = (uint32_t)(kept_bits >> (4 * i)) & 15u;
      uint32_t pa = my_above;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t all = __ballot_sync(0xffffffffu, (m >> q) & 1u);
        pa += __popc(all & below);
        my_above += __popc(all);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if ((m >> q) & 1u) keep[pa++] = row + q;
    }
    if (cs > 1) cluster.sync();  // the others may still read this CTA's shared memory
    return;
  }
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const int at = at0 + 128 * i;
    const uint32_t m = kinds(at);
    const uint32_t mine = __popc(m & 15u) | (__popc(m >> 4) << 16);
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const uint32_t total = __shfl_sync(0xffffffffu, inc, 31);
    uint32_t pa = my_above + ((inc - mine) & 0xffffu), pq = my_at + ((inc - mine) >> 16);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool ab = (m >> q) & 1u, eq = (m >> (4 + q)) & 1u;
      if (ab || (eq && pq < need)) keep[pa + min(pq, need)] = first + at + q;
      pa += ab ? 1u : 0u;
      pq += eq ? 1u : 0u;
    }
    my_above += total & 0xffffu;
    my_at += total >> 16;
  }
  if (cs > 1) cluster.sync();  // the others may still read this CTA's shared memory
}

// Any length: one CTA a row of weights, which it reads again in each of four
// passes over eight bits.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const SelectArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t warp_sum[32];
  __shared__ uint32_t found[2];
  const int c = blockIdx.x, r = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int T = __ldg(a.seq_lens + r);
  if (T < 0 || T > a.weights_rows) {
    if (c == 0 && tid == 0) atomicOr(a.err, PKV_DEVERR_LENGTH);
    T = T < 0 ? 0 : (int)a.weights_rows;
  }
  const uint32_t* w = reinterpret_cast<const uint32_t*>(a.weights) +
                      ((int64_t)r * a.num_kv_heads + c) * a.weights_stride;
  int32_t* keep = a.keep + ((int64_t)r * a.num_kv_heads + c) * a.budget;
  const int kept = min(T, a.budget);
  if (c == 0 && tid == 0) a.new_lens[r] = kept;
  for (int j = kept + tid; j < a.budget; j += kSelThreads) keep[j] = -1;
  if (T <= a.budget) {
    for (int j = tid; j < T; j += kSelThreads) keep[j] = j;
    return;
  }
  const int lo = a.num_sinks, hi = T - a.num_recent;  // candidates: [lo, hi)
  uint32_t need = (uint32_t)(a.budget - a.num_sinks - a.num_recent);  // < hi - lo
  uint32_t prefix = 0, mask = 0;  // the key's bits found so far
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int t = lo + tid; t < hi; t += kSelThreads) {
        const uint32_t key = weight_key(__ldg(w + t));
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid < 32) {  // lane l: bins 8 l .. 8 l + 7, from the top
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) mine += hist[255 - (8 * lane + i)];
        uint32_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        uint32_t before = inc - mine;
        if (before < need && need <= inc) {
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            const uint32_t n = hist[255 - (8 * lane + i)];
            if (need <= before + n) {
              found[0] = 255 - (8 * lane + i);
              found[1] = need - before;
              break;
            }
            before += n;
          }
        }
      }
      __syncthreads();
      prefix |= found[0] << shift;
      mask |= 255u << shift;
      need = found[1];
    }
  } else {
    prefix = 0xffffffffu;  // no candidate is kept: no key is above this one
  }
  // keep every key above `prefix`, and the first `need` at it
  uint32_t above = 0, at = 0;  // so far: kept for certain, and at the key
  for (int base = 0; base < T; base += kSelThreads) {
    const int t = base + tid;
    uint32_t v = 0;
    if (t < T) {
      if (t < lo || t >= hi) {
        v = 1u << 16;
      } else {
        const uint32_t key = weight_key(__ldg(w + t));
        v = key > prefix ? 1u << 16 : (key == prefix ? 1u : 0u);
      }
    }
    uint32_t inc = v;  // counts above in the upper half, at the key in the lower
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    uint32_t pre = 0, total = 0;
    for (int i = 0; i < 32; ++i) {
      const uint32_t x = warp_sum[i];
      if (i < warp) pre += x;
      total += x;
    }
    const uint32_t ex = pre + inc - v;
    const uint32_t my_above = above + (ex >> 16), my_at = at + (ex & 0xffffu);
    if ((v >> 16) || ((v & 1u) && my_at < need)) keep[my_above + min(my_at, need)] = t;
    above += total >> 16;
    at += total & 0xffffu;
    __syncthreads();
  }
}

template <int kThreads>
static cudaError_t launch_select_cluster(const SelectArgs& a, int cs, cudaStream_t stream) {
  const int smem = (int)(((a.weights_rows + cs - 1) / cs + 3) & ~(int64_t)3) * 4;
  auto kern = evict_select_cluster_kernel<kThreads>;
  static SmemAttrCache attr_cache;
  cudaError_t e = ensure_smem_limit(kern, smem, attr_cache);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.num_kv_heads * cs), (unsigned)a.num_seqs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

cudaError_t launch_evict_select(const SelectArgs& a, cudaStream_t stream) {
  // No length passes weights_rows: the smallest cluster whose CTAs hold it.
  // Small CTAs for rows of up to 8192, several to a SM (64 requests: 22.6 us,
  // with 1024 threads 25.6).
  const int64_t most = a.weights_rows;
  if (most <= 8 * kScSlice) {
    int cs = 1;
    while (most > (int64_t)cs * kScSlice) cs *= 2;
    return most <= 8192 ? launch_select_cluster<256>(a, cs, stream)
                        : launch_select_cluster<1024>(a, cs, stream);
  }
  evict_select_kernel<<<dim3((unsigned)a.num_kv_heads, (unsigned)a.num_seqs), kSelThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ compaction
// Row base + keep[j] moves to row base + j, keep ascending (so keep[j] >= j),
// in place.  One CTA walks the rows of one chain -- one (sequence, kv head) of
// K or of V, or some columns of it -- in order, a tile of them at a time.  The
// order that has to hold: a tile's loads, and those of the tiles before it,
// are done before its stores, since its destinations may be their sources.
// Later tiles' loads may run ahead freely: their sources are at or above their
// own destinations, which this tile's stores do not reach.
//
// So each CTA keeps a ring of tiles in shared memory filled by
// cp.async (a plain load would have to arrive before the barrier that orders
// the stores), several tiles ahead, and works out the rows' places further
// ahead still.  Bound by the bytes: every moved row read once and written
// once (64 bf16 requests, 253 MB kept: 85 us, 5.95 TB/s read + written).
// Where the chains are few, a row's columns are dealt to several CTAs and the
// ring is deeper (three fp32 sequences, 7777 rows kept: 20 us, 2.4 TB/s; then
// the order of a chain's tiles bounds it).
namespace {

constexpr uint32_t kCmSkip = 0xffffffffu;             // no row to move here
constexpr int kCmSmall = 8;                           // weights or scales per thread and turn
constexpr int kCmMaxLen = 0x7fff0000;                 // rows of a sequence: turns past the last stay in 32 bits

struct CompactSeq {
  int base, n, len;  // first row, kept rows, rows in all (0: skip)
};

__device__ __forceinline__ CompactSeq compact_seq(const CompactArgs& a, int r, bool report) {
  CompactSeq s;
  s.len = effective_len(__ldg(a.seq_lens + r), a.max_blocks, a.block_size, a.err, report);
  s.base = a.base_lens ? __ldg(a.base_lens + r) : 0;
  s.n = __ldg(a.keep_lens + r);
  const bool ok = s.len <= kCmMaxLen && s.base >= 0 && s.base <= s.len && s.n >= 0 && s.n <= s.len - s.base &&
                  s.n <= a.keep_stride && (!a.weights || s.len <= a.weights_rows);
  if (!ok) {
    if (report) atomicOr(a.err, PKV_DEVERR_LENGTH);
    s.n = 0;
    s.len = s.base = 0;
  }
  return s;
}

// Kept row j, keep[j] = k after keep[j - 1] = prev (-1: none), or -1 where it
// is out of range or order (reported).
__device__ __forceinline__ int kept_row(const CompactArgs& a, const CompactSeq& s, int k, int prev, int j) {
  if (k >= j && k > prev && k < s.len - s.base) return k;
  atomicOr(a.err, PKV_DEVERR_KEEP);
  return -1;
}
__device__ __forceinline__ int kept_before(const int32_t* keep, int j) { return j > 0 ? __ldg(keep + j - 1) : -1; }

// Row t's block, in its table, and place in that block.
__device__ __forceinline__ int block_of(const CompactArgs& a, int t) {
  return a.block_shift >= 0 ? t >> a.block_shift : t / a.block_size;
}
__device__ __forceinline__ int offset_of(const CompactArgs& a, int t) {
  return a.block_shift >= 0 ? t & (a.block_size - 1) : t % a.block_size;
}

__device__ __forceinline__ int table_entry(const CompactArgs& a, int r, int t) {
  return __ldg(a.block_tables + (int64_t)r * a.max_blocks + block_of(a, t));
}

// Pool row of offset `off` of block `blk`, or kCmSkip for a bad id (reported).
// Pool rows are below 2^32 - 1 (the host checks).
__device__ __forceinline__ uint32_t pool_row(const CompactArgs& a, int blk, int off) {
  if (blk >= 0 && (int64_t)blk < a.num_blocks) return (uint32_t)((int64_t)blk * a.block_size + off);
  atomicOr(a.err, PKV_DEVERR_BLOCK);
  return kCmSkip;
}

__device__ __forceinline__ void cp_async16(uint32_t smem, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(g) : "memory");
}

}  // namespace

// kVecs: 16-byte vectors per thread and tile.  kRing: tiles of the ring.
// kPlaces: entries of the ring of places, a power of two >= the rows of kRing +
// 1 tiles (a tile has kThreads at most) and a batch.
template <int kThreads, int kVecs, int kRing, int kPlaces>
__global__ void __launch_bounds__(kThreads) kv_compact_kernel(const CompactArgs a) {
  static_assert(kPlaces >= (kRing + 2) * kThreads, "the ring of places");
  constexpr int kTileVecs = kThreads * kVecs;
  extern __shared__ __align__(128) unsigned char cm_smem[];
  uint4* ring = reinterpret_cast<uint4*>(cm_smem);                               // [kRing][kTileVecs]
  uint2* places = reinterpret_cast<uint2*>(cm_smem + kRing * kTileVecs * 16);  // (from, to) by row
  const int h = blockIdx.x, y = blockIdx.y, r = blockIdx.z;
  const int tid = threadIdx.x, Hkv = a.num_kv_heads, P = a.block_size;
  const CompactSeq s = compact_seq(a, r, h == 0 && y == 0 && tid == 0);
  const int32_t* keep = a.keep + ((int64_t)r * a.keep_heads + (a.keep_heads > 1 ? h : 0)) * a.keep_stride;
  if (y < 2 * a.parts) {
    if (s.n == 0) return;
    unsigned char* pool = y < a.parts ? a.k : a.v;
    // this CTA's columns: `vecs` vectors from c0 on, `rows` (a power of two) rows a tile
    const int per = (a.row_bytes / 16 + a.parts - 1) / a.parts, c0 = (y % a.parts) * per;
    const int vecs = min(per, a.row_bytes / 16 - c0);
    if (vecs <= 0) return;
    const int rows = 1 << (31 - __clz(min(kTileVecs / vecs, kThreads)));
    const int tiles = (s.n + rows - 1) / rows;
    int my_row[kVecs];          // this thread's vectors of a tile: rows,
    unsigned char* col[kVecs];  // and columns in pool row 0
    const uint32_t pitch = (uint32_t)Hkv * a.row_bytes;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int i = tid + u * kThreads;
      my_row[u] = i < rows * vecs ? i / vecs : -1;
      col[u] = pool + (int64_t)h * a.row_bytes + (c0 + i % vecs) * 16;
    }
    // ---- places, in batches of kThreads rows, a row a thread: the kept rows
    // of the batch after next and the block ids of the next one are on their
    // way while a batch is used
    int k_next = -1, k_prev = -1, k_now = -1, b_from = 0, b_to = 0;  // kept rows, block ids
    auto load_keep = [&](int j) {  // looked at a batch later
      if (j < s.n) {
        k_next = __ldg(keep + j);
        k_prev = kept_before(keep, j);
      }
    };
    auto next_keep = [&](int j) { k_now = j < s.n ? kept_row(a, s, k_next, k_prev, j) : -1; };
    auto load_blocks = [&](int j) {
      if (k_now >= 0) {
        b_from = table_entry(a, r, s.base + k_now);
        b_to = table_entry(a, r, s.base + j);
      }
    };
    int filled = 0;  // rows whose places are known
    if (tid * 32 < min(s.n, (kRing + 2) * kThreads))  // the first of them ahead of their turns
      asm volatile("prefetch.global.L2 [%0];" ::"l"(keep + tid * 32));
    load_keep(tid);
    next_keep(tid);
    load_keep(kThreads + tid);
    load_blocks(tid);
    auto fill = [&]() {
      const int j = filled + tid;
      uint2 at = make_uint2(kCmSkip, kCmSkip);
      if (k_now >= 0 && k_now != j) {  // a row already in its place stays
        const uint32_t from = pool_row(a, b_from, offset_of(a, s.base + k_now));
        const uint32_t to = pool_row(a, b_to, offset_of(a, s.base + j));
        if (from != kCmSkip && to != kCmSkip) at = make_uint2(from, to);
      }
      places[j & (kPlaces - 1)] = at;
      filled += kThreads;
      next_keep(filled + tid);
      load_blocks(filled + tid);
      load_keep(filled + kThreads + tid);
    };
    auto issue = [&](int t) {  // this thread's loads of tile t (an empty group past the last)
      if (t < tiles) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
          if (my_row[u] < 0) continue;
          const int j = t * rows + my_row[u];
          const uint32_t from = j < s.n ? places[j & (kPlaces - 1)].x : kCmSkip;
          if (from != kCmSkip)
            cp_async16(smem_u32(ring + (t % kRing) * kTileVecs + u * kThreads + tid),
                       col[u] + (uint64_t)from * pitch);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int ahead = kRing - 1;
    while (filled < min(ahead * rows, s.n)) fill();
    __syncthreads();
    for (int t = 0; t < ahead; ++t) issue(t);
    for (int t = 0; t < tiles; ++t) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
      while (filled < min((t + kRing) * rows, s.n)) fill();
      // tile t has landed for every thread, the places of tile t + kRing - 1
      // are known, and the stores of tile t - 1 have left its ring slot
      __syncthreads();
      issue(t + ahead);
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        if (my_row[u] < 0) continue;
        const int j = t * rows + my_row[u];
        const uint32_t to = j < s.n ? places[j & (kPlaces - 1)].y : kCmSkip;
        if (to != kCmSkip)
          *reinterpret_cast<uint4*>(col[u] + (uint64_t)to * pitch) =
              ring[(t % kRing) * kTileVecs + u * kThreads + tid];
      }
    }
    return;
  }
  // ---- weights, and an MXFP8 pool's scales: a few bytes a row
  constexpr int kTurn = kThreads * kCmSmall;
  if (y == 2 * a.parts && a.weights) {
    float* w = a.weights + ((int64_t)r * Hkv + h) * a.weights_stride + s.base;
    for (int j0 = 0; j0 < s.n; j0 += kTurn) {
      float x[kCmSmall];
      int k[kCmSmall];
#pragma unroll
      for (int u = 0; u < kCmSmall; ++u) {
        const int j = j0 + u * kThreads + tid;
        k[u] = j < s.n ? kept_row(a, s, __ldg(keep + j), kept_before(keep, j), j) : -1;
        if (k[u] == j) k[u] = -1;  // in its place already
      }
#pragma unroll
      for (int u = 0; u < kCmSmall; ++u) {  // a row that K and V do not move: nor its weight
        if (k[u] < 0) continue;
        const int from = table_entry(a, r, s.base + k[u]);
        const int to = table_entry(a, r, s.base + j0 + u * kThreads + tid);
        if (pool_row(a, from, 0) == kCmSkip || pool_row(a, to, 0) == kCmSkip) k[u] = -1;
      }
#pragma unroll
      for (int u = 0; u < kCmSmall; ++u) x[u] = k[u] >= 0 ? w[k[u]] : 0.f;
      __syncthreads();  // the turn's loads are done
#pragma unroll
      for (int u = 0; u < kCmSmall; ++u)
        if (k[u] >= 0) w[j0 + u * kThreads + tid] = x[u];
    }
    __syncthreads();  // every source has been read
    for (int j = s.n + tid; j < s.len - s.base; j += kThreads) w[j] = 0.f;
  } else {
    // scales of K, then of V: [NB, Hkv, P, scale_bytes], scale_bytes a row
    const int v = y - 2 * a.parts - (a.weights ? 1 : 0), sb = a.scale_bytes;
    unsigned char* sc = v == 0 ? a.k_scales : a.v_scales;
    for (int j0 = 0; j0 < s.n; j0 += kTurn) {
      uint32_t from[kCmSmall], to[kCmSmall];
#pragma unroll
      for (int u = 0; u < kCmSmall; ++u) {
        const int j = j0 + u * kThreads + tid;
        const int k = j < s.n ? kept_row(a, s, __ldg(keep + j), kept_before(keep, j), j) : -1;
        from[u] = to[u] = kCmSkip;
        if (k >= 0 && k != j) {
          from[u] = pool_row(a, table_entry(a, r, s.base + k), offset_of(a, s.base + k));
          to[u] = pool_row(a, table_entry(a, r, s.base + j), offset_of(a, s.base + j));
          if (from[u] == kCmSkip) to[u] = kCmSkip;
        }
      }
      auto at = [&](uint32_t row) {
        return sc + (((int64_t)(row / P) * Hkv + h) * P + row % P) * sb;
      };
      for (int b = 0; b < sb; ++b) {  // a byte of every row at a time
        unsigned char x[kCmSmall];
#pragma unroll
        for (int u = 0; u < kCmSmall; ++u)
          if (to[u] != kCmSkip) x[u] = at(from[u])[b];
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kCmSmall; ++u)
          if (to[u] != kCmSkip) at(to[u])[b] = x[u];
      }
    }
  }
}

template <int kThreads, int kVecs, int kRing, int kPlaces>
static cudaError_t launch_compact_t(const CompactArgs& a, unsigned y, cudaStream_t stream) {
  constexpr int smem = kRing * kThreads * kVecs * 16 + kPlaces * 8;
  auto kern = kv_compact_kernel<kThreads, kVecs, kRing, kPlaces>;
  static SmemAttrCache attr_cache;
  cudaError_t e = ensure_smem_limit(kern, smem, attr_cache);
  if (e != cudaSuccess) return e;
  kern<<<dim3((unsigned)a.num_kv_heads, y, (unsigned)a.num_seqs), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_compact(const CompactArgs& args, cudaStream_t stream) {
  CompactArgs a = args;
  // Columns: at most 64 vectors a CTA, and while the chains are fewer than two
  // a SM, halves of at least two vectors (32 bytes, a sector).
  const int vecs = a.row_bytes / 16;
  const int64_t chains = (int64_t)a.num_seqs * a.num_kv_heads * 2;
  a.parts = (vecs + 63) / 64;
  a.block_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.block_size == 1 << i) a.block_shift = i;
  while (chains * a.parts < 304 && vecs % (2 * a.parts) == 0 && vecs / (2 * a.parts) >= 2) a.parts *= 2;
  const unsigned y = 2u * a.parts + (a.weights ? 1u : 0u) + (a.k_scales ? 2u : 0u);
  // A drafted path is one batch of rows at most: a small ring, and more CTAs a
  // SM (64 requests 6.2 us, with four tiles 7.1 us).  Otherwise four CTAs a SM,
  // or one that keeps more on its way where there is no second for every SM
  // (three long fp32 sequences, 96 CTAs: 44 us and 20 us; 14 bf16 ones, 448
  // CTAs: 23.7 us and 29.5 us).
  if (a.keep_stride <= 256) return launch_compact_t<256, 2, 2, 1024>(a, y, stream);
  return chains * a.parts < 304 ? launch_compact_t<1024, 1, 6, 8192>(a, y, stream)
                                : launch_compact_t<256, 2, 4, 2048>(a, y, stream);
}

}  // namespace pkv
