// blocks.cu -- block tables and slot maps of a step, from request lengths.
//
// What it computes (pkv_kv_blocks_update): request r goes from T_r to T'_r
// rows.  With b(T) = ceil(T / P), a shrinking request gives blocks b(T') ..
// b(T) - 1 back, a growing one takes b(T') - b(T) more, and with a window so do
// the blocks that lie wholly behind it.  The free ids are a stack; ids go onto
// it in descending (request, block) order and come off it in ascending order,
// so that a growth and the shrinking that undoes it leave it as it was.  New
// row i of the batch, row j of its request's new ones, gets position T + j and
// slot table[position / P] * P + position % P.
//
// Design (GB300): one CTA.  A batch is a few thousand integers, and everything
// depends on running sums over the requests, so the time is that of a few
// block-wide scans one behind the other, not of bytes; a grid would need a
// launch (or a grid barrier) between them.  Requests are taken 1024 at a time,
// one a thread.  The ids of a chunk's requests are one flat list (a prefix sum
// of their counts): a thread finds its entry's request by bisection, so that
// one request with a thousand blocks costs what a thousand with one do.  The
// slots of many rows (a prompt's) are a second launch over the whole GPU.
#include "common.cuh"
#include "launch.h"

namespace pkv {

namespace {

constexpr int kBlThreads = 1024;
constexpr int kBlWarps = kBlThreads / 32;
// Rows whose slots the one CTA writes itself.
constexpr int64_t kBlOwnRows = 4096;

// Inclusive sum over the CTA's threads; *total receives the sum of all.  `ws`:
// kBlWarps long longs of shared memory, free again when the call returns.
__device__ __forceinline__ long long block_scan(long long x, long long* ws, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) ws[warp] = x;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kBlWarps; ++w) {
    const long long t = ws[w];
    before += w < warp ? t : 0;
    all += t;
  }
  __syncthreads();
  *total = all;
  return before + x;
}

// First index i of the ascending a[0 .. n) with a[i] > x (n: none).
template <typename T>
__device__ __forceinline__ int first_above(const T* a, int n, long long x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if ((long long)a[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// What request r asks for.  bad: its lengths make no sense, nothing changes.
struct Ask {
  int old_len, new_len;
  bool bad;
};
__device__ __forceinline__ Ask read_ask(const BlocksArgs& a, int r, long long cap) {
  Ask k;
  k.old_len = a.seq_lens[r];
  const long long base = a.base_lens ? a.base_lens[r] : 0;
  const long long want = base + a.add[r];
  k.bad = k.old_len < 0 || k.old_len > cap || base < 0 || want < 0 || want > cap || want > INT32_MAX;
  k.new_len = k.bad ? k.old_len : (int)want;
  return k;
}

// Slot and position of row i: those of its request, or -1.
__device__ __forceinline__ void write_row(const BlocksArgs& a, int64_t i) {
  const int32_t* ptr = a.row_ptr;
  int64_t slot = -1;
  int pos = -1;
  if (a.num_seqs > 0 && i < ptr[a.num_seqs]) {
    const int r = first_above(ptr + 1, a.num_seqs, i);
    const int old_len = a.seq_lens[r];
    if (a.out_lens[r] != old_len) {  // it has grown
      pos = old_len + (int)(i - ptr[r]);
      const int b = pos / a.block_size;
      const int32_t id = a.block_tables[(int64_t)r * a.max_blocks + b];
      if (id >= 0 && id < a.num_blocks)
        slot = (int64_t)id * a.block_size + (pos - b * a.block_size);
      else
        pos = -1;
    }
  }
  a.slots[i] = slot;
  if (a.positions) a.positions[i] = pos;
}

__global__ void __launch_bounds__(kBlThreads) blocks_rows_kernel(const BlocksArgs a) {
  const int64_t i = (int64_t)blockIdx.x * kBlThreads + threadIdx.x;
  if (i < a.num_rows) write_row(a, i);
}

__global__ void __launch_bounds__(kBlThreads) blocks_update_kernel(const BlocksArgs a, int own_rows) {
  __shared__ long long ws[kBlWarps];
  __shared__ long long upto[kBlThreads];  // running count of a chunk's ids, by thread
  __shared__ int s_first[kBlThreads], s_next[kBlThreads], s_split[kBlThreads];
  const int t = threadIdx.x, lane = t & 31;
  const int B = a.num_seqs, P = a.block_size;
  const long long cap = (long long)a.max_blocks * P;
  auto blocks_of = [&](int len) { return (int)(((long long)len + P - 1) / P); };

  long long avail = a.count_in[0];
  if (avail < 0 || avail > a.num_blocks) {
    if (t == 0) atomicOr(a.err, PKV_DEVERR_BLOCK);
    avail = avail < 0 ? 0 : a.num_blocks;
  }

  // ---------------------------------------------------------- blocks that go
  // Chunks from the last request to the first; thread t of a chunk takes its
  // request 1023 - t, so that ascending threads are descending requests.
  for (int base = (B - 1) / kBlThreads * kBlThreads; base >= 0 && B > 0; base -= kBlThreads) {
    const int r = base + kBlThreads - 1 - t;
    int hi = 0, n_cut = 0, w_hi = 0, w_lo = 0;
    if (r < B) {
      const Ask k = read_ask(a, r, cap);
      if (k.bad) atomicOr(a.err, PKV_DEVERR_LENGTH);
      if (!k.bad) {
        hi = blocks_of(k.old_len);
        n_cut = max(0, hi - blocks_of(k.new_len));
        if (a.window > 0) {
          // the first row behind the sinks that a decode from here on sees
          const long long lo = (long long)min(k.old_len, k.new_len) - a.window;
          w_lo = blocks_of(a.num_sinks);
          w_hi = lo > 0 ? (int)(lo / P) : 0;
          if (w_hi <= w_lo) w_hi = w_lo = 0;
        }
      }
    }
    // behind the window: what went in earlier calls stands in front of what
    // goes now, so look downwards from the window for the first id that is
    // gone, a warp at a time where there is anything
    if (a.window > 0) {
      const int32_t* row = a.block_tables + (int64_t)(r < B ? r : 0) * a.max_blocks;
      unsigned todo = __ballot_sync(0xffffffffu, w_hi > w_lo && row[w_hi > 0 ? w_hi - 1 : 0] >= 0);
      const int found = __popc(todo & (1u << lane));  // whether this thread's request has some
      if (!found) w_lo = w_hi;
      while (todo) {
        const int l = __ffs(todo) - 1;
        todo &= todo - 1;
        const int rr = __shfl_sync(0xffffffffu, r, l);
        const int top = __shfl_sync(0xffffffffu, w_hi, l), bottom = __shfl_sync(0xffffffffu, w_lo, l);
        const int32_t* rrow = a.block_tables + (int64_t)rr * a.max_blocks;
        int at = top;  // blocks at .. top - 1 are still held
        while (at > bottom) {
          const int j = at - 1 - lane;
          const unsigned gone = __ballot_sync(0xffffffffu, j < bottom || rrow[j] < 0);
          if (gone) {
            at -= __ffs(gone) - 1;
            break;
          }
          at -= 32;
        }
        if (lane == l) w_lo = at;
      }
    }
    long long total;
    const int mine = n_cut + (w_hi - w_lo);
    const long long sum = block_scan(mine, ws, &total);
    upto[t] = sum;
    s_first[t] = hi - 1;   // its topmost block, then downwards
    s_split[t] = n_cut;    // after so many, on from behind the window
    s_next[t] = w_hi - 1;
    __syncthreads();
    for (long long f0 = 0; f0 < total; f0 += kBlThreads) {
      const long long f = f0 + t;
      int32_t id = -1;
      if (f < total) {
        const int o = first_above(upto, kBlThreads, f);
        const int e = (int)(f - (o ? upto[o - 1] : 0));
        const int blk = e < s_split[o] ? s_first[o] - e : s_next[o] - (e - s_split[o]);
        int32_t* at = a.block_tables + (int64_t)(base + kBlThreads - 1 - o) * a.max_blocks + blk;
        id = *at;
        *at = -1;
        if (id >= a.num_blocks) {
          atomicOr(a.err, PKV_DEVERR_BLOCK);
          id = -1;
        }
      }
      long long pushed;
      const long long place = avail + block_scan(id >= 0, ws, &pushed) - 1;
      if (id >= 0) {
        if (place < a.num_blocks)
          a.free_ids[place] = id;
        else
          atomicOr(a.err, PKV_DEVERR_BLOCK);  // more ids than the pool has blocks
      }
      avail = min(avail + pushed, (long long)a.num_blocks);
    }
    __syncthreads();
  }

  // -------------------------------------------------------- blocks that come
  long long rows = 0, taken = 0;  // of the chunks before; taken: asked for so far
  long long used = 0;             // ... and given
  if (t == 0) a.row_ptr[0] = 0;
  for (int base = 0; base < B; base += kBlThreads) {
    const int r = base + t;
    int held = 0, want = 0, n = 0, old_len = 0, new_len = 0;
    if (r < B) {
      const Ask k = read_ask(a, r, cap);
      old_len = k.old_len;
      new_len = k.new_len;
      if (!k.bad && new_len > old_len) {
        n = new_len - old_len;
        held = blocks_of(old_len);
        want = blocks_of(new_len);
      }
    }
    long long total;
    const long long row_end = rows + block_scan(n, ws, &total);
    rows += total;
    if (n > 0 && row_end > a.num_rows) {  // no room for its rows
      atomicOr(a.err, PKV_DEVERR_LENGTH);
      new_len = old_len;
      want = held;
    }
    if (r < B) a.row_ptr[r + 1] = (int32_t)min(row_end, (long long)a.num_rows);
    int demand = want - held;
    const long long sum = taken + block_scan(demand, ws, &total);
    if (demand > 0 && sum > avail) {  // not enough free blocks
      atomicOr(a.err, PKV_DEVERR_POOL);
      new_len = old_len;
    }
    if (r < B) a.out_lens[r] = new_len;
    const bool served = demand > 0 && sum <= avail;
    upto[t] = sum - taken;
    s_first[t] = held;
    s_split[t] = served ? 1 : 0;
    __syncthreads();
    for (long long f = t; f < total; f += kBlThreads) {
      const int o = first_above(upto, kBlThreads, f);
      if (!s_split[o]) continue;
      const int e = (int)(f - (o ? upto[o - 1] : 0));
      int32_t id = a.free_ids[avail - 1 - (taken + f)];
      if (id < 0 || id >= a.num_blocks) {
        atomicOr(a.err, PKV_DEVERR_BLOCK);
        id = -1;
      }
      a.block_tables[(int64_t)(base + o) * a.max_blocks + s_first[o] + e] = id;
    }
    // what the last request served has reached
    long long last = served ? sum : 0;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
    __syncthreads();
    if (lane == 0) ws[t >> 5] = last;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kBlWarps; ++w) used = max(used, ws[w]);
    taken += total;
    __syncthreads();
  }
  if (t == 0) a.count_out[0] = (int32_t)(avail - used);
  if (own_rows) {
    __syncthreads();
    for (int64_t i = t; i < a.num_rows; i += kBlThreads) write_row(a, i);
  }
}

}  // namespace

cudaError_t launch_blocks_update(const BlocksArgs& a, cudaStream_t stream) {
  const int own = a.num_rows <= kBlOwnRows ? 1 : 0;
  blocks_update_kernel<<<1, kBlThreads, 0, stream>>>(a, own);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || own) return e;
  blocks_rows_kernel<<<(unsigned)((a.num_rows + kBlThreads - 1) / kBlThreads), kBlThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
