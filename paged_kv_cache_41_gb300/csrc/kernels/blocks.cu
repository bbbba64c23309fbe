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
// depends on running sums over the requests, so the time is that of a chain of
// loads, scans and barriers, not of bytes; a grid would need a launch (or a
// grid barrier) between its links.  Requests are taken one a thread, as many at
// a time as there are threads: 128, whose barriers and scans are short, where
// the batch and its rows are small, else 1024.  A batch that fits one pass takes its three running sums (ids given
// back, ids taken, rows) in one scan.  The ids of a pass are one flat list: a
// thread finds its entries' request by bisection of the running sums, so that one
// request with a thousand blocks costs what a thousand with one do.  The
// slots of many rows (a prompt's) are a second launch over the whole GPU.
#include "common.cuh"
#include "launch.h"

namespace pkv {

namespace {

constexpr int kBlRowThreads = 256;
// Rows whose slots the one CTA writes itself; more are a second launch's.  By itself
// against that, 1024 threads, us: 8 requests, 1024 rows 5.4 / 6.1, 2048 6.8 / 6.2,
// 4096 9.1 / 6.6; 64 requests, 2048 6.9 / 7.3, 2560 7.9 / 7.4; 256, 2048 5.8 / 7.0, 2560
// 8.2 / 8.2; 512, 2048 6.1 / 7.4, 4096 8.2 / 7.3.
constexpr int64_t kBlOwnRows = 2048;
// Requests (one a thread, one pass) and rows of a call that 128 threads take; 1024
// take any other.  128 against 1024, us: 1 request, 128 rows 4.0 / 5.2, 256 4.7 / 5.2, 320
// 5.6 / 5.4, 512 6.3 / 5.6; 64 requests, 128 rows 3.4 / 4.3, 256 4.0 / 4.2, 320 4.8 /
// 4.4, 512 5.5 / 4.4; 128 requests, 256 rows 4.2 / 4.4, 384 4.8 / 4.4; 192 requests, 192
// rows (two passes) 7.6 / 4.2.
constexpr int kBlFewSeqs = 128;
constexpr int64_t kBlFewRows = 256;

struct Sum3 {
  long long a, b, c;
};
__device__ __forceinline__ Sum3 warp_scan(Sum3 x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ya = __shfl_up_sync(0xffffffffu, x.a, o), yb = __shfl_up_sync(0xffffffffu, x.b, o),
                    yc = __shfl_up_sync(0xffffffffu, x.c, o);
    if (lane >= o) {
      x.a += ya;
      x.b += yb;
      x.c += yc;
    }
  }
  return x;
}
// Inclusive sums over the CTA's threads; *total receives the sums of all.  `ws`:
// kThreads / 32 entries of shared memory, free again when the call returns.
template <int kThreads>
__device__ __forceinline__ Sum3 block_scan(Sum3 x, Sum3* ws, Sum3* total) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  x = warp_scan(x);
  if (lane == 31) ws[warp] = x;
  __syncthreads();
  if constexpr (kWarps <= 4) {
    Sum3 all = {0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const Sum3 y = ws[w];
      if (w == warp) x = {x.a + all.a, x.b + all.b, x.c + all.c};
      all = {all.a + y.a, all.b + y.b, all.c + y.c};
    }
    __syncthreads();
    *total = all;
    return x;
  }
  // the sums of more warps by one of them: all warps reading all sums is a
  // thousand loads of shared memory
  if (warp == 0) {
    const Sum3 y = warp_scan(lane < kWarps ? ws[lane] : Sum3{0, 0, 0});
    __syncwarp();
    if (lane < kWarps) ws[lane] = y;
  }
  __syncthreads();
  *total = ws[kWarps - 1];
  if (warp > 0) {
    const Sum3 before = ws[warp - 1];
    x.a += before.a;
    x.b += before.b;
    x.c += before.c;
  }
  __syncthreads();
  return x;
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

__device__ __forceinline__ int blocks_of(int len, int P) { return (int)(((long long)len + P - 1) / P); }

// Slot and position of row i, row e of the new ones of request r, which goes
// from old_len to new_len rows (none: r < 0, or not grown).
__device__ __forceinline__ void write_row(const BlocksArgs& a, int64_t i, int r, int e, int old_len,
                                          int new_len) {
  int64_t slot = -1;
  int pos = -1;
  if (r >= 0 && new_len != old_len) {
    pos = old_len + e;
    const int b = pos / a.block_size;
    const int32_t id = a.block_tables[(int64_t)r * a.max_blocks + b];
    if (id >= 0 && id < a.num_blocks)
      slot = (int64_t)id * a.block_size + (pos - b * a.block_size);
    else
      pos = -1;
  }
  a.slots[i] = slot;
  if (a.positions) a.positions[i] = pos;
}
// The same from what the update has left in global memory.
__device__ __forceinline__ void write_row(const BlocksArgs& a, int64_t i) {
  const int32_t* ptr = a.row_ptr;
  if (a.num_seqs == 0 || i >= ptr[a.num_seqs]) {
    write_row(a, i, -1, 0, 0, 0);
    return;
  }
  const int r = first_above(ptr + 1, a.num_seqs, i);
  write_row(a, i, r, (int)(i - ptr[r]), a.seq_lens[r], a.out_lens[r]);
}

__global__ void __launch_bounds__(kBlRowThreads) blocks_rows_kernel(const BlocksArgs a) {
  pdl_wait();  // the update's tables, lengths and row ranges
  const int64_t i = (int64_t)blockIdx.x * kBlRowThreads + threadIdx.x;
  if (i < a.num_rows) write_row(a, i);
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) blocks_update_kernel(const BlocksArgs a, int own_rows) {
  __shared__ Sum3 ws[kThreads / 32];
  // running sums by request: of the ids that go, then of those that come; of rows
  __shared__ long long ids_to[kThreads], rows_to[kThreads];
  // what goes: s_cut ids from block s_want on, before them those from block
  // s_wlo on; what comes: from block s_held on, where served
  __shared__ int s_cut[kThreads], s_want[kThreads], s_wlo[kThreads], s_held[kThreads], s_old[kThreads],
      s_new[kThreads];
  constexpr int kPer = kThreads == 128 ? 1 : 2;  // ids of a thread at a time
  const int t = threadIdx.x, lane = t & 31;
  const int B = a.num_seqs, P = a.block_size;
  const long long cap = (long long)a.max_blocks * P;
  const bool single = B <= kThreads;

  long long avail = a.count_in[0];
  if (avail < 0 || avail > a.num_blocks) {
    if (t == 0) atomicOr(a.err, PKV_DEVERR_BLOCK);
    avail = avail < 0 ? 0 : a.num_blocks;
  }

  Ask k;
  int n_go = 0, n_come = 0, n_rows = 0;  // of this thread's request in the pass
  // Read request base + t: what goes (with kGo), what comes.
  auto read = [&](int base, bool report) {
    const int r = base + t;
    n_go = n_come = n_rows = 0;
    int cut = 0, want = 0, held = 0, w_lo = 0, w_hi = 0;
    k = {0, 0, true};
    if (r < B) {
      k = read_ask(a, r, cap);
      if (k.bad && report) atomicOr(a.err, PKV_DEVERR_LENGTH);
      if (!k.bad) {
        held = blocks_of(k.old_len, P);
        want = blocks_of(k.new_len, P);
        cut = max(0, held - want);
        n_come = max(0, want - held);
        n_rows = max(0, k.new_len - k.old_len);
        if (a.window > 0) {
          // the first row behind the sinks that a decode from here on sees
          const long long lo = (long long)min(k.old_len, k.new_len) - a.window;
          w_lo = blocks_of(a.num_sinks, P);
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
      if (!(todo >> lane & 1)) w_lo = w_hi;
      while (todo) {
        const int l = __ffs(todo) - 1;
        todo &= todo - 1;
        const int rr = __shfl_sync(0xffffffffu, r, l);
        const int top = __shfl_sync(0xffffffffu, w_hi, l), bottom = __shfl_sync(0xffffffffu, w_lo, l);
        const int32_t* rrow = a.block_tables + (int64_t)rr * a.max_blocks;
        int at = top;  // blocks at .. top - 1 are still held
        while (at > bottom) {
          const int j = at - 1 - lane;
          const unsigned away = __ballot_sync(0xffffffffu, j < bottom || rrow[j] < 0);
          if (away) {
            at -= __ffs(away) - 1;
            break;
          }
          at -= 32;
        }
        if (lane == l) w_lo = at;
      }
    }
    n_go = cut + (w_hi - w_lo);
    s_cut[t] = cut;
    s_want[t] = want;
    s_wlo[t] = w_lo;
    s_held[t] = held;
  };
  // The ids of a pass that go, `total` of them: entry f of the list (ascending
  // request and block) goes onto the stack behind those after it.
  auto go = [&](int base, long long total) {
    for (long long f0 = total; f0 > 0; f0 -= kPer * kThreads) {
      // entries f0 - 1 - kPer t and those before it, together on their way
      int32_t id[kPer], *at[kPer];
      bool all = true;
      int o = -1;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const long long f = f0 - 1 - kPer * t - e;
        at[e] = nullptr;
        if (f < 0) continue;
        if (o < 0) o = first_above(ids_to, kThreads, f);
        while (o > 0 && ids_to[o - 1] > f) --o;
        const int x = (int)(f - (o ? ids_to[o - 1] : 0));
        const int w = (int)(ids_to[o] - (o ? ids_to[o - 1] : 0)) - s_cut[o];  // of them behind the window
        at[e] = a.block_tables + (int64_t)(base + o) * a.max_blocks +
                (x < w ? s_wlo[o] + x : s_want[o] + (x - w));
      }
#pragma unroll
      for (int e = 0; e < kPer; ++e) id[e] = at[e] ? *at[e] : -1;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (!at[e]) continue;
        *at[e] = -1;
        if (id[e] >= a.num_blocks) {
          atomicOr(a.err, PKV_DEVERR_BLOCK);
          id[e] = -1;
        }
        all = all && id[e] >= 0;
      }
      const long long here = min(f0, (long long)kPer * kThreads);
      if (__syncthreads_and(all)) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const long long place = avail + kPer * t + e;
          if (id[e] < 0) continue;
          if (place < a.num_blocks)
            a.free_ids[place] = id[e];
          else
            atomicOr(a.err, PKV_DEVERR_BLOCK);  // more ids than the pool has blocks
        }
        avail += here;
      } else {
        int mine = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) mine += id[e] >= 0;
        Sum3 pushed;
        long long place = avail + block_scan<kThreads>({mine, 0, 0}, ws, &pushed).a - mine;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          if (id[e] < 0) continue;
          if (place < a.num_blocks)
            a.free_ids[place] = id[e];
          else
            atomicOr(a.err, PKV_DEVERR_BLOCK);
          ++place;
        }
        avail += pushed.a;
      }
      avail = min(avail, (long long)a.num_blocks);
    }
  };

  long long rows = 0, taken = 0, used = 0;  // of the passes before: rows, ids asked for, ids given
  if (t == 0) a.row_ptr[0] = 0;
  // Ids and rows that come in a pass, from their running sums in it.
  auto grow = [&](int base, Sum3 upto, Sum3 total) {
    const int r = base + t;
    const bool crowded = rows + total.c > a.num_rows;  // some rows have no room
    if (crowded) {
      if (n_rows > 0 && rows + upto.c > a.num_rows) {
        atomicOr(a.err, PKV_DEVERR_LENGTH);
        k.new_len = k.old_len;
        n_come = 0;
      }
      Sum3 again;
      upto.b = block_scan<kThreads>({0, n_come, 0}, ws, &again).b;
      total.b = again.b;
    }
    bool served = true;
    if (taken + total.b > avail && n_come > 0 && taken + upto.b > avail) {  // not enough free blocks
      atomicOr(a.err, PKV_DEVERR_POOL);
      k.new_len = k.old_len;
      served = false;
    }
    if (r < B) {
      a.out_lens[r] = k.new_len;
      a.row_ptr[r + 1] = (int32_t)min(rows + upto.c, (long long)a.num_rows);
    }
    ids_to[t] = upto.b;
    rows_to[t] = upto.c;
    s_old[t] = k.old_len;
    s_new[t] = k.new_len;
    // those that are served stand in front of those that are not
    long long got = taken + total.b;
    if (got > avail) {
      Sum3 given;
      block_scan<kThreads>({served ? n_come : 0, 0, 0}, ws, &given);
      got = given.a > 0 ? taken + given.a : 0;
    }
    used = max(used, got);
    __syncthreads();
    for (long long f0 = 0; f0 < total.b; f0 += kPer * kThreads) {
      // entries f0 + kPer t and those behind it
      int32_t id[kPer], *at[kPer];
      int o = -1;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const long long f = f0 + kPer * t + e;
        at[e] = nullptr;
        if (f >= total.b) continue;
        if (o < 0) o = first_above(ids_to, kThreads, f);
        while (ids_to[o] <= f) ++o;
        if (s_new[o] == s_old[o]) continue;  // not served
        at[e] = a.block_tables + (int64_t)(base + o) * a.max_blocks + s_held[o] +
                (int)(f - (o ? ids_to[o - 1] : 0));
        id[e] = a.free_ids[avail - 1 - (taken + f)];
      }
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (!at[e]) continue;
        if (id[e] < 0 || id[e] >= a.num_blocks) {
          atomicOr(a.err, PKV_DEVERR_BLOCK);
          id[e] = -1;
        }
        *at[e] = id[e];
      }
    }
    rows += total.c;
    taken += total.b;
    __syncthreads();
  };

  if (single) {
    Sum3 total;
    read(0, true);
    const Sum3 upto = block_scan<kThreads>({n_go, n_come, n_rows}, ws, &total);
    if (total.a > 0) {
      ids_to[t] = upto.a;
      __syncthreads();
      go(0, total.a);
      __syncthreads();
    }
    grow(0, upto, total);
  } else {
    Sum3 total;
    for (int base = (B - 1) / kThreads * kThreads; base >= 0; base -= kThreads) {
      read(base, true);
      ids_to[t] = block_scan<kThreads>({n_go, 0, 0}, ws, &total).a;
      __syncthreads();
      go(base, total.a);
      __syncthreads();
    }
    for (int base = 0; base < B; base += kThreads) {
      read(base, false);
      const Sum3 upto = block_scan<kThreads>({0, n_come, n_rows}, ws, &total);
      grow(base, upto, total);
    }
  }
  if (t == 0) a.count_out[0] = (int32_t)(avail - used);
  // The decodes read tables and lengths before they wait for the kernel in
  // front of them to be complete, so these are visible before this one ends.
  __threadfence();
  if (!own_rows) return;
  if (single) {
    for (int64_t i = t; i < a.num_rows; i += kThreads) {
      const int o = first_above(rows_to, kThreads, i);
      if (o < B)
        write_row(a, i, o, (int)(i - (o ? rows_to[o - 1] : 0)), s_old[o], s_new[o]);
      else
        write_row(a, i, -1, 0, 0, 0);
    }
  } else {
    for (int64_t i = t; i < a.num_rows; i += kThreads) write_row(a, i);
  }
}

}  // namespace

cudaError_t launch_blocks_update(const BlocksArgs& a, cudaStream_t stream) {
  const int own = a.num_rows <= kBlOwnRows ? 1 : 0;
  // a call without rows gives ids back, of which there may be thousands
  if (a.num_seqs <= kBlFewSeqs && a.num_rows > 0 && a.num_rows <= kBlFewRows)
    blocks_update_kernel<kBlFewSeqs><<<1, kBlFewSeqs, 0, stream>>>(a, own);
  else
    blocks_update_kernel<1024><<<1, 1024, 0, stream>>>(a, own);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || own) return e;
  const int64_t grid = (a.num_rows + kBlRowThreads - 1) / kBlRowThreads;
  return launch_pdl(blocks_rows_kernel, dim3((unsigned)grid), dim3(kBlRowThreads), 0, stream, a);
}

}  // namespace pkv
