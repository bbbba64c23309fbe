// draft_tc.cu -- attention of drafted tokens over a paged bf16 or MXFP8 cache on
// the tcgen05 tensor cores.
//
// What it computes: draft.cu's formula.  For each kv head the n drafted rows'
// G query heads are n G rows of one matrix Q against the same keys, so
//     S [128 rows x 128 keys] = Q . K_tile^T,   O [128 x D] += P . V_tile
// with bf16 operands, fp32 accumulators in TMEM and a softmax state (m, l) in
// fp32 per row; a stage is 128 keys, K and V read once for up to 256 rows.
//
// What bounds it: at head_dim 128 a stage is 64 KiB, 1.47 us of one SM's share
// of the measured copy bandwidth, and 12.6 MFLOP per 128 rows (P in two terms:
// 4.2 of QK, 8.4 of PV), 1.0 us of its share of the measured bf16 rate: the
// bytes up to 128 rows, the MMAs past them.  Measured, 32 query and 8 kv heads:
// 16 requests with trees of 5 to 27 76 us (3.8 TB/s over the call; P in one term
// 66); 64 requests with trees of 64 342 us (1.30 PFLOP/s of MMAs; one term 288);
// MXFP8, 64 query heads, 12 requests 75 us (one term 72).  No pipe is full in any
// of them (64 trees: tensor 58% of its cycles, issue 0.50, DRAM 46%): what is
// left is the latency between the steps of a job, and of a stage's widening.
//
// Design:
//   * the work split, the pieces and their records are the decode's
//     (plan.cuh): one persistent CTA per SM takes an equal contiguous share of
//     the stages of every (sequence, kv head, 256-row) segment, writes whole
//     segments directly and leaves one (O, LSE) record per cut piece, which
//     draft_tc_reduce_kernel merges;
//   * two softmax warpgroups.  A piece of more than 128 rows gives each of them
//     one row tile, both against all of every stage; a piece of up to 128 rows
//     gives them a half of every stage each, against the same rows, and they
//     merge at its end.  (Alternate stages instead of halves keep two
//     stages of the ring under work, and fewer loads in flight: 76 us for 16
//     requests with trees where halves took 71.)
//   * a job is 64 keys, in two S buffers of a group in turn, so that the next
//     job's QK runs under a job's softmax.  TMEM (512 columns): 2 x 2 x 64 of S,
//     2 x 128 of O;
//   * thread t of a group owns row t of its tile (TMEM lane t): no cross-thread
//     reduction.  Warps whose 32 rows hold no drafted row skip the arithmetic;
//   * P goes into the PV as two bf16 terms (one alone errs by up to half a step
//     of each weight, 2^-8, which a few keys of opposite values can lift to the
//     size of the output's own rounding and past it), which overlay its S in
//     TMEM; the row sums take it whole;
//   * one warp streams K and V (TMA, 128-byte swizzle, row-group tiles of
//     launch.h) through a ring of tiles, K0, V0, K1, V1, ..., and each piece's
//     Q as soon as the previous piece's QKs have read theirs; a thread per
//     group issues its MMAs: QK(0), QK(1), PV(0), QK(2), PV(1), ...;
//   * an MXFP8 pool's tiles are filled by eight more warps instead of TMA: they
//     read codes and scales with plain loads, one tile ahead, and store the
//     widened bf16 rows into the ring in the same layout (exact: a code has
//     four significant bits).  No raw copy in shared memory is needed;
//   * only stages that hold drafted rows apply masks: a row's 64-bit mask is
//     shifted into place and selects the scores.  Drafted rows hidden from
//     some rows may hold anything, and 0 * NaN is not 0, so those stages also
//     clear non-finite elements of V, and rows past the last one, in shared
//     memory; a row that does see such an element adds it again at the end
//     (never, in ordinary use);
//   * the exponent base of a row moves only when its maximum grows by more
//     than 2^8 (exact), by a TMEM load/multiply/store of the row's O.
#include <math.h>

#include <atomic>

#include "draft.cuh"
#include "mx_widen.cuh"
#include "plan.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kDtSoftWarps = 8;      // two groups of four
constexpr int kDtWidenWarps = 8;     // MXFP8 pools
// ..., an MMA warp for each, producer, and for MXFP8 an idle warp (registers
// move between whole warpgroups) and the widening warps
constexpr int kDtWidenFirst = kDtSoftWarps + 4;
constexpr int dt_threads(bool mx) { return (mx ? kDtWidenFirst + kDtWidenWarps : kDtSoftWarps + 3) * 32; }
// Registers a thread of the MXFP8 kernel: 96 at launch (20 warps), of which the
// others give some to the softmax warps, whose loop spilled into L2 (the L1 is
// shared memory here; 12 requests, P in one term: 90.7 us, 73.7 so): 128 x 64 +
// 256 x 120 + 256 x 88 = 640 x 96.
constexpr int kDtMxRegs = 96, kDtMxIssueRegs = 64, kDtMxWidenRegs = 88, kDtMxSoftRegs = 120;
static_assert(128 * kDtMxIssueRegs + 256 * kDtMxSoftRegs + 256 * kDtMxWidenRegs <= dt_threads(true) * kDtMxRegs,
              "the warpgroups' registers come from the launch's");
constexpr int kDtJob = 64;           // keys of a job
// Columns of S that a softmax thread holds at once: a job's 64, or 32 (each 32
// are read again for their weights) where the widening warps leave fewer
// registers.
constexpr int dt_chunk(bool mx) { return mx ? 32 : 64; }
// Stage descriptors in flight.  A bf16 stage is described when its ring tiles
// are free.  An MXFP8 one is described once the stage kDtAhead before it has
// been widened; the widening warps send for its codes and then wait for the
// tiles themselves (12 requests, 64 query heads, before the registers moved and
// with P in one term: 90.7 us, described as bf16's
// 96).  So when stage n is described, stage n - 2 has been widened, into a ring
// of 12 tiles at most: the PVs of stage n - 8 are done, and a softmax group,
// which may be a stage without a job of its own behind (the end of a piece,
// where the groups meet), has read stage n - 10's descriptor.
constexpr int dt_descs(bool mx) { return mx ? 10 : 8; }
constexpr int kDtAhead = 2;
constexpr float kDtLn2 = 0.6931471805599453f;

// Stage descriptor flags.
constexpr int kDtStart = 1;   // first stage of a piece
constexpr int kDtEnd = 2;     // last stage of a piece
constexpr int kDtWhole = 4;   // the piece is its whole segment
constexpr int kDtSlot1 = 8;   // a cut piece that is not the CTA's first
constexpr int kDtPair = 16;   // two row tiles: both groups take every stage
constexpr int kDtDone = 32;   // no stage: the end of the CTA's work
constexpr int kDtTail = 64;   // holds drafted rows

constexpr int kDtDraftShift = 16;  // the sequence's drafted rows, above the flags

struct DtDesc {
  int4 a;  // sequence, segment of the sequence, valid keys, flags
  int4 b;  // context rows past the stage's first (may be negative), first query
           // row, rows of the segment, piece number (from 1)
};

// What a piece notes of its drafted rows with non-finite V: [0] the last such
// piece, [1 + j] the last piece whose row j was one (pieces count from 1).  Two
// of them by the piece's parity: some warps may clear a piece's V while others
// still read what the piece before noted.  The piece after that cannot be
// reached before they have: its clearing follows the end of the piece between
// (oend), whose MMAs wait until every softmax warp has left this one (ofree).
// The numbers in 16 bits: one that comes round again has a row looked at once
// more, whose finite elements add nothing.
constexpr int kDtBad = 1 + 64;

template <int D, int kTiles>
struct DtSmem {
  static constexpr int kHalf = kDraftRows * 128;          // 64 columns of a Q tile
  static constexpr int kTile = (D / 64) * kHalf;          // a Q, K or V tile
  static constexpr int kItems = D == 128 ? 7 - kTiles : 12;  // ring tiles
  static constexpr int q_off = 0;
  static constexpr int ring_off = kTiles * kTile;
  static constexpr int exch_off = ring_off + kItems * kTile;  // [2][128] (m, l); the plan's scratch
  static constexpr int desc_off = exch_off + 2 * 128 * 8;
  static constexpr int bar_off = desc_off + dt_descs(true) * (int)sizeof(DtDesc);
  static constexpr int bad_off = bar_off + (2 * kItems + dt_descs(true) + 17 + kDtAhead) * 8;
  static constexpr int tmem_off = bad_off + 2 * kDtBad * 2;
  static constexpr int total = tmem_off + 4;
  static_assert(total <= 227 * 1024, "shared memory of one CTA");
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two weights as bf16 pairs, p = hi + lo to 2^-14.9 of p.  hi is p cut off and lo
// what is left, of p (1 + 2^-20): neither is ever negative, nor 0 (above 2^-106)
// unless p is, so that an infinity of V stays one in hi V + lo V.
__device__ __forceinline__ void split_weights(float p0, float p1, uint32_t& hi, uint32_t& lo) {
  const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
  hi = __byte_perm(b0, b1, 0x7632);
  const float2 minus = make_float2(__uint_as_float((b0 & 0xffff0000u) | 0x80000000u),
                                   __uint_as_float((b1 & 0xffff0000u) | 0x80000000u));
  const float2 left = __ffma2_rn(make_float2(p0, p1), make_float2(1.f + 0x1p-20f, 1.f + 0x1p-20f), minus);
  const __nv_bfloat162 b2 = __floats2bfloat162_rn(left.x, left.y);
  lo = *reinterpret_cast<const uint32_t*>(&b2);
}

// All warps of a warpgroup: from now on each thread has kRegs registers.
template <int kRegs>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// A scale group's E4M3 codes.
struct Codes {
  uint32_t w[8];
};

// Whether any of them is a NaN: its lower seven bits are all set.
__device__ __forceinline__ bool nan_codes(const Codes& x) {
  constexpr uint32_t kLow = 0x7f7f7f7fu, kOne = 0x01010101u;
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) any |= (x.w[i] & kLow) + kOne;
  return (any & 0x80808080u) != 0;
}

// A group's codes (16-byte aligned), the second half before the first if `turned`.
__device__ __forceinline__ Codes load_codes(const uint8_t* p, int turned) {
  const uint4 lo = __ldg(reinterpret_cast<const uint4*>(p) + turned);
  const uint4 hi = __ldg(reinterpret_cast<const uint4*>(p) + (turned ^ 1));
  return Codes{{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
}

// Eight floats to a 32-byte aligned address: one whole sector a thread.
__device__ __forceinline__ void store_sector(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// Bits of a row's mask for the 32 keys 32 i .. 32 i + 31 of a stage whose key
// `mb` is drafted row 0: context keys are seen.
__device__ __forceinline__ uint32_t mask_word(uint64_t mask, int mb, int i) {
  const int sh = 32 * i - mb;  // drafted row of the word's first key
  if (sh >= 64) return 0u;
  if (sh >= 0) return (uint32_t)(mask >> sh);
  if (sh <= -32) return ~0u;
  return (uint32_t)(mask << -sh) | ((1u << -sh) - 1u);
}

}  // namespace

template <int D, int kTiles, bool kMx>
__global__ void __launch_bounds__(dt_threads(kMx), 1)
    draft_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmv, const DraftArgs a) {
  using L = DtSmem<D, kTiles>;
  constexpr int H = D / 64;
  constexpr int kItems = L::kItems;
  constexpr int kDescs = dt_descs(kMx);
  constexpr int kGroupBytes = kRowGroup * H * 128;  // one 8-row group of a K/V tile
  constexpr int kRecRows = kTiles * kDraftRows;
  extern __shared__ __align__(1024) unsigned char dt_smem[];
  unsigned char* sm = dt_smem;
  unsigned char* qs = sm + L::q_off;
  unsigned char* ring = sm + L::ring_off;
  float2* exch = reinterpret_cast<float2*>(sm + L::exch_off);
  DtDesc* descs = reinterpret_cast<DtDesc*>(sm + L::desc_off);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::bar_off);  // a ring tile landed
  uint64_t* freeb = full + kItems;    // its MMAs completed (two commits)
  uint64_t* dfull = freeb + kItems;   // a descriptor was written
  uint64_t* qfull = dfull + kDescs;   // a piece's Q landed
  uint64_t* qfree = qfull + 1;        // its QKs completed (a commit per group)
  uint64_t* sfull = qfree + 1;        // [group][buffer] S written
  uint64_t* pfull = sfull + 4;        // [group][buffer] P written
  uint64_t* pvdone = pfull + 4;       // [group] a PV completed
  uint64_t* oend = pvdone + 2;        // a piece's MMAs completed (a commit per group)
  uint64_t* ofree = oend + 1;         // both groups read its O
  uint64_t* xsync = ofree + 1;        // the groups meet at a piece's end
  uint64_t* vclean = xsync + 1;       // [2] group 0 cleared a tail stage's V for both
  uint64_t* widened = vclean + 2;     // [kDtAhead] MXFP8: a stage has been widened
  volatile uint16_t* bad_rows = reinterpret_cast<volatile uint16_t*>(sm + L::bad_off);  // [2][kDtBad]
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(sm + L::tmem_off);

  // the warp number as a warp-uniform value, for the branches on it
  const int t = threadIdx.x, warp = __shfl_sync(0xffffffffu, t >> 5, 0), lane = t & 31;
  const int c = blockIdx.x, P = a.block_size;
  const int Hkv = a.num_kv_heads, G = a.num_q_heads / Hkv;
  if (t == 0) {
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&full[i], kMx ? kDtWidenWarps : 1);
      mbar_init(&freeb[i], 2);
    }
    for (int i = 0; i < kDescs; ++i) mbar_init(&dfull[i], 1);
    mbar_init(qfull, 1);
    mbar_init(qfree, 2);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 4);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&pvdone[x], 1);
      mbar_init(&vclean[x], 4);
    }
    for (int i = 0; i < kDtAhead; ++i) mbar_init(&widened[i], kDtWidenWarps);
    mbar_init(oend, 2);
    mbar_init(ofree, kDtSoftWarps);
    mbar_init(xsync, kDtSoftWarps);
    fence_barrier_init();
  }
  if (t < 2 * kDtBad) bad_rows[t] = 0;
  if (warp == kDtSoftWarps + 2 && lane == 0) {
    prefetch_tensormap(&tmq);
    if constexpr (!kMx) {
      prefetch_tensormap(&tmk);
      prefetch_tensormap(&tmv);
    }
  }
  if (warp == 0) tc::tmem_alloc(tmem_base, 512);
  pdl_wait();
  pdl_launch_dependents();
  int4 d0;
  const int n =
      plan_cta_stages<dt_threads(kMx), kDraftKeys, 1>(a, reinterpret_cast<long long*>(exch), &d0);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_base;  // S of group x, buffer b at column 128 x + 64 b; O at 256 + 128 x

  if (n <= 0) {
    if (t == 0) a.cut_segs[c] = make_int2(-1, 0);  // nothing to do
  } else if (warp >= kDtSoftWarps && warp < kDtWidenFirst) {
    // setmaxnreg is one instruction of a whole warpgroup: this one takes it
    // together, and then its warps part (MXFP8: the fourth only for this)
    if (kMx) give_registers<kDtMxIssueRegs>();
    if (warp == kDtSoftWarps + 2) {
      // ============================================================ producer
      const int TB = draft_tc_box_rows(P);  // rows per box
      const int j = lane;                   // this lane's box
      const int heads = plan_heads(a);
      int r = d0.x, h = d0.y, i = d0.z;
      DraftSeq s = draft_seq(a, r, false);
      auto stages = [&]() { return s.n > 0 ? (s.ctx + s.n + kDraftKeys - 1) / kDraftKeys : 0; };
      int nt = stages();
      auto next_segment = [&]() {
        i = 0;
        if (++h == heads) {
          h = 0;
          do {
            ++r;
            s = draft_seq(a, r, false);
            nt = stages();
          } while (nt == 0);
        }
      };
      while (i >= nt) {  // the plan may name a segment's end
        const int over = i - nt;
        next_segment();
        i = over;
      }
      auto box_block = [&]() -> int {
        const int row = i * kDraftKeys + j * TB;
        return row < s.ctx + s.n && j * TB < kDraftKeys
                   ? __ldg(a.block_tables + (int64_t)r * a.max_blocks + row / P)
                   : 0;
      };
      int item = 0, pieces = 0;
      bool q_wanted = false;  // a piece's Q is still to be loaded
      int q_row = 0, q_head = 0, q_two = 0;
      int2 cut = make_int2(-1, 0);  // the segment that starts here and runs on into the next CTA
      bool ok = true;
      // lane 0: issue the wanted Q once the previous piece's QKs have read theirs
      auto try_q = [&](bool wait) -> bool {
        if (!q_wanted) return true;
        if (pieces > 1 && !(wait ? mbar_wait(qfree, (pieces - 2) & 1) : mbar_test(qfree, (pieces - 2) & 1)))
          return !wait;
        const int tiles = q_two ? 2 : 1;
        mbar_arrive_expect_tx(qfull, (uint32_t)(tiles * H * a.q_tokens * G * 128));
        for (int x = 0; x < tiles; ++x)
#pragma unroll
          for (int hf = 0; hf < H; ++hf)
            tma_load_3d(qs + x * L::kTile + hf * L::kHalf, &tmq, hf * 64, q_head, q_row + x * (kDraftRows / G),
                        qfull);
        q_wanted = false;
        return true;
      };
      // all lanes: wait for a barrier, and load the wanted Q meanwhile
      int slot = 0;
      uint32_t round = 0;
      auto wait_for = [&](uint64_t* bar, uint32_t n) -> bool {  // the barrier's phase n - 1, none for 0
        int good = 1;
        if (lane == 0) {
          try_q(false);
          if (n > 0) {
            const uint64_t t0 = global_timer_ns();
            while (q_wanted && !(good = mbar_test(bar, (n - 1) & 1)) && global_timer_ns() - t0 <= kWaitLimitNs)
              try_q(false);
            good = mbar_wait(bar, (n - 1) & 1);
          }
        }
        return __shfl_sync(0xffffffffu, good, 0) != 0;
      };
      struct Boxes {
        int group, n, head;  // first row group, boxes, kv head
      };
      // fill the next ring slot
      auto load = [&](const CUtensorMap* tm, const Boxes& x) -> bool {
        if (!wait_for(&freeb[slot], round)) return false;
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], (uint32_t)(x.n * TB * D * 2));
        __syncwarp();
        if (j < x.n)
          tma_load_5d(ring + slot * L::kTile + j * TB * H * 128, tm, 0, 0, 0, x.head, x.group, &full[slot]);
        ++item;
        if (++slot == kItems) {
          slot = 0;
          ++round;
        }
        return true;
      };
      int emitted = 0;
      int blk_next = box_block();
      for (int k = 0; k < n;) {
        const int mt = a.row_tiles > 1 ? h % a.row_tiles : 0;
        const int rows = min(s.n * G - mt * kRecRows, kRecRows);
        if (rows <= 0) {  // the sequence has no rows in this tile: pass its stages over
          k += nt - i;
          if (k >= n) break;
          next_segment();
          blk_next = box_block();
          continue;
        }
        const int kvh = a.row_tiles > 1 ? h / a.row_tiles : h;
        const int t0 = i * kDraftKeys, nvalid = min(kDraftKeys, s.ctx + s.n - t0);
        const int dseg = k - i;  // the CTA's stage that starts the segment
        const bool start = k == 0 || i == 0, end = k == n - 1 || i == nt - 1;
        const bool pair = kTiles > 1 && rows > kDraftRows;
        const int flags = (start ? kDtStart : 0) | (end ? kDtEnd : 0) |
                          (end && i == nt - 1 && dseg >= 0 ? kDtWhole : 0) | (dseg > 0 ? kDtSlot1 : 0) |
                          (pair ? kDtPair : 0) | (t0 + nvalid > s.ctx ? kDtTail : 0) | (s.n << kDtDraftShift);
        const int row0 = s.row0 + mt * (kRecRows / G);
        if (i == 0 && n - k < nt) cut = make_int2(r, h);
        if (start) {
          if (lane == 0 && !try_q(true)) ok = false;  // the piece before this one's, if it still waits
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
          ++pieces;
          q_wanted = true;
          q_row = row0;
          q_head = kvh * G;
          q_two = pair;
        }
        Boxes b;
        b.n = (nvalid + TB - 1) / TB;
        b.head = kvh;
        if (!kMx && j < b.n && (blk_next < 0 || (int64_t)blk_next >= a.num_blocks)) {
          atomicOr(a.err, PKV_DEVERR_BLOCK);
          b.group = (int)a.num_blocks * (P / kRowGroup);  // zero-filled out-of-range box
        } else {
          b.group = blk_next * (P / kRowGroup) + (t0 + j * TB) % P / kRowGroup;
        }
        auto describe = [&](int seq, int seg, int mb) {
          if (lane == 0) {
            DtDesc* d = &descs[emitted % kDescs];
            d->a = make_int4(seq, seg, nvalid, flags);
            d->b = make_int4(mb, row0, rows, pieces);
            mbar_arrive(&dfull[emitted % kDescs]);
          }
        };
        const int seq = r, seg = h, mb = s.ctx - t0;
        if (!kMx) describe(seq, seg, mb);
        ++k;
        if (k < n) {  // the next stage's block ids, under this one's waits
          if (++i == nt) next_segment();
          blk_next = box_block();
        }
        if constexpr (kMx) {
          ok = wait_for(&widened[emitted % kDtAhead], (uint32_t)emitted / kDtAhead);
          if (ok) describe(seq, seg, mb);
        } else {
          ok = load(&tmk, b) && load(&tmv, b);
        }
        if (!ok) break;
        ++emitted;
      }
      if (lane == 0) {
        a.cut_segs[c] = cut;
        if (ok) ok = try_q(true);
        if (ok) {
          descs[emitted % kDescs].a = make_int4(0, 0, 0, kDtDone);
          mbar_arrive(&dfull[emitted % kDescs]);
        } else {
          atomicOr(a.err, PKV_DEVERR_TIMEOUT);
          // copies may still be in flight into the ring and Q: wait for them
          if (!kMx)
            for (int it = item > kItems ? item - kItems : 0; it < item; ++it)
              mbar_wait(&full[it % kItems], (it / kItems) & 1);
          if (pieces > 0 && !q_wanted) mbar_wait(qfull, (pieces - 1) & 1);
        }
      }
    } else if (warp < kDtSoftWarps + 2) {
      // ============================================================ MMA issue
      const int x = warp - kDtSoftWarps;  // of this group's jobs; job j uses S buffer j & 1
      if (tc::elect_one()) {
        const uint32_t idqk = tc::idesc_bf16_f32(kDraftRows, kDtJob, 0, 0) |
                              (a.qscale < 0.f ? tc::kIdescNegateA : 0u);
        constexpr uint32_t kIdPV = tc::idesc_bf16_f32(kDraftRows, D, 0, 1);
        const uint32_t tS = tmem + x * 128, tO = tmem + 256 + x * 128;
        // What a PV needs of its job is kept for the two jobs at most between
        // their QK and their PV: flags, phase << 4, ring slot << 5 of its V.
        constexpr uint32_t kFirst = 1, kSecond = 2, kFrees = 4;
        uint32_t info0 = 0, info1 = 0;
        int jn = 0, pv = 0, pieces = 0;  // QKs and PVs issued, pieces begun
        bool first = true, freed = false;  // no job in the piece yet; O is known to be free
        // descriptors differ in their address field alone
        const uint64_t kdesc = tc::smem_desc_sw128(smem_u32(ring), 16, kGroupBytes);
        const uint64_t vdesc = tc::smem_desc_sw128(smem_u32(ring), 1024, kGroupBytes);
        const uint64_t qdesc = tc::smem_desc_sw128(smem_u32(qs), 16, 1024);
        auto issue_pv = [&]() -> bool {  // of job pv
          const int b = pv & 1;
          const uint32_t q = b ? info1 : info0;
          const uint32_t sl = q >> 5;
          if (!mbar_wait(&full[sl], (q >> 4) & 1)) return false;
          if (!freed) {  // the piece's first PV: the previous piece's O has been read
            if (pieces > 1 && !mbar_wait(ofree, (pieces - 2) & 1)) return false;
            freed = true;
          }
          if (!mbar_wait(&pfull[2 * x + b], (pv >> 1) & 1)) return false;
          tc::fence_after_sync();
          const uint64_t vd = vdesc + sl * (L::kTile >> 4) + ((q & kSecond) ? (8 * kGroupBytes) >> 4 : 0);
#pragma unroll
          for (int k = 0; k < kDtJob / 16; ++k) {  // 16 keys: their hi, then their lo
            const uint32_t tP = tS + b * 64 + 16 * k;
            tc::mma_bf16_ta(tO, tP, vd + ((k * 2 * kGroupBytes) >> 4), kIdPV, (k > 0 || !(q & kFirst)) ? 1u : 0u);
            tc::mma_bf16_ta(tO, tP + 8, vd + ((k * 2 * kGroupBytes) >> 4), kIdPV, 1u);
          }
          tc::commit(&pvdone[x]);
          if (q & kFrees) tc::commit(&freeb[sl]);
          ++pv;
          return true;
        };
        bool ok = true;
        uint32_t slot = 0, phase = 0;  // of the ring item that comes next
        auto advance = [&]() {
          if (++slot == kItems) {
            slot = 0;
            phase ^= 1u;
          }
        };
        for (int e = 0; ok; ++e) {
          uint64_t* db = &dfull[e % kDescs];
          if (!mbar_test(db, (e / kDescs) & 1)) {
            // no QK can be issued ahead of the PVs that are due: issue them first
            while (pv < jn && (ok = issue_pv())) {
            }
            if (!ok || !(ok = mbar_wait(db, (e / kDescs) & 1))) break;
          }
          const int nvalid = descs[e % kDescs].a.z, fl = descs[e % kDescs].a.w;
          if (fl & kDtDone) break;
          if (fl & kDtStart) {
            first = true;
            freed = false;
            if (!(ok = mbar_wait(qfull, pieces & 1))) break;
            ++pieces;
          }
          const uint32_t ksl = slot, kph = phase;
          advance();
          const uint32_t vinfo = (slot << 5) | (phase << 4);
          advance();
          const bool pair = kTiles > 1 && (fl & kDtPair);
          // halves of the stage: both in a pair, half x otherwise
          const int u_lo = pair ? 0 : x, u_hi = pair ? (nvalid > kDtJob ? 2 : 1) : (nvalid > x * kDtJob ? x + 1 : x);
          if (!mbar_test(&full[ksl], kph)) {
            while (pv < jn && (ok = issue_pv())) {
            }
            if (!ok || !(ok = mbar_wait(&full[ksl], kph))) break;
          }
          for (int u = u_lo; u < u_hi; ++u) {
            if (pv + 1 < jn && !(ok = issue_pv())) break;
            const int b = jn & 1;
            tc::fence_after_sync();
            const uint64_t kd = kdesc + ksl * (L::kTile >> 4) + (u ? (8 * kGroupBytes) >> 4 : 0);
            const uint64_t qd = qdesc + (pair ? x * (L::kTile >> 4) : 0);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              tc::mma_bf16(tS + b * 64, qd + (((k >> 2) * L::kHalf + (k & 3) * 32) >> 4),
                           kd + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), idqk, k > 0 ? 1u : 0u);
            tc::commit(&sfull[2 * x + b]);
            const bool last = u == u_hi - 1;
            if (last) tc::commit(&freeb[ksl]);
            const uint32_t q = vinfo | (first ? kFirst : 0) | (u ? kSecond : 0) | (last ? kFrees : 0);
            if (b) info1 = q;
            else info0 = q;
            first = false;
            ++jn;
          }
          if (!ok) break;
          if (u_lo == u_hi) {  // no key of this group's half: give the stage back
            tc::commit(&freeb[ksl]);
            const uint32_t vsl = vinfo >> 5;
            if (!(ok = mbar_wait(&full[vsl], (vinfo >> 4) & 1))) break;
            tc::commit(&freeb[vsl]);
          }
          if (fl & kDtEnd) {
            tc::commit(qfree);
            while (pv < jn && (ok = issue_pv())) {
            }
            if (!ok) break;
            // a piece without a job of this group must not run ahead either
            if (!freed && pieces > 1 && !(ok = mbar_wait(ofree, (pieces - 2) & 1))) break;
            tc::commit(oend);
          }
        }
        if (!ok) atomicOr(a.err, PKV_DEVERR_TIMEOUT);
      }
    }
  } else if (kMx && warp >= kDtWidenFirst) {
    // ============================================================ widening
    give_registers<kDtMxWidenRegs>();
    // A thread takes a scale group, 32 codes, of a row: step i of a tile covers
    // rows kStep i .. of it.  It takes its four chunks of eight codes in an
    // order, `turn`, that puts the stores of eight threads in a row into eight
    // bank groups.  The next tile's loads are out while a tile is widened.
    constexpr int kPerRow = D / 32, kStep = kDtWidenWarps * 32 / kPerRow, kSteps = kDraftKeys / kStep;
    const int wt = t - kDtWidenFirst * 32;
    const int g = wt % kPerRow, row0 = wt / kPerRow, half = g >> 1, turn = (row0 & 3) ^ (2 * half);
    const int shift = (P & (P - 1)) == 0 ? 31 - __clz(P) : -1;  // of a power-of-two block size
    int64_t at[kSteps];  // this thread's groups in the code planes (-1: none), and
    int sat[kSteps];     // how much further on they are in the scale planes
    Codes kx[kSteps], vx[kSteps];
    uint32_t ksc[kSteps], vsc[kSteps];
    int seq = -1, ctx = 0;
    auto places = [&](const int4& da, const int4& db) {
      if (da.x != seq) {
        seq = da.x;
        ctx = __ldg(a.ctx_lens + seq);
      }
      const int kvh = a.row_tiles > 1 ? da.y / a.row_tiles : da.y;
      const int t0 = ctx - db.x + row0;
      const int32_t* table = a.block_tables + (int64_t)seq * a.max_blocks;
      int blk[kSteps], off[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int row = t0 + i * kStep, bi = shift >= 0 ? row >> shift : row / P;
        off[i] = row - bi * P;
        blk[i] = i * kStep + row0 < da.z ? __ldg(table + bi) : -1;
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int64_t base = (int64_t)blk[i] * P * Hkv;  // rows of one head before the block
        at[i] = (base + off[i] * Hkv + kvh) * (D / 32) + g;
        sat[i] = (kvh * P + off[i] - (off[i] * Hkv + kvh)) * (D / 32);
        if (blk[i] < 0 || (int64_t)blk[i] >= a.num_blocks) {
          // any id may stand in the table: a row is one by its number
          if (i * kStep + row0 < da.z && g == 0) atomicOr(a.err, PKV_DEVERR_BLOCK);
          at[i] = -1;
        }
      }
    };
    auto fetch = [&](const void* pool, const uint8_t* scales, Codes (&x)[kSteps], uint32_t (&sc)[kSteps]) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        if (at[i] >= 0) {
          x[i] = load_codes(static_cast<const uint8_t*>(pool) + at[i] * 32, half);
          sc[i] = __ldg(scales + at[i] + sat[i]);
        } else {  // rows past the last one, and of bad blocks
          x[i] = Codes{};
          sc[i] = 0;
        }
      }
    };
    // its chunks' place in a tile: chunk q it takes goes to (q ^ turn) 16 from here on
    const uint32_t dst = (row0 / kRowGroup) * kGroupBytes + half * 1024 + (row0 & 7) * 128 +
                         ((((g & 1) * 4) ^ (row0 & 4)) << 4);
    auto widen = [&](int item, const Codes (&x)[kSteps], const uint32_t (&sc)[kSteps]) -> bool {
      // the tile's last MMAs have read it
      if (item >= kItems && !__all_sync(0xffffffffu, mbar_wait(&freeb[item % kItems], (item / kItems - 1) & 1)))
        return false;
      unsigned char* tile = ring + (size_t)(item % kItems) * L::kTile + dst;
      bool rare = false;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        unsigned char* d = tile + i * (kStep / kRowGroup) * kGroupBytes;
        __nv_bfloat162 s1, s2;
        scale_factors(sc[i], 0, s1, s2);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4*>(d + ((q ^ turn) << 4)) =
              widen8(make_uint2(x[i].w[2 * q], x[i].w[2 * q + 1]), s1, s2, false);
        rare |= sc[i] > 134u || nan_codes(x[i]);
      }
      // Rare: the second factor of scales past 2^7, and the NaN codes
      // s.1111.111, which widen8 takes for numbers, code by code, in few
      // instructions: the warps' loops have to fit the instruction cache.
      if (rare) {
        Codes y[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) y[i] = x[i];
#pragma unroll 1
        for (int n = 0; n < 32; ++n) {
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            const uint32_t code = y[i].w[0] & 0xffu, at16 = place2(code);
            __nv_bfloat162 s1, s2;
            scale_factors(sc[i], 0, s1, s2);
            const __nv_bfloat162 v = __hmul2(__hmul2(*reinterpret_cast<const __nv_bfloat162*>(&at16), s1), s2);
            *reinterpret_cast<uint16_t*>(tile + i * (kStep / kRowGroup) * kGroupBytes +
                                         (((n >> 3) ^ turn) << 4) + (n & 7) * 2) =
                (code & 0x7fu) == 0x7fu ? (uint16_t)0x7fffu : __bfloat16_as_ushort(__low2bfloat16(v));
#pragma unroll
            for (int w = 0; w < 8; ++w) y[i].w[w] = __funnelshift_r(y[i].w[w], w < 7 ? y[i].w[w + 1] : 0u, 8);
          }
        }
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[item % kItems]);
      return true;
    };
    bool ok = true, have = false;
    for (int e = 0;; ++e) {
      if (!have) {
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&dfull[e % kDescs], (e / kDescs) & 1)))) break;
        const DtDesc& d = descs[e % kDescs];
        if (d.a.w & kDtDone) break;
        places(d.a, d.b);
        fetch(a.k, a.k_scales, kx, ksc);
      }
      fetch(a.v, a.v_scales, vx, vsc);
      if (!(ok = widen(2 * e, kx, ksc))) break;
      have = __all_sync(0xffffffffu, mbar_test(&dfull[(e + 1) % kDescs], ((e + 1) / kDescs) & 1));
      if (have) {
        const DtDesc& d = descs[(e + 1) % kDescs];
        have = !(d.a.w & kDtDone);
        if (have) {
          places(d.a, d.b);
          fetch(a.k, a.k_scales, kx, ksc);
        }
      }
      if (!(ok = widen(2 * e + 1, vx, vsc))) break;
      if (lane == 0) mbar_arrive(&widened[e % kDtAhead]);
    }
    if (!ok && lane == 0) atomicOr(a.err, PKV_DEVERR_TIMEOUT);
  } else {
    // ============================================================ softmax
    if (kMx) take_registers<kDtMxSoftRegs>();
    const int x = warp >> 2;
    const int row = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tSx = tmem + x * 128 + lane_base, tOx = tmem + 256 + x * 128 + lane_base;
    // the sign of the scale is in the QK; 1e-37 keeps a hidden score -inf
    // where the scale is 0
    const float cs = fmaxf(fabsf(a.qscale), 1e-37f);
    float m = -INFINITY, l = 0.f;
    uint64_t mask = 0;
    bool live = false, warp_live = false, fresh = true;
    int rowg = 0, jobs = 0, syncs = 0, tails = 0;
    bool ok = true;
    auto wait = [&](uint64_t* b, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(b, parity));
    };
    for (int e = 0;; ++e) {
      if (!(ok = wait(&dfull[e % kDescs], (e / kDescs) & 1))) break;
      const int4 da = descs[e % kDescs].a, db = descs[e % kDescs].b;
      const int fl = da.w;
      if (fl & kDtDone) break;
      const bool pair = kTiles > 1 && (fl & kDtPair);
      const int nvalid = da.z, mb = db.x;
      if (fl & kDtStart) {
        m = -INFINITY;
        l = 0.f;
        fresh = true;
        rowg = (pair ? x * kDraftRows : 0) + row;
        live = rowg < db.z;
        warp_live = __any_sync(0xffffffffu, live);
        DraftSeq s;
        s.n = fl >> kDtDraftShift;
        const int tok0 = a.row_tiles > 1 ? (da.y % a.row_tiles) * (kRecRows / G) : 0;
        s.row0 = db.y - tok0;
        mask = live ? draft_mask(a, s, tok0 + rowg / G) : 0ull;
      }
      {
        const int u_lo = pair ? 0 : x, u_hi = pair ? (nvalid > kDtJob ? 2 : 1) : (nvalid > x * kDtJob ? x + 1 : x);
        for (int u = u_lo; u < u_hi; ++u) {
          const int b = jobs & 1;
          if (!(ok = wait(&sfull[2 * x + b], (jobs >> 1) & 1))) break;
          tc::fence_after_sync();
          if (warp_live) {
            const uint32_t tS = tSx + b * 64;
            constexpr int kChunk = dt_chunk(kMx), kChunks = kDtJob / kChunk;
            uint32_t v[kChunk];
            auto read = [&](int w) {
#pragma unroll
              for (int q = 0; q < kChunk / 32; ++q)
                tc::tmem_ld32(tS + kChunk * w + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(v + 32 * q));
#pragma unroll
              for (int q = 0; q < kChunk / 32; ++q) tc::wait_ld32(*reinterpret_cast<uint32_t(*)[32]>(v + 32 * q));
              if (fl & kDtTail) {
#pragma unroll
                for (int q = 0; q < kChunk / 32; ++q) {
                  const uint32_t bits = mask_word(mask, mb, 2 * u + w * (kChunk / 32) + q);
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    if (!((bits >> i) & 1u)) v[32 * q + i] = __float_as_uint(-INFINITY);
                }
              }
            };
            float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int w = 0; w < kChunks; ++w) {
              read(w);
#pragma unroll
              for (int i = 0; i < kChunk; i += 2)
                mx4[(i >> 1) & 3] = max3(mx4[(i >> 1) & 3], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
            }
            const float mx = cs * fmaxf(max3(mx4[0], mx4[1], mx4[2]), mx4[3]);
            const float m_new = fmaxf(m, mx);
            const bool need = live && m_new > m + 8.0f;
            const float alpha = need ? exp2f(m - m_new) : 1.f;
            if (need) m = m_new;
            const float nm = m == -INFINITY ? 0.f : -m;  // nothing seen yet: every weight is 0
            // ---- P = exp2(c s - m) in bf16 pairs, hi and lo, over the columns
            // of the S that it came from; the sums take it whole
            // (two pairs of sums: with four of them the pair form spills, 353 us
            // for 64 trees of 64 and 342)
            float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            // (not unrolled: MXFP8's two chunks at once spill, 98 us and 75)
#pragma unroll 1
            for (int w = kChunks - 1; w >= 0; --w) {
              if (kChunks > 1) read(w);
#pragma unroll
              for (int q = 0; q < kChunk / 32; ++q) {
                uint32_t pw[32];  // of 16 keys hi, then lo, and of the next 16
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float p0 = exp2f(fmaf(__uint_as_float(v[32 * q + 2 * i]), cs, nm));
                  const float p1 = exp2f(fmaf(__uint_as_float(v[32 * q + 2 * i + 1]), cs, nm));
                  ls[i & 1] = __fadd2_rn(ls[i & 1], make_float2(p0, p1));
                  split_weights(p0, p1, pw[(i & 7) + 16 * (i >> 3)], pw[8 + (i & 7) + 16 * (i >> 3)]);
                }
                tc::tmem_st32(tS + kChunk * w + 32 * q, pw);
              }
            }
            const float2 ls2 = __fadd2_rn(ls[0], ls[1]);
            l = l * alpha + (ls2.x + ls2.y);
            // a new base: once the group's previous PV has added to O under the
            // old one (and no later one has begun), rescale the row
            if (!fresh && __any_sync(0xffffffffu, need)) {
              if (!(ok = wait(&pvdone[x], (jobs - 1) & 1))) break;
              tc::fence_after_sync();
#pragma unroll 1
              for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t o[32];
                tc::tmem_ld32(tOx + c0, o);
                tc::wait_ld32(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tc::tmem_st32(tOx + c0, o);
              }
            }
            tc::wait_st();
          }
          fresh = false;
          // A tail stage's V is cleared, before its first PV, of what the PVs
          // must not multiply: rows past the last one (weight 0, any bytes) and
          // non-finite elements of drafted rows, which some row may not see.
          // In a pair group 0 does it for both, otherwise each in its half.
          if ((fl & kDtTail) && u == u_lo) {
            if (!pair || x == 0) {
              const int vitem = 2 * e + 1;  // K and V of a stage are ring items 2 e and 2 e + 1
              if (!(ok = wait(&full[vitem % kItems], (vitem / kItems) & 1))) break;
              if (row >= mb && (pair || (row >> 6) == x)) {
                unsigned char* vr = ring + (size_t)(vitem % kItems) * L::kTile +
                                    (row / kRowGroup) * kGroupBytes + (row % kRowGroup) * 128;
                bool found = false;
#pragma unroll
                for (int hf = 0; hf < H; ++hf)
#pragma unroll 2
                  for (int ch = 0; ch < 8; ++ch) {
                    uint4* at = reinterpret_cast<uint4*>(vr + hf * 1024 + (ch ^ (row & 7)) * 16);  // other banks than the next rows'
                    if (row >= nvalid) {
                      *at = make_uint4(0u, 0u, 0u, 0u);
                      continue;
                    }
                    const uint4 w = *at;
                    uint32_t q[4] = {w.x, w.y, w.z, w.w};
                    bool any = false;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                      if ((q[i] & 0x7f80u) == 0x7f80u) {
                        q[i] &= 0xffff0000u;
                        any = true;
                      }
                      if ((q[i] & 0x7f800000u) == 0x7f800000u) {
                        q[i] &= 0xffffu;
                        any = true;
                      }
                    }
                    if (any) *at = make_uint4(q[0], q[1], q[2], q[3]);
                    found |= any;
                  }
                if (found) {
                  volatile uint16_t* bad = bad_rows + (db.w & 1) * kDtBad;
                  bad[1 + row - mb] = (uint16_t)db.w;
                  bad[0] = (uint16_t)db.w;
                }
              }
              tc::fence_proxy_async_smem();
              __syncwarp();
              if (pair && lane == 0) mbar_arrive(&vclean[tails & 1]);
            } else if (!(ok = wait(&vclean[tails & 1], (tails >> 1) & 1))) {
              break;
            }
            if (pair) ++tails;
          }
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&pfull[2 * x + b]);
          ++jobs;
        }
        if (!ok) break;
      }
      if (fl & kDtEnd) {
        // ---- a piece's end: O / l and the LSE of each row
        if (!(ok = wait(oend, (db.w - 1) & 1))) break;
        tc::fence_after_sync();
        if (!pair) exch[x * kDraftRows + row] = make_float2(m, l);
        if (!pair || (fl & kDtTail)) {  // the groups' states, and `bad`
          __syncwarp();
          if (lane == 0) mbar_arrive(xsync);
          if (!(ok = wait(xsync, syncs & 1))) break;
          ++syncs;
        }
        if (warp_live) {
          float M = m, Ls = l, f0 = 1.f, f1 = 1.f;
          bool has0 = x == 0, has1 = x == 1;  // accumulators that hold this row's outputs
          if (!pair) {
            const float2 s0 = exch[row], s1 = exch[kDraftRows + row];
            M = fmaxf(s0.x, s1.x);
            const float base = M == -INFINITY ? 0.f : M;
            f0 = exp2f(s0.x - base);
            f1 = exp2f(s1.x - base);
            Ls = f0 * s0.y + f1 * s1.y;
            // a group without a job in the piece (one stage), or without a
            // seen key, has nothing in its O
            has0 = s0.y != 0.f;
            has1 = s1.y != 0.f;
          }
          const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
          f0 *= inv;
          f1 *= inv;
          const float lse2 = Ls == 0.f ? -INFINITY : M + log2f(Ls);
          const int tok = rowg / G, g = rowg % G;
          const int kvh = a.row_tiles > 1 ? da.y / a.row_tiles : da.y;
          const int64_t qh = (int64_t)(db.y + tok) * a.num_q_heads + kvh * G + g;
          const int64_t rec = (2 * (int64_t)c + ((fl & kDtSlot1) ? 1 : 0)) * kRecRows + rowg;
          const bool whole = (fl & kDtWhole) != 0;
          if (live && (pair || x == 0)) {
            if (!whole) a.rec_lse[rec] = lse2;
            else if (a.lse_out) a.lse_out[qh] = lse2 * kDtLn2;
          }
          volatile uint16_t* bad = bad_rows + (db.w & 1) * kDtBad;
          const bool fix = bad[0] == (uint16_t)db.w;
          // columns: all in a pair, this group's half otherwise, 16 at a time
          const int c_lo = pair ? 0 : x * (D / 2), c_hi = pair ? D : c_lo + D / 2;
#pragma unroll 1
          for (int c0 = c_lo; c0 < c_hi; c0 += 16) {
            float o[16];
            uint32_t w0[16], w1[16];
            if (!pair || x == 0) tc::tmem_ld16(tmem + 256 + lane_base + c0, w0);
            if (!pair || x == 1) tc::tmem_ld16(tmem + 384 + lane_base + c0, w1);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              o[i] = has0 ? __uint_as_float(w0[i]) * f0 : 0.f;
              if (has1) o[i] = fmaf(__uint_as_float(w1[i]), f1, o[i]);
            }
            if (fix && live) {  // non-finite elements that this row does see
              for (uint64_t left = mask; left; left &= left - 1) {
                const int jd = __ffsll((long long)left) - 1;
                if (bad[1 + jd] != (uint16_t)db.w) continue;
                const int pos = __ldg(a.ctx_lens + da.x) + jd;
                const int blk = __ldg(a.block_tables + (int64_t)da.x * a.max_blocks + pos / P);
                if (blk < 0 || (int64_t)blk >= a.num_blocks) continue;
                const int64_t vrow = (int64_t)blk * P + pos % P;
                if constexpr (kMx) {
                  const __nv_fp8_e4m3* vp = static_cast<const __nv_fp8_e4m3*>(a.v) + (vrow * Hkv + kvh) * D + c0;
                  const float sc = e8m0_value(__ldg(a.v_scales + (((int64_t)blk * Hkv + kvh) * P + pos % P) * (D / 32) +
                                                    c0 / 32));
#pragma unroll
                  for (int i = 0; i < 16; ++i) {
                    const float x = __bfloat162float(__float2bfloat16_rn((float)vp[i] * sc));
                    if ((__float_as_uint(x) & 0x7f800000u) == 0x7f800000u) o[i] += x;
                  }
                } else {
                  const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(a.v) + (vrow * Hkv + kvh) * D + c0;
#pragma unroll
                  for (int i = 0; i < 16; ++i) {
                    const uint32_t u = __bfloat16_as_ushort(vp[i]);
                    if ((u & 0x7f80u) == 0x7f80u) o[i] += __uint_as_float(u << 16);
                  }
                }
              }
            }
            if (live) {
              if (whole) {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + qh * D + c0);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  uint32_t b[4];
#pragma unroll
                  for (int u = 0; u < 4; ++u) {
                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(o[8 * i + 2 * u], o[8 * i + 2 * u + 1]);
                    b[u] = *reinterpret_cast<const uint32_t*>(&b2);
                  }
                  dst[i] = make_uint4(b[0], b[1], b[2], b[3]);
                }
              } else {
                float* dst = a.rec_o + rec * D + c0;
                store_sector(dst, o);
                store_sector(dst + 8, o + 8);
              }
            }
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(ofree);
      }
    }
    if (!ok && lane == 0) atomicOr(a.err, PKV_DEVERR_TIMEOUT);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// Merge the pieces of the segment that starts in CTA blockIdx.x and runs on
// into later ones, by log-sum-exp: a block per 32 rows, a warp per four of
// them, whose pieces' outputs are loaded together; or, with kShare, a block
// per four rows, whose warps share the pieces.
template <int D, int kTiles, bool kShare>
__global__ void __launch_bounds__(256) draft_tc_reduce_kernel(const DraftArgs a) {
  constexpr int EPL = D / 32;
  constexpr int kRecRows = kTiles * kDraftRows;
  constexpr int kRows = 4, kBatch = kShare ? 4 : 2;  // rows of a warp; pieces loaded at once for each
  pdl_wait();  // the records and the plan are complete
  const int2 seg = a.cut_segs[blockIdx.x];
  if (seg.x < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = seg.x, h = seg.y;
  const long long total = a.plan_pre[a.num_seqs], pre = a.plan_pre[r], u = a.plan_pre[r + 1] - pre;
  const DraftSeq s = draft_seq(a, r, false);
  const int G = a.num_q_heads / a.num_kv_heads;
  const int mt = h % a.row_tiles, kvh = h / a.row_tiles;
  const int row0 = (kShare ? blockIdx.y : blockIdx.y * 8 + warp) * kRows;  // of the segment
  const int rows = min(kRows, s.n * G - mt * kRecRows - row0);
  if (rows <= 0) return;
  const int heads = plan_heads(a);
  const long long su = a.stage_units, pu = a.piece_units;
  const long long nt = (u - pu) / su;
  const long long cw = units_per_cta(total * heads, a.num_ctas, su);
  const long long seg0 = pre * heads + (long long)h * u;
  const int c_first = blockIdx.x, c_last = (int)((seg0 + pu + su * (nt - 1)) / cw);
  // a first piece is in slot 1 of its CTA when that CTA owns an earlier stage
  const bool slot1 = seg0 > 0 && seg0 - su >= (long long)c_first * cw;
  const int np = c_last - c_first + 1;
  auto rec = [&](int i, int k) -> int64_t {  // piece i of row row0 + k
    return (2 * (int64_t)(c_first + i) + (i == 0 && slot1 ? 1 : 0)) * kRecRows + row0 + k;
  };
  float acc[kRows][EPL], M[kRows], Ls[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    M[k] = -INFINITY;
    Ls[k] = 0.f;
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[k][e] = 0.f;
  }
  for (int i0 = kShare ? warp * kBatch : 0; i0 < np; i0 += kShare ? 8 * kBatch : kBatch) {
    float ls[kBatch][kRows], f[kBatch][kRows][EPL];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        ls[i][k] = -INFINITY;
#pragma unroll
        for (int e = 0; e < EPL; ++e) f[i][k][e] = 0.f;
        if (i0 + i >= np || k >= rows) continue;
        ls[i][k] = a.rec_lse[rec(i0 + i, k)];
        const float* p = a.rec_o + rec(i0 + i, k) * D + lane * EPL;
        if constexpr (EPL == 4) {
          const float4 x = *reinterpret_cast<const float4*>(p);
          f[i][k][0] = x.x, f[i][k][1] = x.y, f[i][k][2] = x.z, f[i][k][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(p);
          f[i][k][0] = x.x, f[i][k][1] = x.y;
        }
      }
#pragma unroll
    for (int k = 0; k < kRows; ++k)
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (ls[i][k] == -INFINITY) continue;  // an empty state
        // the running base; a NaN state makes everything NaN
        const float m = fmaxf(M[k], ls[i][k]), w0 = M[k] == m ? 1.f : exp2f(M[k] - m), w1 = exp2f(ls[i][k] - m);
        M[k] = m;
        Ls[k] = Ls[k] * w0 + w1;
#pragma unroll
        for (int e = 0; e < EPL; ++e) acc[k][e] = fmaf(w1, f[i][k][e], acc[k][e] * w0);
      }
  }
  if constexpr (kShare) {  // warp k adds the warps' sums of row k to its own
    __shared__ float2 state[8][kRows];
    __shared__ float sums[8][kRows][D];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (lane == 0) state[warp][k] = make_float2(M[k], Ls[k]);
#pragma unroll
      for (int e = 0; e < EPL; ++e) sums[warp][k][e * 32 + lane] = acc[k][e];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (warp != k) continue;
#pragma unroll 1
      for (int w = 0; w < 8; ++w) {
        const float2 x = state[w][k];
        if (w == warp || x.y == 0.f) continue;  // its own, or nothing
        const float m = fmaxf(M[k], x.x), w0 = M[k] == m ? 1.f : exp2f(M[k] - m), w1 = exp2f(x.x - m);
        M[k] = m;
        Ls[k] = Ls[k] * w0 + x.y * w1;
#pragma unroll
        for (int e = 0; e < EPL; ++e) acc[k][e] = fmaf(w1, sums[w][k][e * 32 + lane], acc[k][e] * w0);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (k >= rows || (kShare && warp != k)) continue;
    const float inv = Ls[k] == 0.f ? 0.f : 1.f / Ls[k];
    const int rowg = mt * kRecRows + row0 + k;
    const int64_t qh = (int64_t)(s.row0 + rowg / G) * a.num_q_heads + kvh * G + rowg % G;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + qh * D + lane * EPL;
    uint32_t o2[EPL / 2];
#pragma unroll
    for (int e = 0; e < EPL / 2; ++e) {
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(acc[k][2 * e] * inv, acc[k][2 * e + 1] * inv);
      o2[e] = *reinterpret_cast<const uint32_t*>(&b2);
    }
    if constexpr (EPL == 4) *reinterpret_cast<uint2*>(out) = make_uint2(o2[0], o2[1]);
    else *reinterpret_cast<uint32_t*>(out) = o2[0];
    if (lane == 0 && a.lse_out)
      a.lse_out[qh] = Ls[k] == 0.f ? -INFINITY : (M[k] + log2f(Ls[k])) * kDtLn2;
  }
}

template <int D, int kTiles, bool kMx>
static cudaError_t launch_draft_tc_t(const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
                                     const DraftArgs& a, cudaStream_t stream) {
  constexpr int smem = DtSmem<D, kTiles>::total;
  auto kern = draft_tc_kernel<D, kTiles, kMx>;
  if constexpr (kMx) {  // with fewer registers at launch the softmax warps would wait for theirs for ever
    static std::atomic<int> regs{0};  // once known; a query that fails is asked again
    if (regs.load(std::memory_order_relaxed) == 0) {
      cudaFuncAttributes f;
      cudaError_t e = cudaFuncGetAttributes(&f, kern);
      if (e != cudaSuccess) return e;
      regs.store(f.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) < kDtMxRegs) return cudaErrorInvalidConfiguration;
  }
  static SmemAttrCache attr_cache;
  cudaError_t e = ensure_smem_limit(kern, smem, attr_cache);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3((unsigned)a.num_ctas), dim3(dt_threads(kMx)), smem, stream, tmq, tmk, tmv, a);
  if (e != cudaSuccess || a.num_ctas == 1) return e;  // one CTA cuts nothing
  const int rows = a.max_draft * (a.num_q_heads / a.num_kv_heads);
  const int most = rows < kTiles * kDraftRows ? rows : kTiles * kDraftRows;
  // Segments of eight pieces or more: one block would merge them one after
  // another (one sequence of 21000 rows, one kv head, 152 pieces: 48.5 us, and
  // 20.1 us shared).
  if (a.num_ctas >= 8ll * a.num_seqs * a.num_kv_heads * a.row_tiles)
    return launch_pdl(draft_tc_reduce_kernel<D, kTiles, true>, dim3((unsigned)a.num_ctas, (unsigned)((most + 3) / 4)),
                      dim3(256), 0, stream, a);
  return launch_pdl(draft_tc_reduce_kernel<D, kTiles, false>,
                    dim3((unsigned)a.num_ctas, (unsigned)((most + 31) / 32)), dim3(256), 0, stream, a);
}

template <int D, bool kMx>
static cudaError_t launch_draft_tc_d(int tiles, const CUtensorMap& tmq, const CUtensorMap& tmk,
                                     const CUtensorMap& tmv, const DraftArgs& a, cudaStream_t stream) {
  return tiles > 1 ? launch_draft_tc_t<D, 2, kMx>(tmq, tmk, tmv, a, stream)
                   : launch_draft_tc_t<D, 1, kMx>(tmq, tmk, tmv, a, stream);
}

cudaError_t launch_draft_tc(int dtype, int head_dim, int tiles, const CUtensorMap& tmq,
                            const CUtensorMap& tmk, const CUtensorMap& tmv, const DraftArgs& a,
                            cudaStream_t stream) {
  if (dtype == PKV_MXFP8)
    return head_dim == 128 ? launch_draft_tc_d<128, true>(tiles, tmq, tmk, tmv, a, stream)
                           : launch_draft_tc_d<64, true>(tiles, tmq, tmk, tmv, a, stream);
  return head_dim == 128 ? launch_draft_tc_d<128, false>(tiles, tmq, tmk, tmv, a, stream)
                         : launch_draft_tc_d<64, false>(tiles, tmq, tmk, tmv, a, stream);
}

}  // namespace pkv
