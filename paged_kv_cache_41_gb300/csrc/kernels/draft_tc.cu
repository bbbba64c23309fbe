// draft_tc.cu -- attention of drafted tokens over a paged bf16 cache on the
// tcgen05 tensor cores.
//
// What it computes: draft.cu's formula.  For each kv head the n drafted rows'
// G query heads are n G rows of one matrix Q against the same keys, so
//     S [128 rows x 128 keys] = Q . K_tile^T,   O [128 x D] += P . V_tile
// with bf16 operands, fp32 accumulators in TMEM and a softmax state (m, l) in
// fp32 per row; a stage is 128 keys, K and V read once for up to 256 rows.
//
// What bounds it: at head_dim 128 a stage is 64 KiB, 1.47 us of one SM's share
// of the measured copy bandwidth, and 8.4 MFLOP per 128 rows, 0.67 us of its
// share of the measured bf16 rate: the bytes, up to 256 rows.
//
// Design:
//   * the work split, the pieces and their records are the decode's
//     (plan.cuh): one persistent CTA per SM takes an equal contiguous share of
//     the stages of every (sequence, kv head, 256-row) segment, writes whole
//     segments directly and leaves one (O, LSE) record per cut piece, which
//     draft_tc_reduce_kernel merges;
//   * two softmax groups, each with its own S and O in TMEM (512 columns).
//     A piece of more than 128 rows gives each of them one row tile, both
//     against every stage; a piece of up to 128 rows gives them alternate
//     stages of the same rows, merged at its end.  Either way one group's
//     softmax runs while the tensor pipe works for the other;
//   * a group is two warpgroups: a thread takes one row (its TMEM lane) and 64
//     of the 128 keys, and meets the row's other thread once a stage, over its
//     maximum.  (One warpgroup a group, 128 keys a thread: the softmax's
//     latency, 4,500 cycles a stage, held the tensor pipe; 700 us for 64
//     requests with trees of 64.)  Warps whose 32 rows hold no drafted row
//     skip the arithmetic;
//   * P is rounded to bf16 (half a step, 2^-8 of each weight, is the size of the
//     output's own rounding) and overlays its S in TMEM, from where
//     the PV MMA reads it; the row sums are taken before the rounding;
//   * one warp streams K and V (TMA, 128-byte swizzle, row-group tiles of
//     launch.h) through a ring of tiles, K0, V0, K1, V1, ..., and each piece's
//     Q as soon as the previous piece's QKs have read theirs; one thread of
//     another issues the MMAs: QK(0), QK(1), PV(0), QK(2), PV(1), ...;
//   * only stages that hold drafted rows apply masks: a row's 64-bit mask is
//     shifted into place and selects the scores.  Drafted rows hidden from
//     some rows may hold anything, and 0 * NaN is not 0, so those stages also
//     clear non-finite elements of V and rows past the last one in shared memory; a row
//     that does see such an element adds it again at the end (never, in
//     ordinary use);
//   * the exponent base of a row moves only when its maximum grows by more
//     than 2^8 (exact), by a TMEM load/multiply/store of the row's O.
#include <math.h>

#include "draft.cuh"
#include "plan.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kDtSoftWarps = 16;     // two groups of eight
constexpr int kDtThreads = (kDtSoftWarps + 2) * 32;  // ..., MMA, producer
constexpr int kDtDescs = 8;          // stage descriptors in flight
constexpr float kDtLn2 = 0.6931471805599453f;

// Stage descriptor flags.
constexpr int kDtStart = 1;   // first stage of a piece
constexpr int kDtEnd = 2;     // last stage of a piece
constexpr int kDtWhole = 4;   // the piece is its whole segment
constexpr int kDtSlot1 = 8;   // a cut piece that is not the CTA's first
constexpr int kDtPair = 16;   // two row tiles: both groups take every stage
constexpr int kDtDone = 32;   // no stage: the end of the CTA's work
constexpr int kDtTail = 64;   // holds drafted rows
constexpr int kDtOdd = 128;   // the stage's first MMA job is group 1's

constexpr int kDtDraftShift = 16;  // the sequence's drafted rows, above the flags

struct DtDesc {
  int4 a;  // sequence, segment of the sequence, valid keys, flags
  int4 b;  // context rows past the stage's first (may be negative), first query
           // row, rows of the segment, piece number (from 1)
};

template <int D, int kTiles>
struct DtSmem {
  static constexpr int kHalf = kDraftRows * 128;          // 64 columns of a Q tile
  static constexpr int kTile = (D / 64) * kHalf;          // a Q, K or V tile
  static constexpr int kItems = D == 128 ? 7 - kTiles : 12;  // ring tiles
  static constexpr int q_off = 0;
  static constexpr int ring_off = kTiles * kTile;
  static constexpr int exch_off = ring_off + kItems * kTile;  // [4][128] floats; the plan's scratch
  static constexpr int desc_off = exch_off + 4 * 128 * 4;
  static constexpr int bar_off = desc_off + kDtDescs * (int)sizeof(DtDesc);
  static constexpr int bad_off = bar_off + (2 * kItems + kDtDescs + 17) * 8;
  static constexpr int tmem_off = bad_off + 65 * 4;
  static constexpr int total = tmem_off + 4;
  static_assert(total <= 227 * 1024, "shared memory of one CTA");
};

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

template <int D, int kTiles>
__global__ void __launch_bounds__(kDtThreads, 1)
    draft_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmv, const DraftArgs a) {
  using L = DtSmem<D, kTiles>;
  constexpr int H = D / 64;
  constexpr int kItems = L::kItems;
  constexpr int kGroupBytes = kRowGroup * H * 128;  // one 8-row group of a K/V tile
  constexpr int kRecRows = kTiles * kDraftRows;
  extern __shared__ __align__(1024) unsigned char dt_smem[];
  unsigned char* sm = dt_smem;
  unsigned char* qs = sm + L::q_off;
  unsigned char* ring = sm + L::ring_off;
  float* exch = reinterpret_cast<float*>(sm + L::exch_off);
  DtDesc* descs = reinterpret_cast<DtDesc*>(sm + L::desc_off);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::bar_off);  // a ring tile landed
  uint64_t* freeb = full + kItems;    // its MMAs completed
  uint64_t* dfull = freeb + kItems;   // a descriptor was written
  uint64_t* qfull = dfull + kDtDescs; // a piece's Q landed
  uint64_t* qfree = qfull + 1;        // its QKs completed
  uint64_t* sfull = qfree + 1;        // [2] S of a group written
  uint64_t* pfull = sfull + 2;        // [2] P of a group written
  uint64_t* oend = pfull + 2;         // a piece's MMAs completed
  uint64_t* ofree = oend + 1;         // both groups read its O
  uint64_t* xsync = ofree + 1;        // the groups meet at a piece's end
  uint64_t* psync = xsync + 1;        // [8] the two warps of the same rows meet
  // a piece's drafted rows with non-finite V: [0] the last such piece, [1 + j]
  // the last piece whose row j was one (pieces count from 1)
  volatile int* bad = reinterpret_cast<volatile int*>(sm + L::bad_off);
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(sm + L::tmem_off);

  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int c = blockIdx.x, P = a.block_size;
  const int Hkv = a.num_kv_heads, G = a.num_q_heads / Hkv;
  if (t == 0) {
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&freeb[i], 1);
    }
    for (int i = 0; i < kDtDescs; ++i) mbar_init(&dfull[i], 1);
    mbar_init(qfull, 1);
    mbar_init(qfree, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sfull[x], 1);
      mbar_init(&pfull[x], 8);
    }
    mbar_init(oend, 1);
    mbar_init(ofree, kDtSoftWarps);
    mbar_init(xsync, kDtSoftWarps);
    for (int i = 0; i < 8; ++i) mbar_init(&psync[i], 2);
    fence_barrier_init();
  }
  if (t < 65) bad[t] = 0;
  if (warp == kDtSoftWarps + 1 && lane == 0) {
    prefetch_tensormap(&tmq);
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
  }
  if (warp == 0) tc::tmem_alloc(tmem_base, 512);
  pdl_wait();
  pdl_launch_dependents();
  int4 d0;
  const int n = plan_cta_stages<kDtThreads, kDraftKeys>(a, reinterpret_cast<long long*>(exch), &d0);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_base;  // S_0, S_1 at columns 0, 128; O_0, O_1 at 256, 384

  if (n <= 0) {
    // nothing to do: only the TMEM to give back
  } else if (warp == kDtSoftWarps + 1) {
    // ============================================================ producer
    const int TB = draft_tc_box_rows(P);  // rows per box
    const int j = lane;                   // this lane's box
    int r = d0.x, h = d0.y, i = d0.z;
    DraftSeq s = draft_seq(a, r, false);
    auto stages = [&]() { return s.n > 0 ? (s.ctx + s.n + kDraftKeys - 1) / kDraftKeys : 0; };
    int nt = stages();
    auto next_segment = [&]() {
      i = 0;
      if (++h == plan_heads(a)) {
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
    auto box_block = [&](int r_, int i_, int len_) -> int {
      const int row = i_ * kDraftKeys + j * TB;
      return row < len_ && j * TB < kDraftKeys
                 ? __ldg(a.block_tables + (int64_t)r_ * a.max_blocks + row / P)
                 : 0;
    };
    int item = 0, pieces = 0, jobs = 0;
    bool q_wanted = false;  // a piece's Q is still to be loaded
    int q_row = 0, q_head = 0, q_two = 0;
    bool ok = true;
    // lane 0: issue the wanted Q once the previous piece's QKs have read theirs
    auto try_q = [&](bool wait) -> bool {
      if (!q_wanted) return true;
      if (pieces > 1 && !(wait ? mbar_wait(qfree, (pieces - 2) & 1) : mbar_try_wait(qfree, (pieces - 2) & 1)))
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
    // all lanes: wait until the next ring slot may be written
    int slot = 0;
    uint32_t round = 0;
    auto wait_slot = [&]() -> bool {
      int good = 1;
      if (lane == 0) {
        try_q(false);
        if (round > 0 && !mbar_try_wait(&freeb[slot], (round - 1) & 1)) {
          const uint64_t t0 = global_timer_ns();
          good = 0;
          do {
            for (int i_ = 0; i_ < 64 && !good; ++i_) {
              try_q(false);
              good = mbar_try_wait(&freeb[slot], (round - 1) & 1);
            }
          } while (!good && global_timer_ns() - t0 <= kWaitLimitNs);
        }
      }
      return __shfl_sync(0xffffffffu, good, 0) != 0;
    };
    struct Boxes {
      int group, n, head;  // first row group, boxes, kv head
    };
    auto load = [&](const CUtensorMap* tm, const Boxes& x) -> bool {
      if (!wait_slot()) return false;
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
    int blk_next = box_block(r, i, s.ctx + s.n);
    for (int k = 0; k < n;) {
      const int rows_all = s.n * G;
      const int mt = a.row_tiles > 1 ? h % a.row_tiles : 0;
      const int rows = min(rows_all - mt * kRecRows, kRecRows);
      const int len = s.ctx + s.n;
      if (rows <= 0) {  // the sequence has no rows in this tile: pass its stages over
        k += nt - i;
        if (k >= n) break;
        next_segment();
        blk_next = box_block(r, i, s.ctx + s.n);
        continue;
      }
      const int kvh = a.row_tiles > 1 ? h / a.row_tiles : h;
      const int t0 = i * kDraftKeys, nvalid = min(kDraftKeys, len - t0);
      const int dseg = k - i;  // the CTA's stage that starts the segment
      const bool start = k == 0 || i == 0, end = k == n - 1 || i == nt - 1;
      const bool pair = kTiles > 1 && rows > kDraftRows;
      const bool tail = t0 + nvalid > s.ctx;
      const int flags = (start ? kDtStart : 0) | (end ? kDtEnd : 0) |
                        (end && i == nt - 1 && dseg >= 0 ? kDtWhole : 0) | (dseg > 0 ? kDtSlot1 : 0) |
                        (pair ? kDtPair : 0) | (tail ? kDtTail : 0) | ((jobs & 1) ? kDtOdd : 0) |
                        (s.n << kDtDraftShift);
      const int row0 = s.row0 + mt * (kRecRows / G);
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
      if (j < b.n && (blk_next < 0 || (int64_t)blk_next >= a.num_blocks)) {
        atomicOr(a.err, PKV_DEVERR_BLOCK);
        b.group = (int)a.num_blocks * (P / kRowGroup);  // zero-filled out-of-range box
      } else {
        b.group = blk_next * (P / kRowGroup) + (t0 + j * TB) % P / kRowGroup;
      }
      if (lane == 0) {
        DtDesc* d = &descs[emitted % kDtDescs];
        d->a = make_int4(r, h, nvalid, flags);
        d->b = make_int4(s.ctx - t0, row0, rows, pieces);
        mbar_arrive(&dfull[emitted % kDtDescs]);
      }
      if (!load(&tmk, b) || !load(&tmv, b)) {
        ok = false;
        break;
      }
      ++emitted;
      jobs += pair ? 2 : 1;
      ++k;
      if (k < n) {
        if (++i == nt) next_segment();
        blk_next = box_block(r, i, s.ctx + s.n);
      }
    }
    if (lane == 0) {
      if (ok) ok = try_q(true);
      if (ok) {
        descs[emitted % kDtDescs].a = make_int4(0, 0, 0, kDtDone);
        mbar_arrive(&dfull[emitted % kDtDescs]);
      } else {
        atomicOr(a.err, PKV_DEVERR_TIMEOUT);
        // copies may still be in flight into the ring and Q: wait for them
        for (int it = item > kItems ? item - kItems : 0; it < item; ++it)
          mbar_wait(&full[it % kItems], (it / kItems) & 1);
        if (pieces > 0 && !q_wanted) mbar_wait(qfull, (pieces - 1) & 1);
      }
    }
  } else if (warp == kDtSoftWarps) {
    // ============================================================ MMA issue
    if (lane == 0) {
      const uint32_t idqk = tc::idesc_bf16_f32(kDraftRows, kDraftKeys, 0, 0) |
                            (a.qscale < 0.f ? tc::kIdescNegateA : 0u);
      constexpr uint32_t kIdPV = tc::idesc_bf16_f32(kDraftRows, D, 0, 1);
      // Jobs alternate between the groups: job j is group j & 1's.  What a PV
      // needs of its job is kept for the two jobs at most between their QK and
      // their PV, in registers: its V's ring slot and phase, and the flags.
      constexpr int kFirst = 1, kPieceFirst = 2, kPieceLast = 4, kFrees = 8;
      uint32_t info0 = 0, info1 = 0;  // flags, phase << 4, slot << 5
      int jn = 0, pv = 0, pieces = 0, pieces_done = 0;  // QKs and PVs issued, pieces begun and finished
      uint32_t fresh = 3;             // bit x: no job of group x in this piece yet
      // descriptors differ in their address field alone
      const uint64_t kdesc = tc::smem_desc_sw128(smem_u32(ring), 16, kGroupBytes);
      const uint64_t vdesc = tc::smem_desc_sw128(smem_u32(ring), 1024, kGroupBytes);
      const uint64_t qdesc = tc::smem_desc_sw128(smem_u32(qs), 16, 1024);
      auto issue_pv = [&]() -> bool {  // of job pv
        const int x = pv & 1;
        const uint32_t q = x ? info1 : info0;
        const uint32_t sl = q >> 5;
        if (!mbar_wait(&pfull[x], (pv >> 1) & 1) || !mbar_wait(&full[sl], (q >> 4) & 1)) return false;
        if ((q & kPieceFirst) && pieces_done > 0 && !mbar_wait(ofree, (pieces_done - 1) & 1)) return false;
        tc::fence_after_sync();
        const uint64_t vd = vdesc + sl * (L::kTile >> 4);
        const uint32_t tO = tmem + 256 + x * 128, tP = tmem + x * 128;
#pragma unroll
        for (int k = 0; k < kDraftKeys / 16; ++k)
          tc::mma_bf16_ta(tO, tP + (k >> 1) * 32 + (k & 1) * 8, vd + ((k * 2 * kGroupBytes) >> 4), kIdPV,
                          (k > 0 || !(q & kFirst)) ? 1u : 0u);
        if (q & kFrees) tc::commit(&freeb[sl]);
        if (q & kPieceLast) {
          tc::commit(oend);
          ++pieces_done;
        }
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
        if (pv + 1 < jn && !(ok = issue_pv())) break;
        if (!(ok = mbar_wait(&dfull[e % kDtDescs], (e / kDtDescs) & 1))) break;
        const int fl = descs[e % kDtDescs].a.w;
        if (fl & kDtDone) break;
        if (fl & kDtStart) {
          fresh = 3;
          if (!(ok = mbar_wait(qfull, pieces & 1))) break;
          ++pieces;
        }
        const uint32_t ksl = slot;
        if (!(ok = mbar_wait(&full[ksl], phase))) break;
        advance();
        const uint32_t vinfo = (slot << 5) | (phase << 4);
        advance();
        const int uses = (kTiles > 1 && (fl & kDtPair)) ? 2 : 1;
        for (int u = 0; u < uses; ++u) {
          if (pv + 1 < jn && !(ok = issue_pv())) break;
          const int x = jn & 1;
          tc::fence_after_sync();
          const uint64_t kd = kdesc + ksl * (L::kTile >> 4), qd = qdesc + u * (L::kTile >> 4);
          const uint32_t tS = tmem + x * 128;
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc::mma_bf16(tS, qd + (((k >> 2) * L::kHalf + (k & 3) * 32) >> 4),
                         kd + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), idqk, k > 0 ? 1u : 0u);
          tc::commit(&sfull[x]);
          const bool last = u == uses - 1;
          if (last) {
            tc::commit(&freeb[ksl]);
            if (fl & kDtEnd) tc::commit(qfree);
          }
          const uint32_t q = vinfo | ((fresh >> x) & 1u ? kFirst : 0) |
                             ((fl & kDtStart) && u == 0 ? kPieceFirst : 0) |
                             ((fl & kDtEnd) && last ? kPieceLast : 0) | (last ? kFrees : 0);
          if (x) info1 = q;
          else info0 = q;
          fresh &= ~(1u << x);
          ++jn;
        }
      }
      while (ok && pv < jn) ok = issue_pv();
      if (!ok) atomicOr(a.err, PKV_DEVERR_TIMEOUT);
    }
  } else {
    // ============================================================ softmax
    const int x = warp >> 3, half = (warp >> 2) & 1;
    const int row = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    // this thread's 64 columns of S; the weights of each 32 overlay their first 16
    const uint32_t tS = tmem + x * 128 + half * 64 + lane_base;
    float* mine = exch + (warp >> 2) * kDraftRows + row;
    const float* other = exch + ((warp >> 2) ^ 1) * kDraftRows + row;
    uint64_t* pair_bar = &psync[(warp >> 3) * 4 + (warp & 3)];
    // the sign of the scale is in the QK; 1e-37 keeps a hidden score -inf
    // where the scale is 0
    const float cs = fmaxf(fabsf(a.qscale), 1e-37f);
    float m = -INFINITY, l = 0.f;
    uint64_t mask = 0;
    bool live = false, warp_live = false;
    bool fresh = true, newpiece = true;  // no job of this group in the piece yet
    int rowg = 0, jobs = 0, syncs = 0, meets = 0;
    bool ok = true;
    auto wait = [&](uint64_t* b, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(b, parity));
    };
    // the two warps of the same rows: what they wrote before is read after
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(pair_bar);
      return wait(pair_bar, meets++ & 1);
    };
    for (int e = 0;; ++e) {
      if (!(ok = wait(&dfull[e % kDtDescs], (e / kDtDescs) & 1))) break;
      const int4 da = descs[e % kDtDescs].a, db = descs[e % kDtDescs].b;
      const int fl = da.w;
      if (fl & kDtDone) break;
      const bool pair = kTiles > 1 && (fl & kDtPair);
      const int first_group = (fl & kDtOdd) ? 1 : 0;  // of the stage's first job
      const int nvalid = da.z, mb = db.x;
      if (fl & kDtStart) {
        m = -INFINITY;
        l = 0.f;
        fresh = newpiece = true;
        rowg = (pair ? x ^ first_group : 0) * kDraftRows + row;
        live = rowg < db.z;
        warp_live = __any_sync(0xffffffffu, live);
        DraftSeq s;
        s.n = fl >> kDtDraftShift;
        const int tok0 = a.row_tiles > 1 ? (da.y % a.row_tiles) * (kRecRows / G) : 0;
        s.row0 = db.y - tok0;
        mask = live ? draft_mask(a, s, tok0 + rowg / G) : 0ull;
      }
      if (pair || x == first_group) {
        if (!(ok = wait(&sfull[x], jobs & 1))) break;
        ++jobs;
        tc::fence_after_sync();
        if (warp_live) {
          // 32 columns at a time (all 64 in registers would spill): both for
          // the maximum, then the second's weights, then the first's, read again
          uint32_t v[32];
          auto hide = [&](int w) {
            if (!(fl & kDtTail)) return;
            const uint32_t bits = mask_word(mask, mb, 2 * half + w);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((bits >> i) & 1u)) v[i] = __float_as_uint(-INFINITY);
          };
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            tc::tmem_ld32(tS + 32 * w, v);
            tc::wait_ld32(v);
            hide(w);
#pragma unroll
            for (int i = 0; i < 32; ++i) mx4[i & 3] = fmaxf(mx4[i & 3], __uint_as_float(v[i]));
          }
          float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
          // the exchange slots were last read at the previous piece's end
          if (newpiece && db.w > 1 && !(ok = wait(ofree, (db.w - 2) & 1))) break;
          *mine = mx;
          if (!(ok = meet())) break;
          mx = cs * fmaxf(mx, *other);
          const float m_new = fmaxf(m, mx);
          const bool need = live && m_new > m + 8.0f;
          const float alpha = need ? exp2f(m - m_new) : 1.f;
          if (need) m = m_new;
          const float nm = m == -INFINITY ? 0.f : -m;  // nothing seen yet: every weight is 0
          // ---- P = exp2(c s - m) in bf16 pairs; the sums take it unrounded
          float2 ls2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int w = 1; w >= 0; --w) {
            if (w == 0) {
              tc::tmem_ld32(tS, v);
              tc::wait_ld32(v);
              hide(0);
            }
            uint32_t pw[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float p0 = exp2f(fmaf(__uint_as_float(v[2 * i]), cs, nm));
              const float p1 = exp2f(fmaf(__uint_as_float(v[2 * i + 1]), cs, nm));
              ls2[i & 1] = __fadd2_rn(ls2[i & 1], make_float2(p0, p1));
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(p0, p1);
              pw[i] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            tc::tmem_st16(tS + 32 * w, pw);
          }
          const float2 ls = __fadd2_rn(ls2[0], ls2[1]);
          l = l * alpha + (ls.x + ls.y);
          // O holds every PV of this group but this job's: its S was computed
          // after them.  The row's two threads rescale half of it each.
          if (!fresh && __any_sync(0xffffffffu, need)) {
            const uint32_t tO = tmem + 256 + x * 128 + half * (D / 2) + lane_base;
#pragma unroll 1
            for (int c0 = 0; c0 < D / 2; c0 += 16) {
              uint32_t o[16];
              tc::tmem_ld16(tO + c0, o);
              tc::wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tc::tmem_st16(tO + c0, o);
            }
          }
          tc::wait_st();
        }
        fresh = newpiece = false;
        // The stage's first job clears what the PVs must not multiply: V rows
        // past the last one (weight 0, any bytes), and non-finite elements of
        // drafted rows, which some row may not see.
        if ((fl & kDtTail) && x == first_group) {
          const int vitem = 2 * e + 1;  // K and V of a stage are ring items 2 e and 2 e + 1
          if (!(ok = wait(&full[vitem % kItems], (vitem / kItems) & 1))) break;
          if (row >= mb) {
            unsigned char* vr = ring + (size_t)(vitem % kItems) * L::kTile + (row / kRowGroup) * kGroupBytes +
                                (row % kRowGroup) * 128;
            bool found = false;
            if (half < H) {  // 64 columns a thread
#pragma unroll 2
              for (int ch = 0; ch < 8; ++ch) {
                uint4* at = reinterpret_cast<uint4*>(vr + half * 1024 + ch * 16);
                if (row >= nvalid) {
                  *at = make_uint4(0u, 0u, 0u, 0u);
                  continue;
                }
                uint4 w = *at;
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
            }
            if (found) {
              bad[1 + row - mb] = db.w;
              bad[0] = db.w;
            }
          }
          tc::fence_proxy_async_smem();
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[x]);
      }
      if (fl & kDtEnd) {
        // ---- a piece's end: O / l and the LSE of each row
        if (!(ok = wait(oend, (db.w - 1) & 1))) break;
        tc::fence_after_sync();
        float M = m, Ls = l, f0 = 1.f, f1 = 1.f;
        bool has0 = x == 0, has1 = x == 1;  // accumulators that hold this row's outputs
        if (warp_live) {
          // the row's sum: its two threads'
          *mine = l;
          if (!(ok = meet())) break;
          Ls = half == 0 ? l + *other : *other + l;
          if (!pair) {  // then the groups' states: (m, sum) of each
            if (!(ok = meet())) break;
            *mine = half == 0 ? m : Ls;
          }
        }
        if (!pair || (fl & kDtTail)) {  // the groups' states, and `bad`
          __syncwarp();
          if (lane == 0) mbar_arrive(xsync);
          if (!(ok = wait(xsync, syncs & 1))) break;
          ++syncs;
        }
        if (warp_live) {
          if (!pair) {
            const float mo = exch[2 * (x ^ 1) * kDraftRows + row], lo = exch[(2 * (x ^ 1) + 1) * kDraftRows + row];
            const float m0 = x == 0 ? m : mo, m1 = x == 0 ? mo : m, l0 = x == 0 ? Ls : lo, l1 = x == 0 ? lo : Ls;
            M = fmaxf(m0, m1);
            const float base = M == -INFINITY ? 0.f : M;
            f0 = exp2f(m0 - base);
            f1 = exp2f(m1 - base);
            Ls = f0 * l0 + f1 * l1;
            // a group without a job in the piece (one stage), or without a
            // seen key, has nothing in its O
            has0 = l0 != 0.f;
            has1 = l1 != 0.f;
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
          if (live && half == 0 && (pair || x == 0)) {
            if (!whole) a.rec_lse[rec] = lse2;
            else if (a.lse_out) a.lse_out[qh] = lse2 * kDtLn2;
          }
          const bool fix = bad[0] == db.w;
          // columns: half of them each in a pair, a quarter otherwise, 16 at a time
          const int span = pair ? D / 2 : D / 4;
          const int c_lo = pair ? half * (D / 2) : (x * 2 + half) * (D / 4);
#pragma unroll 1
          for (int c0 = c_lo; c0 < c_lo + span; c0 += 16) {
            float o[16];
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = 0.f;
            if (!pair || x == 0) {
              tc::tmem_ld16(tmem + 256 + lane_base + c0, w);
              tc::wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (has0) o[i] = __uint_as_float(w[i]) * f0;
            }
            if (!pair || x == 1) {
              tc::tmem_ld16(tmem + 384 + lane_base + c0, w);
              tc::wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (has1) o[i] = fmaf(__uint_as_float(w[i]), f1, o[i]);
            }
            if (fix && live) {  // non-finite elements that this row does see
              for (uint64_t left = mask; left; left &= left - 1) {
                const int jd = __ffsll((long long)left) - 1;
                if (bad[1 + jd] != db.w) continue;
                const int pos = __ldg(a.ctx_lens + da.x) + jd;
                const int blk = __ldg(a.block_tables + (int64_t)da.x * a.max_blocks + pos / P);
                if (blk < 0 || (int64_t)blk >= a.num_blocks) continue;
                const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(a.v) +
                                          (((int64_t)blk * P + pos % P) * Hkv + kvh) * D + c0;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const uint32_t u = __bfloat16_as_ushort(vp[i]);
                  if ((u & 0x7f80u) == 0x7f80u) o[i] += __uint_as_float(u << 16);
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
                float4* dst = reinterpret_cast<float4*>(a.rec_o + rec * D + c0);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
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

// One warp per (sequence, drafted row, query head): merge the pieces of its
// segment by log-sum-exp.  A segment that one CTA covered whole is done.
template <int D, int kTiles>
__global__ void __launch_bounds__(128) draft_tc_reduce_kernel(const DraftArgs a) {
  constexpr int EPL = D / 32;
  constexpr int kRecRows = kTiles * kDraftRows;
  constexpr int kBatch = 4;  // piece outputs loaded at once
  pdl_wait();  // the records and the plan are complete
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.y;
  const int w = blockIdx.x * 4 + warp;
  const DraftSeq s = draft_seq(a, r, false);
  if (w >= s.n * a.num_q_heads) return;
  const int tok = w / a.num_q_heads, qh = w % a.num_q_heads;
  const int G = a.num_q_heads / a.num_kv_heads, g = qh % G;
  const int rowg = tok * G + g, mt = rowg / kRecRows;
  const int heads = plan_heads(a), h = (qh / G) * a.row_tiles + mt;
  const long long su = a.stage_units, pu = a.piece_units;
  const long long S = a.plan_pre[a.num_seqs] * heads;
  const long long pre = a.plan_pre[r], u = a.plan_pre[r + 1] - pre;
  const long long nt = (u - pu) / su;
  const long long cw = units_per_cta(S, a.num_ctas, su);
  const long long seg0 = pre * heads + (long long)h * u;
  const int c_first = (int)((seg0 + pu) / cw), c_last = (int)((seg0 + pu + su * (nt - 1)) / cw);
  if (c_first == c_last) return;
  // a first piece is in slot 1 of its CTA when that CTA owns an earlier stage
  const bool slot1 = seg0 > 0 && seg0 - su >= (long long)c_first * cw;
  const int np = c_last - c_first + 1;
  auto rec = [&](int i) -> int64_t {
    return (2 * (int64_t)(c_first + i) + (i == 0 && slot1 ? 1 : 0)) * kRecRows + rowg % kRecRows;
  };
  float M = -INFINITY;
  for (int i = lane; i < np; i += 32) M = fmaxf(M, a.rec_lse[rec(i)]);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float acc[EPL], Ls = 0.f;
#pragma unroll
  for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
  for (int i0 = 0; i0 < np; i0 += kBatch) {
    float ls[kBatch], f[kBatch][EPL];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      ls[i] = i0 + i < np ? a.rec_lse[rec(i0 + i)] : -INFINITY;
#pragma unroll
      for (int e = 0; e < EPL; ++e) f[i][e] = 0.f;
      if (ls[i] == -INFINITY) continue;  // an empty state
      const float* p = a.rec_o + rec(i0 + i) * D + lane * EPL;
      if constexpr (EPL == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        f[i][0] = x.x, f[i][1] = x.y, f[i][2] = x.z, f[i][3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(p);
        f[i][0] = x.x, f[i][1] = x.y;
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (ls[i] == -INFINITY) continue;
      const float wt = exp2f(ls[i] - M);
      Ls += wt;
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] = fmaf(wt, f[i][e], acc[e]);
    }
  }
  const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
  const int64_t row = (int64_t)(s.row0 + tok) * a.num_q_heads + qh;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * D + lane * EPL;
  uint32_t o2[EPL / 2];
#pragma unroll
  for (int e = 0; e < EPL / 2; ++e) {
    const __nv_bfloat162 b2 = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    o2[e] = *reinterpret_cast<const uint32_t*>(&b2);
  }
  if constexpr (EPL == 4) *reinterpret_cast<uint2*>(out) = make_uint2(o2[0], o2[1]);
  else *reinterpret_cast<uint32_t*>(out) = o2[0];
  if (lane == 0 && a.lse_out) a.lse_out[row] = Ls == 0.f ? -INFINITY : (M + log2f(Ls)) * kDtLn2;
}

template <int D, int kTiles>
static cudaError_t launch_draft_tc_t(const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
                                     const DraftArgs& a, cudaStream_t stream) {
  constexpr int smem = DtSmem<D, kTiles>::total;
  auto kern = draft_tc_kernel<D, kTiles>;
  static SmemAttrCache attr_cache;
  cudaError_t e = ensure_smem_limit(kern, smem, attr_cache);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3((unsigned)a.num_ctas), dim3(kDtThreads), smem, stream, tmq, tmk, tmv, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(draft_tc_reduce_kernel<D, kTiles>,
                    dim3((unsigned)((a.max_draft * a.num_q_heads + 3) / 4), (unsigned)a.num_seqs), dim3(128), 0,
                    stream, a);
}

cudaError_t launch_draft_tc(int head_dim, int tiles, const CUtensorMap& tmq, const CUtensorMap& tmk,
                            const CUtensorMap& tmv, const DraftArgs& a, cudaStream_t stream) {
  if (head_dim == 128)
    return tiles > 1 ? launch_draft_tc_t<128, 2>(tmq, tmk, tmv, a, stream)
                     : launch_draft_tc_t<128, 1>(tmq, tmk, tmv, a, stream);
  return tiles > 1 ? launch_draft_tc_t<64, 2>(tmq, tmk, tmv, a, stream)
                   : launch_draft_tc_t<64, 1>(tmq, tmk, tmv, a, stream);
}

}  // namespace pkv
