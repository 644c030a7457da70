// Shared pieces of the fused attention kernels (attn_prefill_tc.cu and attn_scored_tc.cu): tile
// configuration, units of work, the TMA producers and the MMA issuer.  Not part of the C ABI.
#pragma once

#include "attn_common.cuh"
#include "attn_decode_warp.cuh"
#include "tc_ptx.cuh"

namespace rb {
namespace attn {
namespace {

template <int HD>
struct TcCfg {
  static constexpr int kM = 128;                          // query rows per tile (2 per unit)
  static constexpr int kN = 128;                          // keys per K/V tile
  static constexpr int kPagesPerTile = kN / kPage;        // 8
  static constexpr int kHalves = HD / 64;                 // 128-byte swizzle atoms per row
  static constexpr int kHalfBytes = kN * 128;             // one 64-dim half of a K or V tile
  static constexpr int kTileBytes = kHalves * kHalfBytes;
  static constexpr int kQHalfBytes = kM * 128;
  static constexpr int kQBytes = kHalves * kQHalfBytes;   // one Q tile
  // V tile j is read by the first block of step j, K tile j + 1 by the second half of it, and
  // both slots free at the same point (S of tile j - 1 landing): the deeper ring goes to V
  static constexpr int kStagesK = 2;
  static constexpr int kStagesV = 3;
  static constexpr int kVOffset = kStagesK * kTileBytes;
  static constexpr int kQOffset = kVOffset + kStagesV * kTileBytes;  // Q_A then Q_B
  static constexpr int kUsed = kQOffset + 2 * kQBytes;
  static_assert(8 * DecCfg<HD>::kStages * DecCfg<HD>::kStageBytes <= kUsed,
                "the decode phase's stages must fit in the prefill phase's shared memory");
  // at least 120 KB keeps one CTA per SM (each CTA holds all 512 TMEM columns)
  static constexpr int kSmemBytes = (kUsed + 1024) > 120 * 1024 ? (kUsed + 1024) : 120 * 1024;
  // 3 warpgroups launched at 168 registers per thread (the 64-bit-register pool of one SM for
  // 384 threads); the softmax warpgroups then take 216 and the producer/MMA warpgroup keeps 72:
  // 2 x 128 x 216 + 128 x 72 = 384 x 168.
  static constexpr int kThreads = 384;
  static constexpr int kLaunchRegs = 168;
  static constexpr int kSoftmaxRegs = 216;
  static constexpr int kControlRegs = 72;
  static_assert(2 * 128 * kSoftmaxRegs + 128 * kControlRegs <= kThreads * kLaunchRegs,
                "register split exceeds the launch allocation");
  static constexpr int kMmaWarp = 0;
  static constexpr int kProducerWarp = 1;   // units, Q and K
  static constexpr int kProducerVWarp = 2;  // V (warp 3 only completes the first warpgroup)
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS0 = 0;                   // S_A at 0, S_B at 128
  static constexpr uint32_t kColO0 = 256;                 // O_A at 256, O_B at 256 + HD
  static constexpr int kRing = 4;
  __device__ static constexpr uint32_t col_s(int x) { return kColS0 + 128u * x; }
  __device__ static constexpr uint32_t col_o(int x) { return kColO0 + static_cast<uint32_t>(HD) * x; }
};

// A unit of work: query tokens [tok0, tok0 + 2T) of the request's q (tile A the first T, tile
// B the next T), T = tile_tokens.  In a cascade prefix pass `r` holds the unit's prefix key
// range (the pages are row 0's), the tokens are the whole batch's, key indices are relative to
// the range's first key and no row is masked causally: every row sees keys [0, c].
struct TcUnit {
  int r, h, tok0, t0, q, L, c, n[2], n_kt, pages, valid;
};

// A unit of a scored call.  Its key tiles are [j0, j0 + n_kt) and both query tiles take all of
// them, last to first: with a bias that falls with distance, or with packed documents, a row's
// largest scores are in its last tiles, so its reference settles there, whereas first to last
// it would climb tile by tile (O rescaled each time).  Tile A takes at most one tile that only
// B's rows see.
struct ScoredUnit : TcUnit {
  int j0;         // first key tile
  int lo;         // first key any row sees (none: past the last page)
  int prefix;     // keys every row sees (from its own lo on)
  int lo_max[2];  // largest first key of each tile's rows (rows that see no key left out)
  int odd_first, odd_last;  // key tiles whose V held infinities or NaN that were taken out
};
template <bool kScored>
struct UnitOf {
  using type = TcUnit;
};
template <>
struct UnitOf<true> {
  using type = ScoredUnit;
};

// First page of a unit's keys and the page-table row they are read from.
__device__ __forceinline__ int unit_first_page(const AttnArgs& a, const TcUnit& un) {
  return a.cascade == kPrefixPass ? un.r * (a.prefix_split_keys / kPage) : 0;
}
__device__ __forceinline__ int unit_table_row(const AttnArgs& a, const TcUnit& un) {
  return a.cascade == kPrefixPass ? 0 : un.r;
}

template <bool kScored>
struct TcShared {
  uint64_t unit_full[4], unit_empty[4];
  uint64_t q_full, q_empty;
  uint64_t k_full[TcCfg<128>::kStagesK], k_empty[TcCfg<128>::kStagesK];
  uint64_t v_full[TcCfg<128>::kStagesV], v_empty[TcCfg<128>::kStagesV];
  uint64_t s_full[2], p_full[2], o_done[2], o_free[2];
  uint64_t drain;
  uint64_t dec_bars[8][DecCfg<128>::kStages];  // decode phase: one ring per warp 0..7
  typename UnitOf<kScored>::type units[4];
  uint32_t tmem_base;
  int abort;
  int decode_first;
  int role_rank;  // order in which this CTA took its role: decode-first CTAs are ranks 0..D-1
};

// Bounded wait (a.wait_limit_ns, 1 s unless a test shortened it) that also gives up as soon as
// another role has aborted.  `Relaxed`: for the MMA issuer (see mma_issuer).
template <bool Relaxed = false>
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t phase, volatile int* abort,
                                        const AttnArgs& a) {
  int32_t* err = a.err;
  auto test = [&]() { return Relaxed ? mbar_try_wait_relaxed(bar, phase) : mbar_try_wait(bar, phase); };
#pragma unroll 1
  for (int i = 0; i < 128; ++i)
    if (test()) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  while (true) {
    if (test()) return true;
    if (*abort) return false;
    if (global_timer_ns() - t0 > a.wait_limit_ns) {
      if (atomicExch(const_cast<int*>(abort), 1) == 0) raise_error(err, RB_EBIT_TIMEOUT);
      return false;
    }
  }
}

__device__ __forceinline__ int tiles_for(int c, int jmax) { return (c + jmax + 1 + 127) / 128; }
constexpr int kKeysPerTile = 128;  // keys per K/V tile

__device__ __forceinline__ TcUnit decode_unit(const AttnArgs& a, int u) {
  TcUnit un{};
  const int T = a.tile_tokens;
  if (a.cascade == kPrefixPass) {
    // (key range, kv head, 2T query tokens of the whole batch) against one range of the shared
    // keys [0, P) of row 0; key indices are relative to the range's first key
    const int per_split = a.nkv * ((a.N + 2 * T - 1) / (2 * T));
    const int split = u / per_split, rem = u - split * per_split;
    const int k0 = split * a.prefix_split_keys;
    const int k1 = min(a.prefix_len, k0 + a.prefix_split_keys);
    un.r = split;
    un.h = rem % a.nkv;
    un.tok0 = (rem / a.nkv) * 2 * T;
    un.t0 = 0;
    un.q = a.N;
    un.L = k1 - k0;
    un.c = un.L - 1;
    const int nk = (un.L + kKeysPerTile - 1) / kKeysPerTile;
    un.n[0] = nk;
    un.n[1] = un.tok0 + T < un.q ? nk : 0;
    un.n_kt = nk;
    un.pages = (un.L + kPage - 1) / kPage;
    un.valid = 1;
    return un;
  }
  // the planner lists the (request, pair) entries longest first; the kv heads of one entry
  // are consecutive units
  // (a plain load: a scored launch is resident while the planner still writes the list)
  const int entry = a.pre_list[u / a.nkv];
  const int r = entry >> 16, pair = entry & 0xffff;
  un.r = r;
  un.h = u % a.nkv;
  un.t0 = a.qsl[r];
  un.q = a.qsl[r + 1] - un.t0;
  un.L = a.seq_lens[r];
  un.c = un.L - un.q;
  un.tok0 = pair * 2 * T;
  un.n[0] = tiles_for(un.c, min(un.tok0 + T, un.q) - 1);
  un.n[1] = un.tok0 + T < un.q ? tiles_for(un.c, min(un.tok0 + 2 * T, un.q) - 1) : 0;
  un.n_kt = max(un.n[0], un.n[1]);
  un.pages = (un.L + kPage - 1) / kPage;
  un.valid = 1;
  return un;
}

// Page ids of a unit's K/V tiles for one warp: a 32-page window of the unit's block-table row
// held one id per lane, the next window prefetched; lane l & 7 takes page l & 7 of a tile.
struct PageWindow {
  const AttnArgs& a;
  const int32_t* bt_row;
  int page0, pages, win, bid, bid_next, lane;
  __device__ PageWindow(const AttnArgs& a_, const TcUnit& un, int lane_)
      : a(a_),
        bt_row(a_.block_table + static_cast<size_t>(unit_table_row(a_, un)) * a_.MB),
        page0(unit_first_page(a_, un)),
        pages(un.pages),
        win(0),
        lane(lane_) {
    bid = page(lane);
    bid_next = page(32 + lane);
  }
  __device__ int page(int pg) const {
    return pg < pages ? kernel_page(bt_row, page0 + pg, a.ratio, a.num_blocks, a.null_block)
                      : a.null_block;
  }
  // This lane's page id for tile j (tiles are taken in order).  Pages past the sequence read
  // the null page (masked; V rows zeroed); an invalid id is reported when `report` and replaced
  // by the null page.
  __device__ int tile_page(int j, bool report) {
    const int first = j * kKeysPerTile / kPage;
    if (first - win >= 32) {
      win += 32;
      bid = bid_next;
      bid_next = page(win + 32 + lane);
    }
    int id = __shfl_sync(0xffffffffu, bid, first + (lane & 7) - win);
    const int pg = first + (lane & 7);
    if (pg >= pages) {
      id = a.null_block;
    } else if (id < 0 || id >= a.num_blocks || id == a.null_block) {
      if (report && lane < kKeysPerTile / kPage) raise_error(a.err, RB_EBIT_BLOCK_ID);
      id = a.null_block;
    }
    return id;
  }
};

// A scored unit, by a whole warp: the ordinary unit's rows, and its tokens' key ranges.
__device__ __forceinline__ ScoredUnit scored_unit(const AttnArgs& a, int u, int lane) {
  ScoredUnit un{};
  static_cast<TcUnit&>(un) = decode_unit(a, u);
  const int T = a.tile_tokens;
  un.prefix = key_prefix(a, un.r, un.L);
  int lo = un.pages * kPage;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    int mn = 0x7fffffff, mx = 0;
    if (a.key_start == nullptr) {
      mn = 0;
    } else {
      const int end = min(un.tok0 + (x + 1) * T, un.q);
      for (int j = un.tok0 + x * T + lane; j < end; j += 32) {
        const int k = key_lo(a, un.t0 + j);
        if (k >= max(un.c + j + 1, un.prefix)) continue;
        mn = min(mn, k);
        mx = max(mx, k);
      }
      mn = __reduce_min_sync(0xffffffffu, mn);
      mx = __reduce_max_sync(0xffffffffu, mx);
    }
    un.lo_max[x] = mx;
    lo = min(lo, mn);
  }
  un.lo = lo;
  un.odd_first = 0x7fffffff;
  un.odd_last = -1;
  const int last_tok = min(un.tok0 + 2 * T, un.q) - 1;
  const int n = (max(un.c + last_tok + 1, un.prefix) + kKeysPerTile - 1) / kKeysPerTile;
  un.j0 = min(lo / kKeysPerTile, n - 1);  // at least one tile, also when no row sees a key
  un.n_kt = n - un.j0;
  un.n[0] = un.n_kt;
  un.n[1] = un.tok0 + T < un.q ? un.n_kt : 0;
  return un;
}

// Page ids of a scored unit's K/V tiles for one warp, last tile first: lane l & 7 holds page
// l & 7 of the next two tiles.  Pages before the first visible key (which may be gone from the
// page table) and past the sequence are the null page; their V rows are zeroed.
struct ScoredPages {
  const AttnArgs& a;
  const int32_t* bt_row;
  int first, pages, j0, last, lane, next0, next1;
  __device__ ScoredPages(const AttnArgs& a_, const ScoredUnit& un, int lane_)
      : a(a_),
        bt_row(a_.block_table + static_cast<size_t>(un.r) * a_.MB),
        first(un.lo / kPage),
        pages(un.pages),
        j0(un.j0),
        last(un.j0 + un.n_kt - 1),
        lane(lane_) {
    next0 = page(last);
    next1 = page(last - 1);
  }
  __device__ int page(int tile) const {
    const int pg = tile * (kKeysPerTile / kPage) + (lane & 7);
    return tile >= j0 && pg >= first && pg < pages
               ? kernel_page(bt_row, pg, a.ratio, a.num_blocks, a.null_block)
               : a.null_block;
  }
  __device__ int tile_page(int j, bool report) {  // j-th tile taken
    int id = next0;
    next0 = next1;
    next1 = page(last - j - 2);
    if (id < 0) {
      if (report && lane < kKeysPerTile / kPage) raise_error(a.err, RB_EBIT_BLOCK_ID);
      id = a.null_block;
    }
    return id;
  }
};
template <bool kScored>
struct PagesOf {
  using type = PageWindow;
};
template <>
struct PagesOf<true> {
  using type = ScoredPages;
};

// Producer of units, Q and K (warp 1, whole warp).  It takes units from the global counter
// into the 4-entry unit ring, loads Q_A and Q_B once per unit and each K tile into the K
// ring; lanes 0..7 each issue the boxes of one page of a tile.
template <int HD, bool kScored>
__device__ void producer_qk(const AttnArgs& a, TcShared<kScored>& sh, uint32_t smem_base,
                            const CUtensorMap* qmap, const CUtensorMap* kmap) {
  using C = TcCfg<HD>;
  volatile int* abort = &sh.abort;
  const int lane = threadIdx.x & 31;
  const int n_units = a.header[kHNumPrefillUnits];
  uint32_t it = 0, q_armed = 0, k_armed[C::kStagesK] = {};
  // the unit ring guards plain shared memory (the unit descriptors): acquiring wait
  auto lane0_wait = [&](uint64_t* bar, uint32_t phase) -> bool {
    int ok = 1;
    if (lane == 0) ok = tc_wait(bar, phase, abort, a) ? 1 : 0;
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
  };
  // Q and K slots are read only by tcgen05.mma and written only by TMA: a relaxed test first
  // (an acquiring wait on a long-complete phase cost this warp a few hundred cycles per tile)
  auto slot_wait = [&](uint64_t* bar, uint32_t phase) -> bool {
    int ok = 1;
    if (lane == 0)
      ok = (mbar_test_relaxed(bar, phase) || tc_wait<true>(bar, phase, abort, a)) ? 1 : 0;
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
  };
  for (int k = 0;; ++k) {
    const int slot = k % C::kRing;
    if (!lane0_wait(&sh.unit_empty[slot], ((k / C::kRing) & 1) ^ 1)) break;
    int withhold = 0;
    typename UnitOf<kScored>::type fetched{};
    if constexpr (kScored) {
      int u = 0;
      if (lane == 0) u = atomicAdd(a.header + kHPrefillNext, 1);
      u = __shfl_sync(0xffffffffu, u, 0);
      if (u < n_units) fetched = scored_unit(a, u, lane);
    }
    if (lane == 0) {
      if constexpr (!kScored) {
        const int u = atomicAdd(a.header + kHPrefillNext, 1);
        if (u < n_units) fetched = decode_unit(a, u);
      }
      const auto& un = fetched;
      sh.units[slot] = un;
      // test hook: CTA 0 stops before its first unit reaches the other roles, so their waits
      // for it run out while nothing of that unit has been issued
      withhold = a.withhold_first_unit && blockIdx.x == 0 && k == 0 && un.valid;
      if (!withhold) tc::mbar_arrive(&sh.unit_full[slot]);
    }
    if (__shfl_sync(0xffffffffu, withhold, 0)) break;
    __syncwarp();
    const typename UnitOf<kScored>::type un = sh.units[slot];
    if (!un.valid) break;
    if (!slot_wait(&sh.q_empty, (k & 1) ^ 1)) break;
    if (lane == 0) {
      // one box per 64-dim half of a tile: T tokens x group heads = T * group rows of 128 bytes
      const int nq = un.n[1] > 0 ? 2 : 1;
      mbar_arrive_expect_tx(&sh.q_full, nq * C::kHalves * a.tile_tokens * a.group * 128);
      ++q_armed;
      for (int x = 0; x < nq; ++x)
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_3d(smem_base + C::kQOffset + x * C::kQBytes + hf * C::kQHalfBytes, qmap,
                      &sh.q_full, hf * 64, un.h * a.group, un.t0 + un.tok0 + a.tile_tokens * x);
    }
    typename PagesOf<kScored>::type pw(a, un, lane);
    bool ok = true;
    for (int j = 0; j < un.n_kt; ++j) {
      const int id = pw.tile_page(j, true);
      const uint32_t itk = it + j, st = itk % C::kStagesK;
      if (!slot_wait(&sh.k_empty[st], ((itk / C::kStagesK) & 1) ^ 1)) { ok = false; break; }
      if (lane == 0) {
        mbar_arrive_expect_tx(&sh.k_full[st], C::kTileBytes);
        ++k_armed[st];
      }
      __syncwarp();
      if (lane < C::kPagesPerTile) {
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_3d(smem_base + st * C::kTileBytes + hf * C::kHalfBytes + lane * (kPage * 128),
                      kmap, &sh.k_full[st], hf * 64, un.h, id * kPage);
      }
    }
    if (!ok) break;
    it += un.n_kt;
  }
  if (lane == 0 && *abort) {  // let every copy already issued land before the CTA can exit
    if (q_armed) mbar_wait_bounded(&sh.q_full, (q_armed - 1) & 1, 100000000ull);
    for (int b = 0; b < C::kStagesK; ++b)
      if (k_armed[b]) mbar_wait_bounded(&sh.k_full[b], (k_armed[b] - 1) & 1, 100000000ull);
  }
}

// Producer of V (warp 2, whole warp): follows the unit ring like the other consumers and loads
// each V tile into the V ring.  A warp of its own, so that V tiles are issued as soon as their
// slot frees, not after the next K tile (one warp issuing both took about a whole key-tile step
// for the TMA issue and waits alone, and left V late).
template <int HD, bool kScored>
__device__ void producer_v(const AttnArgs& a, TcShared<kScored>& sh, uint32_t smem_base,
                           const CUtensorMap* vmap) {
  using C = TcCfg<HD>;
  volatile int* abort = &sh.abort;
  const int lane = threadIdx.x & 31;
  uint32_t it = 0, v_armed[C::kStagesV] = {};
  auto lane0_wait = [&](uint64_t* bar, uint32_t phase) -> bool {
    int ok = 1;
    if (lane == 0) ok = tc_wait(bar, phase, abort, a) ? 1 : 0;
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
  };
  auto slot_wait = [&](uint64_t* bar, uint32_t phase) -> bool {
    int ok = 1;
    if (lane == 0)
      ok = (mbar_test_relaxed(bar, phase) || tc_wait<true>(bar, phase, abort, a)) ? 1 : 0;
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
  };
  for (int k = 0;; ++k) {
    const int slot = k % C::kRing;
    if (!lane0_wait(&sh.unit_full[slot], (k / C::kRing) & 1)) break;
    const typename UnitOf<kScored>::type un = sh.units[slot];
    if (!un.valid) break;
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sh.unit_empty[slot]);  // the descriptor is in registers
    typename PagesOf<kScored>::type pw(a, un, lane);
    bool ok = true;
    for (int j = 0; j < un.n_kt; ++j) {
      const int id = pw.tile_page(j, false);
      const uint32_t itv = it + j, st = itv % C::kStagesV;
      if (!slot_wait(&sh.v_empty[st], ((itv / C::kStagesV) & 1) ^ 1)) { ok = false; break; }
      if (lane == 0) {
        mbar_arrive_expect_tx(&sh.v_full[st], C::kTileBytes);
        ++v_armed[st];
      }
      __syncwarp();
      if (lane < C::kPagesPerTile) {
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_3d(smem_base + C::kVOffset + st * C::kTileBytes + hf * C::kHalfBytes +
                          lane * (kPage * 128),
                      vmap, &sh.v_full[st], hf * 64, un.h, id * kPage);
      }
    }
    if (!ok) break;
    it += un.n_kt;
  }
  if (lane == 0 && *abort) {
    for (int b = 0; b < C::kStagesV; ++b)
      if (v_armed[b]) mbar_wait_bounded(&sh.v_full[b], (v_armed[b] - 1) & 1, 100000000ull);
  }
}

template <int HD, bool kScored>
__device__ void mma_issuer(const AttnArgs& a, TcShared<kScored>& sh, uint32_t tmem,
                           uint32_t smem_base) {
  using C = TcCfg<HD>;
  volatile int* abort = &sh.abort;
  constexpr uint32_t idesc_s = tc::make_idesc(128, 128, false);
  constexpr uint32_t idesc_o = tc::make_idesc(128, HD, true);
  uint32_t itk = 0;                       // K/V tiles consumed
  uint32_t tcount[2] = {0, 0};            // S (= P V) tiles per side
  uint32_t ucount[2] = {0, 0};            // units per side that used O
  bool issued = false;
  // Every barrier of the loop below guards data that only tcgen05.mma reads (P and O in tensor
  // memory, Q, K and V that TMA wrote to shared memory), and each wait is followed by
  // tcgen05.fence::after_thread_sync before the MMAs that read it, so the waits are relaxed: an
  // acquiring try_wait behind queued MMAs left the tensor pipe idle ~140 cycles per wait on this
  // GPU, a relaxed one costs nothing.  The unit descriptor is plain shared memory written by the
  // producer warp: its barrier keeps the acquiring wait.
  auto wait = [&](uint64_t* bar, uint32_t phase) { return tc_wait<true>(bar, phase, abort, a); };
  // A wait whose result decides a branch costs the issuing thread a few hundred cycles even when
  // the phase is long complete; so every barrier of one step is first tested at once (the tests
  // issue back to back, one branch on their conjunction) and only a step that finds one not yet
  // complete takes the bounded waits one by one.
  auto test = [](uint64_t* bar, uint32_t phase) { return mbar_test_relaxed(bar, phase); };
  // Shared-memory descriptors are built once: a k-step moves the start address by 32 bytes
  // within a 128-byte swizzle atom, a 64-dim half by a half tile, a stage or a Q tile by whole
  // tiles.  All of these only add to the address field in the descriptor's low word (which no
  // step carries out of), so the MMAs take the two 32-bit halves and add to the low one.
  const uint64_t q_desc0 = tc::sdesc_sw128(smem_base + C::kQOffset, 16, 1024);
  const uint64_t k_desc0 = tc::sdesc_sw128(smem_base, 16, 1024);
  const uint64_t v_desc0 = tc::sdesc_sw128(smem_base + C::kVOffset, C::kHalfBytes, 1024);
  const uint32_t q_lo = static_cast<uint32_t>(q_desc0), k_lo = static_cast<uint32_t>(k_desc0),
                 v_lo = static_cast<uint32_t>(v_desc0);
  const uint32_t q_hi = static_cast<uint32_t>(q_desc0 >> 32),
                 k_hi = static_cast<uint32_t>(k_desc0 >> 32),
                 v_hi = static_cast<uint32_t>(v_desc0 >> 32);
  auto step = [](int ks, uint32_t half_bytes) -> uint32_t {
    return ((ks >> 2) * half_bytes + (ks & 3) * 32) >> 4;
  };
  auto issue_s = [&](int x, uint32_t kt) {  // S_x = Q_x K^T into S_x
    const uint32_t kd = k_lo + (((kt % C::kStagesK) * C::kTileBytes) >> 4);
    const uint32_t qd = q_lo + ((x * C::kQBytes) >> 4);
    const uint32_t d = tmem + C::col_s(x);
    tc::mma_ss_lh(d, qd, q_hi, kd, k_hi, idesc_s, 0u);
#pragma unroll
    for (int ks = 1; ks < HD / 16; ++ks)
      tc::mma_ss_lh_acc(d, qd + step(ks, C::kQHalfBytes), q_hi, kd + step(ks, C::kHalfBytes),
                        k_hi, idesc_s);
    tc::commit(&sh.s_full[x]);
    issued = true;
  };
  // O_x (+)= P_x V.  Only the side's last P V of a unit is committed on its own (o_done): an
  // earlier one is covered by the commit of the S issued after it.
  auto issue_pv = [&](int x, uint32_t kt, bool first, bool last) {
    const uint32_t vd = v_lo + (((kt % C::kStagesV) * C::kTileBytes) >> 4);
    const uint32_t d = tmem + C::col_o(x), p = tmem + C::col_s(x);
    tc::mma_ts_lh(d, p, vd, v_hi, idesc_o, first ? 0u : 1u);
#pragma unroll
    for (int kk = 1; kk < C::kN / 16; ++kk)
      tc::mma_ts_lh_acc(d, p + kk * 8, vd + ((kk * 16 * 128) >> 4), v_hi, idesc_o);
    if (last) tc::commit(&sh.o_done[x]);
  };
  for (int k = 0;; ++k) {
    const int slot = k % C::kRing;
    if (!tc_wait(&sh.unit_full[slot], (k / C::kRing) & 1, abort, a)) break;
    const typename UnitOf<kScored>::type un = sh.units[slot];
    if (!un.valid) break;
    const bool q_k = test(&sh.q_full, k & 1) & test(&sh.k_full[itk % C::kStagesK], (itk / C::kStagesK) & 1);
    if (!q_k && (!wait(&sh.q_full, k & 1) ||
                 !wait(&sh.k_full[itk % C::kStagesK], (itk / C::kStagesK) & 1)))
      break;
    tc::fence_after_sync();
    issue_s(0, itk);
    if (un.n[1] > 0) issue_s(1, itk);
    bool ok = true;
    for (int j = 0; j < un.n_kt && ok; ++j) {
      const uint32_t kt = itk + j;
      bool k_ready = false, v_ready = false;
#pragma unroll
      for (int x = 0; x < 2; ++x) {  // unrolled: the per-side counters stay in registers
        if (j >= un.n[x]) continue;
        // every wait of this side's step first, then one fence before its MMAs
        const bool next_s = j + 1 < un.n[x];
        const bool need_v = !v_ready, need_o = j == 0 && ucount[x] > 0, need_k = next_s && !k_ready;
        const uint32_t ph_p = (tcount[x] + j) & 1, ph_v = (kt / C::kStagesV) & 1,
                       ph_o = (ucount[x] - 1) & 1, ph_k = ((kt + 1) / C::kStagesK) & 1;
        uint64_t* bar_v = &sh.v_full[kt % C::kStagesV];
        uint64_t* bar_k = &sh.k_full[(kt + 1) % C::kStagesK];
        const bool ready = test(&sh.p_full[x], ph_p) & (!need_v || test(bar_v, ph_v)) &
                           (!need_o || test(&sh.o_free[x], ph_o)) & (!need_k || test(bar_k, ph_k));
        if (!ready && (!wait(&sh.p_full[x], ph_p) || (need_v && !wait(bar_v, ph_v)) ||
                       (need_o && !wait(&sh.o_free[x], ph_o)) || (need_k && !wait(bar_k, ph_k)))) {
          ok = false;
          break;
        }
        k_ready = k_ready || next_s;
        v_ready = true;
        tc::fence_after_sync();
        issue_pv(x, kt, j == 0, !next_s);
        if (next_s) issue_s(x, kt + 1);
      }
      if (!ok) break;
    }
    if (!ok) break;
    tc::mbar_arrive(&sh.unit_empty[slot]);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      tcount[x] += un.n[x];
      if (un.n[x] > 0) ++ucount[x];
    }
    itk += un.n_kt;
  }
  if (issued) {  // every MMA and every commit-arrival lands before TMEM and smem are released
    tc::commit(&sh.drain);
    mbar_wait_bounded(&sh.drain, 0, 100000000ull);
  }
}

// Shared-memory barriers of a CTA, by one thread.
template <int HD, bool kScored>
__device__ __forceinline__ void init_barriers(TcShared<kScored>& sh) {
  using C = TcCfg<HD>;
  for (int i = 0; i < C::kRing; ++i) {
    mbar_init(&sh.unit_full[i], 1);
    // the issuer, one lane of each softmax warp and the V producer
    mbar_init(&sh.unit_empty[i], 1 + 8 + 1);
  }
  mbar_init(&sh.q_full, 1);
  mbar_init(&sh.q_empty, 1);
  for (int i = 0; i < C::kStagesK; ++i) {
    mbar_init(&sh.k_full[i], 1);
    mbar_init(&sh.k_empty[i], 1);
  }
  for (int i = 0; i < C::kStagesV; ++i) {
    mbar_init(&sh.v_full[i], 1);
    mbar_init(&sh.v_empty[i], 1);
  }
  for (int i = 0; i < 2; ++i) {
    mbar_init(&sh.s_full[i], 1);
    mbar_init(&sh.p_full[i], 4);  // one lane of each softmax warp
    mbar_init(&sh.o_done[i], 1);
    mbar_init(&sh.o_free[i], 4);
  }
  mbar_init(&sh.drain, 1);
  for (int w = 0; w < 8; ++w)
    for (int st = 0; st < DecCfg<128>::kStages; ++st) mbar_init(&sh.dec_bars[w][st], 1);
  sh.abort = 0;
}

}  // namespace
}  // namespace attn
}  // namespace rb
