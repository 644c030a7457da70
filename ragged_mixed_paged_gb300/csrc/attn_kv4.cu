// rb_paged_attention_kv4: varlen causal GQA attention of a mixed batch over a paged cache held in
// 4 bits.
//
//   o = softmax(scale * q . K) . V,  K = k_scale * s * c,  V = v_scale * s * c  (rb.h's format)
//
// A planner (attn_kv4_plan.cuh) and one persistent launch: the CTAs that the planner gives the decode
// requests take their pages with all 16 warps (attn_kv4_decode.cuh), and every CTA takes prefill
// units.  Prefill unit = (request, kv head, pair of 128-row query tiles):
//   warp 0      one thread issues the MMAs: S = Q K^T (both K-major in shared memory), O += P V (P
//               from TMEM, V MN-major), kind::f16 with fp16 operands;
//   warp 1      takes units and loads Q (TMA);
//   warp 2      copies the cache's bytes of each key tile to shared memory (bulk copies);
//   warps 4, 5  turn the codes of each 128-key K tile into fp16 in the 128-byte-swizzled layout that
//               tcgen05.mma reads; warps 6, 7 the same for V;
//   warps 8-15  softmax and epilogue, a thread per query row.
// fp16 holds every value of the cache exactly, so K and V enter the products unrounded, and P with 11
// bits instead of bf16's 8.  Q comes as bf16: each softmax thread divides its own row by a power of
// two, which makes it exact in fp16 (attn_kv4_decode.cuh), and keeps the factor for its scores.
// A tile is turned once for 256 query rows: 1/2 instruction a value and 4 bytes of shared
// memory traffic, against 512 multiply-adds of the tensor core.
// Values behind the sequence's end are finite whatever a page holds, so their zero weights suffice.
//
// What bounds a prefill unit: the chain of a side's steps.  A key tile takes 4400 cycles: softmax
// 1850 (1024 of them ex2's rate for a row a thread), P V and the next S 1370 at the tensor core's
// rate, the rest notices between the roles; the two sides in turn keep the tensor pipe at 0.53 of
// its rate.  A prompt of 8192 tokens, 32 + 8 heads of 128: 530 us (1.04 PFLOP/s).  Measured when it took
// 536: 433 if nothing were turned; an issuer thread for each side 568; that, and steps of 64 keys with
// S of the next one ahead, 592 (an MMA of 64 columns takes as long as one of 128, which reads as
// much of A); two threads a row, all softmax warps on one side's tile at a time, 596 (ex2 bound).
#include <cfloat>

#include "attn_kv4_decode.cuh"
#include "attn_kv4_plan.cuh"
#include "attn_prefill_tc.cuh"

namespace rb {
namespace attn {
namespace {

using kv4d::hmul2;

constexpr int kPlanThreads = 1024;

// Threads and registers: launched with 128 for each of 512 threads, which the decode phases use; a
// prefill phase gives the softmax warps 184 and the others 72.
constexpr int kThreads = 512, kWarps = 16;
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 184, kControlRegs = 72;
static_assert(256 * kSoftmaxRegs + 256 * kControlRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr int kTurnWarp = 4, kSoftmaxWarp = 8;  // the first ones
constexpr int kRawSlots = 3;                    // half tiles of the cache's bytes on their way

__global__ void __launch_bounds__(kPlanThreads) kv4_plan_kernel(AttnArgs a, int head_dim) {
  grid_release();  // the attention launch sets itself up meanwhile
  kv4_plan_body(a, head_dim, kWarps);
}

struct Kv4Shared {
  uint64_t unit_full[4], unit_empty[4];
  uint64_t q_full[2], q_ready[2], q_empty;  // Q landed (bf16), Q turned (fp16), per side
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], o_done[2], o_free[2];
  uint64_t raw_full[2][kRawSlots], raw_empty[2][kRawSlots];  // K and V
  uint64_t drain;
  TcUnit units[4];
  uint32_t tmem_base;
  int abort;
};

__host__ __device__ constexpr uint32_t make_idesc_f16(int M, int N, bool b_mn_major) {
  return tc::make_idesc(M, N, b_mn_major) & ~((1u << 7) | (1u << 10));  // A and B fp16, not bf16
}

// The warps that turn tiles read the cache's bytes from rings of pages in shared memory.  Loops are kept
// rolled, and K and V share their code: straight-line code of several roles runs at the rate of
// instruction fetch (a tile's half unrolled took 8000 cycles, ten times its instructions).
template <int HD>
struct Kv4Cfg {
  using C = TcCfg<HD>;
  static constexpr int kStagesK = 2, kStagesV = 2;
  static constexpr int kVOffset = kStagesK * C::kTileBytes;
  static constexpr int kQOffset = kVOffset + kStagesV * C::kTileBytes;  // Q_A then Q_B
  static constexpr int kRawOffset = kQOffset + 2 * C::kQBytes;
  static constexpr int kRawBytes = C::kPagesPerTile / 2 * 9 * HD;  // K or V of half a tile
  static constexpr int kUsed = kRawOffset + 2 * kRawSlots * kRawBytes;
  static constexpr int kDecode = kWarps * kv4d::Ring<HD>::kWarpBytes;
  static constexpr int kMost = kUsed > kDecode ? kUsed : kDecode;
  // at least 120 KB keeps one CTA per SM (each CTA holds all 512 TMEM columns)
  static constexpr int kSmemBytes = (kMost + 1024) > 120 * 1024 ? (kMost + 1024) : 120 * 1024;
};

// A lane's part in turning pages into fp16 rows of a tile (128 keys x 128 bytes, 128-byte swizzle, one
// such block per 64 values): it takes runs of 32 values, a quarter (half, for heads of 64) of a
// token, four 16-byte stores each, of token `tok` and for heads of 128 of tok + 8.  A head of 128 has
// its quarters in two blocks of the same banks: the upper two take their pieces in the order 2, 3,
// 0, 1.  The places do not change, so they are worked out once.
template <int HD>
struct Turner {
  static constexpr int kParts = HD / 32, kTokens = 32 / kParts;
  int code, scale, scale_run, scale_next, row, piece[4];  // bytes from the page; from the tile's row and in it
  uint32_t first, second;          // which of a run's two scales a piece takes (byte selectors)
  bool upper;
  __device__ Turner(int lane, bool values) {
    const int part = lane % kParts, tok = lane / kParts;
    upper = part >= 2;
    code = tok * (HD / 2) + part * 16;
    scale = 8 * HD + (values ? 2 * part * kPage + tok : tok * (HD / 16) + 2 * part);
    scale_next = values ? kPage : 1;
    scale_run = kTokens * (values ? 1 : HD / 16);
    row = (part >> 1) * (HD == 128 ? TcCfg<HD>::kHalfBytes : 0) + tok * 128;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      piece[k] = row + ((((part & 1) * 4 + (upper ? k ^ 2 : k)) ^ (tok & 7)) << 4);
    first = upper ? 0x3232 : 0x1010;
    second = upper ? 0x1010 : 0x3232;
  }
  // One page, whose first row of the tile is at `rows`.
  __device__ __forceinline__ void page(const uint8_t* from, uint8_t* rows) const {
#pragma unroll
    for (int i = 0; i < kPage / kTokens; ++i) {  // (rows 8 apart have the same swizzle)
      const uint4 c = *reinterpret_cast<const uint4*>(from + code + i * kTokens * (HD / 2));
      const uint8_t* sp = from + scale + i * scale_run;
      const uint32_t sb = sp[0] | static_cast<uint32_t>(sp[scale_next]) << 8;
      const uint32_t s2 = kv4d::scales2<0x4140>(sb);
      const uint32_t w[4] = {upper ? c.z : c.x, upper ? c.w : c.y, upper ? c.x : c.z,
                             upper ? c.y : c.w};
      const uint32_t m0 = __byte_perm(s2, 0, first), m1 = __byte_perm(s2, 0, second);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t h[4];
        kv4::values8(w[k], h);
        const uint32_t m = k < 2 ? m0 : m1;
        *reinterpret_cast<uint4*>(rows + piece[k] + i * kTokens * 128) =
            make_uint4(hmul2(h[0], m), hmul2(h[1], m), hmul2(h[2], m), hmul2(h[3], m));
      }
    }
  }
};

// One contiguous copy into shared memory, its bytes counted on `bar`.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const uint8_t* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Warp 2: the cache's bytes of each half tile (four pages) of each unit, K and V, into a ring of
// kRawSlots half tiles.  A bulk copy a page: 16-byte cp.async starves beside the MMAs, which read
// shared memory at its full rate (pages five ahead came 6000 cycles late).
template <int HD>
__device__ __forceinline__ void producer_raw(const Kv4Args& g4, Kv4Shared& sh, uint32_t raw_at) {
  using C = TcCfg<HD>;
  using K4 = Kv4Cfg<HD>;
  const AttnArgs& a = g4.a;
  volatile int* abort = &sh.abort;
  constexpr int kHalf = C::kPagesPerTile / 2, kBytes = 9 * HD;
  const int lane = threadIdx.x & 31;
  const int kv = lane >> 2 & 1;  // lanes 0-3 copy K, 4-7 V
  const uint8_t* cache = kv ? g4.v : g4.k;
  uint32_t count = 0;  // half tiles so far
  bool ok = true;
  for (int k = 0; ok; ++k) {
    const int slot = k % C::kRing;
    int go = 1;
    if (lane == 0) go = tc_wait(&sh.unit_full[slot], (k / C::kRing) & 1, abort, a) ? 1 : 0;
    if (!__shfl_sync(0xffffffffu, go, 0)) break;
    const TcUnit un = sh.units[slot];
    if (!un.valid) break;
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sh.unit_empty[slot]);  // the descriptor is in registers
    PageWindow pw(a, un, lane);
    int id = 0;
#pragma unroll 1
    for (int i = 0; i < 2 * un.n_kt; ++i, ++count) {
      if ((i & 1) == 0) id = pw.tile_page(i >> 1, true);
      const int mine = __shfl_sync(0xffffffffu, id, (i & 1) * kHalf + (lane & 3));
      const uint32_t st = count % kRawSlots;
      if ((lane & 3) == 0 && lane < 8) {
        go = tc_wait(&sh.raw_empty[kv][st], ((count / kRawSlots) & 1) ^ 1, abort, a) ? 1 : 0;
        if (go) mbar_arrive_expect_tx(&sh.raw_full[kv][st], kHalf * kBytes);
      }
      const bool armed_k = __shfl_sync(0xffffffffu, go, 0), armed_v = __shfl_sync(0xffffffffu, go, 4);
      // (what is armed is copied, so that its barrier completes whatever happens)
      if (lane < 8 && (kv ? armed_v : armed_k))
        bulk_copy(raw_at + (2 * st + kv) * K4::kRawBytes + (lane & 3) * kBytes,
                  cache + (static_cast<size_t>(mine) * a.nkv + un.h) * kBytes, kBytes,
                  &sh.raw_full[kv][st]);
      if (!(armed_k && armed_v)) { ok = false; break; }
    }
  }
  if (lane == 0 && *abort)  // let the copies already issued land before the CTA can exit
#pragma unroll 1
    for (uint32_t i = 0; i < kRawSlots && i < count + 1; ++i) {
      const uint32_t c = count - i;  // (the one after the last may be armed in part)
      for (int w = 0; w < 2; ++w)
        mbar_wait_bounded(&sh.raw_full[w][c % kRawSlots], (c / kRawSlots) & 1, 1000000ull);
    }
  __syncwarp();
}

// A warp of the two that turn K (V): two pages of each half tile, into a ring of kStages tiles.
template <int HD, int kStages>
__device__ __forceinline__ void turn_tiles(const AttnArgs& a, Kv4Shared& sh, bool values, uint8_t* ring,
                                           const uint8_t* raw, uint64_t* full, uint64_t* empty) {
  using C = TcCfg<HD>;
  using K4 = Kv4Cfg<HD>;
  volatile int* abort = &sh.abort;
  constexpr int kBytes = 9 * HD, kHalf = C::kPagesPerTile / 2;
  const int lane = threadIdx.x & 31, page = (threadIdx.x >> 5 & 1) * (kHalf / 2);
  const Turner<HD> turner(lane, values);
  uint32_t it = 0, count = 0;
  auto wait = [&](uint64_t* bar, uint32_t phase) -> bool {
    const bool done = tc_wait(bar, phase, abort, a);
    return !__any_sync(0xffffffffu, !done);
  };
  bool ok = true;
  for (int k = 0; ok; ++k) {
    const int slot = k % C::kRing;
    if (!wait(&sh.unit_full[slot], (k / C::kRing) & 1)) break;
    const int tiles = sh.units[slot].n_kt, valid = sh.units[slot].valid;
    if (!valid) break;
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sh.unit_empty[slot]);
#pragma unroll 1
    for (int i = 0; i < 2 * tiles; ++i, ++count) {
      const uint32_t tile = it + (i >> 1), st = tile % kStages, from = count % kRawSlots;
      if (!wait(&sh.raw_full[values][from], (count / kRawSlots) & 1) ||
          ((i & 1) == 0 && !wait(&empty[st], ((tile / kStages) & 1) ^ 1))) {
        ok = false;
        break;
      }
      const uint8_t* src = raw + (2 * from + values) * K4::kRawBytes;
#pragma unroll 1
      for (int p = page; p < page + kHalf / 2; ++p)
        turner.page(src + p * kBytes,
                    ring + st * C::kTileBytes + ((i & 1) * kHalf + p) * (kPage * 128));
      if (i & 1) fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&sh.raw_empty[values][from]);
        if (i & 1) tc::mbar_arrive(&full[st]);
      }
    }
    it += tiles;
  }
}

// Warp 1: units and Q.
template <int HD>
__device__ void producer_q4(const AttnArgs& a, Kv4Shared& sh, uint32_t smem_base,
                            const CUtensorMap* qmap) {
  using C = TcCfg<HD>;
  using K4 = Kv4Cfg<HD>;
  volatile int* abort = &sh.abort;
  const int lane = threadIdx.x & 31;
  const int n_units = a.header[kHNumPrefillUnits];
  uint32_t q_armed[2] = {0, 0};
  if (lane == 0) {
    for (int k = 0;; ++k) {
      const int slot = k % C::kRing;
      if (!tc_wait(&sh.unit_empty[slot], ((k / C::kRing) & 1) ^ 1, abort, a)) break;
      const int u = atomicAdd(a.header + kHPrefillNext, 1);
      TcUnit un{};
      if (u < n_units) un = decode_unit(a, u);
      sh.units[slot] = un;
      // test hook: CTA 0 stops before its first unit reaches the other roles
      if (a.withhold_first_unit && blockIdx.x == 0 && k == 0 && un.valid) break;
      tc::mbar_arrive(&sh.unit_full[slot]);
      if (!un.valid) break;
      if (!tc_wait(&sh.q_empty, (k & 1) ^ 1, abort, a)) break;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (un.n[x] == 0) continue;
        mbar_arrive_expect_tx(&sh.q_full[x], C::kHalves * a.tile_tokens * a.group * 128);
        ++q_armed[x];
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_3d(smem_base + K4::kQOffset + x * C::kQBytes + hf * C::kQHalfBytes, qmap,
                      &sh.q_full[x], hf * 64, un.h * a.group, un.t0 + un.tok0 + a.tile_tokens * x);
      }
    }
    if (*abort)  // let the copies already issued land before the CTA can exit
      for (int x = 0; x < 2; ++x)
        if (q_armed[x]) mbar_wait_bounded(&sh.q_full[x], (q_armed[x] - 1) & 1, 100000000ull);
  }
  __syncwarp();
}

// The MMA issuer (one thread).  Q, K and V are written to shared memory by ordinary stores, whose
// threads make them visible to the tensor core (a proxy fence) and then arrive: the issuer's waits for
// them acquire, so that its MMAs come after those stores.  P and O are in tensor memory, whose
// accesses tcgen05.fence::after_thread_sync orders behind a relaxed wait.  (A prompt of 8192 tokens:
// 536 us then, 538 with P tested first, 542 with relaxed tests and one acquiring fence a step.)
template <int HD>
__device__ void mma_issuer4(const AttnArgs& a, Kv4Shared& sh, uint32_t tmem, uint32_t smem_base) {
  using C = TcCfg<HD>;
  using K4 = Kv4Cfg<HD>;
  volatile int* abort = &sh.abort;
  constexpr uint32_t idesc_s = make_idesc_f16(128, 128, false);
  constexpr uint32_t idesc_o = make_idesc_f16(128, HD, true);
  static_assert(K4::kStagesK == 2 && K4::kStagesV == 2, "stages are taken by parity");
  uint32_t itk = 0;               // K/V tiles so far
  uint32_t ph_s = 0, ph_u = 0;    // bit x: parity of side x's S tiles and units so far
  uint32_t used = 0;              // bit x: side x had a unit
  // Loops stay rolled: this thread's code runs once a step beside the loops of other roles, and
  // straight-line it waits for its instructions.  A wait whose result decides a branch costs a few
  // hundred cycles even when the phase is long complete, so the barriers of one step are tested
  // together and waited for one by one only if one of them is not complete.
  auto test = [](uint64_t* bar, uint32_t phase) { return mbar_test_relaxed(bar, phase); };
  auto test_acquire = [](uint64_t* bar, uint32_t phase) { return mbar_test(bar, phase); };
  auto relaxed = [&](uint64_t* bar, uint32_t phase) { return tc_wait<true>(bar, phase, abort, a); };
  auto acquire = [&](uint64_t* bar, uint32_t phase) { return tc_wait(bar, phase, abort, a); };
  const uint64_t q_desc = tc::sdesc_sw128(smem_base + K4::kQOffset, 16, 1024);
  const uint64_t v_desc = tc::sdesc_sw128(smem_base + K4::kVOffset, C::kHalfBytes, 1024);
  const uint32_t q_lo = static_cast<uint32_t>(q_desc), v_lo = static_cast<uint32_t>(v_desc);
  const uint32_t k_lo = static_cast<uint32_t>(tc::sdesc_sw128(smem_base, 16, 1024));
  const uint32_t hi = static_cast<uint32_t>(q_desc >> 32);  // the same for all
  auto issue_s = [&](int x, uint32_t kt) {  // S_x = Q_x K^T
    uint32_t kd = k_lo + (((kt & 1) * C::kTileBytes) >> 4), qd = q_lo + ((x * C::kQBytes) >> 4);
    const uint32_t d = tmem + C::col_s(x);
#pragma unroll 1
    for (int half = 0; half < C::kHalves; ++half) {
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        tc::mma_ss_lh(d, qd + ks * 2, hi, kd + ks * 2, hi, idesc_s, half + ks > 0 ? 1u : 0u);
      qd += C::kQHalfBytes >> 4;
      kd += C::kHalfBytes >> 4;
    }
    tc::commit(&sh.s_full[x]);
  };
  auto issue_pv = [&](int x, uint32_t kt, bool first, bool last) {  // O_x (+)= P_x V
    uint32_t vd = v_lo + (((kt & 1) * C::kTileBytes) >> 4), p = tmem + C::col_s(x);
    const uint32_t d = tmem + C::col_o(x);
#pragma unroll 1
    for (int kk = 0; kk < C::kN / 64; ++kk) {
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        tc::mma_ts_lh(d, p + ks * 8, vd + ((ks * 16 * 128) >> 4), hi, idesc_o,
                      first && kk + ks == 0 ? 0u : 1u);
      p += 32;
      vd += (64 * 128) >> 4;
    }
    if (last) tc::commit(&sh.o_done[x]);
  };
  for (int k = 0;; ++k) {
    const int slot = k % C::kRing;
    if (!acquire(&sh.unit_full[slot], (k / C::kRing) & 1)) break;
    const int n0 = sh.units[slot].n[0], n1 = sh.units[slot].n[1];
    if (!sh.units[slot].valid) break;
    const int steps = max(n0, n1);
    if (!acquire(&sh.k_full[itk & 1], (itk >> 1) & 1)) break;
    bool ok = true;
#pragma unroll 1
    for (int x = 0; x < (n1 > 0 ? 2 : 1) && ok; ++x) {
      ok = acquire(&sh.q_ready[x], ph_u >> x & 1);
      if (!ok) break;
      tc::fence_after_sync();
      issue_s(x, itk);
    }
    for (int j = 0; j < steps && ok; ++j) {
      const uint32_t kt = itk + j;
#pragma unroll 1
      for (int x = 0; x < 2; ++x) {
        const int n = x ? n1 : n0;
        if (j >= n) continue;
        const bool next_s = j + 1 < n, need_o = j == 0 && (used >> x & 1);
        uint64_t* bar_v = &sh.v_full[kt & 1];
        uint64_t* bar_k = &sh.k_full[(kt + 1) & 1];
        const uint32_t ph_v = (kt >> 1) & 1, ph_k = ((kt + 1) >> 1) & 1;
        const uint32_t ph_p = ph_s >> x & 1, ph_o = (ph_u >> x & 1) ^ 1;
        // (P last: it comes last, and what is tested after it delays the MMAs)
        const bool ready = test_acquire(bar_v, ph_v) & (!next_s || test_acquire(bar_k, ph_k)) &
                           (!need_o || test(&sh.o_free[x], ph_o)) & test(&sh.p_full[x], ph_p);
        if (!ready && (!acquire(bar_v, ph_v) || (need_o && !relaxed(&sh.o_free[x], ph_o)) ||
                       (next_s && !acquire(bar_k, ph_k)) || !relaxed(&sh.p_full[x], ph_p))) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        issue_pv(x, kt, j == 0, !next_s);
        if (next_s) issue_s(x, kt + 1);
        ph_s ^= 1u << x;
      }
    }
    if (!ok) break;
    tc::mbar_arrive(&sh.unit_empty[slot]);
    ph_u ^= n1 > 0 ? 3u : 1u;
    used |= n1 > 0 ? 3u : 1u;
    itk += steps;
  }
  // every MMA and every commit-arrival lands before TMEM and smem are released
  tc::commit(&sh.drain);
  mbar_wait_bounded(&sh.drain, 0, 100000000ull);
}

// Columns of a tile that a softmax thread takes at a time.
constexpr int kCols = 32;
// Largest sum of their exponents: P stays below 2^15 in fp16.
constexpr float kSumLimit = 32768.f;

__device__ __forceinline__ void load_scores(uint32_t at, float (&s)[kCols]) {
#pragma unroll
  for (int c = 0; c < kCols / 32; ++c)
    tc::ld32(at + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * c));
  tc::wait_ld();
}
__device__ __forceinline__ void store_weights(uint32_t at, const uint32_t (&p)[kCols / 2]) {
#pragma unroll
  for (int c = 0; c < kCols / 32; ++c)
    tc::st16(at + 16 * c, *reinterpret_cast<const uint32_t(*)[16]>(p + 16 * c));
}

// O (if it holds anything: S of this tile, issued after the tiles before, has landed) and P of the
// tile's columns before c0, times alpha (in fp32: it may be below fp16's range).  The stores have
// landed when it returns: it may be called again for the same tile.
template <int HD>
__device__ __forceinline__ void rescale(uint32_t col_s, uint32_t col_o, int c0, bool has_o,
                                        float alpha) {
  if (has_o) {
#pragma unroll 1
    for (int c = 0; c < HD; c += 16) {
      uint32_t r[16];
      tc::ld16(col_o + c, r);
      tc::wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
      tc::st16(col_o + c, r);
    }
  }
#pragma unroll 1
  for (int c = 0; c < c0 / 2; c += 16) {
    uint32_t r[16];
    tc::wait_st();
    tc::ld16(col_s + c, r);
    tc::wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
      r[i] = kv4d::pack_f16x2(v.x * alpha, v.y * alpha);
    }
    tc::st16(col_s + c, r);
  }
  tc::wait_st();
}

// The two functions below are out of line.  They take a row's reference and sum by value and return
// them: by address the loop that calls them keeps both in memory (a prompt of 8192 tokens 571 us
// instead of 531).
//
// A warp's rows take a new reference where their scores of columns [c0, c0 + kCols) exceed the old
// one: O, the sum and the row's P of the columns before move by a power of two.  Rare, but for a
// row's first columns.  (All rows at once: each by itself comes here far more often, and a prompt of
// 8192 tokens takes 606 us instead of 530.)
template <int HD>
__device__ __noinline__ float2 move_reference(uint32_t col_s, uint32_t col_o, int c0, int seen,
                                              float scale, bool has_o, float old, float l) {
  float top = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < kCols; c += 16) {
    uint32_t r[16];
    tc::ld16(col_s + c0 + c, r);
    tc::wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float v = __uint_as_float(r[i]);
      top = c0 + c + i < seen ? fmaxf(top, v) : top;
    }
  }
  const float next = fmaxf(old, ceilf(top * scale));
  const float alpha = next > old ? fast_exp2(old - next) : 1.f;
  rescale<HD>(col_s, col_o, c0, has_o, alpha);
  return make_float2(next, l * alpha);
}

// Largest factor of the raw products (below 2^13) whose scores leave whole references exact in fp32.
// (A row of 128 values of 16 at most has one of about 2^9, over k_scale 1.)
constexpr float kNearScale = 0x1p11f;

// P of a tile for a warp that has a row of a larger factor, whose scores may pass 2^24.  A reference is
// one of the raw products then, which is taken off them before the factor, so that their differences
// keep their bits.
template <int HD>
__device__ __noinline__ float2 far_tile(uint32_t col_s, uint32_t col_o, int seen, float scale,
                                        bool has_o, float ref, float l) {
  constexpr float kGrowth = 8.f;  // P stays below 2^(kPShift + kGrowth)
#pragma unroll 1
  for (int c0 = 0; c0 < TcCfg<HD>::kN; c0 += kCols) {
    float s[kCols], top = -INFINITY;
    load_scores(col_s + c0, s);
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      s[i] = c0 + i < seen ? s[i] : -INFINITY;
      top = fmaxf(top, s[i]);
    }
    float alpha = 1.f;
    if (top > -INFINITY && (ref == -INFINITY || (top - ref) * scale > kGrowth)) {
      alpha = fast_exp2((ref - top) * scale);
      ref = top;
    }
    l *= alpha;
    if (__any_sync(0xffffffffu, alpha != 1.f)) rescale<HD>(col_s, col_o, c0, has_o, alpha);
    const float base = ref == -INFINITY ? 0.f : ref;
    uint32_t pk[kCols / 2];
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) {
      const float p = fast_exp2(fmaf(s[2 * i] - base, scale, kPShift));
      const float q = fast_exp2(fmaf(s[2 * i + 1] - base, scale, kPShift));
      l += p + q;
      pk[i] = kv4d::pack_f16x2(p, q);
    }
    store_weights(col_s + c0 / 2, pk);
  }
  return make_float2(ref, l);
}

// Softmax and epilogue of tile x (0 = A, 1 = B); thread t = row t of the tile = TMEM lane t.
// Exponents are taken against a reference that lags the row's maximum, as in the ordinary launch
// (attn_prefill_tc.cu), but kCols columns at a time in a rolled loop, P going over columns that are
// read already.
template <int HD>
__device__ void softmax_kv4(const Kv4Args& g4, Kv4Shared& sh, uint32_t tmem, uint8_t* smem_ptr,
                            int x) {
  using C = TcCfg<HD>;
  using K4 = Kv4Cfg<HD>;
  const AttnArgs& a = g4.a;
  volatile int* abort = &sh.abort;
  const int t = threadIdx.x & 127;
  const uint32_t lane_off = static_cast<uint32_t>((t >> 5) * 32) << 16;
  const uint32_t col_s = tmem + lane_off + C::col_s(x), col_o = tmem + lane_off + C::col_o(x);
  uint32_t tc_x = 0, itk = 0, uc_x = 0;  // S tiles, K/V tiles and units (with n > 0) of this side
  auto wait_all = [&](uint64_t* bar, uint32_t phase) -> bool {
    const bool ok = tc_wait(bar, phase, abort, a);
    return !__any_sync(0xffffffffu, !ok);
  };
  const bool lane0 = (t & 31) == 0;
  auto arrive_warp = [&](uint64_t* bar) {
    __syncwarp();
    if (lane0) tc::mbar_arrive(bar);
  };
  for (int k = 0;; ++k) {
    const int slot = k % C::kRing;
    if (!wait_all(&sh.unit_full[slot], (k / C::kRing) & 1)) break;
    const TcUnit un = sh.units[slot];
    if (!un.valid) break;
    const int n = un.n[x];
    // row t: token tok_base + t / group, head t % group of the kv head's group; the other rows hold
    // no query and are masked out
    const int tok_base = un.tok0 + a.tile_tokens * x;
    const int rows_used = a.tile_tokens * a.group;
    const int jt_in = t / a.group;
    const bool valid = t < rows_used && tok_base + jt_in < un.q;
    const int jt = valid ? tok_base + jt_in : 0;
    const int hh = valid ? t - jt_in * a.group : 0;
    const int lim = valid ? un.c + jt : -1;
    const int lim_min = un.c + tok_base;
    const bool partial = rows_used < C::kM || tok_base + a.tile_tokens > un.q;
    const bool releases = x == (un.n[1] > 0 ? 1 : 0);
    bool ok = true;
    float scale = a.scale_log2 * kv4d::kScaleUnit;
    if (n > 0) {  // this row of Q to fp16, in place
      if (!wait_all(&sh.q_full[x], uc_x & 1)) break;
      uint8_t* row = smem_ptr + K4::kQOffset + x * C::kQBytes + t * 128;
      uint4 w[HD / 8];
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) {
        w[i] = *reinterpret_cast<const uint4*>(row + (i >> 3) * C::kQHalfBytes +
                                               (((i & 7) ^ (t & 7)) << 4));
        const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          top = fmax3(top, fabsf(__uint_as_float(v[e] << 16)),
                      fabsf(__uint_as_float(v[e] & 0xffff0000u)));
      }
      float down, up;
      kv4d::power_of(top, &down, &up);
      scale = kv4d::score_scale(up, scale);
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) {
        uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = kv4d::pack_f16x2(__uint_as_float(v[e] << 16) * down,
                                  __uint_as_float(v[e] & 0xffff0000u) * down);
        *reinterpret_cast<uint4*>(row + (i >> 3) * C::kQHalfBytes +
                                  (((i & 7) ^ (t & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
      }
      fence_proxy_async_smem();
      arrive_warp(&sh.q_ready[x]);
    }
    const bool far = __any_sync(0xffffffffu, valid && scale > kNearScale);
    // running reference (log2 units, a whole number; if far, a raw product) and sum; a row without a
    // query starts at 0
    float m_ref = valid ? -INFINITY : 0.f, l = 0.f;
    for (int j = 0; j < n; ++j) {
      const uint32_t tj = tc_x + j;
      if (!wait_all(&sh.s_full[x], tj & 1)) { ok = false; break; }
      if (releases && t == 0) {
        const uint32_t kt = itk + j;
        tc::mbar_arrive(&sh.k_empty[kt % K4::kStagesK]);
        if (j > 0) tc::mbar_arrive(&sh.v_empty[(kt - 1) % K4::kStagesV]);
        if (j + 1 == n) tc::mbar_arrive(&sh.q_empty);
      }
      tc::fence_after_sync();
      const int kv_base = j * C::kN;
      const bool masked = partial || kv_base + C::kN - 1 > lim_min;
      // keys of the tile that this row sees
      const int seen = masked ? lim + 1 - kv_base : C::kN;
      const float2 sc2 = make_float2(scale, scale);
      if (far) {
        const float2 next = far_tile<HD>(col_s, col_o, seen, scale, j > 0, m_ref, l);
        m_ref = next.x;
        l = next.y;
      }
#pragma unroll 1
      for (int c0 = far ? C::kN : 0; c0 < C::kN; c0 += kCols) {
        float s[kCols];
        load_scores(col_s + c0, s);
        if (masked) {
#pragma unroll
          for (int i = 0; i < kCols; ++i) s[i] = c0 + i < seen ? s[i] : -INFINITY;
        }
        uint32_t pk[kCols / 2];
        auto exponents = [&]() -> float {
          const float mu = m_ref == -INFINITY ? 0.f : m_ref - kPShift;
          const float2 nmu2 = make_float2(-mu, -mu);
          float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int i = 0; i < kCols / 2; ++i) {
            const float2 e = __ffma2_rn(make_float2(s[2 * i], s[2 * i + 1]), sc2, nmu2);
            const float2 p = make_float2(fast_exp2(e.x), fast_exp2(e.y));
            rs[i & 1] = __fadd2_rn(rs[i & 1], p);
            pk[i] = kv4d::pack_f16x2(p.x, p.y);
          }
          const float2 r = __fadd2_rn(rs[0], rs[1]);
          return r.x + r.y;
        };
        float sum = exponents();
        // the row's first columns, and any that exceed the reference by too much
        if (__any_sync(0xffffffffu, !(sum <= kSumLimit) || m_ref == -INFINITY)) {
          const float2 next = move_reference<HD>(col_s, col_o, c0, seen, scale, j > 0, m_ref, l);
          m_ref = next.x;
          l = next.y;
          sum = exponents();
        }
        l += sum;
        store_weights(col_s + c0 / 2, pk);
      }
      tc::wait_st();
      tc::fence_before_sync();
      arrive_warp(&sh.p_full[x]);
    }
    if (!ok) break;
    const uint32_t kt_last = itk + un.n_kt - 1;
    itk += un.n_kt;
    if (n > 0) {
      if (!wait_all(&sh.o_done[x], uc_x & 1)) break;  // the unit's last P V is in O
      if (releases && t == 0) tc::mbar_arrive(&sh.v_empty[kt_last % K4::kStagesV]);
      ++uc_x;
      tc_x += n;
      tc::fence_after_sync();
      const float wa = g4.v_scale * kv4d::kScaleUnit / l;  // (nothing but -inf: 0 / 0)
      uint32_t pk[HD / 2];
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        tc::ld32(col_o + c * 32, o);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          pk[16 * c + i] =
              pack_bf16x2(__uint_as_float(o[2 * i]) * wa, __uint_as_float(o[2 * i + 1]) * wa);
      }
      tc::fence_before_sync();
      arrive_warp(&sh.o_free[x]);
      if (valid) {
        __nv_bfloat16* dst =
            a.out + (static_cast<size_t>(un.t0 + jt) * a.nh + un.h * a.group + hh) * HD;
        if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
#pragma unroll
          for (int v = 0; v < HD / 16; ++v)
            st_global_v8(dst + 16 * v, pk[8 * v], pk[8 * v + 1], pk[8 * v + 2], pk[8 * v + 3],
                         pk[8 * v + 4], pk[8 * v + 5], pk[8 * v + 6], pk[8 * v + 7]);
        } else {
#pragma unroll
          for (int v = 0; v < HD / 8; ++v)
            reinterpret_cast<uint4*>(dst)[v] = make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
        }
      }
    }
    arrive_warp(&sh.unit_empty[slot]);
  }
}

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kv4_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ Kv4Args g4) {
  using C = TcCfg<HD>;
  using K4 = Kv4Cfg<HD>;
  const AttnArgs& a = g4.a;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Kv4Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  if (tid == 32 && a.N_pad > 0) prefetch_tmap(&qmap);
  if (tid == 0) {
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(&sh.unit_full[i], 1);
      mbar_init(&sh.unit_empty[i], 1 + 8 + 4 + 1);  // issuer; softmax, turning, copying warps
    }
    mbar_init(&sh.q_empty, 1);
    for (int i = 0; i < K4::kStagesK; ++i) {
      mbar_init(&sh.k_full[i], 2);
      mbar_init(&sh.k_empty[i], 1);
    }
    for (int i = 0; i < K4::kStagesV; ++i) {
      mbar_init(&sh.v_full[i], 2);
      mbar_init(&sh.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_ready[i], 4);  // one lane of each softmax warp of the side
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.o_done[i], 1);
      mbar_init(&sh.o_free[i], 4);
    }
    for (int w = 0; w < 2; ++w)
      for (int i = 0; i < kRawSlots; ++i) {
        mbar_init(&sh.raw_full[w][i], 1);
        mbar_init(&sh.raw_empty[w][i], 2);
      }
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    fence_barrier_init();
  }
  if (warp == C::kMmaWarp) {
    tc::tmem_alloc(&sh.tmem_base, C::kTmemCols);
    tc::tmem_relinquish();
  }
  kv4_clear_padding(a, HD);  // (what ran before the planner is done)
  grid_wait();  // the planner's results
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem_base;

  // The first CTAs take the decode requests' pages (the stream's warps spread over them); every CTA
  // then takes prefill units.
  const int decode_ctas = a.header[kHDecodeCtas];
  const int rank = static_cast<int>(blockIdx.x);
  if (rank < decode_ctas) {
    decode_warp_kv4<HD>(g4, base_ptr + warp * kv4d::Ring<HD>::kWarpBytes,
                        warp * decode_ctas + rank);
    fence_proxy_async_smem();  // the rings' ordinary accesses before the tiles' asynchronous ones
  }
  if (a.header[kHNumPrefillUnits] > 0) {
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp < kSoftmaxWarp) {
      fewer_registers<kControlRegs>();
      if (warp == C::kMmaWarp) {
        if ((tid & 31) == 0) mma_issuer4<HD>(a, sh, tmem, base);
        __syncwarp();
      } else if (warp == 1) {
        producer_q4<HD>(a, sh, base, &qmap);
      } else if (warp == 2) {
        producer_raw<HD>(g4, sh, base + K4::kRawOffset);
      } else if (warp >= kTurnWarp) {
        const bool values = warp >= kTurnWarp + 2;
        turn_tiles<HD, K4::kStagesK>(a, sh, values, base_ptr + (values ? K4::kVOffset : 0),
                                     base_ptr + K4::kRawOffset, values ? sh.v_full : sh.k_full,
                                     values ? sh.v_empty : sh.k_empty);
      }
      __syncwarp();
    } else {
      more_registers<kSoftmaxRegs>();
      softmax_kv4<HD>(g4, sh, tmem, base_ptr, (warp - kSoftmaxWarp) >> 2);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == C::kMmaWarp) {
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int HD>
rb_status launch_kv4(const Kv4Args& g4, const CUtensorMap& qmap, cudaStream_t s) {
  using C = TcCfg<HD>;
  using K4 = Kv4Cfg<HD>;
  static bool configured[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return RB_ERR_CUDA;
  if (!configured[dev]) {
    if (cudaFuncSetAttribute(attn_kv4_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             K4::kSmemBytes) != cudaSuccess)
      return RB_ERR_CUDA;
    configured[dev] = true;
  }
  return launch_overlapped(attn_kv4_kernel<HD>, max(1, device_sm_count()), kThreads,
                           K4::kSmemBytes, s, qmap, g4);
}

}  // namespace
}  // namespace attn
}  // namespace rb

extern "C" rb_status rb_paged_attention_kv4(
    const rb_dims* dims, int32_t num_reqs, int32_t num_tokens, int32_t num_tokens_padded,
    const void* d_q, const void* d_k_cache, const void* d_v_cache, const int32_t* d_block_table,
    const int32_t* d_query_start_loc, const int32_t* d_seq_lens, float softmax_scale,
    float k_scale, float v_scale, void* d_out, void* d_workspace, size_t workspace_bytes,
    int32_t* d_error_word, void* stream) {
  rb::CallRange range_("rb_paged_attention_kv4");
  using namespace rb;
  using namespace rb::attn;
  AttnSetup su;
  rb_status st = attn_setup(dims, num_reqs, num_tokens, num_tokens_padded, d_q, d_k_cache,
                            d_v_cache, d_block_table, d_query_start_loc, d_seq_lens,
                            softmax_scale, d_out, d_workspace, workspace_bytes, d_error_word,
                            &su);
  if (st != RB_OK) return st;
  AttnArgs& a = su.a;
  const float scale = softmax_scale * k_scale * 1.4426950408889634f;
  if (!(softmax_scale > 0.f) || !kv4::layer_scale_ok(k_scale) || !kv4::layer_scale_ok(v_scale) ||
      !std::isfinite(scale * kv4d::kScaleUnit) || !(softmax_scale * k_scale >= FLT_MIN))
    return RB_ERR_INVALID_ARG;  // (a subnormal product has lost bits)
  // the units' list holds 16 bits of request and 16 of tile pair, the decode stream 31 of pages
  if (a.R > 32768 || a.N / (2 * a.tile_tokens) > 65535 || a.R * a.kp_cap > 0x7fffffffLL)
    return RB_ERR_CAPACITY;
  a.scale_log2 = scale;
  if (a.N_pad > 0 &&
      !encode_q_tensor_map(&su.qmap, a.q, su.head_dim, a.nh, a.N_pad, a.group))
    return RB_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  kv4_plan_kernel<<<1, kPlanThreads, 0, s>>>(a, su.head_dim);
  if (last_launch_status() != RB_OK) return RB_ERR_CUDA;
  note_launches(1);
  if (a.R == 0) return RB_OK;
  const Kv4Args g4{a, static_cast<const uint8_t*>(d_k_cache),
                   static_cast<const uint8_t*>(d_v_cache), v_scale};
  return su.head_dim == 128 ? launch_kv4<128>(g4, su.qmap, s) : launch_kv4<64>(g4, su.qmap, s);
}
