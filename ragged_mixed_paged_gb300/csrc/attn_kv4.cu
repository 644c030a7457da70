// rb_paged_attention_kv4: varlen causal GQA attention of a mixed batch over a paged cache held in
// 4 bits.
//
//   o = softmax(scale * q . K) . V,  K = k_scale * s * c,  V = v_scale * s * c  (rb.h's format)
//
// The planner and the shape of the launch are the 16-bit cache's (attention.cu,
// attn_prefill_tc.cu): one persistent launch in which every CTA runs decode units
// (attn_kv4_decode.cuh) and prefill units, the kind the planner gave it first.
//
// Prefill unit = (request, kv head, pair of 128-row query tiles); 12 warps:
//   warp 1      takes units, loads Q (TMA), and turns the codes of each 128-key K tile into fp16 in
//               the 128-byte-swizzled layout that tcgen05.mma reads;
//   warp 2      does the same for V;
//   warp 0      one thread issues the MMAs: S = Q K^T (both K-major in shared memory), O += P V (P
//               from TMEM, V MN-major), kind::f16 with fp16 operands;
//   warps 4-11  softmax and epilogue, a thread per query row.
// fp16 holds every value of the cache exactly, so K and V enter the products unrounded, and P with 11
// bits instead of bf16's 8.  Q comes as bf16: each softmax thread divides its own row by a power of
// two, which makes it exact in fp16 (attn_kv4_decode.cuh), and keeps the factor for its scores.
// A tile is turned once for 256 query rows: 1/2 instruction a value and 4 bytes of shared
// memory traffic, against 512 multiply-adds of the tensor core.
// Values behind the sequence's end are finite whatever a page holds, so their zero weights suffice.
#include "attn_kv4_decode.cuh"
#include "attn_plan.cuh"
#include "attn_prefill_tc.cuh"

namespace rb {
namespace attn {
namespace {

using kv4d::hmul2;

constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads) kv4_plan_kernel(AttnArgs a, int head_dim) {
  plan_body<false>(a, head_dim, ReqSrc{a.qsl, a.seq_lens, nullptr});
}

struct Kv4Shared {
  uint64_t unit_full[4], unit_empty[4];
  uint64_t q_full[2], q_ready[2], q_empty;  // Q landed (bf16), Q turned (fp16), per side
  uint64_t k_full[TcCfg<128>::kStagesK], k_empty[TcCfg<128>::kStagesK];
  uint64_t v_full[TcCfg<128>::kStagesV], v_empty[TcCfg<128>::kStagesV];
  uint64_t s_full[2], p_full[2], o_done[2], o_free[2];
  uint64_t drain;
  TcUnit units[4];
  uint32_t tmem_base;
  int abort;
  int decode_first;
  int role_rank;
};

// Largest sum of one tile's exponents (128 keys of a row): P stays below 2^15 in fp16.
constexpr float kSumLimit = 32768.f;

__host__ __device__ constexpr uint32_t make_idesc_f16(int M, int N, bool b_mn_major) {
  return tc::make_idesc(M, N, b_mn_major) & ~((1u << 7) | (1u << 10));  // A and B fp16, not bf16
}

// One lane's bytes of a page of one kv head: kRows runs of 32 codes with their two scales.
template <int HD>
struct Codes {
  static constexpr int kRows = HD / 64;
  uint4 c[kRows];
  uint32_t s[kRows];
};

// Lane's run of 32 values: token and place in the head, of run i of a page.
template <int HD>
__device__ __forceinline__ int run_token(int lane, int i) {
  return HD == 128 ? i * 8 + (lane >> 2) : lane >> 1;
}
template <int HD>
__device__ __forceinline__ int run_part(int lane) {
  return HD == 128 ? lane & 3 : lane & 1;
}

template <int HD, bool kValues>
__device__ __forceinline__ void load_codes(Codes<HD>& b, const uint8_t* page, int lane) {
  const int part = run_part<HD>(lane);
#pragma unroll
  for (int i = 0; i < Codes<HD>::kRows; ++i) {
    const int tok = run_token<HD>(lane, i);
    b.c[i] = __ldg(reinterpret_cast<const uint4*>(page + tok * (HD / 2) + part * 16));
    const uint8_t* s = page + 8 * HD;
    if constexpr (kValues)
      b.s[i] = __ldg(s + 2 * part * kPage + tok) |
               static_cast<uint32_t>(__ldg(s + (2 * part + 1) * kPage + tok)) << 8;
    else
      b.s[i] = __ldg(reinterpret_cast<const uint16_t*>(s + tok * (HD / 16) + 2 * part));
  }
}

// Turns the runs into fp16 rows of a tile (128 keys x 128 bytes, 128-byte swizzle, one such block per
// 64 values): four 16-byte stores a run.  A head of 128 has its runs in two blocks of the same
// banks: the upper two parts take their pieces in the order 2, 3, 0, 1.
template <int HD>
__device__ __forceinline__ void store_codes(const Codes<HD>& b, uint8_t* tile, int page, int lane) {
  using C = TcCfg<HD>;
  const int part = run_part<HD>(lane);
  const bool upper = HD == 128 && part >= 2;
#pragma unroll
  for (int i = 0; i < Codes<HD>::kRows; ++i) {
    const int row = page * kPage + run_token<HD>(lane, i);
    const uint4 c = b.c[i];
    const uint32_t w[4] = {upper ? c.z : c.x, upper ? c.w : c.y, upper ? c.x : c.z,
                           upper ? c.y : c.w};
    const uint32_t s2 = kv4d::scales2(b.s[i]);
    const uint32_t first = upper ? kv4d::high2(s2) : kv4d::low2(s2);
    const uint32_t second = upper ? kv4d::low2(s2) : kv4d::high2(s2);
    uint8_t* dst = tile + (part >> 1) * (HD == 128 ? C::kHalfBytes : 0) + row * 128;
    const int chunk = (part & 1) * 4 + (upper ? 2 : 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t h[4];
      kv4::values8(w[k], h);
      const uint32_t m = k < 2 ? first : second;
      *reinterpret_cast<uint4*>(dst + (((chunk ^ k) ^ (row & 7)) << 4)) =
          make_uint4(hmul2(h[0], m), hmul2(h[1], m), hmul2(h[2], m), hmul2(h[3], m));
    }
  }
}

// Turns a unit's tiles one after the other into a ring of `kStages` tiles; false: gave up.  The
// codes of kAhead pages are on their way in registers, across the tiles.
template <int HD, bool kValues, int kStages>
__device__ __forceinline__ bool produce_tiles(const Kv4Args& g4, const TcUnit& un, uint8_t* ring,
                                              uint64_t* full, uint64_t* empty, uint32_t it,
                                              volatile int* abort, int lane) {
  using C = TcCfg<HD>;
  const AttnArgs& a = g4.a;
  constexpr int kAhead = 4;
  const uint8_t* cache = kValues ? g4.v : g4.k;
  PageWindow pw(a, un, lane);
  auto at = [&](int id, int page) {
    return cache + (static_cast<size_t>(__shfl_sync(0xffffffffu, id, page)) * a.nkv + un.h) *
                       kv4::page_bytes(HD);
  };
  int id = pw.tile_page(0, !kValues);
  Codes<HD> buf[kAhead];
#pragma unroll
  for (int p = 0; p < kAhead; ++p) load_codes<HD, kValues>(buf[p], at(id, p), lane);
  for (int j = 0; j < un.n_kt; ++j) {
    const uint32_t tile = it + j, st = tile % kStages;
    const int next = j + 1 < un.n_kt ? pw.tile_page(j + 1, !kValues) : id;
    int ok = 1;
    if (lane == 0) ok = tc_wait(&empty[st], ((tile / kStages) & 1) ^ 1, abort, a) ? 1 : 0;
    if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
    uint8_t* dst = ring + st * C::kTileBytes;
#pragma unroll
    for (int p = 0; p < C::kPagesPerTile; ++p) {
      store_codes<HD>(buf[p % kAhead], dst, p, lane);
      const int n = p + kAhead;
      load_codes<HD, kValues>(buf[p % kAhead],
                              n < C::kPagesPerTile ? at(id, n) : at(next, n - C::kPagesPerTile),
                              lane);
    }
    id = next;
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&full[st]);
  }
  return true;
}

// Warp 1: units, Q and K.
template <int HD>
__device__ void producer_qk4(const Kv4Args& g4, Kv4Shared& sh, uint32_t smem_base,
                             uint8_t* smem_ptr, const CUtensorMap* qmap) {
  using C = TcCfg<HD>;
  const AttnArgs& a = g4.a;
  volatile int* abort = &sh.abort;
  const int lane = threadIdx.x & 31;
  const int n_units = a.header[kHNumPrefillUnits];
  uint32_t it = 0, q_armed[2] = {0, 0};
  auto lane0_wait = [&](uint64_t* bar, uint32_t phase) -> bool {
    int ok = 1;
    if (lane == 0) ok = tc_wait(bar, phase, abort, a) ? 1 : 0;
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
  };
  for (int k = 0;; ++k) {
    const int slot = k % C::kRing;
    if (!lane0_wait(&sh.unit_empty[slot], ((k / C::kRing) & 1) ^ 1)) break;
    int withhold = 0;
    if (lane == 0) {
      const int u = atomicAdd(a.header + kHPrefillNext, 1);
      TcUnit un{};
      if (u < n_units) un = decode_unit(a, u);
      sh.units[slot] = un;
      // test hook: CTA 0 stops before its first unit reaches the other roles
      withhold = a.withhold_first_unit && blockIdx.x == 0 && k == 0 && un.valid;
      if (!withhold) tc::mbar_arrive(&sh.unit_full[slot]);
    }
    if (__shfl_sync(0xffffffffu, withhold, 0)) break;
    __syncwarp();
    const TcUnit un = sh.units[slot];
    if (!un.valid) break;
    if (!lane0_wait(&sh.q_empty, (k & 1) ^ 1)) break;
    if (lane == 0) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (un.n[x] == 0) continue;
        mbar_arrive_expect_tx(&sh.q_full[x], C::kHalves * a.tile_tokens * a.group * 128);
        ++q_armed[x];
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_3d(smem_base + C::kQOffset + x * C::kQBytes + hf * C::kQHalfBytes, qmap,
                      &sh.q_full[x], hf * 64, un.h * a.group, un.t0 + un.tok0 + a.tile_tokens * x);
      }
    }
    __syncwarp();
    if (!produce_tiles<HD, false, C::kStagesK>(g4, un, smem_ptr, sh.k_full, sh.k_empty, it, abort,
                                               lane))
      break;
    it += un.n_kt;
  }
  if (lane == 0 && *abort) {  // let the copies already issued land before the CTA can exit
    for (int x = 0; x < 2; ++x)
      if (q_armed[x]) mbar_wait_bounded(&sh.q_full[x], (q_armed[x] - 1) & 1, 100000000ull);
  }
}

// Warp 2: V.
template <int HD>
__device__ void producer_v4(const Kv4Args& g4, Kv4Shared& sh, uint8_t* smem_ptr) {
  using C = TcCfg<HD>;
  volatile int* abort = &sh.abort;
  const int lane = threadIdx.x & 31;
  uint32_t it = 0;
  for (int k = 0;; ++k) {
    const int slot = k % C::kRing;
    int ok = 1;
    if (lane == 0) ok = tc_wait(&sh.unit_full[slot], (k / C::kRing) & 1, abort, g4.a) ? 1 : 0;
    if (!__shfl_sync(0xffffffffu, ok, 0)) break;
    const TcUnit un = sh.units[slot];
    if (!un.valid) break;
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sh.unit_empty[slot]);  // the descriptor is in registers
    if (!produce_tiles<HD, true, C::kStagesV>(g4, un, smem_ptr + C::kVOffset, sh.v_full,
                                              sh.v_empty, it, abort, lane))
      break;
    it += un.n_kt;
  }
}

// The MMA issuer (one thread).  K and V are written by ordinary stores of other warps, which fence
// them for the tensor core before they arrive; the waits for them acquire.  P, O and S are tensor
// memory, ordered by tcgen05 fences, and their waits are relaxed (an acquiring wait behind queued
// MMAs idles the tensor pipe).
template <int HD>
__device__ void mma_issuer4(const AttnArgs& a, Kv4Shared& sh, uint32_t tmem, uint32_t smem_base) {
  using C = TcCfg<HD>;
  volatile int* abort = &sh.abort;
  constexpr uint32_t idesc_s = make_idesc_f16(128, 128, false);
  constexpr uint32_t idesc_o = make_idesc_f16(128, HD, true);
  uint32_t itk = 0, tcount[2] = {0, 0}, ucount[2] = {0, 0};
  bool issued = false;
  auto relaxed = [&](uint64_t* bar, uint32_t phase) {
    return mbar_test_relaxed(bar, phase) || tc_wait<true>(bar, phase, abort, a);
  };
  auto acquire = [&](uint64_t* bar, uint32_t phase) { return tc_wait(bar, phase, abort, a); };
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
  auto issue_s = [&](int x, uint32_t kt) {  // S_x = Q_x K^T
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
  auto issue_pv = [&](int x, uint32_t kt, bool first, bool last) {  // O_x (+)= P_x V
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
    if (!acquire(&sh.unit_full[slot], (k / C::kRing) & 1)) break;
    const TcUnit un = sh.units[slot];
    if (!un.valid) break;
    if (!acquire(&sh.k_full[itk % C::kStagesK], (itk / C::kStagesK) & 1)) break;
    bool ok = true;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (!ok || un.n[x] == 0) continue;
      if (!acquire(&sh.q_ready[x], ucount[x] & 1)) { ok = false; continue; }
      tc::fence_after_sync();
      issue_s(x, itk);
    }
    for (int j = 0; j < un.n_kt && ok; ++j) {
      const uint32_t kt = itk + j;
      bool k_ready = false, v_ready = false;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (j >= un.n[x]) continue;
        const bool next_s = j + 1 < un.n[x];
        const bool need_v = !v_ready, need_o = j == 0 && ucount[x] > 0, need_k = next_s && !k_ready;
        uint64_t* bar_v = &sh.v_full[kt % C::kStagesV];
        uint64_t* bar_k = &sh.k_full[(kt + 1) % C::kStagesK];
        const uint32_t ph_v = (kt / C::kStagesV) & 1, ph_k = ((kt + 1) / C::kStagesK) & 1;
        if ((need_v && !acquire(bar_v, ph_v)) || (need_k && !acquire(bar_k, ph_k)) ||
            (need_o && !relaxed(&sh.o_free[x], (ucount[x] - 1) & 1)) ||
            !relaxed(&sh.p_full[x], (tcount[x] + j) & 1)) {
          ok = false;
          break;
        }
        k_ready = k_ready || next_s;
        v_ready = true;
        tc::fence_after_sync();
        issue_pv(x, kt, j == 0, !next_s);
        if (next_s) issue_s(x, kt + 1);
      }
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

// Softmax and epilogue of tile x (0 = A, 1 = B); thread t = row t of the tile = TMEM lane t.  The
// reference and its rescaling are those of the ordinary launch (attn_prefill_tc.cu).
template <int HD>
__device__ void softmax_kv4(const Kv4Args& g4, Kv4Shared& sh, uint32_t tmem, uint8_t* smem_ptr,
                            int x) {
  using C = TcCfg<HD>;
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
    float scale = a.scale_log2;
    if (n > 0) {  // this row of Q to fp16, in place
      if (!wait_all(&sh.q_full[x], uc_x & 1)) break;
      uint8_t* row = smem_ptr + C::kQOffset + x * C::kQBytes + t * 128;
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
      scale *= up;
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
    // running reference (log2 domain) and sum; a row without a query starts at 0
    float m_ref = valid ? -INFINITY : 0.f, l = 0.f;
    for (int j = 0; j < n; ++j) {
      const uint32_t tj = tc_x + j;
      if (!wait_all(&sh.s_full[x], tj & 1)) { ok = false; break; }
      if (releases && t == 0) {
        const uint32_t kt = itk + j;
        tc::mbar_arrive(&sh.k_empty[kt % C::kStagesK]);
        if (j > 0) tc::mbar_arrive(&sh.v_empty[(kt - 1) % C::kStagesV]);
        if (j + 1 == n) tc::mbar_arrive(&sh.q_empty);
      }
      tc::fence_after_sync();
      float s[128];
      {
        uint32_t r0[32], r1[32], r2[32], r3[32];
        tc::ld32(col_s + 0, r0);
        tc::ld32(col_s + 32, r1);
        tc::ld32(col_s + 64, r2);
        tc::ld32(col_s + 96, r3);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          s[i] = __uint_as_float(r0[i]);
          s[32 + i] = __uint_as_float(r1[i]);
          s[64 + i] = __uint_as_float(r2[i]);
          s[96 + i] = __uint_as_float(r3[i]);
        }
      }
      const int kv_base = j * C::kN;
      if (partial || kv_base + C::kN - 1 > lim_min) {
#pragma unroll
        for (int i = 0; i < 128; ++i) s[i] = (kv_base + i <= lim) ? s[i] : -INFINITY;
      }
      auto take_tile_max = [&]() {
        float mx[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mx[i] = fmax3(s[i], s[8 + i], s[16 + i]);
#pragma unroll
        for (int g = 3; g + 1 < 16; g += 2)
#pragma unroll
          for (int i = 0; i < 8; ++i) mx[i] = fmax3(mx[i], s[8 * g + i], s[8 * g + 8 + i]);
#pragma unroll
        for (int i = 0; i < 8; ++i) mx[i] = fmaxf(mx[i], s[120 + i]);
        const float m_tile = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]),
                                   fmaxf(mx[6], mx[7])) *
                             scale;
        const bool need = m_tile > m_ref;
        if (__any_sync(0xffffffffu, need)) {
          const float m_new = need ? m_tile : m_ref;
          const float alpha = fast_exp2(m_ref - m_new);
          if (j > 0) {  // O holds P_{j-1} V_{j-1}: S_j, issued after it, has landed
            uint32_t r[32];
#pragma unroll
            for (int c = 0; c < HD / 32; ++c) {
              tc::ld32(col_o + c * 32, r);
              tc::wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
              tc::st32(col_o + c * 32, r);
            }
            tc::wait_st();
          }
          l *= alpha;
          m_ref = m_new;
        }
      };
      if (__any_sync(0xffffffffu, m_ref == -INFINITY)) take_tile_max();
      // exponents and the row sum two columns at a time; P (fp16) goes over the S columns
      auto exponents = [&]() -> float {
        const float mu = m_ref == -INFINITY ? 0.f : m_ref - kPShift;
        const float2 sc2 = make_float2(scale, scale), nmu2 = make_float2(-mu, -mu);
        float2 rs[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                        make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 e = __ffma2_rn(make_float2(s[c * 32 + 2 * i], s[c * 32 + 2 * i + 1]),
                                        sc2, nmu2);
            const float2 p = make_float2(fast_exp2(e.x), fast_exp2(e.y));
            rs[i & 3] = __fadd2_rn(rs[i & 3], p);
            pk[i] = kv4d::pack_f16x2(p.x, p.y);
          }
          tc::st16(col_s + c * 16, pk);
        }
        const float2 rs01 = __fadd2_rn(rs[0], rs[1]), rs23 = __fadd2_rn(rs[2], rs[3]);
        const float2 rsum = __fadd2_rn(rs01, rs23);
        return rsum.x + rsum.y;
      };
      float rsum = exponents();
      if (__any_sync(0xffffffffu, !(rsum <= kSumLimit))) {  // rare: re-reference this tile
        tc::wait_st();
        take_tile_max();
        rsum = exponents();
      }
      tc::wait_st();
      tc::fence_before_sync();
      arrive_warp(&sh.p_full[x]);
      l += rsum;
    }
    if (!ok) break;
    const uint32_t kt_last = itk + un.n_kt - 1;
    itk += un.n_kt;
    if (n > 0) {
      if (!wait_all(&sh.o_done[x], uc_x & 1)) break;  // the unit's last P V is in O
      if (releases && t == 0) tc::mbar_arrive(&sh.v_empty[kt_last % C::kStagesV]);
      ++uc_x;
      tc_x += n;
      tc::fence_after_sync();
      uint32_t o[HD];
#pragma unroll
      for (int c = 0; c < HD / 32; ++c)
        tc::ld32(col_o + c * 32, *reinterpret_cast<uint32_t(*)[32]>(o + c * 32));
      tc::wait_ld();
      tc::fence_before_sync();
      arrive_warp(&sh.o_free[x]);
      if (valid) {
        const float wa = l > 0.f ? g4.v_scale / l : l * 0.f;  // (NaN stays NaN)
        uint32_t pk[HD / 2];
#pragma unroll
        for (int i = 0; i < HD / 2; ++i)
          pk[i] = pack_bf16x2(__uint_as_float(o[2 * i]) * wa, __uint_as_float(o[2 * i + 1]) * wa);
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

template <int HD>
__global__ void __launch_bounds__(TcCfg<HD>::kThreads, 1)
    attn_kv4_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ Kv4Args g4) {
  using C = TcCfg<HD>;
  const AttnArgs& a = g4.a;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Kv4Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  if (tid == 32) prefetch_tmap(&qmap);
  if (tid == 0) {
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(&sh.unit_full[i], 1);
      mbar_init(&sh.unit_empty[i], 1 + 8 + 1);  // issuer, one lane of each softmax warp, V
    }
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
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_ready[i], 4);  // one lane of each softmax warp of the side
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.o_done[i], 1);
      mbar_init(&sh.o_free[i], 4);
    }
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    sh.role_rank = atomicAdd(a.header + kHRoleNext, 1);
    sh.decode_first = sh.role_rank < a.header[kHDecodeCtas];
    fence_barrier_init();
  }
  if (warp == C::kMmaWarp) {
    tc::tmem_alloc(&sh.tmem_base, C::kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem_base;

  // the planner's kind of work first, then the other; each register class in a loop of its own
  const bool decode_first = sh.decode_first != 0;
  auto phase_end = [] {
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
  };
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kControlRegs));
    for (int phase = 0; phase < 2; ++phase) {
      if ((phase == 0) != decode_first) {
        if (warp == C::kProducerWarp) {
          producer_qk4<HD>(g4, sh, base, base_ptr, &qmap);
        } else if (warp == C::kProducerVWarp) {
          producer_v4<HD>(g4, sh, base_ptr);
        } else if (warp == C::kMmaWarp) {
          if ((tid & 31) == 0) mma_issuer4<HD>(a, sh, tmem, base);
        }
      }
      phase_end();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    for (int phase = 0; phase < 2; ++phase) {
      if ((phase == 0) == decode_first)
        decode_warp_kv4<HD>(g4, decode_first ? sh.role_rank * a.decode_warps_per_cta + warp - 4
                                             : -1);
      else
        softmax_kv4<HD>(g4, sh, tmem, base_ptr, (warp >> 2) - 1);
      phase_end();
    }
  }
  if (warp == C::kMmaWarp) {
    __syncwarp();
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int HD>
rb_status launch_kv4(const Kv4Args& g4, const CUtensorMap& qmap, cudaStream_t s) {
  using C = TcCfg<HD>;
  static bool configured[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return RB_ERR_CUDA;
  if (!configured[dev]) {
    if (cudaFuncSetAttribute(attn_kv4_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmemBytes) != cudaSuccess)
      return RB_ERR_CUDA;
    configured[dev] = true;
  }
  attn_kv4_kernel<HD><<<max(1, device_sm_count()), C::kThreads, C::kSmemBytes, s>>>(qmap, g4);
  if (last_launch_status() != RB_OK) return RB_ERR_CUDA;
  note_launches(1);
  return RB_OK;
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
  if (!(softmax_scale > 0.f) || !std::isfinite(k_scale) || !std::isfinite(v_scale) ||
      !(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(scale) || !(scale > 0.f))
    return RB_ERR_INVALID_ARG;
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
