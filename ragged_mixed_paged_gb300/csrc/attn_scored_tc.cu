// The fused attention launch with score rules (rb_paged_attention_scored): capped scores, a bias
// that falls with distance, and a key range [lo, hi) per query token.
//
// Units, roles, producers and MMA issuer are those of the ordinary launch (attn_prefill_tc.cu);
// key tiles are taken last to first (ScoredUnit).  The softmax differs.  A ruled score costs up
// to four more multiply-adds, and straight-line code for a row's 128 scores ran at the rate of
// instruction fetch: a third of an instruction per cycle and scheduler, with 8 softmax warps and
// with 16 alike, and the same loop of 16 columns unrolled is a quarter slower than rolled.  So a
// row's scores are read from tensor memory 64 columns at a time by a loop of two rounds, and P
// goes over columns already read.  A score above the running reference by more than kGrowth is met
// when its columns are read: reference, sum, O and the row's P so far then move by a power of
// two, which is exact in bf16.
//
// What bounds this form is the chain of a side's tile: S lands, softmax, P stored, P V and the
// next S issued, each waiting for all 128 columns of the one before.  On four chunks of 1024 over
// 4096 cached tokens nothing is busy half the time (tensor pipe 47 % without a rule, 37 capped, 40
// biased; issue slots 32 to 37 %), and warps wait for data (long scoreboard, 2.2 to 3.1 per
// instruction issued) far more than for instructions (0.5 to 0.6).
//
// Measured on four chunks of 1-2 k tokens over up to 16 k cached ones (32 / 8 heads of 128; the
// ordinary launch 646 us, 0.74 of the bf16 rate): no rule 710 us, soft cap 925, distance bias 854.
// With all 128 scores kept in registers and the maximum taken once per tile: 695, 1102, 828; in
// rounds of 16 columns 961, 1037, 1064; of 32 763, 949, 892; with the next columns' loads ahead of
// the current ones' work (twice the code) 850, 992, 985 for 32.
#include <type_traits>

#include "attn_prefill_tc.cuh"

namespace rb {
namespace attn {
namespace {

// How far (log2 units) a score may lie above its row's reference.
constexpr float kGrowth = 20.f;
// Capped scores lie within +-cap_log2 (a bias that falls with distance only lowers them), so up to
// kMaxBoundedCap a row needs no maximum.  Its reference starts where a score of -cap_log2, the least
// that a row's largest can be (biased: its own key's, if it sees that one), weighs 2^-31 or more and
// one of +cap_log2 at most 2^118, and rises by a power of two when a tile's 128 columns sum to more
// than 2^kGrowth.  So the weights that O takes neither vanish nor, tile by tile, sum to more than
// that, whichever end of the cap a row's scores lie at.  (A reference that never moved had V up to
// 2^80 and down to 2^-26 at the ends of a cap of 50; the check costs 3 %, 900 -> 925 us below.)
constexpr float kMaxBoundedCap = 74.f, kCapLow = 30.f;
constexpr float kLargeSum = 1048576.f;  // 2^kGrowth
constexpr int kCols = 64;  // columns taken at a time

// Softmax and epilogue of tile x (0 = A, 1 = B); thread t = row t of the tile = TMEM lane t.
template <int HD, int kRules>
__device__ void softmax_scored(const AttnArgs& a, TcShared<true>& sh, uint32_t tmem,
                               uint8_t* smem_ptr, int x) {
  using C = TcCfg<HD>;
  constexpr bool kCap = (kRules & kCapped) != 0, kBias = (kRules & kBiased) != 0;
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
  // factors as register pairs (two-at-a-time instructions take no operand from constant memory;
  // the empty asm keeps them from being fetched again per use)
  auto pair_of = [](float v) {
    float2 p = make_float2(v, v);
    asm volatile("" : "+f"(p.x), "+f"(p.y));
    return p;
  };
  float2 scale2 = make_float2(0.f, 0.f), cap2[4];
  if constexpr (kCap) {
#pragma unroll
    for (int k = 0; k < 4; ++k) cap2[k] = pair_of(a.cap_poly[k]);
  } else {
    scale2 = pair_of(a.scale_log2);
  }
  for (int k = 0;; ++k) {
    const int slot = k % C::kRing;
    if (!wait_all(&sh.unit_full[slot], (k / C::kRing) & 1)) break;
    const ScoredUnit un = sh.units[slot];
    if (!un.valid) break;
    const int n = un.n[x];
    // row t of this tile: token tok_base + t / group, head t % group of the kv head's group;
    // rows past T * group (a group that does not divide 128) or past the last token hold no
    // query: they may compute anything, have no say in the warp's votes and are never stored
    const int tok_base = un.tok0 + a.tile_tokens * x;
    const int rows_used = a.tile_tokens * a.group;
    const int jt_in = t / a.group;
    const bool valid = t < rows_used && tok_base + jt_in < un.q;
    const int jt = valid ? tok_base + jt_in : 0;
    const int hh = valid ? t - jt_in * a.group : 0;
    const int pos = un.c + jt;
    // the row's keys [lo, hi), its slope, and the smallest hi of the tile's rows
    int lo = 0, hi = 0;
    bool blind = false;
    float slope = 0.f;
    if (valid) {
      lo = key_lo(a, un.t0 + jt);
      hi = max(pos + 1, un.prefix);
      // A row that sees no key takes the unit's keys as its own, so that it does not make every
      // tile a masked one, and writes zeros in the end.
      if (lo >= hi) {
        blind = true;
        lo = 0;
      }
      if constexpr (kBias) slope = __ldg(a.slopes + un.h * a.group + hh) * 1.4426950408889634f;
    }
    const int hi_min = max(un.c + tok_base + 1, un.prefix);
    bool bounded = false;
    if constexpr (kCap) {
      bounded = a.cap_log2 <= kMaxBoundedCap;
      if constexpr (kBias)
        bounded = bounded && __all_sync(0xffffffffu, slope >= 0.f && lo <= pos);
    }
    // The side that reads the unit's K/V tiles last (B, or A when B is empty) hands the Q, K and
    // V slots back to the producers as its S tiles land.
    const bool releases = x == (un.n[1] > 0 ? 1 : 0);
    // Running reference (log2 units, a whole number) and sum.  A row that has seen no key is at
    // -inf (or where it starts); one without a query stays at +inf, where no score moves it.
    // (Masking such rows' keys made every tile of a group like 6 or 7 a masked one: prompts of 300
    // to 1500 tokens with 12 / 2 heads of 64 and a bias 97 us, so 83.)
    const float cap_s = valid ? a.cap_s : INFINITY;
    float m_ref = !valid    ? INFINITY
                  : bounded ? ceilf(fminf(a.cap_log2, kCapLow - a.cap_log2))
                            : -INFINITY;
    float l = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const uint32_t tj = tc_x + j;
      if (!wait_all(&sh.s_full[x], tj & 1)) { ok = false; break; }
      if (releases && t == 0) {
        const uint32_t kt = itk + j;
        tc::mbar_arrive(&sh.k_empty[kt % C::kStagesK]);
        if (j > 0) tc::mbar_arrive(&sh.v_empty[(kt - 1) % C::kStagesV]);
        if (j + 1 == n) tc::mbar_arrive(&sh.q_empty);
      }
      const int kv_base = (un.j0 + n - 1 - j) * C::kN;  // first key of the tile
      {
        // V of the tile, by tile A for both sides: keys at or past the end of the sequence and
        // before the unit's first visible one may hold anything (zeroed); of keys that some rows
        // of the unit see and others do not, what is not finite is taken out and noted.
        const bool unknown = kv_base + C::kN > un.L || kv_base < un.lo;
        const bool mixed = kv_base < max(un.lo_max[0], un.lo_max[1]) ||
                           kv_base + C::kN > max(un.c + un.tok0 + 1, un.prefix);
        if (x == 0 && (unknown || mixed)) {
          const uint32_t kt = itk + j, sv = kt % C::kStagesV;
          if (!wait_all(&sh.v_full[sv], (kt / C::kStagesV) & 1)) { ok = false; break; }
          uint8_t* v = smem_ptr + C::kVOffset + sv * C::kTileBytes;
          if (t >= un.L - kv_base || t < un.lo - kv_base) {
#pragma unroll 1
            for (int hf = 0; hf < C::kHalves; ++hf)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4*>(v + hf * C::kHalfBytes + t * 128 + c * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
          }
          if (mixed) {  // this warp's 32 keys, 512 bytes at a time
            __syncwarp();
            bool odd = false;
            for (int hf = 0; hf < C::kHalves; ++hf)
              odd |= take_out_not_finite(v + hf * C::kHalfBytes + (t >> 5) * 32 * 128, 8, 512);
            if (odd && lane0) {
              atomicMin(&sh.units[slot].odd_first, kv_base / C::kN);
              atomicMax(&sh.units[slot].odd_last, kv_base / C::kN);
              __threadfence_block();
            }
          }
        }
      }
      tc::fence_after_sync();
      const bool masked = kv_base < un.lo_max[x] || kv_base + C::kN > hi_min;
      // a key past its query, where the distance changes sign, needs |p - k| taken
      const bool past = kBias && kv_base + C::kN > un.c + tok_base + 1;
      const unsigned seen0 = static_cast<unsigned>(kv_base - lo), n_seen = hi - lo;
      float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};

      // Multiplies what the warp's rows took before round c by alpha (1: a row that stays).
      auto rescale = [&](float alpha, int c) {
        tc::wait_st();
#pragma unroll 1
        for (int p = 0; p < c * (kCols / 32); ++p) {  // P of the rounds before
          uint32_t r[16];
          tc::ld16(col_s + p * 16, r);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            r[i] = pack_bf16x2(__uint_as_float(r[i] << 16) * alpha,
                               __uint_as_float(r[i] & 0xffff0000u) * alpha);
          tc::st16(col_s + p * 16, r);
        }
        if (j > 0) {  // O holds P_{j-1} V_{j-1}: S_j, issued after it, has landed
#pragma unroll 1
          for (int p = 0; p < HD / 16; ++p) {
            uint32_t r[16];
            tc::ld16(col_o + p * 16, r);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
            tc::st16(col_o + p * 16, r);
          }
        }
        tc::wait_st();
        l *= alpha;
        rs[0] = __fmul2_rn(rs[0], make_float2(alpha, alpha));
        rs[1] = __fmul2_rn(rs[1], make_float2(alpha, alpha));
      };
      // Raises the reference above `top`, the largest of a row's scores in round c, for the rows
      // of the warp that need it.
      auto move_reference = [&](float top, int c) {
        const bool need = top > m_ref + kGrowth;
        const float m_new = need ? ceilf(top) : m_ref;
        // (-inf before the first key: alpha 0)
        rescale(need ? fast_exp2(m_ref - m_new) : 1.f, c);
        m_ref = m_new;
      };
#pragma unroll 1
      for (int c = 0; c < C::kN / kCols; ++c) {
        // columns kCols c ..: raw scores
        float s[kCols];
        {
          uint32_t r0[32], r1[32];
          tc::ld32(col_s + c * kCols, r0);
          tc::ld32(col_s + c * kCols + 32, r1);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            s[i] = __uint_as_float(r0[i]);
            s[32 + i] = __uint_as_float(r1[i]);
          }
        }
        bool plain_cap = false;  // capped by the polynomial, against a fixed reference
        if constexpr (kCap) {
          float top = fmaxf(fabsf(s[0]), fabsf(s[1]));
#pragma unroll
          for (int i = 2; i < kCols; i += 2) top = fmax3(top, fabsf(s[i]), fabsf(s[i + 1]));
          plain_cap = bounded && !__any_sync(0xffffffffu, top > cap_s);
        }
        float b[kCols];  // bias, less the reference where that is fixed
        if constexpr (kBias) {
          const float d0 = static_cast<float>(kv_base + kCols * c - pos);
          const float add = plain_cap ? -m_ref : 0.f;
          if (past) {
#pragma unroll
            for (int i = 0; i < kCols; ++i)
              b[i] = fmaf(-slope, fabsf(d0 + static_cast<float>(i)), add);
          } else {  // every key at or before the row's own: slope * (k - p)
            const float b0 = fmaf(slope, d0, add);
#pragma unroll
            for (int i = 0; i < kCols; ++i) b[i] = fmaf(slope, static_cast<float>(i), b0);
          }
        }
        auto mask = [&]() {
#pragma unroll
          for (int i = 0; i < kCols; ++i)
            s[i] = seen0 + kCols * c + i < n_seen ? s[i] : -INFINITY;
        };
        // s: the exponents
        if (kCap && plain_cap) {
#pragma unroll
          for (int i = 0; i < kCols; i += 2) {
            const float2 y = make_float2(s[i], s[i + 1]), z = __fmul2_rn(y, y);
            float2 f = __ffma2_rn(cap2[3], z, cap2[2]);
            f = __ffma2_rn(f, z, cap2[1]);
            f = __ffma2_rn(f, z, cap2[0]);
            const float2 e = __ffma2_rn(y, f, kBias ? make_float2(b[i], b[i + 1])
                                                    : make_float2(-m_ref, -m_ref));
            s[i] = e.x;
            s[i + 1] = e.y;
          }
          if (masked) mask();
        } else {
          // ruled scores in log2 units (kMasked: raw), masked, then less a reference that may have
          // to move
          if constexpr (kCap) {
            cap_scores(a, s);
            if constexpr (kBias) {
#pragma unroll
              for (int i = 0; i < kCols; ++i) s[i] += b[i];
            }
          } else if constexpr (kBias) {
#pragma unroll
            for (int i = 0; i < kCols; i += 2) {
              const float2 y = __ffma2_rn(make_float2(s[i], s[i + 1]), scale2,
                                          make_float2(b[i], b[i + 1]));
              s[i] = y.x;
              s[i + 1] = y.y;
            }
          }
          if (masked) mask();
          if (!(kCap && bounded)) {
            float top = fmaxf(s[0], s[1]);
#pragma unroll
            for (int i = 2; i < kCols; i += 2) top = fmax3(top, s[i], s[i + 1]);
            if constexpr (kRules == kMasked) top *= a.scale_log2;
            if (__builtin_expect(__any_sync(0xffffffffu, top > m_ref + kGrowth), 0))
              move_reference(top, c);
          }
          const float mu = m_ref == -INFINITY ? 0.f : m_ref;
          const float2 nmu2 = make_float2(-mu, -mu);
#pragma unroll
          for (int i = 0; i < kCols; i += 2) {
            const float2 y = make_float2(s[i], s[i + 1]);
            const float2 e = kRules == kMasked ? __ffma2_rn(y, scale2, nmu2) : __fadd2_rn(y, nmu2);
            s[i] = e.x;
            s[i + 1] = e.y;
          }
        }
        uint32_t pk[kCols / 2];
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) {
          const float2 p = make_float2(fast_exp2(s[2 * i]), fast_exp2(s[2 * i + 1]));
          rs[i & 1] = __fadd2_rn(rs[i & 1], p);
          pk[i] = pack_bf16x2(p.x, p.y);
        }
        tc::st32(col_s + c * (kCols / 2), pk);
      }
      tc::wait_st();
      float2 r = __fadd2_rn(rs[0], rs[1]);
      if (kCap && bounded) {
        const float sum = r.x + r.y;
        const bool need = sum > kLargeSum;
        if (__builtin_expect(__any_sync(0xffffffffu, need), 0)) {
          // by the sum's power of two, at most 2^125
          const int up = need ? (__float_as_int(sum) >> 23) - 127 : 0;
          const float alpha = __int_as_float((127 - up) << 23);
          rescale(alpha, C::kN / kCols);
          r = __fmul2_rn(r, make_float2(alpha, alpha));
          m_ref += static_cast<float>(up);
        }
      }
      // P_j overwrites the S columns P_{j-1} V_{j-1} read: that product is done, since S_j (the
      // MMA after it) has landed
      tc::fence_before_sync();
      arrive_warp(&sh.p_full[x]);
      l += r.x + r.y;
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
      // the whole O row into registers at once; O is then free for the next unit's P V while
      // this row is scaled and stored
      uint32_t o[HD];
#pragma unroll
      for (int c = 0; c < HD / 32; ++c)
        tc::ld32(col_o + c * 32, *reinterpret_cast<uint32_t(*)[32]>(o + c * 32));
      tc::wait_ld();
      tc::fence_before_sync();
      arrive_warp(&sh.o_free[x]);
      if (valid) {
        const float w = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // (a NaN sum stays one)
        uint32_t pk[HD / 2];
#pragma unroll
        for (int i = 0; i < HD / 2; ++i)
          pk[i] = blind ? 0u
                        : pack_bf16x2(__uint_as_float(o[2 * i]) * w,
                                      __uint_as_float(o[2 * i + 1]) * w);
        __nv_bfloat16* dst =
            a.out + (static_cast<size_t>(un.t0 + jt) * a.nh + un.h * a.group + hh) * HD;
        // 32-byte stores when the output is 32-byte aligned, else 16-byte ones
        if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
#pragma unroll
          for (int v = 0; v < HD / 16; ++v)
            st_global_v8(dst + 16 * v, pk[8 * v], pk[8 * v + 1], pk[8 * v + 2], pk[8 * v + 3],
                         pk[8 * v + 4], pk[8 * v + 5], pk[8 * v + 6], pk[8 * v + 7]);
        } else {
#pragma unroll
          for (int v = 0; v < HD / 8; ++v)
            reinterpret_cast<uint4*>(dst)[v] =
                make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
        }
        // V's infinities and NaN that were taken out
        const volatile auto& now = sh.units[slot];
        if (now.odd_last >= 0 && !blind)
          add_not_finite(a, un.r, un.h, max(lo, now.odd_first * C::kN),
                         min(hi, (now.odd_last + 1) * C::kN), HD, dst);
      }
    }
    arrive_warp(&sh.unit_empty[slot]);
  }
}

template <int HD, int kRules>
__global__ void __launch_bounds__(TcCfg<HD>::kThreads, 1)
    attn_scored_tc_kernel(const __grid_constant__ CUtensorMap qmap,
                          const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap, const AttnArgs a) {
  using C = TcCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ TcShared<true> sh;
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  if (tid == 32) {  // the three descriptors every role's first copies use
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  if (tid == 0) {
    init_barriers<HD>(sh);
    fence_barrier_init();
  }
  if (warp == C::kMmaWarp) {
    tc::tmem_alloc(&sh.tmem_base, C::kTmemCols);
    tc::tmem_relinquish();
  }
  grid_wait();  // launched beside the planner: its results from here on
  if (tid == 0) {
    sh.role_rank = atomicAdd(a.header + kHRoleNext, 1);
    sh.decode_first = sh.role_rank < a.header[kHDecodeCtas];
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem_base;

  // Two phases, as in the ordinary launch: the kind of work the planner assigned this CTA, then
  // the other kind until its queue is empty too.  Decode runs on warps 4-11.
  const bool decode_first = sh.decode_first != 0;
  auto phase_end = [] {
    fence_proxy_async_smem();  // generic smem traffic of this phase before the next one's TMA
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
  };
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kControlRegs));
    for (int phase = 0; phase < 2; ++phase) {
      if ((phase == 0) != decode_first) {
        if (warp == C::kProducerWarp) {
          producer_qk<HD, true>(a, sh, base, &qmap, &kmap);
        } else if (warp == C::kProducerVWarp) {
          producer_v<HD, true>(a, sh, base, &vmap);
        } else if (warp == C::kMmaWarp) {
          if ((tid & 31) == 0) mma_issuer<HD, true>(a, sh, tmem, base);
        }
      }
      phase_end();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    for (int phase = 0; phase < 2; ++phase) {
      if ((phase == 0) == decode_first) {
        using D = DecCfg<HD>;
        const int w = warp - 4;
        // a decode-first CTA's warps start on units rank x 8 + w without the counter
        decode_warp<HD, kRules>(&kmap, &vmap, a, sh.dec_bars[w],
                                base + w * D::kStages * D::kStageBytes,
                                base_ptr + w * D::kStages * D::kStageBytes,
                                decode_first ? sh.role_rank * a.decode_warps_per_cta + w : -1);
      } else {
        softmax_scored<HD, kRules>(a, sh, tmem, base_ptr, (warp >> 2) - 1);
      }
      phase_end();
    }
  }
  if (warp == C::kMmaWarp) {
    __syncwarp();
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int HD, int kRules>
rb_status launch_rules(const AttnArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                       const CUtensorMap& vmap, cudaStream_t s) {
  using C = TcCfg<HD>;
  static bool configured[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return RB_ERR_CUDA;
  if (!configured[dev]) {
    if (cudaFuncSetAttribute(attn_scored_tc_kernel<HD, kRules>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmemBytes) != cudaSuccess)
      return RB_ERR_CUDA;
    configured[dev] = true;
  }
  return launch_overlapped(attn_scored_tc_kernel<HD, kRules>, max(1, device_sm_count()),
                           C::kThreads, C::kSmemBytes, s, qmap, kmap, vmap, a);
}

}  // namespace

rb_status launch_scored_tc(const AttnArgs& a, int head_dim, const CUtensorMap& qmap,
                           const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t s) {
  auto launch = [&](auto rules) {
    constexpr int kRules = decltype(rules)::value;
    return head_dim == 128 ? launch_rules<128, kRules>(a, qmap, kmap, vmap, s)
                           : launch_rules<64, kRules>(a, qmap, kmap, vmap, s);
  };
  switch (a.rules) {
    case kMasked: return launch(std::integral_constant<int, kMasked>{});
    case kMasked | kCapped: return launch(std::integral_constant<int, kMasked | kCapped>{});
    case kMasked | kBiased: return launch(std::integral_constant<int, kMasked | kBiased>{});
    default: return launch(std::integral_constant<int, kMasked | kCapped | kBiased>{});
  }
}

}  // namespace attn
}  // namespace rb
