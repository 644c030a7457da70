// Prefill / chunk attention on the 5th-generation tensor cores (tcgen05 + TMEM).
//
// The same persistent launch also runs the split-KV decode units (attn_decode_warp.cuh): the
// planner assigns each CTA a first kind of work (decode or prefill) so HBM-bound and
// tensor-bound units run side by side; a CTA whose queue empties helps with the other one.
//
// Prefill unit = (request, kv head, pair of 128-row query tiles A and B); rows are (query token,
// head of the group) pairs, token-major, so every K/V tile serves the whole query-head group
// and both tiles of the pair.  A tile holds T = 128 / group whole tokens (T * group rows; for a
// group that does not divide 128 the last rows hold no query and are masked out).  One CTA per
// SM (persistent; units pulled from an atomic counter, the most expensive pair of each request
// first), 12 warps with fixed roles (the single-thread MMA issuer is warp 0, the oldest warp of
// its SM sub-partition, which shares that scheduler with one softmax warp of each tile):
//   warp 1     TMA producer of units, Q and K: fetches units into a 4-entry ring, loads Q_A and
//              Q_B once per unit (3-D boxes {64 dims, group heads, T tokens}) and each 128-key
//              K tile (8 pages x 128-byte boxes, 128B swizzle, one page per lane) into a
//              2-stage K ring (K is freed once S is done);
//   warp 2     TMA producer of V: the same boxes into a 3-stage V ring;
//   warp 0     allocates all 512 TMEM columns (S_A, S_B, O_A, O_B); one thread issues the MMAs
//              in the order S_A(0) S_B(0) | PV_A(0) S_A(1) | PV_B(0) S_B(1) | PV_A(1) ...
//              S = Q K^T: M=128, N=128, K=hd, both operands K-major in shared memory;
//              O += P V:  M=128, N=hd,  K=128, P read from TMEM, V MN-major in shared memory;
//              so one tile's softmax runs while the tensor core works on the other tile;
//   warps 4-7  softmax of tile A, warps 8-11 softmax of tile B; thread t = query row t: reads its
//              S row from TMEM, masks causally, takes exponents against a running reference
//              (log2 domain) and keeps their sum, writes P (bf16) back over the S columns.  The
//              reference is the row's first-tile maximum and moves (O rescaled in TMEM, the
//              tile's exponents taken again) only when a tile's sum exceeds 2^20 (exact either
//              way: P and the sum share the reference), so a common tile takes no row maximum.
//              The epilogue reads O, divides by the sum, stores bf16 rows.  The side that reads
//              every K/V tile of the unit (B, or A alone) hands the Q, K and V slots back to the
//              producers as its S tiles land, so the issuer commits only S, O and its drain.
// All mbarrier waits are bounded; a timeout sets RB_EBIT_TIMEOUT, every role stops, in-flight
// copies and MMAs are drained with bounded waits and TMEM is freed before the CTA exits.
#include "attn_prefill_tc.cuh"

namespace rb {
namespace attn {
namespace {

// Largest sum of one tile's exponents (128 keys of one row) taken against a lagging reference:
// P <= 2^20 keeps P V and the row sum far inside fp32 and bf16 range.
constexpr float kSumLimit = 1048576.f;

// Softmax and epilogue of tile x (0 = A, 1 = B); thread t = row t of the tile = TMEM lane t.
template <int HD>
__device__ void softmax_wg(const AttnArgs& a, TcShared<false>& sh, uint32_t tmem, uint8_t* smem_ptr,
                           int x) {
  using C = TcCfg<HD>;
  volatile int* abort = &sh.abort;
  const int t = threadIdx.x & 127;
  const uint32_t lane_off = static_cast<uint32_t>((t >> 5) * 32) << 16;
  const uint32_t col_s = tmem + lane_off + C::col_s(x), col_o = tmem + lane_off + C::col_o(x);
  uint32_t tc_x = 0, itk = 0, uc_x = 0;  // S tiles, K/V tiles and units (with n > 0) of this side
  auto wait_all = [&](uint64_t* bar, uint32_t phase) -> bool {
    const bool ok = tc_wait(bar, phase, abort, a);
    return !__any_sync(0xffffffffu, !ok);
  };
  // One lane of each warp arrives for the warp: 128 arrivals on one barrier load the barrier
  // unit that the MMA issuer's waits go through.
  const bool lane0 = (t & 31) == 0;
  auto arrive_warp = [&](uint64_t* bar) {
    __syncwarp();
    if (lane0) tc::mbar_arrive(bar);
  };
  // s_full of tile j tracks every MMA issued before S_j, P V of tile j - 1 among them; o_done
  // completes once per unit of this side, after its last P V.
  for (int k = 0;; ++k) {
    const int slot = k % C::kRing;
    if (!wait_all(&sh.unit_full[slot], (k / C::kRing) & 1)) break;
    const TcUnit un = sh.units[slot];
    if (!un.valid) break;
    const int n = un.n[x];
    // row t of this tile: token tok_base + t / group, head t % group of the kv head's group;
    // rows past T * group (a group that does not divide 128) or past the last token hold no
    // query: every key is masked for them and they are never stored
    const int tok_base = un.tok0 + a.tile_tokens * x;
    const int rows_used = a.tile_tokens * a.group;
    const int jt_in = t / a.group;
    const bool valid = t < rows_used && tok_base + jt_in < un.q;
    const int jt = valid ? tok_base + jt_in : 0;
    const int hh = valid ? t - jt_in * a.group : 0;
    const bool causal = a.cascade != kPrefixPass;
    const int lim = !valid ? -1 : (causal ? un.c + jt : un.c);
    const int lim_min = causal ? un.c + tok_base : un.c;
    const bool partial = rows_used < C::kM || tok_base + a.tile_tokens > un.q;
    // The side that reads every K/V tile of the unit (B, or A when B is empty: B's rows come
    // later, so it sees at least A's keys) hands the Q, K and V slots back to the producers:
    // its S of tile j landing means every MMA issued before that S has completed, S_A of tile
    // j and both P V of tile j - 1 among them; its last P V landing (o_done) frees the last V.
    // This keeps those arrivals off the MMA issuer, whose commits are its critical path.
    const bool releases = x == (un.n[1] > 0 ? 1 : 0);
    // running reference (log2 domain) and sum; a row without a query starts at 0, so that only
    // rows with visible keys take the first tile's maximum
    float m_ref = valid ? -INFINITY : 0.f, l = 0.f;
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
      // The exponents are taken against the running reference m_ref, not against this tile's
      // maximum: any reference gives the same softmax, since P and the sum share it.  The row
      // maximum is taken only (a) on the first tile of a row and (b) when the tile's sum of
      // exponents shows the reference lagging the row's maximum by more than log2 of
      // kSumLimit (or overflowing); then O and the sum are rescaled to the new reference and
      // the tile's exponents are taken again.  So P <= kSumLimit always, and the common tile
      // skips the maximum over its 128 columns.
      auto take_tile_max = [&]() {
        // eight running maxima over the 16 groups of 8 columns, three-input max instructions
        float mx[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mx[k] = fmax3(s[k], s[8 + k], s[16 + k]);
#pragma unroll
        for (int g = 3; g + 1 < 16; g += 2)
#pragma unroll
          for (int k = 0; k < 8; ++k) mx[k] = fmax3(mx[k], s[8 * g + k], s[8 * g + 8 + k]);
#pragma unroll
        for (int k = 0; k < 8; ++k) mx[k] = fmaxf(mx[k], s[120 + k]);
        // scores are scaled inside the exponent: max and mask commute with a positive scale
        const float m_tile = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]),
                                   fmaxf(mx[6], mx[7])) *
                             a.scale_log2;
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
      // keys at or past the end of the sequence may hold anything: zero their V rows (only the
      // unit's last K/V tile can reach them; tile A zeroes it when it uses that tile)
      if (kv_base + C::kN > un.L && (x == 0 || j >= un.n[0])) {
        const uint32_t kt = itk + j, sv = kt % C::kStagesV;
        if (!wait_all(&sh.v_full[sv], (kt / C::kStagesV) & 1)) { ok = false; break; }
        const int kmin = max(un.L - kv_base, 0);
        if (t >= kmin) {
          uint8_t* vrow = smem_ptr + C::kVOffset + sv * C::kTileBytes + t * 128;
#pragma unroll
          for (int hf = 0; hf < C::kHalves; ++hf)
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<uint4*>(vrow + hf * C::kHalfBytes + c * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
        }
      }
      // exponents and the row sum two columns at a time with the paired fp32 FMA / add
      // instructions; P (bf16) goes over the S columns
      auto exponents = [&]() -> float {
        const float mu = m_ref == -INFINITY ? 0.f : m_ref;
        const float2 sc2 = make_float2(a.scale_log2, a.scale_log2), nmu2 = make_float2(-mu, -mu);
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
            pk[i] = pack_bf16x2(p.x, p.y);
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
      // P_j overwrites the S columns P_{j-1} V_{j-1} read: that product is done, since S_j (the
      // MMA after it) has landed
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
      // the whole O row into registers at once; O is then free for the next unit's P V while
      // this row is scaled and stored
      uint32_t o[HD];
#pragma unroll
      for (int c = 0; c < HD / 32; ++c)
        tc::ld32(col_o + c * 32, *reinterpret_cast<uint32_t(*)[32]>(o + c * 32));
      tc::wait_ld();
      tc::fence_before_sync();
      arrive_warp(&sh.o_free[x]);
      const size_t orow = static_cast<size_t>(un.t0 + jt) * a.nh + un.h * a.group + hh;
      // rows are written with 32-byte stores when the output is 32-byte aligned (a warp's
      // rows are scattered: fewer, whole-sector stores), else 16-byte ones
      if (a.cascade == kPrefixPass) {
        // shared-prefix row: normalised fp32 output and its log-sum-exp, merged later
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const size_t prow = static_cast<size_t>(un.r) * a.N * a.nh + orow;
        float* dst = a.pre_o + prow * HD;
        if (valid) {
#pragma unroll
          for (int i = 0; i < HD; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
          if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
#pragma unroll
            for (int v = 0; v < HD / 8; ++v)
              st_global_v8(dst + 8 * v, o[8 * v], o[8 * v + 1], o[8 * v + 2], o[8 * v + 3],
                           o[8 * v + 4], o[8 * v + 5], o[8 * v + 6], o[8 * v + 7]);
          } else {
#pragma unroll
            for (int v = 0; v < HD / 4; ++v)
              reinterpret_cast<uint4*>(dst)[v] = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
          }
          a.pre_lse[prow] = l > 0.f ? m_ref + __log2f(l) : -INFINITY;
        }
      } else if (valid) {
        // out = O * wa + sum over prefix key ranges of (shared-prefix row) * wp (cascade only)
        float wa = 1.f / l;
        float wp[kMaxPrefixSplits];
        const bool cas = a.cascade == kSuffixPass;
        if (cas) wa = cascade_weights(a, orow, m_ref, l, wp);
        else if (!(l > 0.f)) wa = 0.f;
#pragma unroll
        for (int i = 0; i < HD; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * wa);
        if (cas) {
#pragma unroll
          for (int ps = 0; ps < kMaxPrefixSplits; ++ps) {
            if (ps >= a.prefix_splits) break;
            const float4* o1 = reinterpret_cast<const float4*>(cascade_row<HD>(a, ps, orow));
#pragma unroll
            for (int v = 0; v < HD / 4; ++v) {
              const float4 e = __ldg(o1 + v);
              o[4 * v + 0] = __float_as_uint(__uint_as_float(o[4 * v + 0]) + e.x * wp[ps]);
              o[4 * v + 1] = __float_as_uint(__uint_as_float(o[4 * v + 1]) + e.y * wp[ps]);
              o[4 * v + 2] = __float_as_uint(__uint_as_float(o[4 * v + 2]) + e.z * wp[ps]);
              o[4 * v + 3] = __float_as_uint(__uint_as_float(o[4 * v + 3]) + e.w * wp[ps]);
            }
          }
        }
        uint32_t pk[HD / 2];
#pragma unroll
        for (int i = 0; i < HD / 2; ++i)
          pk[i] = pack_bf16x2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
        __nv_bfloat16* dst = a.out + orow * HD;
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
    attn_prefill_tc_kernel(const __grid_constant__ CUtensorMap qmap,
                           const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap, const AttnArgs a) {
  using C = TcCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ TcShared<false> sh;
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

  // Two phases: the kind of work the planner assigned this CTA first, then the other kind
  // until its queue is empty too.  The decode phase runs on warps 4-11, each with its own ring of
  // decode stages in the same shared memory the prefill phase uses.  Each register class keeps
  // its own loop so the code after setmaxnreg stays within that class's budget.
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
          producer_qk<HD, false>(a, sh, base, &qmap, &kmap);
        } else if (warp == C::kProducerVWarp) {
          producer_v<HD, false>(a, sh, base, &vmap);
        } else if (warp == C::kMmaWarp) {
          if ((tid & 31) == 0) mma_issuer<HD, false>(a, sh, tmem, base);
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
        decode_warp<HD>(&kmap, &vmap, a, sh.dec_bars[w], base + w * D::kStages * D::kStageBytes,
                        base_ptr + w * D::kStages * D::kStageBytes,
                        decode_first ? sh.role_rank * a.decode_warps_per_cta + w : -1);
      } else {
        softmax_wg<HD>(a, sh, tmem, base_ptr, (warp >> 2) - 1);
      }
      phase_end();
    }
  }
  if (warp == C::kMmaWarp) {
    __syncwarp();
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int HD>
rb_status launch_hd(const AttnArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                    const CUtensorMap& vmap, cudaStream_t s) {
  using C = TcCfg<HD>;
  static bool configured[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return RB_ERR_CUDA;
  if (!configured[dev]) {
    if (cudaFuncSetAttribute(attn_prefill_tc_kernel<HD>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmemBytes) != cudaSuccess)
      return RB_ERR_CUDA;
    configured[dev] = true;
  }
  const int grid = max(1, device_sm_count());
  attn_prefill_tc_kernel<HD><<<grid, C::kThreads, C::kSmemBytes, s>>>(qmap, kmap, vmap, a);
  if (last_launch_status() != RB_OK) return RB_ERR_CUDA;
  note_launches(1);
  return RB_OK;
}

}  // namespace

rb_status launch_prefill_tc(const AttnArgs& a, int head_dim, const CUtensorMap& qmap,
                            const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t s) {
  if (is_scored(a.rules)) return launch_scored_tc(a, head_dim, qmap, kmap, vmap, s);
  return head_dim == 128 ? launch_hd<128>(a, qmap, kmap, vmap, s)
                         : launch_hd<64>(a, qmap, kmap, vmap, s);
}

}  // namespace attn
}  // namespace rb
