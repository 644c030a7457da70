// Shared definitions of the paged-attention kernels (planner, split-KV decode, prefill tiles,
// split combine).  Not part of the C ABI.
#pragma once

#include "rb_internal.cuh"

namespace rb {
namespace attn {

constexpr int kMaxCols = 8;          // decode columns: (query token, head of the group) pairs
constexpr int kMaxTargetUnits = 8192;
constexpr int kMinSplitPages = 8;
constexpr int kPage = 16;            // tokens per KV page (the only page size these kernels take)

enum HeaderField : int {
  kHNumDecodeUnits = 0,
  kHNumPrefillUnits = 1,
  kHDecodeNext = 2,
  kHPrefillNext = 3,
  kHSplitPages = 4,
  kHDecodeCtas = 5,  // fused kernel: CTAs that start on decode units
  kHRoleNext = 6,    // fused kernel: role ticket counter
  kHeaderInts = 32
};

// Workspace: [header][decode unit offsets R+1][prefill unit offsets R+1]
//            [finished-split counters R x nkv][prefill pair list][partial (m, l)][partial o]
struct WsLayout {
  size_t header, dec_off, pre_off, done, pre_list, part_ml, part_o, total;
  long long max_units;
};

// Prefill (request, tile pair) entries a batch can have: a pair covers 2 * (128 / group) >= 16
// query tokens for groups up to 16, so sum over requests of ceil(q_i / pair tokens)
// <= N / 16 + R.
__host__ __device__ inline long long max_prefill_pairs(int num_reqs, int num_tokens) {
  return static_cast<long long>(num_tokens) / 16 + num_reqs + 1;
}

inline WsLayout ws_layout(int head_dim, int num_kv_heads, int num_reqs, int num_tokens) {
  WsLayout w{};
  size_t off = 0;
  auto take = [&off](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) & ~static_cast<size_t>(255);
    return o;
  };
  w.max_units = kMaxTargetUnits + static_cast<long long>(num_kv_heads) * num_reqs;
  w.header = take(kHeaderInts * sizeof(int32_t));
  w.dec_off = take(static_cast<size_t>(num_reqs + 1) * sizeof(int32_t));
  w.pre_off = take(static_cast<size_t>(num_reqs + 1) * sizeof(int32_t));
  w.done = take(static_cast<size_t>(num_reqs) * num_kv_heads * sizeof(int32_t));
  w.pre_list = take(static_cast<size_t>(max_prefill_pairs(num_reqs, num_tokens)) * sizeof(int32_t));
  w.part_ml = take(static_cast<size_t>(w.max_units) * kMaxCols * sizeof(float2));
  w.part_o = take(static_cast<size_t>(w.max_units) * kMaxCols * head_dim * sizeof(float));
  w.total = off;
  return w;
}

// Cascade attention ("第8章 ModelRunner…", "8.3.2.5 Cascade Attention"): a prefix pass runs every
// query row against the P keys all requests share (no mask: P <= every request's cached
// length), a suffix pass runs the ordinary causal attention over keys [P, seq_len) and merges
// the prefix result into each row by log-sum-exp before the single bf16 rounding.
enum CascadePass : int { kNoCascade = 0, kPrefixPass = 1, kSuffixPass = 2 };
constexpr int kMaxPrefixSplits = 4;  // the prefix keys may be cut into this many ranges

// Extra workspace of a cascade call, after the ordinary layout: shifted sequence lengths and,
// per prefix key range, the prefix pass's normalised outputs (fp32) with their log2-domain
// log-sum-exp.
struct CascadeLayout {
  size_t lens, lse, o, total;
};

inline CascadeLayout cascade_layout(int head_dim, int num_q_heads, int num_kv_heads, int num_reqs,
                                    int num_tokens) {
  CascadeLayout c{};
  size_t off = ws_layout(head_dim, num_kv_heads, num_reqs, num_tokens).total;
  auto take = [&off](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) & ~static_cast<size_t>(255);
    return o;
  };
  c.lens = take(static_cast<size_t>(num_reqs) * sizeof(int32_t));
  c.lse = take(static_cast<size_t>(kMaxPrefixSplits) * num_tokens * num_q_heads * sizeof(float));
  c.o = take(static_cast<size_t>(kMaxPrefixSplits) * num_tokens * num_q_heads * head_dim *
             sizeof(float));
  c.total = off;
  return c;
}

struct AttnArgs {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  const int32_t* block_table;
  const int32_t* qsl;
  const int32_t* seq_lens;
  int32_t* header;
  int32_t* dec_off;
  int32_t* pre_off;
  int32_t* done;  // per (request, kv head): decode splits finished so far
  int32_t* pre_list;  // tcgen05 prefill (request, pair) entries, longest first: r * 65536 + pair
  float2* part_ml;
  float* part_o;
  int R, N, N_pad, nh, nkv, group, MB, num_blocks, null_block;
  int ratio;  // kernel pages per page-table entry (manager block)
  int target_units;
  int tile_tokens;  // query tokens per 128-row tcgen05 tile: 128 / group (whole tokens only)
  int fused_ctas;  // > 0: decode and prefill share one launch of this many CTAs (one per SM)
  int decode_warps_per_cta;  // decode warps per CTA in the launch that runs decode units
  float scale_log2;
  int32_t* err;
  long long kp_cap;   // kernel pages a row may span (max_blocks_per_req * ratio, less a shift)
  int cascade;        // CascadePass
  int prefix_len;     // prefix pass: the shared keys [0, P) of row 0
  int prefix_splits;  // key ranges of the prefix pass (1 .. kMaxPrefixSplits)
  int prefix_split_keys;  // keys per range (a multiple of 128)
  float* pre_o;       // [splits, N, nh, HD] prefix-pass outputs per key range, normalised
  float* pre_lse;     // [splits, N, nh] their log-sum-exp (log2 units of the scaled scores)
  // limit of the fused launch's bounded waits, and (tests only) CTA 0's producer withholding
  // the arrival of its first prefill unit so that the waits for it run out
  unsigned long long wait_limit_ns;
  int withhold_first_unit;
  // score rules (rb_paged_attention_scored); the ordinary kernels do not read them
  int rules;                 // Rules the kernel applies
  const __nv_bfloat16* v;    // V cache
  float cap_in, cap_log2;    // softcap: score = cap_log2 * tanh(cap_in * q.k) in log2 units
  float cap_poly[4];         // the same as s * (cap_poly[0] + s^2 (cap_poly[1] + ...)), s = q.k
  float cap_z, cap_s;        // for s^2 up to cap_z, |s| up to cap_s
  const float* slopes;       // [nh] distance bias -slope * |p - k|, or null
  const int32_t* key_start;  // [N] first visible key of each query token, or null
  const int32_t* prefix;     // [R] keys every query of the request sees, or null
};

// What a kernel instance applies, so that each rule's code (and its registers) is only in the
// kernels of the calls that ask for it: kOrdinary is rb_paged_attention, kMasked adds the key
// ranges, and the other two the soft cap and the distance bias on top of them.
enum Rules : int { kOrdinary = 0, kMasked = 1, kCapped = 2, kBiased = 4 };
__host__ __device__ constexpr bool is_scored(int rules) { return rules != kOrdinary; }

// The keys a query token at position p of a request of length L may see are [lo, hi):
// lo = key_start (0 without one), hi = min(L, max(p + 1, prefix)); none when lo >= hi.
__device__ __forceinline__ int key_lo(const AttnArgs& a, int token) {
  return a.key_start != nullptr ? max(0, __ldg(a.key_start + token)) : 0;
}
__device__ __forceinline__ int key_prefix(const AttnArgs& a, int r, int L) {
  return a.prefix != nullptr ? min(L, max(0, __ldg(a.prefix + r))) : 0;
}

// First page a scored decode request (request r, q query tokens from flat token t0, length L) reads:
// the one of the first key that any of its tokens sees, but always a page of the request, so
// that a request whose tokens see nothing still has a unit that writes its zero rows.
__device__ __forceinline__ int scored_first_page(const AttnArgs& a, int r, int t0, int q, int L) {
  if (a.key_start == nullptr) return 0;
  const int prefix = key_prefix(a, r, L);
  int lo = 0x7fffffff;
#pragma unroll 1
  for (int j = 0; j < q; ++j) {
    const int k = key_lo(a, t0 + j);
    if (k < max(L - q + j + 1, prefix)) lo = min(lo, k);
  }
  return min(lo / kPage, (L + kPage - 1) / kPage - 1);
}

// A product of probability 0 with an infinite or NaN value is NaN, so where only some queries of
// a tile (or page) see a key, a V that is not finite would reach the others' rows.  Such elements
// are taken out of the staged V (set to 0) and added, as they are, to the results of the rows
// that see the key: any positive weight times infinity or NaN is that.  (Out of line: rare, and
// kept out of the attention loops' registers and instruction stream.)
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {  // bit 15 of each bf16 half
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
__device__ __forceinline__ bool not_finite(const uint4& w) {
  return ((not_finite(w.x) | not_finite(w.y)) | (not_finite(w.z) | not_finite(w.w))) != 0;
}
__device__ __forceinline__ uint32_t finite_halves(uint32_t w) {  // the others set to 0
  const uint32_t f = not_finite(w);
  return w & ~((f & 0x8000u ? 0xffffu : 0u) | (f & 0x80000000u ? 0xffff0000u : 0u));
}
// A warp takes what is not finite out of `count` runs of 512 bytes, `stride` apart, of staged V;
// returns whether there was any.
static __device__ __noinline__ bool take_out_not_finite(uint8_t* p, int count, int stride) {
  p += (threadIdx.x & 31) * 16;
  bool odd = false;
#pragma unroll 8
  for (int i = 0; i < count; ++i) {
    const uint4 w = *reinterpret_cast<const uint4*>(p + i * stride);
    odd |= ((not_finite(w.x) | not_finite(w.y)) | (not_finite(w.z) | not_finite(w.w))) != 0;
  }
  if (!__any_sync(0xffffffffu, odd)) return false;
  for (int i = 0; i < count; ++i) {
    uint4* q = reinterpret_cast<uint4*>(p + i * stride);
    const uint4 w = *q;
    *q = make_uint4(finite_halves(w.x), finite_halves(w.y), finite_halves(w.z),
                    finite_halves(w.w));
  }
  fence_proxy_async_smem();
  __syncwarp();
  return true;
}
// V row of a request's key, or null where its page id is invalid.
__device__ __forceinline__ const __nv_bfloat16* v_row(const AttnArgs& a, int r, int h, int key,
                                                      int head_dim) {
  const int id = kernel_page(a.block_table + static_cast<size_t>(r) * a.MB, key / kPage, a.ratio,
                             a.num_blocks, a.null_block);
  if (id < 0) return nullptr;
  return a.v + ((static_cast<size_t>(id) * kPage + key % kPage) * a.nkv + h) * head_dim;
}
// One thread adds the infinities and NaN in V of keys [k0, k1) to its output row.
static __device__ __noinline__ void add_not_finite(const AttnArgs& a, int r, int h, int k0, int k1,
                                                   int head_dim, __nv_bfloat16* out) {
  for (int key = k0; key < k1; ++key) {
    const __nv_bfloat16* v = v_row(a, r, h, key, head_dim);
    if (v == nullptr) continue;
    for (int d = 0; d < head_dim; ++d) {
      const float x = __bfloat162float(v[d]);
      if (!isfinite(x)) out[d] = __float2bfloat16_rn(__bfloat162float(out[d]) + x);
    }
  }
}

// Capped scores (log2 units): cap_log2 * tanh(u), u = cap_in * s.  For u^2 <= z tanh(u) = u P(u^2)
// with P(0) = 1 of degree 3, the least maximum relative error of that form on [0, z]:
// multiply-adds two at a time and no trip to the SFU, which the exponents keep busy.  Larger |u|:
// tanh(u) = 1 - 2 / (1 + e^2u), two SFU operations (e^2u = inf or 0 gives +-1), with an error of
// 1.5e-7 from u = 0.3 on.
// The error counts cap_log2 times, and 2^-11 log2 units move a probability by an eleventh of what
// rounding it to bf16 does.  z = 1/2 (an error of 5.2e-6 in tanh) stays below that up to
// cap_log2 = 93, a cap of 64; above, P is the one for z = 1/10 (5.5e-9), which leaves the
// exponential form's error (2^-12 at a cap of 1000) and, from caps of thousands on, the fp32
// rounding of scores of that size.
struct TanhPoly {
  float c[4], z;
};
constexpr TanhPoly kTanhWide = {{1.0f, -0.3329871892929077f, 0.12897320091724396f,
                                 -0.03759901970624924f}, 0.5f};
constexpr TanhPoly kTanhNarrow = {{1.0f, -0.33332962386243388f, 0.13310651554494919f,
                                   -0.04998707773147634f}, 0.1f};
constexpr float kTanhWideCap = 93.f;  // cap_log2

// kCount raw products, in place.  Both forms are evaluated and one chosen per score: tiles and
// pages that need their scores in place are few.
template <int kCount>
__device__ __forceinline__ void cap_scores(const AttnArgs& a, float (&s)[kCount]) {
  const float in2 = a.cap_in * (2.f * 1.4426950408889634f);
#pragma unroll
  for (int i = 0; i < kCount; ++i) {
    const float z = s[i] * s[i];
    float f = fmaf(a.cap_poly[3], z, a.cap_poly[2]);
    f = fmaf(f, z, a.cap_poly[1]);
    f = fmaf(f, z, a.cap_poly[0]);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fast_exp2(s[i] * in2) + 1.f));
    s[i] = z > a.cap_z ? fmaf(-2.f * a.cap_log2, r, a.cap_log2) : s[i] * f;  // (NaN stays NaN)
  }
}

// Test hook behind rb_debug_attention_wait_limit: the wait limit and withhold flag of every
// later attention call (process-wide).
void debug_wait_settings(unsigned long long* limit_ns, int* withhold);

// Weights that merge a suffix-pass row (accumulator relative to running max m, sum l; log2
// units) with the prefix-pass rows of the same (token, head) (one per key range: log-sum-exp
// lse_s, normalised o_s): out = acc * (return value) + sum_s o_s * w[s].
__device__ __forceinline__ float cascade_weights(const AttnArgs& a, size_t row, float m, float l,
                                                 float* w) {
  const size_t stride = static_cast<size_t>(a.N) * a.nh;
  float lse[kMaxPrefixSplits];
  float mx = l > 0.f ? m : -INFINITY;
#pragma unroll
  for (int s = 0; s < kMaxPrefixSplits; ++s) {
    lse[s] = s < a.prefix_splits ? __ldg(a.pre_lse + s * stride + row) : -INFINITY;
    mx = fmaxf(mx, lse[s]);
  }
  if (mx == -INFINITY) {
#pragma unroll
    for (int s = 0; s < kMaxPrefixSplits; ++s) w[s] = 0.f;
    return 0.f;
  }
  const float wa = l > 0.f ? fast_exp2(m - mx) : 0.f;
  float den = l * wa;
#pragma unroll
  for (int s = 0; s < kMaxPrefixSplits; ++s) {
    w[s] = lse[s] == -INFINITY ? 0.f : fast_exp2(lse[s] - mx);
    den += w[s];
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
#pragma unroll
  for (int s = 0; s < kMaxPrefixSplits; ++s) w[s] *= inv;
  return wa * inv;
}

// Prefix-pass output row of key range s for (token, head) row `row`.
template <int HD>
__device__ __forceinline__ const float* cascade_row(const AttnArgs& a, int s, size_t row) {
  return a.pre_o + (static_cast<size_t>(s) * a.N * a.nh + row) * HD;
}

// Request classes shared by the planner and the kernels.
__host__ __device__ inline bool is_decode_class(int q, int group) {
  return q >= 1 && q * group <= kMaxCols;
}

// Host side of one attention call: checked arguments, kernel arguments and TMA descriptors.
struct AttnSetup {
  AttnArgs a;
  PageGeom g;
  int head_dim, num_kv_heads;
  const void* k_cache;
  const void* v_cache;
  long long num_slots;
  CUtensorMap qmap, kmap, vmap;
};

// Host checks and kernel arguments of rb_paged_attention (no launch, no driver call).
rb_status attn_setup(const rb_dims* dims, int32_t num_reqs, int32_t num_tokens,
                     int32_t num_tokens_padded, const void* d_q, const void* d_k_cache,
                     const void* d_v_cache, const int32_t* d_block_table,
                     const int32_t* d_query_start_loc, const int32_t* d_seq_lens,
                     float softmax_scale, void* d_out, void* d_workspace, size_t workspace_bytes,
                     int32_t* d_error_word, AttnSetup* su);
// Encodes the TMA descriptors of a set-up call.
rb_status attn_encode_maps(AttnSetup* su);
// Enqueues what follows the planner: the fused decode + prefill launch.
rb_status attn_main(const AttnSetup& su, cudaStream_t s);

// Adds rb_paged_attention_scored's rules to a set-up call.
rb_status attn_set_rules(AttnSetup* su, const rb_score_rules* rules, float softmax_scale);

rb_status launch_scored_tc(const AttnArgs& a, int head_dim, const CUtensorMap& qmap,
                           const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t s);
rb_status launch_prefill_tc(const AttnArgs& a, int head_dim, const CUtensorMap& qmap,
                            const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t s);

}  // namespace attn
}  // namespace rb
