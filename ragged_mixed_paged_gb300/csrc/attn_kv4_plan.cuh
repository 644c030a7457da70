// The planner of the attention over a 4-bit cache, one CTA.  Not part of the C ABI.
#pragma once

#include "attn_plan.cuh"

namespace rb {
namespace attn {

// Finish-time model (this GPU, cold caches, heads of 128; fitted to whole-launch times): a CTA
// decodes 12.5 pages of one kv head a microsecond, a prefill unit of n key tiles takes 6 + 2.7 n.
constexpr float kKv4PagesPerUs = 12.5f, kKv4UnitUs = 6.f, kKv4TileUs = 2.7f;
// Pages of a decode warp: at least kMinPages, and enough that a (request, kv head)'s pieces cost no
// more to merge than its pages take (attn_plan.cuh's rule for splits).
constexpr int kKv4MinPages = 4;

// Validates the metadata, counts the decode requests' pages (a.dec_off: of one kv head, before each
// request) and lists the prefill units longest first, divides the CTAs between the two, clears the
// merge counters and writes the padding rows of the output as zeros.
__device__ __forceinline__ void kv4_plan_body(const AttnArgs& a, int head_dim, int warps_per_cta) {
  __shared__ int s_longest, s_pre_max, s_bin[kTileBins];
  __shared__ float s_pre_us;
  const int tid = threadIdx.x, nthreads = blockDim.x, lane = tid & 31;
  const int per = (a.R + nthreads - 1) / nthreads;  // the same for every thread
  const int lo = min(tid * per, a.R), hi = min(lo + per, a.R);
  const ReqSrc src{a.qsl, a.seq_lens, nullptr};
  // a thread's first requests are kept; the others are read again
  constexpr int kCache = 2;
  ReqInfo cache[kCache];
#pragma unroll
  for (int k = 0; k < kCache; ++k)
    cache[k] = lo + k < hi ? req_info<false>(a, src, lo + k) : ReqInfo{false, 0, 0, 0};
  auto get = [&](int k) {
    return k == 0 ? cache[0] : k == 1 ? cache[1] : req_info<false>(a, src, lo + k);
  };
  for (int i = tid; i < kTileBins; i += nthreads) s_bin[i] = 0;
  if (tid == 0) {
    s_longest = s_pre_max = 0;
    s_pre_us = 0.f;
  }
  int bits = tid == 0 && (a.qsl[0] != 0 || a.qsl[a.R] != a.N) ? RB_EBIT_ATTN_META : 0;
  int pages = 0, pairs = 0, longest = 0;
#pragma unroll 1
  for (int k = 0; lo + k < hi; ++k) {
    const ReqInfo x = get(k);
    if (!x.ok) bits |= RB_EBIT_ATTN_META;
    else if (is_decode_class(x.q, a.group)) {
      pages += x.pages;
      longest = max(longest, x.pages);
    } else if (x.q > 0) {
      pairs += prefill_pairs(x.q, a.tile_tokens);
    }
  }
  int at, ex_pairs, total, total_pairs;
  block_scan2(pages, pairs, &at, &ex_pairs, &total, &total_pairs);
#pragma unroll 1
  for (int k = 0; lo + k < hi; ++k) {
    const ReqInfo x = get(k);
    a.dec_off[lo + k] = at;
    if (x.ok && is_decode_class(x.q, a.group)) at += x.pages;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0 && longest) atomicMax(&s_longest, longest);

  if (total_pairs > 0) {  // a counting sort of the (request, pair) entries by key tiles
    auto each_pair = [&](auto&& body) {  // body(r, key tiles, pair); a request's spread over a warp
#pragma unroll 1
      for (int k = 0; k < per; ++k) {
        const ReqInfo x = lo + k < hi ? get(k) : ReqInfo{false, 0, 0, 0};
        const int n = x.ok && x.q > 0 && !is_decode_class(x.q, a.group)
                          ? prefill_pairs(x.q, a.tile_tokens) : 0;
        for (unsigned m = __ballot_sync(0xffffffffu, n > 0); m; m &= m - 1) {
          const int from = __ffs(m) - 1;
          const int r = __shfl_sync(0xffffffffu, lo + k, from);
          const int q = __shfl_sync(0xffffffffu, x.q, from);
          const int c = __shfl_sync(0xffffffffu, x.L - x.q, from);
          const int np = __shfl_sync(0xffffffffu, n, from);
          for (int p = lane; p < np; p += 32) body(r, pair_key_tiles(c, q, a.tile_tokens, p), p);
        }
      }
    };
    float us = 0.f;
    int most = 0;
    each_pair([&](int, int n, int) {
      atomicAdd(&s_bin[min(n, kTileBins - 1)], 1);
      us += kKv4UnitUs + kKv4TileUs * n;
      most = max(most, n);
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) us += __shfl_xor_sync(0xffffffffu, us, o);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0 && most > 0) {
      atomicAdd(&s_pre_us, us);
      atomicMax(&s_pre_max, most);
    }
    __syncthreads();
    // bins in descending order: where each one's entries start in the list
    const int per_bin = (kTileBins + nthreads - 1) / nthreads;
    int count = 0, start, all, none0, none1;
    for (int i = 0; i < per_bin; ++i) {
      const int b = kTileBins - 1 - (tid * per_bin + i);
      if (b >= 0) count += s_bin[b];
    }
    block_scan2(count, 0, &start, &none0, &all, &none1);
    for (int i = 0; i < per_bin; ++i) {
      const int b = kTileBins - 1 - (tid * per_bin + i);
      if (b < 0) continue;
      const int c = s_bin[b];
      s_bin[b] = start;
      start += c;
    }
    __syncthreads();
    each_pair([&](int r, int n, int p) {
      a.pre_list[atomicAdd(&s_bin[min(n, kTileBins - 1)], 1)] = r * 65536 + p;
    });
  }
  __syncthreads();
  if (tid == 0) {
    const int ctas = a.fused_ctas;
    const long long work = static_cast<long long>(total) * a.nkv;
    int decode_ctas = 0, warps = 0;
    if (work > 0) {
      // Both kinds together take (their SM time) / ctas, or the longest unit.  The decode CTAs then
      // go on with prefill units, the shortest ones by then, so they are to be done with their own
      // after 3/4 of that.
      const float scale = static_cast<float>(head_dim) / 128.f;
      const float dec = static_cast<float>(work) * scale / kKv4PagesPerUs, pre = s_pre_us * a.nkv;
      const float end = fmaxf((dec + pre) / ctas, kKv4UnitUs + kKv4TileUs * s_pre_max);
      decode_ctas = total_pairs == 0 ? ctas
                                     : min(ctas, static_cast<int>(dec / (0.75f * end)) + 1);
      const int least = max(kKv4MinPages,
                            static_cast<int>(sqrtf(kSplitCost * static_cast<float>(s_longest))));
      warps = static_cast<int>(min(static_cast<long long>(decode_ctas) * warps_per_cta,
                                   (work + least - 1) / least));
      warps = min(warps, kMaxTargetUnits / 2);  // (two partials a warp)
    }
    a.dec_off[a.R] = total;
    a.header[kHNumDecodeUnits] = warps;
    a.header[kHNumPrefillUnits] = total_pairs * a.nkv;
    a.header[kHPrefillNext] = 0;
    a.header[kHDecodeCtas] = decode_ctas;
    a.header[kHRoleNext] = 0;
  }
  for (int i = tid; i < a.R * a.nkv; i += nthreads) a.done[i] = 0;
  // rows of padding tokens are written as zeros
  const long long row16 = static_cast<long long>(a.nh) * head_dim * 2 / 16;
  int4* out = reinterpret_cast<int4*>(a.out);
  for (long long i = a.N * row16 + tid; i < a.N_pad * row16; i += nthreads)
    out[i] = make_int4(0, 0, 0, 0);
  if (bits) raise_error(a.err, bits);
}

}  // namespace attn
}  // namespace rb
