// The planner of the attention over a 4-bit cache, one CTA.  Not part of the C ABI.
#pragma once

#include "attn_plan.cuh"

namespace rb {
namespace attn {

// Finish-time model (this GPU, cold caches, heads of 128; fitted to whole-launch times): a CTA
// decodes 14.5 pages of one kv head a microsecond (twice as many of heads of 64), a prefill unit of n
// key tiles takes 6 + 2.4 n, whatever its heads and whether it has one side or two.  It divides the CTAs,
// so that what it is off by costs time alone.
constexpr float kKv4PagesPerUs = 14.5f, kKv4UnitUs = 6.f, kKv4TileUs = 2.4f;
// Pages of a decode warp: at least kMinPages (64 decodes of 100 to 500 tokens: 25 us, 29 with 4), and
// enough that a (request, kv head)'s pieces cost no more to merge than its pages take
// (attn_plan.cuh's rule for splits); an even number, because a step takes two.  It sets the count of
// warps, over which the stream is cut in equal parts: they are even where it divides (24 decodes of
// 4000 tokens, 20 pages a warp instead of 19.7: 58 -> 46 us), near it elsewhere.
constexpr int kKv4MinPages = 6;

// Rows of padding tokens are written as zeros, by every CTA that calls this.
__device__ __forceinline__ void kv4_clear_padding(const AttnArgs& a, int head_dim) {
  const long long row16 = static_cast<long long>(a.nh) * head_dim * 2 / 16;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  int4* out = reinterpret_cast<int4*>(a.out);
  for (long long i = a.N * row16 + static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
       i < a.N_pad * row16; i += step)
    out[i] = make_int4(0, 0, 0, 0);
}

// Validates the metadata, counts the decode requests' pages (a.dec_off: of one kv head, before each
// request) and lists the prefill units longest first, divides the CTAs between the two and clears
// the merge counters.  Requests are taken a thread
// each, as many as there are threads at a time; of the prefill ones among them each is then a warp's,
// whose lanes take its units (a request a lane, the fourteen of a small batch were one warp's: 9 us
// instead of 7).
__device__ __forceinline__ void kv4_plan_body(const AttnArgs& a, int head_dim, int warps_per_cta) {
  constexpr int kMaxThreads = 1024;
  __shared__ int s_longest, s_pre_max, s_pre_units, s_list, s_bin[kTileBins];
  __shared__ int s_r[kMaxThreads], s_q[kMaxThreads], s_c[kMaxThreads];  // prefill requests
  __shared__ unsigned s_pre_tiles;
  const int tid = threadIdx.x, nthreads = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const ReqSrc src{a.qsl, a.seq_lens, nullptr};
  auto info = [&](int r) {  // (a length near 2^31, which rounding up to pages would overflow, is none)
    if (a.seq_lens[r] > 0x7ffffff0) return ReqInfo{false, 0, 0, 0};
    return req_info<false>(a, src, r);
  };
  for (int i = tid; i < kTileBins; i += nthreads) s_bin[i] = 0;
  if (tid == 0) {
    s_longest = s_pre_max = s_pre_units = s_list = 0;
    s_pre_tiles = 0;
  }
  int bits = tid == 0 && (a.qsl[0] != 0 || a.qsl[a.R] != a.N) ? RB_EBIT_ATTN_META : 0;
  __syncthreads();
  auto is_prefill = [&](const ReqInfo& x) {
    return x.ok && x.q > 0 && !is_decode_class(x.q, a.group);
  };
  auto put = [&](int r, const ReqInfo& x) {
    if (!is_prefill(x)) return;
    const int i = atomicAdd(&s_list, 1);
    s_r[i] = r;
    s_q[i] = x.q;
    s_c[i] = x.L - x.q;
  };
  auto each_unit = [&](auto&& body) {  // body(r, key tiles, pair) of the listed requests
    for (int i = warp; i < s_list; i += nthreads / 32) {
      const int r = s_r[i], q = s_q[i], c = s_c[i], n = prefill_pairs(q, a.tile_tokens);
      for (int p = lane; p < n; p += 32) body(r, pair_key_tiles(c, q, a.tile_tokens, p), p);
    }
  };
  int total = 0, longest = 0, most = 0, units = 0;
  unsigned tiles = 0;  // (sums of integers: the plan does not depend on the atomics' order)
#pragma unroll 1
  for (int base = 0; base < a.R; base += nthreads) {
    const int r = base + tid;
    const ReqInfo x = r < a.R ? info(r) : ReqInfo{true, 0, 0, 0};
    if (!x.ok) bits |= RB_EBIT_ATTN_META;
    const int pages = x.ok && is_decode_class(x.q, a.group) ? x.pages : 0;
    longest = max(longest, pages);
    put(r, x);
    int at, none0, sum, none1;
    block_scan2(pages, 0, &at, &none0, &sum, &none1);  // (with barriers: the list is whole)
    if (r < a.R) a.dec_off[r] = total + at;
    total += sum;
    each_unit([&](int, int n, int) {
      atomicAdd(&s_bin[min(n, kTileBins - 1)], 1);
      tiles += n;
      most = max(most, n);
      ++units;
    });
    __syncthreads();
    if (base + nthreads < a.R && tid == 0) s_list = 0;
    __syncthreads();
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  most = __reduce_max_sync(0xffffffffu, most);
  units = __reduce_add_sync(0xffffffffu, units);
  tiles = __reduce_add_sync(0xffffffffu, tiles);
  if (lane == 0 && longest) atomicMax(&s_longest, longest);
  if (lane == 0 && units) {
    atomicMax(&s_pre_max, most);
    atomicAdd(&s_pre_units, units);
    atomicAdd(&s_pre_tiles, tiles);
  }
  __syncthreads();
  int total_pairs = s_pre_units;
  if (total_pairs > max_prefill_pairs(a.R, a.N)) {  // rows that several requests claim: no list
    total_pairs = 0;
    bits |= RB_EBIT_ATTN_META;
  }

  if (total_pairs > 0) {  // a counting sort of the units by key tiles, longest first
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
    auto list_units = [&] {
      each_unit([&](int r, int n, int p) {
        a.pre_list[atomicAdd(&s_bin[min(n, kTileBins - 1)], 1)] = r * 65536 + p;
      });
    };
    if (a.R <= nthreads) {
      list_units();
    } else {  // the requests once more
#pragma unroll 1
      for (int base = 0; base < a.R; base += nthreads) {
        __syncthreads();
        if (tid == 0) s_list = 0;
        __syncthreads();
        if (base + tid < a.R) put(base + tid, info(base + tid));
        __syncthreads();
        list_units();
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    const int ctas = a.fused_ctas;
    const long long work = static_cast<long long>(total) * a.nkv;
    int decode_ctas = 0, warps = 0;
    if (work > 0) {
      // Both kinds together take (their SM time) / ctas, or the longest unit.  The decode CTAs then
      // go on with prefill units, the shortest ones by then, so they are to be done with their own
      // after 3/4 of that (flat: 1/2 to 19/20 gave the large mix, now 411 us, 425 to 431 when it was
      // fitted, other mixes 166 to 176 and 869 to 884).
      const float scale = static_cast<float>(head_dim) / 128.f;
      const float dec = static_cast<float>(work) * scale / kKv4PagesPerUs;
      const float pre = (kKv4UnitUs * total_pairs + kKv4TileUs * s_pre_tiles) * a.nkv;
      const float end = fmaxf((dec + pre) / ctas, kKv4UnitUs + kKv4TileUs * s_pre_max);
      decode_ctas = total_pairs == 0 ? ctas
                                     : min(ctas, static_cast<int>(dec / (0.75f * end)) + 1);
      const int least = max(kKv4MinPages,
                            static_cast<int>(sqrtf(kSplitCost * static_cast<float>(s_longest))));
      const long long most = static_cast<long long>(decode_ctas) * warps_per_cta;
      long long pages = max(static_cast<long long>(least), (work + most - 1) / most);
      pages += pages & 1;
      warps = static_cast<int>((work + pages - 1) / pages);
      warps = min(warps, kMaxTargetUnits / 2);  // (two partials a warp)
    }
    a.dec_off[a.R] = total;
    a.header[kHNumDecodeUnits] = warps;
    a.header[kHNumPrefillUnits] = total_pairs * a.nkv;
    a.header[kHPrefillNext] = 0;
    a.header[kHDecodeCtas] = decode_ctas;
  }
  for (int i = tid; i < a.R * a.nkv; i += nthreads) a.done[i] = 0;
  if (a.R == 0) kv4_clear_padding(a, head_dim);  // (nothing else is launched)
  if (bits) raise_error(a.err, bits);
}

}  // namespace attn
}  // namespace rb
