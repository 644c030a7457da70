// Page management of the paged KV cache: rb_pages_count, rb_pages_copy, rb_pages_fork,
// rb_pages_free and rb_pages_compact.
//
// The state is the persistent batch's page table (d_block_table, d_num_blocks) and one reference
// count per page-table entry id: the number of rows that hold the page, 0 for a free page.
// "A page" here is what one page-table entry names: a kernel page, or a manager block of r.
//
//   copy     dst[i] <- src[i], whole pages of K and V
//   fork     a new row shares the full pages of another (count + 1) and gets its own copy of
//            the partial last page, on the lowest free page
//   free     count - 1 for every page of a row
//   compact  the L live pages move into the L lowest ids: live page number j above them goes to
//            free page number j below, and the table entries follow
//
// Copies move whole 16-byte chunks and are bound by HBM (2 x page bytes); everything else is a
// few dependent passes over the counts and is bound by latency, so each call is few launches: one
// for copy and free, two (a plan by one CTA or one cluster, then the grid that copies) for fork
// and compact.  A launch may be resident while the one before it still writes what it reads, so
// nothing here is read through the non-coherent path (__ldg).
#include <cooperative_groups.h>

#include "rb_internal.cuh"

namespace rb {
namespace {

namespace cg = cooperative_groups;

constexpr int kCopyThreads = 256;
constexpr int kCheckThreads = 1024;
constexpr int kClusterCtas = 8;     // free and compact's plan: one cluster
constexpr int kCopyPerSm = 32;      // CTAs of a copy per SM, most of them queued

struct PageArgs {
  int rows, MB, entries, null_entry, page_tokens;
  long long page_chunks;   // 16-byte chunks of one page of K (or V)
  int token_chunks;        // 16-byte chunks of one token's row of K (or V)
  int32_t* table;
  int32_t* num_blocks;
  int32_t* ref;
  int4* k;
  int4* v;
  int32_t* err;
};

// Workspace: [mark / code: entries][list a: entries][list b: entries][header]
struct PagesWs {
  int32_t *code, *movers, *holes, *header;
};
constexpr int kHeaderInts = 16;  // [0]: the fork plan holds; [1]: pages compact moves

__host__ __device__ inline size_t up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

inline size_t ws_bytes(int entries, int rows) {
  const size_t list = up(sizeof(int32_t) * static_cast<size_t>(entries > rows ? entries : rows));
  return 3 * list + up(kHeaderInts * sizeof(int32_t));
}

inline PagesWs ws_of(void* p, int entries, int rows) {
  const size_t list = up(sizeof(int32_t) * static_cast<size_t>(entries > rows ? entries : rows));
  unsigned char* b = static_cast<unsigned char*>(p);
  PagesWs w;
  w.code = reinterpret_cast<int32_t*>(b);
  w.movers = reinterpret_cast<int32_t*>(b + list);
  w.holes = reinterpret_cast<int32_t*>(b + 2 * list);
  w.header = reinterpret_cast<int32_t*>(b + 3 * list);
  return w;
}

__device__ __forceinline__ bool valid_page(const PageArgs& a, int id) {
  return id >= 0 && id < a.entries && id != a.null_entry;
}

// 16-byte chunks [first, last) of a page by one CTA's threads, kUnroll loads in flight each.
template <int kUnroll>
__device__ __forceinline__ void copy_chunks(int4* dst, const int4* src, long long first,
                                            long long last, int tid, int threads) {
  for (long long i = first + tid; i < last; i += kUnroll * threads) {
    int4 x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (i + u * threads < last) x[u] = src[i + u * threads];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (i + u * threads < last) dst[i + u * threads] = x[u];
  }
}

// K and V of n pages, page src(i) to page dst(i) (negative: skipped), by CTAs `cta` of `ctas`.  A
// unit of work is kUnroll chunks per thread of one page; `once(i)` runs in one thread for each i.
template <int kUnroll, class Src, class Dst, class Once>
__device__ __forceinline__ void copy_units(const PageArgs& a, long long n, int cta, int ctas,
                                           Src&& src, Dst&& dst, Once&& once) {
  const int tid = threadIdx.x, threads = blockDim.x;
  const long long chunk = static_cast<long long>(kUnroll) * threads;
  const long long parts = (a.page_chunks + chunk - 1) / chunk, units = 2 * n * parts;
  for (long long u = cta; u < units; u += ctas) {
    const long long i = u / (2 * parts), rest = u - i * 2 * parts;
    const int s = src(i), d = dst(i);
    if (s < 0 || d < 0) continue;
    if (rest == 0 && tid == 0) once(i);
    int4* base = rest >= parts ? a.v : a.k;
    const long long c0 = (rest >= parts ? rest - parts : rest) * chunk;
    copy_chunks<kUnroll>(base + d * a.page_chunks, base + s * a.page_chunks, c0,
                         min(a.page_chunks, c0 + chunk), tid, threads);
  }
}

// Few pages are cut into many small units, so that every CTA has one; many pages are copied with
// four 16-byte loads in flight per thread.  Measured on 8191 pairs of 2 x 32 KiB pages with
// 256-thread CTAs: 178 us (6.0 TB/s) with 8 CTAs per SM, each taking many units, 164 us (6.5
// TB/s) with 32 per SM, most of them queued; 16-byte loads eight at a time 170 and 164 us; bulk
// copies through shared memory 166 us at their best shape, up to 237 us at others.
template <class Src, class Dst, class Once>
__device__ __forceinline__ void copy_pages(const PageArgs& a, long long n, int cta, int ctas,
                                           Src&& src, Dst&& dst, Once&& once) {
  const long long wide = 4LL * blockDim.x;
  if (2 * n * ((a.page_chunks + wide - 1) / wide) >= ctas)
    copy_units<4>(a, n, cta, ctas, src, dst, once);
  else
    copy_units<1>(a, n, cta, ctas, src, dst, once);
}

// ------------------------------------------------------------------------------------- count
__global__ void __launch_bounds__(256) pages_count_kernel(PageArgs a) {
  for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const int n = a.num_blocks[r];
    if (n < 0 || n > a.MB) {
      if (threadIdx.x == 0) raise_error(a.err, RB_EBIT_ROW);
      continue;
    }
    for (int j = threadIdx.x; j < n; j += blockDim.x) {
      const int id = a.table[static_cast<size_t>(r) * a.MB + j];
      if (valid_page(a, id)) atomicAdd(a.ref + id, 1);
      else raise_error(a.err, RB_EBIT_BLOCK_ID);
    }
  }
}

// -------------------------------------------------------------------------------------- copy
constexpr int kSource = 1 << 30;  // bit of a page's mark: it is a source

// CTA 0 checks the pairs (a destination twice, or also a source) while the others copy: where
// it finds one the error bit is set and the pages' contents are unspecified.
__global__ void __launch_bounds__(kCopyThreads)
    pages_copy_kernel(PageArgs a, int n, const int32_t* src, const int32_t* dst, int32_t* mark) {
  grid_wait();
  const int tid = threadIdx.x;
  if (blockIdx.x == 0) {
    // eight pairs per thread and round, so that the three passes stay shorter than the copies
    constexpr int kPer = 8;
    int bits = 0;
    auto each = [&](auto&& fn) {
      for (int base = tid; base < n; base += kPer * kCopyThreads) {
        int s[kPer], d[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int i = base + k * kCopyThreads;
          s[k] = i < n ? src[i] : -1;
          d[k] = i < n ? dst[i] : -1;
        }
        fn(s, d);
      }
    };
    each([&](const int (&s)[kPer], const int (&d)[kPer]) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (s[k] < 0 || d[k] < 0) continue;  // skipped pair
        if (!valid_page(a, s[k]) || !valid_page(a, d[k])) {
          bits |= RB_EBIT_BLOCK_ID;
          continue;
        }
        mark[s[k]] = 0;
        mark[d[k]] = 0;
      }
    });
    __syncthreads();
    each([&](const int (&s)[kPer], const int (&d)[kPer]) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (!valid_page(a, s[k]) || !valid_page(a, d[k])) continue;
        atomicOr(mark + s[k], kSource);
        if (atomicAdd(mark + d[k], 1) & (kSource - 1)) bits |= RB_EBIT_PAGE_PAIR;
      }
    });
    __syncthreads();
    each([&](const int (&s)[kPer], const int (&d)[kPer]) {
      int m[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        m[k] = valid_page(a, s[k]) && valid_page(a, d[k]) ? __ldcg(mark + d[k]) : 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (m[k] & kSource) bits |= RB_EBIT_PAGE_PAIR;
    });
    if (bits) raise_error(a.err, bits);
    return;
  }
  auto page = [&](const int32_t* list, long long i) {
    const int id = list[i];
    return valid_page(a, id) ? id : -1;
  };
  copy_pages(
      a, n, blockIdx.x - 1, gridDim.x - 1, [&](long long i) { return page(src, i); },
      [&](long long i) { return page(dst, i); }, [](long long) {});
}

// Exclusive prefix sum over the block; *total gets the block's sum.
__device__ int block_prefix(int v, int* tmp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = lane < nw ? tmp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    if (lane < nw) tmp[lane] = w;
  }
  __syncthreads();
  const int before = (warp == 0 ? 0 : tmp[warp - 1]) + x - v;
  *total = tmp[nw - 1];
  __syncthreads();
  return before;
}

// -------------------------------------------------------------------------------------- fork
// Validates every fork, then hands the lowest free pages, in the order of the forks, to those
// that end inside a page (fresh[i], else -1).  On an error nothing is changed by either launch.
__global__ void __launch_bounds__(kCheckThreads)
    fork_plan_kernel(PageArgs a, int n, const int32_t* src, const int32_t* dst,
                     const int32_t* cached, int32_t* claim, int32_t* fresh, int32_t* free_list,
                     int32_t* header) {
  __shared__ int tmp[32];
  __shared__ int s_bits;
  grid_wait();
  const int tid = threadIdx.x;
  grid_release();
  if (tid == 0) s_bits = 0;
  for (int r = tid; r < a.rows; r += kCheckThreads) claim[r] = 0;
  __syncthreads();
  int bits = 0, need = 0;
  for (int base = 0; base < n; base += kCheckThreads) {
    const int i = base + tid;
    int wants = 0;
    if (i < n) {
      const int s = src[i], d = dst[i];
      if (s < 0 || s >= a.rows || d < 0 || d >= a.rows || s == d) {
        bits |= RB_EBIT_ROW;
      } else {
        const int c = cached[s], held = a.num_blocks[s];
        const long long pages = (static_cast<long long>(c) + a.page_tokens - 1) / a.page_tokens;
        if (c < 0 || held < 0 || held > a.MB || pages > held) bits |= RB_EBIT_ROW;
        if (a.num_blocks[d] != 0 || atomicExch(claim + d, 1) != 0) bits |= RB_EBIT_ROW;
        wants = c >= 0 && c % a.page_tokens != 0;
      }
    }
    int total;
    const int at = block_prefix(wants, tmp, &total);
    if (i < n) fresh[i] = wants ? need + at : -1;  // number of its free page, for now
    need += total;
  }
  // the need lowest free pages
  __syncthreads();
  constexpr int kPer = 16;  // counts per thread and round: 16 loads in flight, one block scan
  int found = 0;
  for (int base = 0; base < a.entries && found < need; base += kPer * kCheckThreads) {
    const int id0 = base + kPer * tid;
    unsigned free_bits = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int id = id0 + k;
      if (id < a.entries && id != a.null_entry && a.ref[id] == 0) free_bits |= 1u << k;
    }
    int total;
    int at = found + block_prefix(__popc(free_bits), tmp, &total);
    for (; free_bits != 0 && at < need; free_bits &= free_bits - 1)
      free_list[at++] = id0 + __ffs(free_bits) - 1;
    found += total;
  }
  found = min(found, need);
  if (found < need) bits |= RB_EBIT_NO_PAGE;
  if (bits) atomicOr(&s_bits, bits);
  __syncthreads();
  if (tid == 0) {
    header[0] = s_bits == 0;
    if (s_bits) raise_error(a.err, s_bits);
  }
  for (int i = tid; i < n; i += kCheckThreads)
    if (fresh[i] >= 0 && fresh[i] < found) fresh[i] = free_list[fresh[i]];
}

__global__ void __launch_bounds__(kCopyThreads)
    fork_apply_kernel(PageArgs a, int n, const int32_t* src, const int32_t* dst,
                      const int32_t* cached, const int32_t* fresh, const int32_t* header) {
  grid_wait();
  if (!header[0]) return;
  const int i = blockIdx.x, tid = threadIdx.x;
  const int s = src[i], d = dst[i], c = cached[s];
  const int full = c / a.page_tokens, tail = c - full * a.page_tokens;
  const int32_t* from = a.table + static_cast<size_t>(s) * a.MB;
  int32_t* to = a.table + static_cast<size_t>(d) * a.MB;
  for (int j = tid; j < full; j += kCopyThreads) {
    const int id = from[j];
    to[j] = id;
    if (valid_page(a, id)) atomicAdd(a.ref + id, 1);
    else raise_error(a.err, RB_EBIT_BLOCK_ID);
  }
  if (tail > 0) {
    const int old = from[full], page = fresh[i];
    if (tid == 0) {
      to[full] = page;
      a.ref[page] = 1;
      if (!valid_page(a, old)) raise_error(a.err, RB_EBIT_BLOCK_ID);
    }
    if (valid_page(a, old)) {
      const long long count = static_cast<long long>(tail) * a.token_chunks;
      copy_chunks<4>(a.k + page * a.page_chunks, a.k + old * a.page_chunks, 0, count, tid,
                     kCopyThreads);
      copy_chunks<4>(a.v + page * a.page_chunks, a.v + old * a.page_chunks, 0, count, tid,
                     kCopyThreads);
    }
  }
  if (tid == 0) a.num_blocks[d] = full + (tail > 0);
}

// -------------------------------------------------------------------------------------- free
// One cluster of 8 CTAs, a warp per row: the CTAs' numbers of freed pages meet in shared memory,
// so the total needs no cleared counter (a memset before the launch cost more than the launch).
__global__ void __launch_bounds__(kCheckThreads) __cluster_dims__(kClusterCtas, 1, 1)
    pages_free_kernel(PageArgs a, int n, const int32_t* list, int32_t* num_freed) {
  __shared__ int s_freed;
  grid_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) s_freed = 0;
  __syncthreads();
  int freed = 0, bits = 0;
  constexpr int kWarps = kCheckThreads / 32;
  for (int i = (threadIdx.x >> 5) * kClusterCtas + blockIdx.x; i < n; i += kWarps * kClusterCtas) {
    const int r = list[i];
    if (r < 0 || r >= a.rows) {
      bits |= RB_EBIT_ROW;
      continue;
    }
    // the first warp to take the row's count frees it; a row named twice is then empty.  A count
    // that no row can have stays where it is.
    int held = 0;
    if (lane == 0) {
      held = a.num_blocks[r];
      if (held > 0 && held <= a.MB) held = atomicCAS(a.num_blocks + r, held, 0);
    }
    held = __shfl_sync(0xffffffffu, held, 0);
    if (held < 0 || held > a.MB) {
      bits |= RB_EBIT_ROW;
      continue;
    }
    int32_t* row = a.table + static_cast<size_t>(r) * a.MB;
    auto drop = [&](int id) {
      if (!valid_page(a, id)) {
        bits |= RB_EBIT_BLOCK_ID;
        return;
      }
      const int was = atomicSub(a.ref + id, 1);
      if (was < 1) {
        atomicAdd(a.ref + id, 1);
        bits |= RB_EBIT_PAGE_REF;
      }
      freed += was == 1;
    };
    constexpr int kPer = 4;
    for (int j = lane; j < held; j += kPer * 32) {
      int id[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (j + 32 * k < held) id[k] = row[j + 32 * k];
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (j + 32 * k < held) {
          row[j + 32 * k] = -1;
          drop(id[k]);
        }
    }
  }
  if (bits) raise_error(a.err, bits);
  if (num_freed == nullptr) return;
  freed = __reduce_add_sync(0xffffffffu, freed);
  if (lane == 0 && freed) atomicAdd(&s_freed, freed);
  cluster.sync();
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    int sum = lane < kClusterCtas ? *cluster.map_shared_rank(&s_freed, lane) : 0;
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) *num_freed = sum;
  }
  cluster.sync();  // nobody leaves while its sum may be read
}

// ----------------------------------------------------------------------------------- compact
__device__ __forceinline__ int is_live(const PageArgs& a, int id) {
  return id < a.entries && id != a.null_entry && a.ref[id] > 0;
}

// Plan, by one cluster: each CTA counts the live pages of its range of ids, the counts meet in
// shared memory, and each CTA classifies its ids (code[id] = id where it stays or is the reserved
// page, -1 if free, -2 - m for mover number m) and lists movers and holes.  A cooperative grid that
// did plan and copies in one launch took 10 us more host time than the two launches.
__global__ void __launch_bounds__(kCheckThreads) __cluster_dims__(kClusterCtas, 1, 1)
    compact_plan_kernel(PageArgs a, PagesWs w, int32_t* num_live) {
  __shared__ int tmp[32];
  __shared__ int s_count, s_low;
  grid_wait();
  cg::cluster_group cluster = cg::this_cluster();
  grid_release();
  const int tid = threadIdx.x, lane = tid & 31, cta = blockIdx.x;
  const int per = (a.entries + kClusterCtas - 1) / kClusterCtas;
  const int begin = min(a.entries, cta * per), end = min(a.entries, begin + per);
  if (tid == 0) s_count = s_low = 0;
  __syncthreads();
  int n = 0, bits = 0;
#pragma unroll 4
  for (int id = begin + tid; id < end; id += kCheckThreads) {
    const int held = id != a.null_entry ? a.ref[id] : 0;
    n += held > 0;
    if (held < 0) bits |= RB_EBIT_PAGE_REF;
  }
  if (bits) raise_error(a.err, bits);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0 && n) atomicAdd(&s_count, n);
  cluster.sync();
  // live pages in all, below this range, and already in the packed region: every id below
  // `limit` but the reserved page
  int before = 0, total = 0, low = 0;
  int counts[kClusterCtas];
#pragma unroll
  for (int c = 0; c < kClusterCtas; ++c) {
    counts[c] = *cluster.map_shared_rank(&s_count, c);
    total += counts[c];
    before += c < cta ? counts[c] : 0;
  }
  const int limit = total + (a.null_entry <= total);
  const int part = limit / per;  // the range partly inside
#pragma unroll
  for (int c = 0; c < kClusterCtas; ++c) low += c < part ? counts[c] : 0;
  n = 0;
#pragma unroll 4
  for (int id = part * per + tid; id < min(limit, a.entries); id += kCheckThreads)
    n += is_live(a, id);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0 && n) atomicAdd(&s_low, n);
  __syncthreads();
  low += s_low;
  if (cta == 0 && tid == 0) {
    w.header[1] = total - low;
    if (num_live != nullptr) *num_live = total;
  }
  constexpr int kPer = 4;  // ids per thread and block scan
  int rank = before;       // live pages below the id
  for (int base = begin; base < end; base += kPer * kCheckThreads) {
    const int id0 = base + kPer * tid;
    unsigned live = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (id0 + k < end && is_live(a, id0 + k)) live |= 1u << k;
    int all;
    int mine = rank + block_prefix(__popc(live), tmp, &all);
    rank += all;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int id = id0 + k;
      if (id >= end) break;
      int code = -1;
      if (id == a.null_entry) {
        code = id;
      } else if (live >> k & 1) {
        code = id < limit ? id : -2 - (mine - low);
        if (id >= limit) w.movers[mine - low] = id;
        ++mine;
      } else if (id < limit) {
        w.holes[id - (id > a.null_entry) - mine] = id;
      }
      w.code[id] = code;
    }
  }
  cluster.sync();  // nobody leaves while its count may be read
}

// The table's entries and the map, by the first `table_ctas` CTAs; the pages, by the others.
__global__ void __launch_bounds__(kCopyThreads)
    compact_move_kernel(PageArgs a, PagesWs w, int32_t* page_map, int table_ctas) {
  const int tid = threadIdx.x;
  grid_wait();
  auto moved = [&](int id) {
    const int c = w.code[id];
    return c <= -2 ? w.holes[-2 - c] : c;
  };
  if (static_cast<int>(blockIdx.x) < table_ctas) {
    for (int r = blockIdx.x; r < a.rows; r += table_ctas) {
      const int n = a.num_blocks[r];
      if (n < 0 || n > a.MB) {
        if (tid == 0) raise_error(a.err, RB_EBIT_ROW);
        continue;
      }
      for (int j = tid; j < n; j += kCopyThreads) {
        int32_t* e = a.table + static_cast<size_t>(r) * a.MB + j;
        const int id = *e;
        const int to = valid_page(a, id) ? moved(id) : -1;
        if (to < 0) raise_error(a.err, RB_EBIT_BLOCK_ID);
        else if (to != id) *e = to;
      }
    }
    if (page_map != nullptr)
      for (int id = blockIdx.x * kCopyThreads + tid; id < a.entries;
           id += table_ctas * kCopyThreads)
        page_map[id] = moved(id);
    return;
  }
  copy_pages(
      a, w.header[1], blockIdx.x - table_ctas, gridDim.x - table_ctas,
      [&](long long i) { return w.movers[i]; }, [&](long long i) { return w.holes[i]; },
      [&](long long i) {  // (nothing in this launch reads the counts)
        a.ref[w.holes[i]] = a.ref[w.movers[i]];
        a.ref[w.movers[i]] = 0;
      });
}

// ---------------------------------------------------------------------------------- host side
// CTAs of a grid that copies at most `pages` pages.
int copy_grid(const PageArgs& a, long long pages) {
  const long long units = 2 * pages * ((a.page_chunks + kCopyThreads - 1) / kCopyThreads);
  const long long most = static_cast<long long>(kCopyPerSm) * max(1, device_sm_count());
  return static_cast<int>(units < most ? units : most);
}

// Checks what every entry point shares and fills `a`.  `tables`, the caches and the workspace
// are checked only where the entry point uses them.
rb_status setup(const rb_dims* dims, const rb_page_tables* t, bool use_tables, void* d_k,
                void* d_v, bool use_cache, void* ws, size_t ws_size, bool use_ws, int32_t* err,
                PageArgs* a) {
  if (dims == nullptr) return RB_ERR_INVALID_ARG;
  const rb_dims& d = *dims;
  PageGeom g;
  if (page_geom_of(d, &g) != RB_OK || d.block_size < 1 || d.num_kv_heads < 1 ||
      d.head_dim < 1 || d.max_num_reqs < 0)
    return RB_ERR_INVALID_ARG;
  const long long row = 2LL * d.num_kv_heads * d.head_dim;  // bytes of a token's K (or V)
  const long long tokens = static_cast<long long>(d.block_size) * g.ratio;
  if (row % 16 != 0) return RB_ERR_UNSUPPORTED;
  if (tokens > 0x7fffffffLL || row / 16 > 0x7fffffffLL) return RB_ERR_UNSUPPORTED;
  *a = PageArgs{};
  a->entries = g.num_blocks / g.ratio;
  a->null_entry = g.null_block / g.ratio;
  a->page_tokens = static_cast<int>(tokens);
  a->token_chunks = static_cast<int>(row / 16);
  a->page_chunks = tokens * a->token_chunks;
  a->MB = d.max_blocks_per_req;
  a->err = err;
  if (use_tables) {
    if (t == nullptr || t->reserved != 0 || t->num_rows < 0) return RB_ERR_INVALID_ARG;
    if (t->num_rows > d.max_num_reqs) return RB_ERR_CAPACITY;
    if (t->d_block_table == nullptr || t->d_num_blocks == nullptr || t->d_ref_count == nullptr)
      return RB_ERR_INVALID_ARG;
    a->rows = t->num_rows;
    a->table = t->d_block_table;
    a->num_blocks = t->d_num_blocks;
    a->ref = t->d_ref_count;
  }
  if (use_cache) {
    if (d_k == nullptr || d_v == nullptr || !aligned16(d_k) || !aligned16(d_v))
      return RB_ERR_INVALID_ARG;
    a->k = static_cast<int4*>(d_k);
    a->v = static_cast<int4*>(d_v);
  }
  if (use_ws) {
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return RB_ERR_INVALID_ARG;
    if (ws_size < ws_bytes(a->entries, d.max_num_reqs)) return RB_ERR_CAPACITY;
  }
  return RB_OK;
}

}  // namespace
}  // namespace rb

extern "C" size_t rb_pages_workspace_size(const rb_dims* dims) {
  using namespace rb;
  PageGeom g;
  if (dims == nullptr || page_geom_of(*dims, &g) != RB_OK || dims->max_num_reqs < 0) return 0;
  return ws_bytes(g.num_blocks / g.ratio, dims->max_num_reqs);
}

extern "C" rb_status rb_pages_count(const rb_dims* dims, const rb_page_tables* tables,
                                    int32_t* d_error_word, void* stream) {
  rb::CallRange range_("rb_pages_count");
  using namespace rb;
  PageArgs a;
  rb_status st = setup(dims, tables, true, nullptr, nullptr, false, nullptr, 0, false,
                       d_error_word, &a);
  if (st != RB_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(a.ref, 0, sizeof(int32_t) * static_cast<size_t>(a.entries), s) !=
      cudaSuccess)
    return RB_ERR_CUDA;
  if (a.rows == 0) return RB_OK;
  pages_count_kernel<<<a.rows, 256, 0, s>>>(a);
  if (last_launch_status() != RB_OK) return RB_ERR_CUDA;
  note_launches(1);
  return RB_OK;
}

extern "C" rb_status rb_pages_copy(const rb_dims* dims, int32_t num_pairs, const int32_t* d_src,
                                   const int32_t* d_dst, void* d_k_cache, void* d_v_cache,
                                   void* d_workspace, size_t workspace_bytes,
                                   int32_t* d_error_word, void* stream) {
  rb::CallRange range_("rb_pages_copy");
  using namespace rb;
  PageArgs a;
  rb_status st = setup(dims, nullptr, false, d_k_cache, d_v_cache, true, d_workspace,
                       workspace_bytes, true, d_error_word, &a);
  if (st != RB_OK) return st;
  if (num_pairs < 0) return RB_ERR_INVALID_ARG;
  if (num_pairs > a.entries) return RB_ERR_CAPACITY;
  if (num_pairs == 0) return RB_OK;
  if (d_src == nullptr || d_dst == nullptr) return RB_ERR_INVALID_ARG;
  const int grid = 1 + copy_grid(a, num_pairs);
  return launch_overlapped(pages_copy_kernel, grid, kCopyThreads, 0,
                           static_cast<cudaStream_t>(stream), a, num_pairs, d_src, d_dst,
                           ws_of(d_workspace, a.entries, dims->max_num_reqs).code);
}

extern "C" rb_status rb_pages_fork(const rb_dims* dims, const rb_page_tables* tables,
                                   int32_t num_forks, const int32_t* d_src_rows,
                                   const int32_t* d_dst_rows, const int32_t* d_num_cached,
                                   void* d_k_cache, void* d_v_cache, void* d_workspace,
                                   size_t workspace_bytes, int32_t* d_error_word, void* stream) {
  rb::CallRange range_("rb_pages_fork");
  using namespace rb;
  PageArgs a;
  rb_status st = setup(dims, tables, true, d_k_cache, d_v_cache, true, d_workspace,
                       workspace_bytes, true, d_error_word, &a);
  if (st != RB_OK) return st;
  if (num_forks < 0) return RB_ERR_INVALID_ARG;
  if (num_forks > a.rows) return RB_ERR_CAPACITY;
  if (num_forks == 0) return RB_OK;
  if (d_src_rows == nullptr || d_dst_rows == nullptr || d_num_cached == nullptr)
    return RB_ERR_INVALID_ARG;
  const PagesWs w = ws_of(d_workspace, a.entries, dims->max_num_reqs);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = launch_overlapped(fork_plan_kernel, 1, kCheckThreads, 0, s, a, num_forks, d_src_rows,
                         d_dst_rows, d_num_cached, w.code, w.movers, w.holes, w.header);
  if (st != RB_OK) return st;
  return launch_overlapped(fork_apply_kernel, num_forks, kCopyThreads, 0, s, a, num_forks,
                           d_src_rows, d_dst_rows, d_num_cached, w.movers, w.header);
}

extern "C" rb_status rb_pages_free(const rb_dims* dims, const rb_page_tables* tables,
                                   int32_t num_free, const int32_t* d_rows, int32_t* d_num_freed,
                                   int32_t* d_error_word, void* stream) {
  rb::CallRange range_("rb_pages_free");
  using namespace rb;
  PageArgs a;
  rb_status st = setup(dims, tables, true, nullptr, nullptr, false, nullptr, 0, false,
                       d_error_word, &a);
  if (st != RB_OK) return st;
  if (num_free < 0 || (num_free > 0 && d_rows == nullptr)) return RB_ERR_INVALID_ARG;
  if (num_free == 0 && d_num_freed == nullptr) return RB_OK;
  return launch_overlapped(pages_free_kernel, kClusterCtas, kCheckThreads, 0,
                           static_cast<cudaStream_t>(stream), a, num_free, d_rows, d_num_freed);
}

extern "C" rb_status rb_pages_compact(const rb_dims* dims, const rb_page_tables* tables,
                                      int32_t* d_page_map, int32_t* d_num_live, void* d_k_cache,
                                      void* d_v_cache, void* d_workspace, size_t workspace_bytes,
                                      int32_t* d_error_word, void* stream) {
  rb::CallRange range_("rb_pages_compact");
  using namespace rb;
  PageArgs a;
  rb_status st = setup(dims, tables, true, d_k_cache, d_v_cache, true, d_workspace,
                       workspace_bytes, true, d_error_word, &a);
  if (st != RB_OK) return st;
  const PagesWs w = ws_of(d_workspace, a.entries, dims->max_num_reqs);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = launch_overlapped(compact_plan_kernel, kClusterCtas, kCheckThreads, 0, s, a, w,
                         d_num_live);
  if (st != RB_OK) return st;
  const int table_ctas =
      min(max(a.rows, (a.entries + 4095) / 4096), max(1, device_sm_count()));
  // at most half of the pages move
  const int grid = table_ctas + copy_grid(a, a.entries / 2);
  return launch_overlapped(compact_move_kernel, grid, kCopyThreads, 0, s, a, w, d_page_map,
                           table_ctas);
}
