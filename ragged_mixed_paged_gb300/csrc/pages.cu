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
// few dependent passes over the counts and is bound by latency.
#include "rb_internal.cuh"

namespace rb {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCheckThreads = 1024;
constexpr int kScan = 2048;  // reference counts per CTA of a compaction's passes

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

// Workspace: [mark / code: entries][list a: entries][list b: entries][chunk counts][header]
struct PagesWs {
  int32_t *code, *movers, *holes, *counts, *header;
};
enum HeaderInt : int { kHOk = 0, kHMoves = 1, kHLive = 2, kHInts = 16 };

__host__ __device__ inline size_t up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

inline size_t ws_bytes(int entries, int rows) {
  const size_t list = up(sizeof(int32_t) * static_cast<size_t>(entries > rows ? entries : rows));
  const size_t counts = up(sizeof(int32_t) * (static_cast<size_t>(entries) / kScan + 2));
  return 3 * list + counts + up(kHInts * sizeof(int32_t));
}

inline PagesWs ws_of(void* p, int entries, int rows) {
  const size_t list = up(sizeof(int32_t) * static_cast<size_t>(entries > rows ? entries : rows));
  const size_t counts = up(sizeof(int32_t) * (static_cast<size_t>(entries) / kScan + 2));
  unsigned char* b = static_cast<unsigned char*>(p);
  PagesWs w;
  w.code = reinterpret_cast<int32_t*>(b);
  w.movers = reinterpret_cast<int32_t*>(b + list);
  w.holes = reinterpret_cast<int32_t*>(b + 2 * list);
  w.counts = reinterpret_cast<int32_t*>(b + 3 * list);
  w.header = reinterpret_cast<int32_t*>(b + 3 * list + counts);
  return w;
}

__device__ __forceinline__ bool valid_page(const PageArgs& a, int id) {
  return id >= 0 && id < a.entries && id != a.null_entry;
}

// One page-sized run of 16-byte chunks, by one CTA's threads.
__device__ __forceinline__ void copy_chunks(int4* dst, const int4* src, long long first,
                                            long long last, int tid, int threads) {
  constexpr int kUnroll = 4;
  long long i = first + tid;
  for (; i + (kUnroll - 1) * threads < last; i += kUnroll * threads) {
    int4 x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) x[u] = src[i + u * threads];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) dst[i + u * threads] = x[u];
  }
  for (; i < last; i += threads) dst[i] = src[i];
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
// CTA 0 checks the pairs (a destination twice, or also a source) while the others copy: where
// it finds one the error bit is set and the pages' contents are unspecified.
__global__ void __launch_bounds__(kCopyThreads)
    pages_copy_kernel(PageArgs a, int n, const int32_t* src, const int32_t* dst, int32_t* mark) {
  const int tid = threadIdx.x;
  if (blockIdx.x == 0) {
    int bits = 0;
    for (int i = tid; i < n; i += kCopyThreads) {
      const int s = src[i], d = dst[i];
      if (s < 0 || d < 0) continue;  // skipped pair
      if (!valid_page(a, s) || !valid_page(a, d)) {
        bits |= RB_EBIT_BLOCK_ID;
        continue;
      }
      mark[s] = 0;
      mark[d] = 0;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kCopyThreads) {
      const int s = src[i], d = dst[i];
      if (!valid_page(a, s) || !valid_page(a, d)) continue;
      atomicOr(mark + s, 1 << 30);
      if (atomicAdd(mark + d, 1) & 0xffffff) bits |= RB_EBIT_PAGE_PAIR;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kCopyThreads) {
      const int s = src[i], d = dst[i];
      if (valid_page(a, s) && valid_page(a, d) && (__ldcg(mark + d) & (1 << 30)))
        bits |= RB_EBIT_PAGE_PAIR;
    }
    if (bits) raise_error(a.err, bits);
    return;
  }
  const int first = blockIdx.x - 1, step = gridDim.x - 1;
  const long long chunk = 4 * kCopyThreads;
  const long long parts = (a.page_chunks + chunk - 1) / chunk;
  const long long units = 2LL * n * parts;
  for (long long u = first; u < units; u += step) {
    const long long i = u / (2 * parts), rest = u - i * 2 * parts;
    const int s = __ldg(src + i), d = __ldg(dst + i);
    if (!valid_page(a, s) || !valid_page(a, d)) continue;
    int4* base = rest >= parts ? a.v : a.k;
    const long long c0 = (rest >= parts ? rest - parts : rest) * chunk;
    copy_chunks(base + d * a.page_chunks, base + s * a.page_chunks, c0,
                min(a.page_chunks, c0 + chunk), tid, kCopyThreads);
  }
}

// Exclusive prefix sum over a block of kCheckThreads threads; *total gets the block's sum.
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
  const int tid = threadIdx.x;
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
  int found = 0;
  for (int base = 0; base < a.entries && found < need; base += kCheckThreads) {
    const int id = base + tid;
    const int is_free = id < a.entries && id != a.null_entry && a.ref[id] == 0;
    int total;
    const int at = found + block_prefix(is_free, tmp, &total);
    if (is_free && at < need) free_list[at] = id;
    found += total;
  }
  if (found < need) bits |= RB_EBIT_NO_PAGE;
  if (bits) atomicOr(&s_bits, bits);
  __syncthreads();
  if (tid == 0) {
    header[kHOk] = s_bits == 0;
    if (s_bits) raise_error(a.err, s_bits);
  }
  for (int i = tid; i < n; i += kCheckThreads)
    if (fresh[i] >= 0 && fresh[i] < found) fresh[i] = free_list[fresh[i]];
}

__global__ void __launch_bounds__(kCopyThreads)
    fork_apply_kernel(PageArgs a, int n, const int32_t* src, const int32_t* dst,
                      const int32_t* cached, const int32_t* fresh, const int32_t* header) {
  if (!header[kHOk]) return;
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
      copy_chunks(a.k + page * a.page_chunks, a.k + old * a.page_chunks, 0, count, tid,
                  kCopyThreads);
      copy_chunks(a.v + page * a.page_chunks, a.v + old * a.page_chunks, 0, count, tid,
                  kCopyThreads);
    }
  }
  if (tid == 0) a.num_blocks[d] = full + (tail > 0);
}

// -------------------------------------------------------------------------------------- free
__global__ void __launch_bounds__(256)
    pages_free_kernel(PageArgs a, const int32_t* list, int32_t* num_freed) {
  __shared__ int s_n;
  const int r = list[blockIdx.x];
  if (r < 0 || r >= a.rows) {
    if (threadIdx.x == 0) raise_error(a.err, RB_EBIT_ROW);
    return;
  }
  // the first CTA to take the row's count frees it; a row named twice is then empty
  if (threadIdx.x == 0) s_n = atomicExch(a.num_blocks + r, 0);
  __syncthreads();
  const int n = s_n;
  if (n < 0 || n > a.MB) {
    if (threadIdx.x == 0) raise_error(a.err, RB_EBIT_ROW);
    return;
  }
  int freed = 0;
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    int32_t* e = a.table + static_cast<size_t>(r) * a.MB + j;
    const int id = *e;
    *e = -1;
    if (!valid_page(a, id)) {
      raise_error(a.err, RB_EBIT_BLOCK_ID);
      continue;
    }
    const int was = atomicSub(a.ref + id, 1);
    if (was < 1) {
      atomicAdd(a.ref + id, 1);
      raise_error(a.err, RB_EBIT_PAGE_REF);
    }
    freed += was == 1;
  }
  if (num_freed != nullptr) {
    for (int o = 16; o > 0; o >>= 1) freed += __shfl_xor_sync(0xffffffffu, freed, o);
    if ((threadIdx.x & 31) == 0 && freed) atomicAdd(num_freed, freed);
  }
}

// ----------------------------------------------------------------------------------- compact
__device__ __forceinline__ int is_live(const PageArgs& a, int id) {
  return id < a.entries && id != a.null_entry && a.ref[id] > 0;
}

__global__ void __launch_bounds__(kCheckThreads)
    compact_count_kernel(PageArgs a, int32_t* counts) {
  __shared__ int s_n;
  if (threadIdx.x == 0) s_n = 0;
  __syncthreads();
  int n = 0, bits = 0;
  for (int k = threadIdx.x; k < kScan; k += kCheckThreads) {
    const int id = blockIdx.x * kScan + k;
    n += is_live(a, id);
    if (id < a.entries && id != a.null_entry && a.ref[id] < 0) bits |= RB_EBIT_PAGE_REF;
  }
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  if ((threadIdx.x & 31) == 0) atomicAdd(&s_n, n);
  __syncthreads();
  if (threadIdx.x == 0) counts[blockIdx.x] = s_n;
  if (bits) raise_error(a.err, bits);
}

// Classifies the ids of one chunk: code[id] = id (stays, or the null page), -1 (free), or
// -2 - m for mover number m; lists the movers and the holes they go to.
__global__ void __launch_bounds__(kCheckThreads)
    compact_list_kernel(PageArgs a, PagesWs w, int chunks, int32_t* num_live) {
  __shared__ int tmp[32];
  __shared__ int s_before, s_total, s_low;
  const int tid = threadIdx.x;
  // live pages in all, and before this chunk
  if (tid == 0) s_before = s_total = s_low = 0;
  __syncthreads();
  int before = 0, total = 0;
  for (int c = tid; c < chunks; c += kCheckThreads) {
    const int n = w.counts[c];
    total += n;
    before += c < static_cast<int>(blockIdx.x) ? n : 0;
  }
  atomicAdd(&s_before, before);
  atomicAdd(&s_total, total);
  __syncthreads();
  before = s_before;
  total = s_total;
  // the packed region is every id below `limit` but the null page; live pages already in it
  const int limit = total + (a.null_entry <= total);
  const int at = limit / kScan;  // its last chunk, partly inside
  int low = 0;
  for (int c = tid; c < min(at, chunks); c += kCheckThreads) low += w.counts[c];
  for (int id = at * kScan + tid; id < min(limit, a.entries); id += kCheckThreads)
    low += is_live(a, id);
  atomicAdd(&s_low, low);
  __syncthreads();
  low = s_low;
  if (blockIdx.x == 0 && tid == 0) {
    w.header[kHMoves] = total - low;
    if (num_live != nullptr) *num_live = total;
  }
  int rank = before;  // live pages below the id
  for (int k = 0; k < kScan; k += kCheckThreads) {
    const int id = blockIdx.x * kScan + k + tid;
    const int live = is_live(a, id);
    int all;
    const int mine = rank + block_prefix(live, tmp, &all);
    rank += all;
    if (id >= a.entries) continue;
    int code = -1;
    if (id == a.null_entry) {
      code = id;
    } else if (live) {
      code = id < limit ? id : -2 - (mine - low);
      if (id >= limit) w.movers[mine - low] = id;
    } else if (id < limit) {
      w.holes[id - (id > a.null_entry) - mine] = id;
    }
    w.code[id] = code;
  }
}

__global__ void __launch_bounds__(kCopyThreads)
    compact_move_kernel(PageArgs a, PagesWs w, int32_t* page_map, int table_ctas) {
  const int tid = threadIdx.x;
  auto moved = [&](int id) {
    const int c = w.code[id];
    return c <= -2 ? w.holes[-2 - c] : c;
  };
  if (static_cast<int>(blockIdx.x) < table_ctas) {
    // the page table's entries, and the map
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
  const int moves = w.header[kHMoves];
  const long long chunk = 4 * kCopyThreads;
  const long long parts = (a.page_chunks + chunk - 1) / chunk;
  const long long units = 2LL * moves * parts;
  for (long long u = blockIdx.x - table_ctas; u < units; u += gridDim.x - table_ctas) {
    const long long i = u / (2 * parts), rest = u - i * 2 * parts;
    const int s = w.movers[i], d = w.holes[i];
    if (rest == 0 && tid == 0) {
      a.ref[d] = a.ref[s];
      a.ref[s] = 0;
    }
    int4* base = rest >= parts ? a.v : a.k;
    const long long c0 = (rest >= parts ? rest - parts : rest) * chunk;
    copy_chunks(base + d * a.page_chunks, base + s * a.page_chunks, c0,
                min(a.page_chunks, c0 + chunk), tid, kCopyThreads);
  }
}

// ---------------------------------------------------------------------------------- host side
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
  const long long chunk = 4 * kCopyThreads;
  const long long units = 2LL * num_pairs * ((a.page_chunks + chunk - 1) / chunk);
  const long long most = 8LL * max(1, device_sm_count());
  const int grid = 1 + static_cast<int>(units < most ? units : most);
  pages_copy_kernel<<<grid, kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      a, num_pairs, d_src, d_dst, ws_of(d_workspace, a.entries, dims->max_num_reqs).code);
  if (last_launch_status() != RB_OK) return RB_ERR_CUDA;
  note_launches(1);
  return RB_OK;
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
  fork_plan_kernel<<<1, kCheckThreads, 0, s>>>(a, num_forks, d_src_rows, d_dst_rows,
                                               d_num_cached, w.code, w.movers, w.holes,
                                               w.header);
  if (last_launch_status() != RB_OK) return RB_ERR_CUDA;
  note_launches(1);
  fork_apply_kernel<<<num_forks, kCopyThreads, 0, s>>>(a, num_forks, d_src_rows, d_dst_rows,
                                                       d_num_cached, w.movers, w.header);
  if (last_launch_status() != RB_OK) return RB_ERR_CUDA;
  note_launches(1);
  return RB_OK;
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d_num_freed != nullptr && cudaMemsetAsync(d_num_freed, 0, sizeof(int32_t), s) != cudaSuccess)
    return RB_ERR_CUDA;
  if (num_free == 0) return RB_OK;
  pages_free_kernel<<<num_free, 256, 0, s>>>(a, d_rows, d_num_freed);
  if (last_launch_status() != RB_OK) return RB_ERR_CUDA;
  note_launches(1);
  return RB_OK;
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
  const int chunks = (a.entries + kScan - 1) / kScan;
  compact_count_kernel<<<chunks, kCheckThreads, 0, s>>>(a, w.counts);
  if (last_launch_status() != RB_OK) return RB_ERR_CUDA;
  note_launches(1);
  compact_list_kernel<<<chunks, kCheckThreads, 0, s>>>(a, w, chunks, d_num_live);
  if (last_launch_status() != RB_OK) return RB_ERR_CUDA;
  note_launches(1);
  const int sms = max(1, device_sm_count());
  const int table_ctas = min(max(a.rows, 1), sms);
  compact_move_kernel<<<table_ctas + 8 * sms, kCopyThreads, 0, s>>>(a, w, d_page_map, table_ctas);
  if (last_launch_status() != RB_OK) return RB_ERR_CUDA;
  note_launches(1);
  return RB_OK;
}
